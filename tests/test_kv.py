"""The 8-bit key/value cache on the CPU: the plain implementation's own pins,
and what the entry points refuse before any GPU call."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import arena_compaction_amd as ac
from kv_plain import Cache, least_exp, nearest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


def test_plain_exponents_and_codes():
    assert least_exp(448.0, E4M3) == 0 and least_exp(448.1, E4M3) == 1 and least_exp(224.0, E4M3) == -1
    assert least_exp(127.0, INT8) == 0 and least_exp(127.5, INT8) == 1 and least_exp(0.0, INT8) == -64
    x = torch.tensor([0.4, 0.5, 1.5, 2.5, -126.6, 300.0, float("nan"), float("-inf")], dtype=torch.float64)
    assert nearest(x, INT8).tolist() == [0, 0, 2, 2, -127, 127, 0, -127]
    x = torch.tensor([448.0, 500.0, 17.0, 19.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -0.3], dtype=torch.float64)
    assert nearest(x, E4M3).float().tolist() == [448.0, 448.0, 16.0, 20.0, 2.0 ** -9, 0.0, 2.0 ** -8, -0.3125]
    assert torch.isnan(nearest(torch.tensor([float("nan")], dtype=torch.float64), E4M3).float()).all()


def test_plain_cache_reads_back_what_it_holds():
    c = Cache([2], 2, 64, INT8)
    x = torch.arange(-63, 65).float()[:, None, None].expand(128, 2, 64) / 4
    c.append(0, 0, x[:70], x[:70])
    c.append(0, 70, x[70:], x[70:])
    k, v, ok = c.numbers(0, 128, 1)
    assert ok.all() and torch.equal(k, x[:, 0].double()) and torch.equal(v, k)


def test_page_bytes():
    assert ac.defrag_kv_page_bytes(1, 64) == 8192 + 32
    assert ac.defrag_kv_page_bytes(8, 128) == 8 * 128 * 128 + 64
    for bad in ((0, 64), (1, 80), (1, 0), (70000, 64)):
        with pytest.raises(ac.DefragError):
            ac.defrag_kv_page_bytes(*bad)


def _args(cls, **change):
    """Arguments that pass every check (addresses are never followed)."""
    c = ac.defrag_kv_cache(0x10000, 1 << 30, 0x20000, 16, 0x30000, 4, 2, 64, 0, None)
    for k in [k for k in change if k in ("arena_dev", "pages_dev", "page_stride", "lens_dev", "batch", "heads",
                                         "dim", "codes", "n_invalid_dev")]:
        setattr(c, k, change.pop(k))
    if cls is ac.defrag_kv_append_args:
        a = cls(ctypes.pointer(c), 0x40000, 0x50000, 128, 64, 128, 64, 0, 1, 4, None, None, None, None, 0)
    elif cls is ac.defrag_kv_attend_args:
        a = cls(ctypes.pointer(c), 0x40000, 512, 64, 0, 4, 4, None, 1, 1024, 0.125, 0, 0x50000, None, None, 0)
    else:
        a = cls(ctypes.pointer(c), 128, 1024, 4, 16, 0x40000, 0x50000, 0x60000, 1024, 0x70000, 0x80000, 128, 0x90000)
    for k, v in change.items():
        setattr(a, k, v)
    return a


CACHE_FAULTS = [dict(heads=0), dict(dim=80), dict(dim=0), dict(codes=2), dict(codes=-1), dict(batch=70000),
                dict(arena_dev=0x10010), dict(arena_dev=None), dict(pages_dev=None), dict(pages_dev=0x20004),
                dict(lens_dev=None), dict(page_stride=1 << 40)]


@pytest.mark.parametrize("fault", CACHE_FAULTS + [
    dict(k_dev=None), dict(v_dev=0x50001), dict(dtype=2), dict(max_new=0), dict(max_new=5), dict(tokens=3),
    dict(tokens=1 << 40, starts_dev=0x1000), dict(weight_dev=0x1002), dict(n_invalid_dev=0x1004)])
def test_append_refusals(fault):
    a = _args(ac.defrag_kv_append_args, **fault)
    assert ac.lib.defrag_kv_append(ctypes.byref(a), None) == ac.DEFRAG_EINVAL


@pytest.mark.parametrize("fault", CACHE_FAULTS + [
    dict(q_dev=None), dict(out_dev=None), dict(out_dev=0x50008), dict(dtype=-1), dict(group=0), dict(group=257),
    dict(max_new=0), dict(max_new=5), dict(tokens=5), dict(max_len=1025), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(weight_dev=0x1000, weight_stride=1023), dict(lse_dev=0x1002)])
def test_attend_refusals(fault):
    a = _args(ac.defrag_kv_attend_args, **fault)
    assert ac.lib.defrag_kv_attend_workspace_bytes(ctypes.byref(a)) == 0
    assert ac.lib.defrag_kv_attend(ctypes.byref(a), ctypes.c_void_p(0x100000), 1 << 40, None) == ac.DEFRAG_EINVAL


@pytest.mark.parametrize("fault", CACHE_FAULTS + [
    dict(budget=0), dict(budget=100), dict(budget=0xFFFFFFC0), dict(budget=(1 << 25) + 64), dict(max_len=1025), dict(weight_stride=1000),
    dict(weight_out_stride=127), dict(recent=-1), dict(pos_dev=None), dict(next_pos_dev=None),
    dict(weight_out_dev=None), dict(lens_out_dev=0x90002)])
def test_evict_refusals(fault):
    a = _args(ac.defrag_kv_evict_args, **fault)
    assert ac.lib.defrag_kv_evict_workspace_bytes(ctypes.byref(a)) == 0
    assert ac.lib.defrag_kv_evict(ctypes.byref(a), ctypes.c_void_p(0x100000), 1 << 40, None) == ac.DEFRAG_EINVAL


def test_workspace_refusals():
    for cls, size, call in ((ac.defrag_kv_attend_args, ac.lib.defrag_kv_attend_workspace_bytes, ac.lib.defrag_kv_attend),
                            (ac.defrag_kv_evict_args, ac.lib.defrag_kv_evict_workspace_bytes, ac.lib.defrag_kv_evict)):
        a = _args(cls, **({"max_len": 1024, "weight_dev": 0x1000, "weight_stride": 1024}
                          if cls is ac.defrag_kv_attend_args else {}))
        need = size(ctypes.byref(a))
        assert need >= 256
        for ws, n in ((None, need), (0x100010, need), (0x100000, 255)):
            assert call(ctypes.byref(a), ctypes.c_void_p(ws), n, None) == ac.DEFRAG_EWORKSPACE
    assert ac.lib.defrag_kv_append(None, None) == ac.DEFRAG_EINVAL
    assert ac.lib.defrag_kv_attend(None, None, 0, None) == ac.DEFRAG_EINVAL
    assert ac.lib.defrag_kv_evict(None, None, 0, None) == ac.DEFRAG_EINVAL


def test_binding_refuses_before_any_call():
    arena = torch.zeros(1 << 16, dtype=torch.uint8)
    pages, lens = torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    plane, place = torch.zeros(2, 2, 200), torch.zeros(2, 2, 200, dtype=torch.int32)
    for bad in (x.float(), x[0], x):                        # type, shape, host memory
        with pytest.raises(ValueError, match="k:"):
            ac.defrag_kv_append(arena, pages, lens, bad, x, E4M3)
        with pytest.raises(ValueError, match="q:"):
            ac.defrag_kv_attend(arena, pages, lens, bad, 2, E4M3)
    with pytest.raises(ValueError, match="codes"):
        ac._kv_cache(arena, pages, lens, 2, 64, torch.uint8, None)
    with pytest.raises(ValueError, match="lens"):
        ac._kv_cache(arena, pages, lens.long(), 2, 64, E4M3, None)
    with pytest.raises(ValueError, match="pages"):
        ac._kv_cache(arena, pages[0], lens, 2, 64, E4M3, None)
    with pytest.raises(ValueError, match="starts"):
        ac._kv_new(None, None, 3, 2, arena)
    with pytest.raises(ValueError, match="starts"):
        ac._kv_new(torch.zeros(2, dtype=torch.int32), None, 3, 2, arena)
    with pytest.raises(ValueError, match="weight"):
        ac._kv_plane(plane[:1], arena, torch.float32, (2, 2), "weight")
    with pytest.raises(ValueError, match="weight"):
        ac._kv_plane(plane.double(), arena, torch.float32, (2, 2), "weight")
    with pytest.raises(ValueError):
        ac.defrag_kv_evict(arena, pages, lens, 64, plane, place, plane, place, lens, 64, E4M3)   # host memory
    with pytest.raises(ValueError, match="weight"):
        ac.defrag_kv_evict(arena, pages, lens, 64, plane[0], place, plane, place, lens, 64, E4M3)


def test_structs_match_the_header():
    structs = {k: getattr(ac, k) for k in ("defrag_kv_cache", "defrag_kv_append_args", "defrag_kv_attend_args",
                                           "defrag_kv_evict_args")}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "arena_compaction.h"', 'int main(void) {']
    for name, cls in structs.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    lines += ['printf("page %d\\n", DEFRAG_KV_PAGE_TOKENS);', 'return 0; }']
    with tempfile.TemporaryDirectory() as tmp:
        src, exe = os.path.join(tmp, "layout.c"), os.path.join(tmp, "layout")
        open(src, "w").write("\n".join(lines))
        subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include",
                        src, "-o", exe], check=True)
        got = dict(x.rsplit(" ", 1) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(got["page"]) == ac.KV_PAGE_TOKENS
    for name, cls in structs.items():
        assert int(got[name]) == ctypes.sizeof(cls), name
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, f"{name}.{f}"
