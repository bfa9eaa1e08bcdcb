"""Rotary append, attention with terms and accept on the CPU: the plain
implementation's own pins, and what the entry points refuse before any GPU
call (no arguments here would be launched)."""
import ctypes
import math

import pytest
import torch

import arena_compaction_amd as ac
from kv_more_plain import PAGE, Cache, accept, attend, rotate, tree, walk, words_of
from kv_plain import attend as causal_attend
from test_kv import CACHE_FAULTS, _args

E4M3, INT8 = torch.float8_e4m3fn, torch.int8


# ---- the plain implementation

def test_plain_rotation():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 5.0, 6.0]]])
    freq = torch.tensor([math.pi / 2, math.pi], dtype=torch.float64)
    halves = rotate(x, torch.tensor([1]), freq, False)[0, 0]
    assert torch.allclose(halves, torch.tensor([-3.0, -2.0, 1.0, -4.0, 5.0, 6.0], dtype=torch.float64))
    neighbours = rotate(x, torch.tensor([1]), freq, True)[0, 0]
    assert torch.allclose(neighbours, torch.tensor([-2.0, 1.0, -3.0, -4.0, 5.0, 6.0], dtype=torch.float64))


def test_plain_rotation_keeps_distances():
    """Scores of rotated queries and keys go by the difference of their positions alone."""
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(2, 1, 64, generator=gen)
    freq = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    scores = [float((rotate(x[:1], torch.tensor([p]), freq, False) * rotate(x[1:], torch.tensor([p + 9]), freq, False)).sum())
              for p in (0, 5, 1000)]
    assert max(scores) - min(scores) < 1e-10


def test_plain_words():
    seen = torch.zeros(2, 70, dtype=torch.bool)
    seen[0, 0] = seen[0, 63] = seen[1, 64] = seen[1, 69] = True
    assert words_of(seen).tolist() == [[1 | -(1 << 63), 0], [0, 1 | 1 << 5]]
    assert words_of(seen, 3).shape == (2, 3)


def test_plain_attention_without_terms_is_causal():
    c = Cache([2], 1, 64, INT8)
    c.fill_random([90], 1)
    q = torch.randn(5, 2, 64, generator=torch.Generator().manual_seed(2))
    want = causal_attend(c, [90], q, 2, [5], 0.125)
    same = torch.ones(5, 5, dtype=torch.bool).tril()
    for mask in (None, [same]):
        got = attend(c, [90], q, 2, [5], 0.125, mask)
        for i in (0, 2, 4):
            assert torch.allclose(got[i], want[i], rtol=1e-12, atol=1e-12)


def test_plain_accept():
    gen = torch.Generator().manual_seed(3)
    up, seen, depth = tree(30, 3, gen)
    path = walk(up, gen)
    assert path == sorted(path) and all(bool(seen[b, a]) for a, b in zip(path, path[1:]))
    assert [depth[i] for i in path] == list(range(len(path)))
    c = Cache([2], 2, 64, INT8)
    c.fill_random([80], 1, spread=4)
    before = [c.numbers(0, 80, h) for h in (0, 1)]
    pos = torch.arange(128, dtype=torch.int32).expand(1, 2, 128).clone()
    assert accept(c, [80], [30], [path], None, pos) == [50 + len(path)]
    for h in (0, 1):
        k, v, _ = c.numbers(0, 50 + len(path), h)
        scale = max(float(x) for j in (0, 1) for x in c.head(int(c.pages[0, j]), h)[2])
        src = list(range(50)) + [50 + i for i in path]
        assert pos[0, h, : len(src)].tolist() == src
        assert (k - before[h][0][src]).abs().max() <= scale and (v - before[h][1][src]).abs().max() <= scale


# ---- refusals

def _rotary(**change):
    r = {k: change.pop(k) for k in list(change) if k in ("freq_dev", "rotary_dim", "interleaved", "token_pos_dev", "q_dev", "q_row",
                                                        "q_head", "out_dev", "out_row", "out_head", "q_heads")}
    a = _args(ac.defrag_kv_append_args, **change)
    out = ac.defrag_kv_rotary_args(ctypes.pointer(a), 0xA0000, 64, 0, None, 0xB0000, 512, 64, 0xC0000, 512, 64, 8, 0)
    for k, v in r.items():
        setattr(out, k, v)
    return out


@pytest.mark.parametrize("fault", CACHE_FAULTS + [
    dict(k_dev=None), dict(v_dev=0x50001), dict(dtype=2), dict(max_new=0), dict(max_new=5), dict(tokens=3),
    dict(freq_dev=None), dict(freq_dev=0xA0004), dict(rotary_dim=0), dict(rotary_dim=4), dict(rotary_dim=12), dict(rotary_dim=72),
    dict(interleaved=2), dict(interleaved=-1), dict(token_pos_dev=0x1002), dict(q_dev=None), dict(q_dev=0xB0001), dict(out_dev=None),
    dict(out_dev=0xC0001), dict(q_heads=8 * 65534), dict(heads=65528, q_heads=65),
    # rows of the output that overlap one another
    dict(out_row=0), dict(out_head=0), dict(out_head=63), dict(out_row=511), dict(out_row=64, out_head=255), dict(out_row=-511),
    # outputs over inputs
    dict(out_dev=0xB0000, out_row=513), dict(out_dev=0xB0000, out_head=-64), dict(out_dev=0xB0000 + 128), dict(out_dev=0x40010),
    dict(out_dev=0x50000 - 64), dict(out_dev=0x20000), dict(out_dev=0x30008), dict(out_dev=0xA0080), dict(out_dev=0x8000040),
    dict(out_dev=0xC0000, weight_dev=0xC0100, weight_stride=8), dict(out_dev=0xC0000, pos_dev=0xC0FF0, weight_stride=8),
    dict(token_pos_dev=0xC0000), dict(first_pos_dev=0xC0FFC), dict(out_dev=0xC0000, starts_dev=0xC0004),
    # between another's rows: queries of 8 heads into rows 2 heads wide
    dict(q_dev=0xB0000, q_row=640, out_dev=0xB0000 + 1024, out_row=640)])
def test_rotary_refusals(fault):
    r = _rotary(**{"arena_dev": 0x8000000, **fault})
    assert ac.lib.defrag_kv_append_rotary(ctypes.byref(r), None) == ac.DEFRAG_EINVAL


def test_rotary_refuses_null():
    assert ac.lib.defrag_kv_append_rotary(None, None) == ac.DEFRAG_EINVAL
    r = _rotary()
    r.append = None
    assert ac.lib.defrag_kv_append_rotary(ctypes.byref(r), None) == ac.DEFRAG_EINVAL


def _terms(**change):
    t = ac.defrag_kv_terms(0xA0000, 1, 30.0, 0, 0xB0000, 0xC0000, 1024)
    for k, v in change.items():
        setattr(t, k, v)
    return t


def terms_say(args, **change):
    """(bytes the query asks for, what the call says without a workspace)."""
    a = _args(ac.defrag_kv_attend_args, **{**dict(group=4, weight_dev=0x8000000, weight_stride=1024), **args})
    t = _terms(**change)
    need = ac.lib.defrag_kv_attend_terms_workspace_bytes(ctypes.byref(a), ctypes.byref(t))
    assert need != 1, "would be launched"
    return need, ac.lib.defrag_kv_attend_terms(ctypes.byref(a), ctypes.byref(t), None, 0, None)


REFUSED = (0, ac.DEFRAG_EINVAL)


@pytest.mark.parametrize("fault", CACHE_FAULTS + [
    dict(q_dev=None), dict(out_dev=None), dict(dtype=-1), dict(group=0), dict(max_new=0), dict(max_len=1025),
    dict(scale=float("nan")), dict(weight_stride=1023), dict(lse_dev=0x1002)])
def test_terms_refuse_what_attend_refuses(fault):
    assert terms_say(fault) == REFUSED


@pytest.mark.parametrize("fault", [
    dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(cap=2.0 ** -65), dict(cap=2.0 ** 65),
    dict(mask_dev=0xA0004), dict(mask_words=0), dict(mask_words=(1 << 23) + 1), dict(slopes_dev=0xB0002), dict(pos_dev=0xC0002),
    dict(pos_stride=1023), dict(pos_stride=0), dict(pos_stride=1 << 40)])
def test_terms_refusals(fault):
    assert terms_say({}, **fault) == REFUSED


def test_terms_positions_are_needed_up_to_a_pages_end():
    assert terms_say(dict(max_len=961), pos_stride=1023) == REFUSED
    assert terms_say(dict(max_len=960), pos_stride=960)[1] == ac.DEFRAG_EWORKSPACE
    assert terms_say(dict(max_len=961), pos_dev=None, pos_stride=0)[1] == ac.DEFRAG_EWORKSPACE


def test_terms_mask_words():
    sizes = dict(tokens=300, max_new=129, starts_dev=0x1000)
    for words, said in ((2, ac.DEFRAG_EINVAL), (3, ac.DEFRAG_EWORKSPACE), (9, ac.DEFRAG_EWORKSPACE)):
        assert terms_say({**sizes, "out_dev": 0x50000000, "q_dev": 0x60000000}, mask_words=words)[1] == said


@pytest.mark.parametrize("args,change", [
    (dict(out_dev=0xA0000), {}), (dict(lse_dev=0xA0010), {}), (dict(out_dev=0xB0000), {}), (dict(weight_dev=0xC0000), {}),
    (dict(lse_dev=0xC0FF0), {}), (dict(), dict(mask_dev=0x50FF8)), (dict(), dict(slopes_dev=0x8000000)),
    (dict(out_dev=0x40000), {})])
def test_terms_refuse_outputs_over_inputs(args, change):
    assert terms_say(args, **change) == REFUSED


def test_terms_take_all_or_none():
    for change in (dict(), dict(mask_dev=None, mask_words=0), dict(cap=0.0), dict(slopes_dev=None), dict(pos_dev=None),
                   dict(mask_dev=None, cap=0.0, slopes_dev=None, pos_dev=None, mask_words=0, pos_stride=0)):
        need, said = terms_say({}, **change)
        assert need > 1 and said == ac.DEFRAG_EWORKSPACE
    a = _args(ac.defrag_kv_attend_args)
    assert ac.lib.defrag_kv_attend_terms_workspace_bytes(ctypes.byref(a), None) == 0
    assert ac.lib.defrag_kv_attend_terms(ctypes.byref(a), None, None, 0, None) == ac.DEFRAG_EINVAL
    assert ac.lib.defrag_kv_attend_terms(None, ctypes.byref(_terms()), None, 0, None) == ac.DEFRAG_EINVAL


def test_workspaces_of_attend_and_of_terms():
    """The bytes that attend asks for, but of short caches, which terms leave whole."""
    def both(**sizes):
        sizes = {**dict(weight_dev=0x8000000, weight_stride=4096, page_stride=64, max_len=4096), **sizes}
        need = ac.lib.defrag_kv_attend_workspace_bytes(ctypes.byref(_args(ac.defrag_kv_attend_args, **sizes)))
        return need, terms_say(sizes, mask_words=11, pos_stride=4096, pos_dev=0x20000000)[0]
    for sizes in (dict(group=4), dict(group=16, weight_dev=None), dict(group=4, max_len=1025), dict(group=4, dim=192, max_len=1024),
                  dict(group=4, batch=1, tokens=700, max_new=700, starts_dev=0x1000, q_dev=0x4000000, out_dev=0x5000000)):
        need, terms = both(**sizes)
        assert need > 1 and terms == need
    need, terms = both(group=4, max_len=1024)
    assert 1 < terms < need


def _accept(**change):
    c = ac.defrag_kv_cache(0x8000000, 1 << 20, 0x20000, 16, 0x30000, 4, 2, 64, 0, None)
    for k in [k for k in change if k in ("arena_dev", "pages_dev", "page_stride", "lens_dev", "batch", "heads", "dim", "codes",
                                         "n_invalid_dev")]:
        setattr(c, k, change.pop(k))
    a = ac.defrag_kv_accept_args(ctypes.pointer(c), 40, 0x40000, 16, 0, 0x50000, 16, 0x60000, 0x70000, 0x80000, 1024, 0x90000)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("fault", CACHE_FAULTS + [
    dict(n_invalid_dev=0x1004), dict(tokens=1 << 40), dict(starts_dev=None), dict(starts_dev=0x40002), dict(max_new=0), dict(max_new=41),
    dict(path_dev=None), dict(path_dev=0x50002), dict(path_stride=(1 << 32) + 1), dict(kept_dev=None), dict(kept_dev=0x60002),
    dict(weight_dev=0x70002), dict(pos_dev=0x80002), dict(lens_out_dev=None), dict(lens_out_dev=0x90002),
    dict(lens_out_dev=0x30000), dict(lens_out_dev=0x3000C), dict(lens_out_dev=0x40010), dict(lens_out_dev=0x500FC),
    dict(lens_out_dev=0x60004), dict(lens_out_dev=0x20000), dict(lens_out_dev=0x77FFC), dict(pos_dev=0x70010), dict(weight_dev=0x50000),
    dict(pos_dev=0x60000), dict(lens_out_dev=0x8000010), dict(weight_dev=0x8000000 + (1 << 20) - 4)])
def test_accept_refusals(fault):
    a = _accept(**fault)
    assert ac.lib.defrag_kv_accept(ctypes.byref(a), None) == ac.DEFRAG_EINVAL
    assert ac.lib.defrag_kv_accept(None, None) == ac.DEFRAG_EINVAL


def test_binding_refuses():
    """Tensors on the CPU, of other types and shapes."""
    arena, pages, lens = torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    k = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ac.defrag_kv_append_rotary(arena, pages, lens, k, k, E4M3, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        ac.defrag_kv_attend_terms(arena, pages, lens, k, 1, E4M3, cap=3.0)
    with pytest.raises(ValueError):
        ac.defrag_kv_accept(arena, pages, lens, torch.zeros(2, 4, dtype=torch.int32), lens, lens.clone(), 1, 64, E4M3)
    assert PAGE == ac.KV_PAGE_TOKENS


APPEND_FAULTS = [   # rows of 4 x 2 x 8 numbers from 0x800000 on are 0x100 bytes
    dict(weight_dev=0x800000, pos_dev=0x800000), dict(weight_dev=0x800000, pos_dev=0x8000FC),
    dict(weight_dev=0x800000, first_pos_dev=0x8000F4), dict(pos_dev=0x800000, first_pos_dev=0x800010),
    dict(pos_dev=0x20000), dict(weight_dev=0x30008), dict(pos_dev=0x40010), dict(weight_dev=0x50000 - 4),
    dict(pos_dev=0x800000, starts_dev=0x800000)]
ROTARY_FAULTS = [
    dict(pos_dev=0x800000, token_pos_dev=0x8000F0), dict(weight_dev=0x800000, token_pos_dev=0x800000),
    dict(pos_dev=0x800000, freq_dev=0x800080), dict(weight_dev=0x800000 - 4, freq_dev=0x800000)]


@pytest.mark.parametrize("fault", APPEND_FAULTS + [dict(weight_dev=0x30010, weight_stride=1 << 60)])
def test_append_refuses_planes_over_what_it_reads(fault):
    a = _args(ac.defrag_kv_append_args, **{"arena_dev": 0x8000000, "weight_stride": 8, **fault})
    said = ac.lib.defrag_kv_append(ctypes.byref(a), None)
    assert said == ac.DEFRAG_EINVAL


@pytest.mark.parametrize("queries", [dict(), dict(q_heads=0, q_dev=None, out_dev=None)])
@pytest.mark.parametrize("fault", APPEND_FAULTS + ROTARY_FAULTS)
def test_rotary_refuses_planes_over_what_it_reads(fault, queries):
    r = _rotary(**{"arena_dev": 0x8000000, "weight_stride": 8, **fault, **queries})
    assert ac.lib.defrag_kv_append_rotary(ctypes.byref(r), None) == ac.DEFRAG_EINVAL


@pytest.mark.parametrize("fault", [dict(pos_dev=0xB0100), dict(weight_dev=0xB0000 + 8 * 64 * 2 * 4 - 4)])
def test_rotary_refuses_planes_over_queries(fault):
    r = _rotary(**{"arena_dev": 0x8000000, "weight_stride": 8, **fault})
    assert ac.lib.defrag_kv_append_rotary(ctypes.byref(r), None) == ac.DEFRAG_EINVAL


@pytest.mark.parametrize("cap", [1e-50, -1e-46, 5e-324])
def test_binding_refuses_a_cap_that_its_field_would_make_none(cap):
    """Below what a float32 holds: 0 there would mean that there is no cap."""
    arena, pages, lens = torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ac.DefragError):
        ac.defrag_kv_attend_terms(arena, pages, lens, q, 1, E4M3, cap=cap)


@pytest.mark.parametrize("batch,max_new,group,dim,pieces", [
    (34, 1, 4, 128, 2), (48, 1, 4, 96, 2), (33, 1, 4, 128, 1), (49, 1, 4, 128, 1), (40, 1, 4, 64, 1), (40, 5, 4, 128, 1),
    (40, 5, 4, 96, 1), (40, 1, 4, 192, 1)])
def test_terms_cut_long_caches_in_two_where_that_was_measured_to_gain(batch, max_new, group, dim, pieces):
    """8 heads, 8000 tokens: two pieces for 272 to 384 (sequence, head)s of up to 16 rows and 96 or 128 dimensions."""
    tokens = batch * max_new
    a = _args(ac.defrag_kv_attend_args, batch=batch, heads=8, dim=dim, page_stride=125, tokens=tokens, starts_dev=0x1000, max_new=max_new,
              group=group, max_len=8000, q_dev=0x20000000, out_dev=0x30000000, weight_dev=None)
    need = ac.lib.defrag_kv_attend_terms_workspace_bytes(ctypes.byref(a), ctypes.byref(_terms(mask_dev=None, mask_words=0, slopes_dev=None,
                                                                                               pos_dev=None)))
    parts = pieces * tokens * 8 * group * (dim + 2) * 4 if pieces > 1 else 1
    assert need == (parts + 255) // 256 * 256 if pieces > 1 else need == 1
