"""Sizes of the key/value cache's calls at their limits: what the size query
accepts the call accepts, and nothing is launched here (the workspace is
missing, or the arguments are refused)."""
import ctypes

import pytest

import arena_compaction_amd as ac
from test_kv import _args


def attend_says(**change):
    """(bytes the query asks for, what the call says without a workspace)."""
    apart = {"q_dev": 1 << 46, "out_dev": 1 << 47, "weight_dev": 1 << 55, "weight_stride": 1 << 30}
    a = _args(ac.defrag_kv_attend_args, **{**apart, **change})
    need = ac.lib.defrag_kv_attend_workspace_bytes(ctypes.byref(a))
    assert need != 1, "would be launched"
    return need, ac.lib.defrag_kv_attend(ctypes.byref(a), None, 0, None)


ACCEPTED = [
    # a prompt of 131,072 tokens, 128 query heads
    dict(batch=1, heads=8, group=16, dim=128, tokens=131072, max_new=131072, starts_dev=0x1000, page_stride=2048, max_len=131072),
    # 64 prompts of 4096 tokens, max_new as the binding's default has it
    dict(batch=64, heads=8, group=8, dim=64, tokens=262144, max_new=262144, starts_dev=0x1000, page_stride=64, max_len=4096),
    # drafts over a table for 131,072 tokens
    dict(batch=64, heads=32, group=4, dim=128, tokens=512, max_new=8, starts_dev=0x1000, page_stride=2048, max_len=131072),
    # more than 2^23 workgroups of 512 lanes
    dict(batch=64, heads=64, group=8, dim=256, tokens=262145, max_new=262145, starts_dev=0x1000, page_stride=64, max_len=4096)]


@pytest.mark.parametrize("sizes", ACCEPTED)
def test_attend_takes_ordinary_sizes(sizes):
    need, said = attend_says(**sizes)
    assert need > 1 and said == ac.DEFRAG_EWORKSPACE


LIMITS = [  # the largest that is taken, and the next
    # query rows of a head
    (dict(batch=1, heads=1, group=256, tokens=0x7FFFFC, max_new=0x7FFFFC, starts_dev=0x1000), dict(tokens=0x7FFFFD, max_new=0x7FFFFD)),
    # query rows of a call
    (dict(batch=64, heads=128, group=1, tokens=1 << 29, max_new=1, starts_dev=0x1000), dict(heads=129)),
    # workgroups over the rows
    (dict(batch=65535, heads=255, group=1, tokens=65535, max_new=16384, starts_dev=0x1000), dict(max_new=16385)),
    # workgroups over the pages
    (dict(batch=65535, heads=32, group=1, tokens=65535, max_new=33, starts_dev=0x1000, page_stride=2048, max_len=65536), dict(max_len=65537)),
    # kept scores
    (dict(batch=4, heads=65535, group=1, tokens=4, max_new=1, page_stride=2048, max_len=130560), dict(max_len=130561)),
    # heads over all
    (dict(batch=4, heads=13107, group=5, tokens=4, max_new=1), dict(heads=13108))]


@pytest.mark.parametrize("sizes,more", LIMITS)
def test_attend_limits(sizes, more):
    need, said = attend_says(**sizes)
    assert need > 1 and said == ac.DEFRAG_EWORKSPACE
    assert attend_says(**{**sizes, **more}) == (0, ac.DEFRAG_EINVAL)


@pytest.mark.parametrize("cls,query", [(ac.defrag_kv_attend_args, ac.lib.defrag_kv_attend_workspace_bytes),
                                       (ac.defrag_kv_evict_args, ac.lib.defrag_kv_evict_workspace_bytes)])
def test_queries_refuse_the_counter_that_the_calls_refuse(cls, query):
    assert query(ctypes.byref(_args(cls, n_invalid_dev=0x1008))) > 0
    assert query(ctypes.byref(_args(cls, n_invalid_dev=0x1004))) == 0


def test_append_refuses_a_grid_of_two_to_the_32_lanes():
    """2^23 pages of 512 lanes each; one page fewer, or tokens for one page fewer, would fit."""
    a = _args(ac.defrag_kv_append_args, dim=256, page_stride=1 << 23, tokens=1 << 29, max_new=1 << 29, starts_dev=0x1000)
    assert ac.lib.defrag_kv_append(ctypes.byref(a), None) == ac.DEFRAG_EINVAL


@pytest.mark.parametrize("change", [
    dict(lens_out_dev=0x30000), dict(lens_out_dev=0x3000C), dict(lens_out_dev=0x40000),      # lens, next_pos
    dict(next_pos_dev=0x9000C), dict(lens_out_dev=0x20010), dict(lens_out_dev=0x50000),      # pages, weight
    dict(weight_out_dev=0x50004), dict(weight_out_dev=0x50000), dict(pos_out_dev=0x67FFC),   # shifted, another stride
    dict(pos_out_dev=0x70800), dict(weight_out_dev=0x60000, weight_out_stride=1024),
    dict(weight_out_dev=0x50000, weight_out_stride=1024, pos_out_dev=0x50000)])
def test_evict_refuses_outputs_over_inputs(change):
    a = _args(ac.defrag_kv_evict_args, **change)
    assert ac.lib.defrag_kv_evict_workspace_bytes(ctypes.byref(a)) == 0
    assert ac.lib.defrag_kv_evict(ctypes.byref(a), None, 0, None) == ac.DEFRAG_EINVAL


@pytest.mark.parametrize("change", [
    dict(weight_out_dev=0x50000, weight_out_stride=1024), dict(pos_out_dev=0x60000, weight_out_stride=1024),
    dict(lens_out_dev=0x30010), dict(weight_out_dev=0x58000), dict(next_pos_dev=0x30000)])
def test_evict_takes_planes_in_place_and_neighbours(change):
    a = _args(ac.defrag_kv_evict_args, **change)
    assert ac.lib.defrag_kv_evict_workspace_bytes(ctypes.byref(a)) > 1
    assert ac.lib.defrag_kv_evict(ctypes.byref(a), None, 0, None) == ac.DEFRAG_EWORKSPACE


@pytest.mark.parametrize("change", [
    dict(out_dev=0x40000), dict(out_dev=0x40FF0), dict(out_dev=0x3F810), dict(out_dev=0x40000, q_row=-512, q_dev=0x40C00),  # q
    dict(lse_dev=0x40010), dict(lse_dev=0x507F0), dict(lse_dev=0x30004), dict(out_dev=0x30000), dict(out_dev=0x20000),
    dict(lse_dev=0x10FC), dict(weight_dev=0x50000), dict(weight_dev=0x48000 - 4 * 4 * 2 * 1024 + 16, q_dev=0x48000),
    dict(starts_dev=0x50010)])
def test_attend_refuses_outputs_over_inputs(change):
    """q holds 4 x 8 x 64 numbers from 0x40000 on, out as many from 0x50000, the weights 4 x 2 x 1024 from 0x1000."""
    sizes = dict(group=4, weight_dev=0x1000, weight_stride=1024, **{k: v for k, v in change.items() if k != "weight_dev"})
    sizes["weight_dev"] = change.get("weight_dev", 0x1000)
    a = _args(ac.defrag_kv_attend_args, **sizes)
    assert ac.lib.defrag_kv_attend_workspace_bytes(ctypes.byref(a)) == 0
    assert ac.lib.defrag_kv_attend(ctypes.byref(a), None, 0, None) == ac.DEFRAG_EINVAL


@pytest.mark.parametrize("change", [
    dict(out_dev=0x41000), dict(out_dev=0x3F000), dict(lse_dev=0x51000), dict(lse_dev=0x50000 - 128),
    dict(out_dev=0x41000, q_row=-512, q_dev=0x40C00), dict(out_dev=0x40400, tokens=1, batch=1, max_new=1)])
def test_attend_takes_outputs_beside_inputs(change):
    a = _args(ac.defrag_kv_attend_args, **{**dict(group=4, weight_dev=0x1000, weight_stride=1024), **change})
    assert ac.lib.defrag_kv_attend_workspace_bytes(ctypes.byref(a)) > 1
    assert ac.lib.defrag_kv_attend(ctypes.byref(a), None, 0, None) == ac.DEFRAG_EWORKSPACE


def test_binding_refuses_numbers_that_do_not_fit():
    """ctypes cuts a number to its field: 2^32 + 1 heads would be one."""
    for heads, dim in (((1 << 32) + 1, 64), (1, (1 << 32) + 64), (-1, 64)):
        with pytest.raises(ac.DefragError):
            ac.defrag_kv_page_bytes(heads, dim)
    assert ac._kv_int(0xFFFFFFFF, "x") == 0xFFFFFFFF and ac._kv_int(-5, "x", -5, 5) == -5
    for bad in (-1, 1 << 32):
        with pytest.raises(ac.DefragError, match="x = "):
            ac._kv_int(bad, "x")
