"""Attention over caches of many parts and of many pages a part, sequences of
very different sizes in one call, and ranges of new tokens that are none.
Long caches repeat a few pages (pages that are only read may be shared)."""
import pytest
import torch

from kv_plain import PAGE, Cache, attend
from test_kv_gpu import HALF, check_attend, queries

pytestmark = pytest.mark.gpu
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


@pytest.fixture(scope="module")
def ac():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import arena_compaction_amd
    return arena_compaction_amd


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def repeated(heads, dim, codes, n, last=1.0, far=None):
    """n tokens over 7 pages in turn and a last one of its own, whose keys are `last` times larger; with `far` its
    values are 2^far times larger and 0 in the upper half of the dimensions."""
    pages = -(-n // PAGE)
    c = Cache([8], heads, dim, codes, fill=0x7F)
    c.fill_random([7 * PAGE], 111, spread=2)
    gen = torch.Generator().manual_seed(112)
    k, v = torch.randn(2, n - (pages - 1) * PAGE, heads, dim, generator=gen).unbind()
    if far is not None:
        v = v * 2.0 ** far
        v[..., dim // 2:] = 0.0
    c.append_page(0, 7, k * last, v)
    c.pages = torch.cat([c.pages[:, torch.arange(pages - 1) % 7], c.pages[:, 7:]], 1)
    return c


@pytest.mark.parametrize("group,dim,codes,dtype,count", [
    (2, 64, E4M3, torch.bfloat16, 1), (8, 128, INT8, torch.float16, 1), (1, 64, INT8, torch.float16, 7),
    (4, 96, E4M3, torch.bfloat16, 6), (3, 256, INT8, torch.bfloat16, 2), (20, 64, E4M3, torch.float16, 2)])
@pytest.mark.parametrize("last", [0.25, 3.0])
def test_attend_more_than_256_parts(ac, group, dim, codes, dtype, count, last):
    """One head: every four pages are a part, and a row's parts are read in two turns; the last part may hold the
    largest score, so that everything before it is scaled again."""
    n = 67 * 1024 + 5
    c = repeated(1, dim, codes, n, last)
    q = queries(count, group, dim, dtype, 113)
    assert check_attend(ac, c, [n], q, group, [count])[1] == 0


@pytest.mark.parametrize("group,dim,codes,dtype,count,weight,far", [
    (2, 64, E4M3, torch.bfloat16, 1, True, None), (3, 128, INT8, torch.float16, 4, False, None),
    (4, 64, INT8, torch.float16, 6, True, None), (1, 64, E4M3, torch.bfloat16, 40, True, None),
    (2, 64, E4M3, torch.bfloat16, 1, False, 40), (1, 64, INT8, torch.bfloat16, 40, False, 40)])
@pytest.mark.parametrize("pages", [260, 800])
def test_attend_256_pages_a_part(ac, pages, group, dim, codes, dtype, count, weight, far):
    """So many sequences that a long cache is cut in few pieces, at 256 pages the latest, the most that a wave's
    lanes hold (or, of many rows, not at all)."""
    B, heads, n = 260, 2, pages * PAGE + 17
    c = repeated(heads, dim, codes, n, 2.0, far)
    q = queries(count, heads * group, dim, dtype, 114)
    w = torch.zeros(B, heads, c.pages.shape[1] * PAGE, device="cuda") if weight else None
    lse = torch.empty(B * count, heads * group, device="cuda")
    out = ac.defrag_kv_attend(c.arena.cuda(), c.pages.repeat(B, 1).cuda(), ints([n] * B), q.repeat(B, 1, 1).cuda(), heads, codes,
                              starts=ints([count * b for b in range(B + 1)]), max_new=count, lse=lse, weight=w)
    for x in (out.unflatten(0, (B, count)), lse.unflatten(0, (B, count))) + ((w,) if weight else ()):
        assert torch.equal(x, x[:1].expand_as(x))
    want, bound, lse_, lbound, add, wbound = attend(c, [n], q, group, [count], dim ** -0.5)
    if far is not None:   # 2^8 lies between a band's scales: weights to 2^-30 instead of 2^-38
        v = torch.stack([c.numbers(0, n, h)[1].abs().sum(0) for h in range(heads)])
        bound = bound + v.repeat_interleave(group, 0) * 2.0 ** -30
    err = (out[:count].double().cpu() - want).abs()
    assert (err <= bound * (1 + HALF[dtype]) + want.abs() * HALF[dtype] + 2.0 ** -25).all()
    assert ((lse[:count].double().cpu() - lse_).abs() <= lbound + 2.0 ** -22).all()
    if weight:
        got = w[0].double().cpu()
        assert ((got[:, :n] - add[0]).abs() <= wbound[0] + add[0] * 2.0 ** -23).all() and not got[:, n:].any()


@pytest.mark.parametrize("heads,group,dim,codes,dtype", [
    (2, 4, 64, E4M3, torch.bfloat16), (1, 3, 128, INT8, torch.float16), (2, 2, 192, E4M3, torch.float16)])
@pytest.mark.parametrize("max_len", [None, 5001])
def test_attend_single_tokens_beside_a_prompt(ac, heads, group, dim, codes, dtype, max_len):
    """One call with a prompt, single tokens over long and short caches, a draft and sequences that bring nothing."""
    lens, counts = [300, 5001, 1, 64, 900, 200, 0, 2500], [300, 1, 1, 1, 0, 5, 0, 1]
    c = Cache([-(-n // PAGE) for n in lens], heads, dim, codes, fill=0x7F)
    c.fill_random(lens, 115, spread=2)
    q = queries(sum(counts), heads * group, dim, dtype, 116)
    assert check_attend(ac, c, lens, q, group, counts, max_len=max_len)[1] == 0


def test_attend_starts_that_are_none(ac):
    """A range that does not ascend inside the queries, or brings more than max_new, brings nothing: its sequence
    gives no weight, rows of no sequence are not written, and the other sequences are as they should be."""
    c = Cache([1, 1, 1], 1, 64, INT8)
    c.fill_random([9, 9, 9], 117)
    q = queries(4, 2, 64, torch.float16, 118)
    for starts, good in (([0, 1, 2, 9], [0, 1]), ([-1, 1, 2, 4], [1, 2]), ([0, 4, 4, 4], [1, 2]), ([3, 1, 2, 4], [1, 2]),
                         ([0, 1, 1, 4], [0, 1, 2]), ([1, 2, 3, 3], [0, 1, 2])):
        n = torch.zeros(1, dtype=torch.int64, device="cuda")
        out, w = torch.full((4, 2, 64), 5.0, dtype=torch.float16, device="cuda"), torch.zeros(3, 1, 64, device="cuda")
        lse = torch.full((4, 2), 5.0, device="cuda")
        ac.defrag_kv_attend(c.arena.cuda(), c.pages.cuda(), ints([9, 9, 9]), q.cuda(), 1, INT8, starts=ints(starts), max_new=3,
                            out=out, lse=lse, weight=w, n_invalid=n)
        assert int(n) == 3 - len(good), starts
        out, lse, w, written = out.cpu(), lse.cpu(), w.double().cpu(), torch.zeros(4, dtype=torch.bool)
        for b in range(3):
            lo, hi = starts[b], starts[b + 1]
            if b not in good:
                assert not w[b].any(), starts
                continue
            one = Cache.__new__(Cache)
            one.__dict__.update(c.__dict__)
            one.pages = c.pages[b: b + 1]
            want, bound, lse_, lbound, add, wbound = attend(one, [9], q[lo:hi], 2, [hi - lo], 64 ** -0.5)
            assert ((out[lo:hi].double() - want).abs() <= bound * 1.001 + want.abs() * 2.0 ** -11 + 2.0 ** -25).all(), starts
            assert ((lse[lo:hi].double() - lse_).abs() <= lbound + 2.0 ** -22).all(), starts
            assert ((w[b, 0, :9] - add[0, 0]).abs() <= wbound[0, 0] + add[0, 0] * 2.0 ** -23).all() and not w[b, 0, 9:].any(), starts
            written[lo:hi] = True
        assert (out[~written] == 5.0).all() and (lse[~written] == 5.0).all(), starts
