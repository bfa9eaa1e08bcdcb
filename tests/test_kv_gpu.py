"""The 8-bit key/value cache on the GPU against plain 64-bit arithmetic.

Codes, scales, positions and lengths are compared exactly; attention within
the bounds that kv_plain.attend derives, plus half a step of the output's
type (bf16 2^-8, fp16 2^-11 of the value)."""
import itertools
import math

import pytest
import torch

from kv_plain import PAGE, Cache, attend, evict

pytestmark = pytest.mark.gpu
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def ac():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import arena_compaction_amd
    return arena_compaction_amd


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts_of(counts):
    return ints([0] + list(itertools.accumulate(counts)))


def queries(n, heads, dim, dtype, seed, layout="packed"):
    gen = torch.Generator().manual_seed(seed)
    if layout == "packed":
        return torch.randn(n, heads, dim, generator=gen).to(dtype)
    if layout == "slice":       # of a fused projection
        return torch.randn(n, heads + 4, dim, generator=gen).to(dtype)[:, 2: 2 + heads]
    if layout == "heads first":
        return torch.randn(heads, n, dim, generator=gen).to(dtype).transpose(0, 1)
    wide = torch.randn(n, heads, dim + 3, generator=gen).to(dtype)  # rows that are not 16-byte aligned
    return wide[:, :, 1: 1 + dim]


def on_gpu(x):
    """The same strides on the GPU."""
    y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
    return y.copy_(x)


def check_attend(ac, c, lens, q, group, counts, scale=None, weight=True, lens_gpu=None, **kw):
    scale = c.D ** -0.5 if scale is None else scale
    want, bound, lse, lbound, add, wbound = attend(c, lens, q, group, counts, scale)
    qg = on_gpu(q) if not q.is_contiguous() else q.cuda()
    got_lse = torch.full((q.shape[0], q.shape[1]), 7.0, device="cuda")
    places = c.pages.shape[1] * PAGE + 3
    gen = torch.Generator().manual_seed(5)
    before = torch.rand(len(lens), c.H, places, generator=gen)
    w = before.cuda() if weight else None
    bad = torch.full((1,), 9, dtype=torch.int64, device="cuda")
    out = ac.defrag_kv_attend(c.arena.cuda(), c.pages.cuda(), ints(lens) if lens_gpu is None else lens_gpu, qg, c.H,
                              c.codes, starts=starts_of(counts), scale=scale, lse=got_lse, weight=w, n_invalid=bad, **kw)
    torch.cuda.synchronize()
    got = out.double().cpu()
    # a result outside the type's range is its infinity
    past = torch.isinf(got) & (want * got.sign() + bound >= torch.finfo(q.dtype).max)
    err = torch.where(past, 0.0, got - want).abs()
    tol = bound * (1 + HALF[q.dtype]) + want.abs() * HALF[q.dtype] + 2.0 ** -25
    assert (err <= tol).all(), f"out: {(err / tol).max()} of the bound"
    got = got_lse.double().cpu()
    assert torch.equal(torch.isinf(got), torch.isinf(lse))
    assert ((got - lse).abs().nan_to_num() <= lbound + 2.0 ** -22).all(), "lse"
    if weight:
        n = add.shape[2]
        after = w.double().cpu()
        exp = before.double()
        exp[:, :, :n] += add
        tol = torch.full_like(exp, 0.0)
        tol[:, :, :n] = wbound + exp[:, :, :n] * 2.0 ** -23
        assert ((after - exp).abs() <= tol).all(), "weight"
    return out, int(bad)


SHAPES = [  # heads, group, dim, codes, dtype
    (1, 1, 64, E4M3, torch.bfloat16), (2, 4, 64, INT8, torch.float16), (3, 3, 96, INT8, torch.bfloat16),
    (2, 7, 96, E4M3, torch.float16), (2, 16, 128, E4M3, torch.bfloat16), (1, 17, 128, INT8, torch.float16),
    (4, 2, 192, E4M3, torch.float16), (1, 8, 192, INT8, torch.bfloat16), (1, 6, 256, E4M3, torch.bfloat16),
    (2, 24, 256, INT8, torch.float16)]


@pytest.mark.parametrize("heads,group,dim,codes,dtype", SHAPES)
def test_attend_one_token(ac, heads, group, dim, codes, dtype):
    lens = [1, 63, 64, 65, 128, 129, 300, 2, 517]
    c = Cache([-(-n // PAGE) for n in lens], heads, dim, codes, fill=0x7F)
    c.fill_random(lens, 1, spread=6)
    q = queries(len(lens), heads * group, dim, dtype, 2, "slice")
    assert check_attend(ac, c, lens, q, group, [1] * len(lens))[1] == 0


@pytest.mark.parametrize("heads,group,dim,codes,dtype", SHAPES)
def test_attend_ragged_rows(ac, heads, group, dim, codes, dtype):
    lens, counts = [5, 200, 64, 130, 0, 77, 3], [5, 7, 0, 66, 0, 77, 1]
    c = Cache([-(-n // PAGE) for n in lens], heads, dim, codes, fill=0x7F)
    c.fill_random(lens, 3, spread=3)
    q = queries(sum(counts), heads * group, dim, dtype, 4, "heads first")
    assert check_attend(ac, c, lens, q, group, counts, max_new=77)[1] == 0


@pytest.mark.parametrize("dtype,codes", [(torch.bfloat16, E4M3), (torch.float16, INT8)])
@pytest.mark.parametrize("count", [1, 5, 40, 150])
def test_attend_split_cache(ac, dtype, codes, count):
    """A long cache, cut into pieces; pages whose scales lie far apart."""
    lens = [4999, 1]
    c = Cache([-(-n // PAGE) for n in lens], 2, 64, codes, fill=0x7F)
    c.fill_random(lens, 5, spread=20)
    q = queries(count + 1, 8, 64, dtype, 6, "unaligned")
    assert check_attend(ac, c, lens, q, 4, [count, 1])[1] == 0


@pytest.mark.parametrize("weight", [False, True])
def test_attend_many_rows(ac, weight):
    for past, count, group, dim, codes, dtype in ((0, 333, 4, 64, E4M3, torch.bfloat16), (190, 257, 2, 128, INT8, torch.float16),
                                                  (1000, 100, 3, 96, E4M3, torch.float16), (63, 130, 8, 256, INT8, torch.bfloat16),
                                                  (64, 97, 5, 192, E4M3, torch.bfloat16)):
        lens = [past + count, count, past + 1]
        c = Cache([-(-n // PAGE) for n in lens], 2, dim, codes, fill=0x7F)
        c.fill_random(lens, 7, spread=2)
        q = queries(2 * count + 1, 2 * group, dim, dtype, 8)
        assert check_attend(ac, c, lens, q, group, [count, count, 1], weight=weight)[1] == 0


@pytest.mark.parametrize("heads,group,dim,codes,dtype", SHAPES)
@pytest.mark.parametrize("count", [17, 18, 31, 33])
def test_attend_weights_of_part_tiles(ac, heads, group, dim, codes, dtype, count):
    """Rows that do not fill their last tile of 16, of the last sequence: no row behind them is there to be read."""
    lens, counts = [40, 65 + count], [3, count]
    c = Cache([-(-n // PAGE) for n in lens], heads, dim, codes, fill=0x7F)
    c.fill_random(lens, 41, spread=2)
    q = queries(sum(counts), heads * group, dim, dtype, 42)
    assert check_attend(ac, c, lens, q, group, counts, max_new=count)[1] == 0


@pytest.mark.parametrize("dim,codes,dtype", [(64, E4M3, torch.float16), (128, INT8, torch.bfloat16), (256, E4M3, torch.bfloat16)])
def test_attend_weights_in_pieces(ac, dim, codes, dtype):
    """Few heads and many rows: each page's weights are made in pieces of the rows, ends of which see nothing of it."""
    lens, counts = [700, 130, 0, 450], [611, 129, 0, 1]
    c = Cache([-(-n // PAGE) for n in lens], 1, dim, codes, fill=0x7F)
    c.fill_random(lens, 43, spread=2)
    q = queries(sum(counts), 7, dim, dtype, 44)
    assert check_attend(ac, c, lens, q, 7, counts, max_new=611)[1] == 0


def test_attend_large_scores(ac):
    """One token takes all the weight; others lie far below it."""
    for dtype, codes in ((torch.bfloat16, INT8), (torch.float16, E4M3)):
        c = Cache([6], 1, 128, codes)
        c.fill_random([350], 9, size=4.0)
        q = queries(9, 4, 128, dtype, 10) * 8
        check_attend(ac, c, [350], q, 4, [9], scale=1.0)
        check_attend(ac, c, [350], q, 4, [9], scale=-0.25)
        check_attend(ac, c, [350], q, 4, [9], scale=0.0)


def test_attend_rows_that_see_nothing(ac):
    """More new tokens than the cache holds: the first rows see no token."""
    lens, counts = [3, 0, 70], [5, 2, 72]
    c = Cache([1, 0, 2], 2, 64, E4M3, stride=2, fill=0x7F)
    c.fill_random(lens, 11)
    q = queries(sum(counts), 4, 64, torch.bfloat16, 12)
    out, bad = check_attend(ac, c, lens, q, 2, counts)
    assert bad == 0 and (out[:2] == 0).all() and (out[5:9] == 0).all()


def test_attend_later_tokens_without_numbers(ac):
    """NaN keys of tokens that a row may not see do not reach it; of the ones
    that see it, every output is NaN."""
    c = Cache([2], 1, 64, E4M3)
    c.fill_random([100], 13)
    k, _, _ = c.head(int(c.pages[0, 1]), 0)
    k.view(torch.uint8)[97 - 64] = 0x7F
    q = queries(8, 2, 64, torch.float16, 14).cuda()
    got = ac.defrag_kv_attend(c.arena.cuda(), c.pages.cuda(), ints([100]), q, 1, E4M3, starts=ints([0, 8])).cpu()
    k.view(torch.uint8)[97 - 64] = 0
    want = attend(c, [100], q.cpu(), 2, [8], 64 ** -0.5)[0]
    # token t sees places up to 92 + t: the first five do not see place 97
    assert ((got.double() - want)[:5].abs() <= want[:5].abs() * 2.0 ** -9 + 2.0 ** -9).all()
    assert torch.isnan(got[5:]).all()


def test_attend_later_values_without_numbers(ac):
    """The same for values: a NaN reaches its own dimension alone, in the rows
    that see its token."""
    for count, group in ((8, 2), (40, 3)):
        c = Cache([2], 1, 64, E4M3)
        c.fill_random([100], 13)
        _, v, _ = c.head(int(c.pages[0, 1]), 0)
        was = v.view(torch.uint8)[97 - 64, 7].item()
        v.view(torch.uint8)[97 - 64, 7] = 0x7F
        q = queries(count, group, 64, torch.float16, 14).cuda()
        got = ac.defrag_kv_attend(c.arena.cuda(), c.pages.cuda(), ints([100]), q, 1, E4M3, starts=ints([0, count])).cpu()
        v.view(torch.uint8)[97 - 64, 7] = was
        want = attend(c, [100], q.cpu(), group, [count], 64 ** -0.5)[0]
        nan = torch.zeros(want.shape, dtype=torch.bool)
        nan[97 - (100 - count):, :, 7] = True
        assert torch.equal(torch.isnan(got), nan)
        assert ((got.double() - want)[~nan].abs() <= want[~nan].abs() * 2.0 ** -9 + 2.0 ** -9).all()


def test_attend_bad_pages_and_lengths(ac):
    """Entries that are no page are passed over and counted; a length that is
    out of range counts as one, and its rows see nothing."""
    lens = [300, 70, 40, 129]
    c = Cache([5, 2, 1, 3], 2, 64, INT8, stride=5)
    c.fill_random(lens, 15)
    c.pages[0, 1] = -1
    c.pages[0, 4] += 8                       # off the 32-byte grid
    c.pages[1, 0] = c.arena.numel() - 64     # ends behind the arena
    c.pages[3, 2] = 1 << 62
    for counts in ([1, 1, 1, 1], [3, 30, 1, 20]):
        q = queries(sum(counts), 6, 64, torch.float16, 16)
        assert check_attend(ac, c, lens, q, 3, counts)[1] == 4
    seen = [300, 70, 0, 129]
    for n in (-3, 5 * PAGE + 1, 2 ** 31 - 1):
        counts = [1, 1, 1, 1]
        q = queries(4, 6, 64, torch.float16, 16)
        out, bad = check_attend(ac, c, seen, q, 3, counts, lens_gpu=ints([300, 70, n, 129]))
        assert bad == 5 and (out[2] == 0).all()


def test_attend_bad_starts(ac):
    """Ranges that do not ascend inside the queries bring nothing."""
    c = Cache([1, 1, 1], 1, 64, INT8)
    c.fill_random([9, 9, 9], 17)
    q = queries(4, 2, 64, torch.float16, 18).cuda()
    for starts, bad in (([0, 1, 2, 9], 1), ([-1, 1, 2, 4], 1), ([0, 3, 2, 4], 1), ([0, 4, 4, 4], 1)):
        n = torch.zeros(1, dtype=torch.int64, device="cuda")
        out = torch.full_like(q, 5.0)
        w = torch.zeros(3, 1, 64, device="cuda")
        ac.defrag_kv_attend(c.arena.cuda(), c.pages.cuda(), ints([9, 9, 9]), q, 1, INT8, starts=ints(starts), max_new=3,
                            out=out, weight=w, n_invalid=n)
        assert int(n) == bad, starts
        assert torch.isfinite(out).all() and torch.isfinite(w).all()


def test_attend_nothing(ac):
    c = Cache([1], 1, 64, E4M3)
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert ac.defrag_kv_attend(c.arena.cuda(), c.pages.cuda(), ints([5]), q, 1, E4M3, starts=ints([0, 0])).shape == q.shape
    assert ac.defrag_kv_attend(c.arena.cuda(), c.pages[:0].cuda(), none, q, 1, E4M3).shape == q.shape
    ac.defrag_kv_append(c.arena.cuda(), c.pages[:0].cuda(), none, q, q, E4M3)


def test_attend_repeats_bit_for_bit(ac):
    lens, counts = [700, 90, 2000], [3, 90, 1]
    c = Cache([-(-n // PAGE) for n in lens], 2, 128, E4M3)
    c.fill_random(lens, 19)
    q = queries(sum(counts), 8, 128, torch.bfloat16, 20).cuda()
    arena, pages, first = c.arena.cuda(), c.pages.cuda(), None
    for _ in range(3):
        w, lse = torch.zeros(3, 2, 2048, device="cuda"), torch.empty(sum(counts), 8, device="cuda")
        out = ac.defrag_kv_attend(arena, pages, ints(lens), q, 2, E4M3, starts=starts_of(counts), lse=lse, weight=w)
        now = [out.clone(), lse, w]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


# ---- append ---------------------------------------------------------------

def check_append(ac, c, lens, counts, k, v, layout=None, **kw):
    """The kernel's arena against the plain one, byte for byte but for what
    stands for the same number."""
    arena = c.arena.cuda()
    B, places = len(lens), c.pages.shape[1] * PAGE
    w = torch.full((B, c.H, places), 3.0, device="cuda")
    pos = torch.full((B, c.H, places), -9, dtype=torch.int32, device="cuda")
    first = [17 * b for b in range(B)]
    ac.defrag_kv_append(arena, c.pages.cuda(), ints(lens), k if k.is_cuda else on_gpu(k), v if v.is_cuda else on_gpu(v), c.codes,
                        starts=starts_of(counts), weight=w, pos=pos, first_pos=ints(first), **kw)
    at = 0
    for b, (n, t) in enumerate(zip(lens, counts)):
        c.append(b, n, k[at: at + t].cpu(), v[at: at + t].cpu())
        line = torch.arange(places)
        new = (line >= n) & (line < n + t)
        assert torch.equal(w[b].cpu(), torch.where(new, 0.0, 3.0).expand(c.H, -1))
        assert torch.equal(pos[b].cpu(), torch.where(new, first[b] + line - n, -9).int().expand(c.H, -1))
        at += t
    same(c, arena)


def same(c, arena):
    got = arena.cpu()
    diff = (got != c.arena).nonzero()[:, 0]
    if diff.numel():   # -0 and +0, or two NaNs
        x, y = got[diff].view(c.codes).float(), c.arena[diff].view(c.codes).float()
        assert ((x == y) | (torch.isnan(x) & torch.isnan(y))).all(), diff[:10]


@pytest.mark.parametrize("heads,group,dim,codes,dtype", SHAPES)
def test_append(ac, heads, group, dim, codes, dtype):
    lens, counts = [0, 1, 63, 64, 65, 130, 5, 60], [1, 1, 1, 1, 130, 66, 0, 8]
    c = Cache([-(-(n + t) // PAGE) for n, t in zip(lens, counts)], heads, dim, codes, fill=0x7F)
    c.fill_random(lens, 21)
    gen = torch.Generator().manual_seed(22)
    x = torch.randn(sum(counts), 2 * heads, dim, generator=gen) * torch.exp(torch.randn(sum(counts), 1, 1, generator=gen) * 2)
    x = x.to(dtype)
    check_append(ac, c, lens, counts, x[:, :heads], x[:, heads:])


def test_append_layouts(ac):
    for layout in ("packed", "slice", "heads first", "unaligned"):
        lens, counts = [10, 100], [40, 70]
        c = Cache([1, 3], 3, 96, INT8)
        c.fill_random(lens, 23)
        k, v = (queries(110, 3, 96, torch.float16, s, layout) for s in (24, 25))
        check_append(ac, c, lens, counts, k, v, max_new=70)


@pytest.mark.parametrize("codes", [E4M3, INT8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_odd_numbers(ac, codes, dtype):
    """Zeros, infinities, NaN, the least and the largest numbers of a type."""
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    rows = [[0.0] * 8, [math.inf, 1.0, -2.0, 0.1, 0, 0, 0, 0], [math.nan, 1.0, -math.inf, 3.0, 0, 0, 0, 0],
            [big, -big, 1.0, tiny, 0, 0, 0, 0], [tiny, -tiny, tiny / 4, 0, 0, 0, 0, 0], [math.inf] * 8,
            [448.0, 449.0, 127.0, 127.5, -448.0, 0.5, 1.5, 2.5]]
    for x in rows:
        x = torch.tensor(x * 8).to(dtype).expand(3, 1, 64).contiguous()
        for n in (0, 62):
            c = Cache([2], 1, 64, codes, seed=n)
            c.fill_random([n], 26, size=2.0 ** 5)
            check_append(ac, c, [n], [3], x, -x)


def test_append_refuses_bad_pages(ac):
    """Bad entries are counted; nothing outside the good pages changes."""
    c = Cache([2, 2, 2], 2, 64, INT8, stride=2)
    c.fill_random([60, 60, 60], 27)
    c.pages[1, 1] = c.arena.numel() - 32
    x = queries(30, 2, 64, torch.float16, 28)
    arena, n = c.arena.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda")
    # the second's tokens behind its bad page, and the third whole, are left out
    ac.defrag_kv_append(arena, c.pages.cuda(), ints([60, 60, 120]), x.cuda(), x.cuda(), INT8, starts=ints([0, 10, 20, 30]), n_invalid=n)
    assert int(n) == 2
    c.append(0, 60, x[:10], x[:10])
    c.append(1, 60, x[10:14], x[10:14])
    same(c, arena)
    for bad in ([0, 10, 5, 30], [0, 10, 20, 31], [-1, 0, 0, 0]):
        ac.defrag_kv_append(arena, c.pages.cuda(), ints([128, 128, 128]), x.cuda(), x.cuda(), INT8, starts=ints(bad), n_invalid=n)
        assert int(n) >= 1
    same(c, arena)


# ---- evict ----------------------------------------------------------------

def check_evict(ac, c, lens, budget, weight, pos, sink=0, recent=0, next_pos=None, **kw):
    arena, B = c.arena.cuda(), len(lens)
    places = budget + 5
    wo = torch.full((B, c.H, places), -3.0, device="cuda")
    po = torch.full((B, c.H, places), -9, dtype=torch.int32, device="cuda")
    lo = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    bad = torch.full((1,), 4, dtype=torch.int64, device="cuda")
    nxt = lens if next_pos is None else next_pos
    ac.defrag_kv_evict(arena, c.pages.cuda(), ints(lens), budget, weight.cuda(), pos.cuda(), wo, po, lo, c.D, c.codes,
                       sink=sink, recent=recent, next_pos=ints(nxt), n_invalid=bad, **kw)
    kw_, kp, kl = evict(c, lens, budget, weight, pos, sink, recent, nxt)
    assert lo.tolist() == kl and int(bad) == 0
    for b, h in kw_:
        n = kl[b]
        assert po[b, h, :n].tolist() == kp[b, h] and (po[b, h, n:] == -9).all()
        w = torch.tensor(kw_[b, h])
        assert torch.equal(wo[b, h, :n].cpu().nan_to_num(nan=7e7), w.nan_to_num(nan=7e7)) and (wo[b, h, n:] == -3).all()
    same(c, arena)


def plane(B, H, n, seed, zeros=0.2, ties=False):
    gen = torch.Generator().manual_seed(seed)
    w = torch.exp(2 * torch.randn(B, H, n, generator=gen))
    if ties:
        w = torch.randint(0, 3, (B, H, n), generator=gen).float()
    w = w * (torch.rand(B, H, n, generator=gen) >= zeros)
    pos = torch.rand(B, H, n, generator=gen).argsort(-1).int()
    return w, pos


@pytest.mark.parametrize("heads,group,dim,codes,dtype", SHAPES)
def test_evict(ac, heads, group, dim, codes, dtype):
    lens = [0, 1, 64, 127, 128, 129, 300, 200]
    c = Cache([-(-n // PAGE) for n in lens], heads, dim, codes, fill=0x7F)
    c.fill_random(lens, 31, spread=5)
    w, pos = plane(len(lens), heads, 300, 32)
    check_evict(ac, c, lens, 128, w, pos, sink=4, recent=20)


@pytest.mark.parametrize("codes", [E4M3, INT8])
@pytest.mark.parametrize("sink,recent", [(0, 0), (1, 0), (300, 0), (0, 1 << 30), (5, 150)])
def test_evict_ties_and_safe_tokens(ac, codes, sink, recent):
    """Equal weights go to the lowest place; more safe tokens than the budget."""
    lens = [320, 201, 193]
    c = Cache([5, 4, 4], 2, 64, codes)
    c.fill_random(lens, 33)
    for ties in (True, False):
        w, pos = plane(3, 2, 320, 34, ties=ties)
        check_evict(ac, c, lens, 192, w, pos, sink=sink, recent=recent)


def test_evict_odd_weights(ac):
    """NaN, infinities, both zeros, negative and tiny weights."""
    odd = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, -1.0, 1e-42, -1e-42, 1e38, 1.0])
    gen = torch.Generator().manual_seed(35)
    for budget in (64, 128, 192):
        c = Cache([4], 2, 64, INT8)
        c.fill_random([250], 36)
        w = odd[torch.randint(0, 10, (1, 2, 256), generator=gen)]
        check_evict(ac, c, [250], budget, w, plane(1, 2, 256, 37)[1], sink=2, recent=9)


def test_evict_long(ac):
    for n, budget in ((5000, 1024), (4097, 4096), (4160, 64)):
        c = Cache([-(-n // PAGE)], 1, 64, E4M3)
        c.fill_random([n], 38, spread=4)
        w, pos = plane(1, 1, n, 39)
        check_evict(ac, c, [n], budget, w, pos, sink=4, recent=32, next_pos=[n + 11])


@pytest.mark.parametrize("n,budget,ties", [(16385, 64, False), (20000, 8256, True), (40007, 30016, False),
                                           (70000, 192, True)])
def test_evict_longer_rows(ac, n, budget, ties):
    """Rows that several workgroups share, beside shorter ones."""
    lens = [n, 100, budget, min(n, budget + 1), n - 4321]
    c = Cache([-(-x // PAGE) for x in lens], 1, 64, INT8)
    gen = torch.Generator().manual_seed(44)
    for b in range(len(lens)):
        for j in range(-(-lens[b] // PAGE)):
            k, v, sc = c.head(int(c.pages[b, j]), 0)
            for x in (k, v):
                x.copy_(torch.randint(-127, 128, x.shape, generator=gen).to(torch.int8))
            sc.copy_(2.0 ** torch.randint(-3, 3, (2,), generator=gen))
    w, pos = plane(5, 1, n, 45, ties=ties)
    check_evict(ac, c, lens, budget, w, pos, sink=4, recent=32 if ties else budget * 3)


def test_evict_longer_rows_bad_pages(ac):
    n = 20000
    c = Cache([-(-n // PAGE), 1], 2, 64, INT8)
    c.fill_random([64, 60], 46)
    c.pages[0, 5], c.pages[0, 200] = -1, c.arena.numel()
    w, pos = plane(2, 2, n, 47)
    arena, bad = c.arena.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda")
    wo, po = torch.zeros(2, 2, 64, device="cuda"), torch.zeros(2, 2, 64, dtype=torch.int32, device="cuda")
    lo = torch.full((2,), 77, dtype=torch.int32, device="cuda")
    ac.defrag_kv_evict(arena, c.pages.cuda(), ints([n, 60]), 64, w.cuda(), pos.cuda(), wo, po, lo, 64, INT8, n_invalid=bad)
    assert int(bad) == 2 and lo.tolist() == [77, 60] and (wo[0] == 0).all() and torch.equal(wo[1, :, :60].cpu(), w[1, :, :60])
    same(c, arena)


def test_evict_leaves_bad_sequences_alone(ac):
    c = Cache([3, 3, 3], 2, 64, INT8, stride=3)
    c.fill_random([190, 190, 190], 41)
    c.pages[1, 2] = -1
    w, pos = plane(3, 2, 192, 42)
    arena, n = c.arena.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda")
    wo, po = torch.zeros(3, 2, 64, device="cuda"), torch.zeros(3, 2, 64, dtype=torch.int32, device="cuda")
    lo = torch.full((3,), 77, dtype=torch.int32, device="cuda")
    ac.defrag_kv_evict(arena, c.pages.cuda(), ints([193, 190, -1]), 64, w.cuda(), pos.cuda(), wo, po, lo, 64, INT8, n_invalid=n)
    assert int(n) == 3 and lo.tolist() == [77, 77, 77] and (wo == 0).all()
    same(c, arena)


# ---- together -------------------------------------------------------------

def test_other_stream_and_graph(ac):
    """append + attend + evict on a side stream and captured into a graph,
    replayed with eager work between: every replay equals the eager run."""
    H, G, D, B = 2, 4, 64, 3
    lens = [100, 63, 250]
    c = Cache([4, 4, 5], H, D, E4M3, stride=5)
    c.fill_random(lens, 51)
    x = queries(B, (G + 2) * H, D, torch.bfloat16, 52).cuda()
    q, k, v = x[:, : G * H], x[:, G * H: (G + 1) * H], x[:, (G + 1) * H:]
    base, pages, old = c.arena.cuda(), c.pages.cuda(), ints(lens)
    w0, pos0 = (t.cuda() for t in plane(B, H, 320, 53))
    arena, w, pos = base.clone(), w0.clone(), pos0.clone()
    wo, po, lo = torch.zeros(B, H, 128, device="cuda"), torch.zeros(B, H, 128, dtype=torch.int32, device="cuda"), ints([0] * B)
    out, bad, new = torch.empty_like(q), torch.zeros(1, dtype=torch.int64, device="cuda"), old + 1

    def reset():
        arena.copy_(base), w.copy_(w0), pos.copy_(pos0), wo.zero_(), po.zero_(), lo.zero_(), out.zero_()

    def step(stream=None):
        ac.defrag_kv_append(arena, pages, old, k, v, E4M3, weight=w, pos=pos, n_invalid=bad, stream=stream)
        ac.defrag_kv_attend(arena, pages, new, q, H, E4M3, out=out, weight=w, stream=stream)
        ac.defrag_kv_evict(arena, pages, new, 128, w, pos, wo, po, lo, D, E4M3, sink=2, recent=8, next_pos=new, stream=stream)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (arena, w, pos, wo, po, lo, out, bad)]

    reset()
    step()
    want = results()
    side = torch.cuda.Stream()
    reset()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    assert all(torch.equal(a, b) for a, b in zip(want, results()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        reset()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, results()))
        reset()
        step()
        assert all(torch.equal(a, b) for a, b in zip(want, results()))


def test_offsets_past_32_bits(ac):
    """Pages behind the first 4 GiB of the arena."""
    base = (1 << 32) + 4096
    c = Cache([3, 3], 2, 64, INT8, stride=3)
    c.fill_random([130, 140], 61)
    big = torch.empty(base + c.arena.numel(), dtype=torch.uint8, device="cuda")
    big[base:] = c.arena.cuda()
    pages = torch.where(c.pages >= 0, c.pages + base, c.pages).cuda()
    x = queries(2, 2, 64, torch.float16, 62)
    ac.defrag_kv_append(big, pages, ints([130, 140]), x.cuda(), x.cuda(), INT8)
    for b in range(2):
        c.append(b, [130, 140][b], x[b: b + 1], x[b: b + 1])
    same(c, big[base:])
    q = queries(2, 4, 64, torch.float16, 63)
    want, bound = attend(c, [131, 141], q, 2, [1, 1], 0.125)[:2]
    got = ac.defrag_kv_attend(big, pages, ints([131, 141]), q.cuda(), 2, INT8).double().cpu()
    assert ((got - want).abs() <= bound * 2 + want.abs() * 2.0 ** -11 + 2.0 ** -25).all()
    w, pos = plane(2, 2, 192, 64)
    wo, po, lo = torch.zeros(2, 2, 64, device="cuda"), torch.zeros(2, 2, 64, dtype=torch.int32, device="cuda"), ints([0, 0])
    ac.defrag_kv_evict(big, pages, ints([131, 141]), 64, w.cuda(), pos.cuda(), wo, po, lo, 64, INT8)
    evict(c, [131, 141], 64, w, pos, 0, 0, [131, 141])
    same(c, big[base:])


def test_example(ac):
    """The example: generation, eviction and compaction of one arena (it checks
    that attention over the moved pages gives the same bits)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "kv_cache.py")
    spec = importlib.util.spec_from_file_location("kv_cache_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    report = example.main(["--steps", "300", "--batch", "3", "--heads", "2", "--dim", "64", "--budget", "128",
                           "--slack", "64"])
    assert len(report) >= 2 and all(after == 0.0 for _, _, after in report)
    assert any(frag > 0.0 for _, frag, _ in report)
