"""The 8-bit key/value cache on the GPU at the ends of its ranges: scales far
apart, scores without numbers, grids past one axis, lengths past one part.

Codes, scales, positions and lengths are compared exactly; attention within
the bounds that kv_plain.attend derives, plus half a step of the output's type
(bf16 2^-8, fp16 2^-11 of the value)."""
import math

import math

import pytest
import torch

from kv_plain import PAGE, Cache, attend, evict
from test_kv_gpu import queries

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


def same_pages(c, arena):
    """Every head of every page: scales bit for bit, codes as the numbers they stand for."""
    got = Cache.__new__(Cache)
    got.__dict__.update(c.__dict__)
    got.arena = arena.cpu()
    for off in c.pages[c.pages >= 0].tolist():
        for h in range(c.H):
            for a, b, what in zip(got.head(off, h), c.head(off, h), ("keys", "values", "scales")):
                if what == "scales":
                    assert torch.equal(a.view(torch.int32), b.view(torch.int32)), (off, h, a, b)
                else:
                    a, b = a.float(), b.float()
                    assert ((a == b) | (torch.isnan(a) & torch.isnan(b))).all(), (off, h, what)


# ---- evict: a kept token of zeros beside dropped ones of another size ------

@pytest.mark.parametrize("codes", [E4M3, INT8])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("power", [64, 65, 75, 100, 126])
@pytest.mark.parametrize("beside", ["zeros", "small", "nan"])
def test_evict_zeros_of_a_large_scale(ac, codes, dim, power, beside):
    """Pages of numbers up to 2^power keep tokens of zeros alone: beside more
    zeros, numbers of 2^-60, or codes that are no number (which stay so)."""
    c = Cache([3], 2, dim, codes)
    gen = torch.Generator().manual_seed(power)
    weight = torch.zeros(1, 2, 192)
    for j in range(3):
        x = torch.randn(2, PAGE, 2, dim, generator=gen).clamp(-1.5, 1.5) * 2.0 ** power
        x[:, j::3] = 0.0       # a third of the tokens: the ones that stay
        weight[0, :, j * PAGE + j: (j + 1) * PAGE: 3] = 1.0
        if j == 2 and beside == "small":
            x = torch.randn(2, PAGE, 2, dim, generator=gen) * 2.0 ** -60
        c.append_page(0, j, x[0], x[1])
        if beside == "nan" and codes == E4M3:
            for h in range(2):
                k, v, _ = c.head(int(c.pages[0, j]), h)
                k.view(torch.uint8)[j + 3, 5] = 0x7F
                v.view(torch.uint8)[j + 3, 6] = 0xFF
    weight[:, :, 0] = 2.0
    pos = torch.arange(192, dtype=torch.int32).expand(1, 2, 192).contiguous()
    arena = c.arena.cuda()
    wo, po = torch.zeros(1, 2, 64, device="cuda"), torch.zeros(1, 2, 64, dtype=torch.int32, device="cuda")
    lo = ints([0])
    ac.defrag_kv_evict(arena, c.pages.cuda(), ints([192]), 64, weight.cuda(), pos.cuda(), wo, po, lo, dim, codes)
    kw, kp, _ = evict(c, [192], 64, weight, pos, 0, 0, [192])
    assert lo.tolist() == [64] and all(po[0, h].tolist() == kp[0, h] for h in range(2))
    if beside == "zeros":
        assert not c.head(int(c.pages[0, 0]), 0)[0].float().any()
    same_pages(c, arena)


# ---- attend: rows whose every score is -infinity ----------------------------

@pytest.mark.parametrize("heads,group,dim,codes,dtype,past,count", [
    (2, 1, 64, E4M3, torch.bfloat16, 60, 40),       # many rows, weights from the keys again
    (1, 4, 128, INT8, torch.float16, 700, 80),      # in pieces, the cache cut
    (1, 2, 256, E4M3, torch.float16, 3, 200),
    (2, 2, 64, INT8, torch.bfloat16, 300, 5),       # few rows, from the keys again
    (2, 2, 64, E4M3, torch.float16, 300, 2),        # from kept scores
    (1, 8, 192, E4M3, torch.bfloat16, 4990, 1)])    # from kept scores, the cache cut
def test_attend_rows_of_minus_infinity(ac, heads, group, dim, codes, dtype, past, count):
    """Their sums are empty: output 0, logarithm -infinity, and no weight for
    any token from them; the others are as they would be without them."""
    n = past + count
    c = Cache([-(-n // PAGE)], heads, dim, codes, fill=0x7F)
    c.fill_random([n], 71)
    for off in c.pages[0].tolist():
        for h in range(heads):
            c.head(off, h)[0].view(torch.uint8)[:, 0] = 0x30   # e4m3 0.5, int8 48: above 0
    gen = torch.Generator().manual_seed(72)
    q = torch.randn(count, heads * group, dim, generator=gen).to(dtype)
    none = torch.zeros(count, heads * group, dtype=torch.bool)
    none[::3, ::2] = True
    calm = torch.where(none[..., None], torch.zeros_like(q), q)
    q = calm.clone()
    q[..., 0] = torch.where(none, -math.inf, q[..., 0])
    out_, bound, lse_, lbound, _, wbound = attend(c, [n], calm, group, [count], dim ** -0.5)
    add = torch.zeros(heads, n, dtype=torch.float64)
    for h in range(heads):
        k = c.numbers(0, n, h)[0]
        for g in range(group):
            s = calm[:, h * group + g].double() @ k.t() * dim ** -0.5
            s = s.masked_fill(torch.arange(n)[None, :] > past + torch.arange(count)[:, None], -math.inf)
            add[h] += torch.softmax(s, -1)[~none[:, h * group + g]].sum(0)
    lse = torch.empty(count, heads * group, device="cuda")
    w = torch.full((1, heads, c.pages.shape[1] * PAGE + 3), 0.25, device="cuda")
    out = ac.defrag_kv_attend(c.arena.cuda(), c.pages.cuda(), ints([n]), q.cuda(), heads, codes, starts=ints([0, count]),
                              lse=lse, weight=w).double().cpu()
    lse, w = lse.double().cpu(), w[0].double().cpu()
    assert (out[none] == 0).all() and (lse[none] == -math.inf).all()
    assert ((out - out_).abs() <= bound * (1 + HALF[dtype]) + out_.abs() * HALF[dtype] + 2.0 ** -25)[~none].all()
    assert ((lse - lse_).abs() <= lbound + 2.0 ** -22)[~none].all()
    assert ((w[:, :n] - 0.25 - add).abs() <= wbound[0] + (add + 0.25) * 2.0 ** -23).all() and (w[:, n:] == 0.25).all()


# ---- attend: value scales far apart -----------------------------------------

def far_apart(heads, dim, codes, n, power, where):
    """Pages of large values that are 0 in the upper half of the dimensions, and pages of small ones."""
    pages = -(-n // PAGE)
    c = Cache([pages], heads, dim, codes, fill=0x7F)
    gen = torch.Generator().manual_seed(81)
    for j in range(pages):
        k, v = torch.randn(2, min(PAGE, n - j * PAGE), heads, dim, generator=gen).unbind()
        large = {"first": j == 0, "between": j % 3 == 1, "steps": j % 4 != 3, "waves": j // 4 % 3 == 0}[where]
        if large:
            v[..., dim // 2:] = 0.0
            v *= 2.0 ** (power if where != "steps" else power * (3 - j % 4) / 3)
        c.append_page(0, j, k, v)
    return c


def check_far_apart(c, out, lse, q, group, n):
    """A weight may be off by 2^-30 of the row's largest instead of kv_plain's
    2^-38: 2^8 lies between a band's scales."""
    count, dtype = q.shape[0], q.dtype
    want, bound, lse_, lbound, _, _ = attend(c, [n], q, group, [count], c.D ** -0.5)
    floor = torch.stack([c.numbers(0, n, h)[1].abs().sum(0) for h in range(c.H)]).repeat_interleave(group, 0) * 2.0 ** -30
    out, lse = out.double().cpu(), lse.double().cpu()
    past = torch.isinf(out) & (want * out.sign() + bound >= torch.finfo(dtype).max)
    err = torch.where(past, 0.0, out - want).abs()
    tol = (bound + floor) * (1 + HALF[dtype]) + want.abs() * HALF[dtype] + 2.0 ** -25
    assert (err <= tol).all(), f"{(err / tol).max()} of the bound"
    assert ((lse - lse_).abs() <= lbound + 2.0 ** -22).all()


@pytest.mark.parametrize("heads,group,dim,codes,dtype,n,count", [
    (1, 4, 64, INT8, torch.bfloat16, 400, 100), (1, 3, 128, E4M3, torch.float16, 400, 150),
    (1, 2, 64, E4M3, torch.bfloat16, 4300, 70), (1, 2, 192, INT8, torch.float16, 300, 40),
    (2, 2, 96, E4M3, torch.bfloat16, 300, 90), (1, 2, 256, E4M3, torch.bfloat16, 500, 60)])
@pytest.mark.parametrize("power", [12, 31, 50, 100])
@pytest.mark.parametrize("where", ["first", "between", "steps"])
def test_attend_value_scales_far_apart(ac, heads, group, dim, codes, dtype, n, count, power, where):
    """Where the large pages are 0 the small ones alone make the output, to its
    full accuracy wherever the large ones lie: many rows."""
    c = far_apart(heads, dim, codes, n, power, where)
    q = queries(count, heads * group, dim, dtype, 82)
    lse = torch.empty(count, heads * group, device="cuda")
    out = ac.defrag_kv_attend(c.arena.cuda(), c.pages.cuda(), ints([n]), q.cuda(), heads, codes, starts=ints([0, count]), lse=lse)
    check_far_apart(c, out, lse, q, group, n)


@pytest.mark.parametrize("heads,group,dim,codes,dtype,count", [
    (2, 2, 64, E4M3, torch.bfloat16, 1), (1, 4, 128, INT8, torch.float16, 5), (2, 8, 96, E4M3, torch.float16, 4),
    (1, 4, 192, INT8, torch.bfloat16, 2), (1, 4, 256, E4M3, torch.float16, 3)])
@pytest.mark.parametrize("power", [12, 31, 50, 100])
@pytest.mark.parametrize("where", ["first", "waves", "steps"])
def test_attend_value_scales_far_apart_few_rows(ac, heads, group, dim, codes, dtype, count, power, where):
    """The same for few rows, of so many sequences (over the same pages) that a wave has several pages."""
    n, B = 1500, 520 // heads
    c = far_apart(heads, dim, codes, n, power, where)
    q = queries(count, heads * group, dim, dtype, 83)
    lse = torch.empty(B * count, heads * group, device="cuda")
    out = ac.defrag_kv_attend(c.arena.cuda(), c.pages.repeat(B, 1).cuda(), ints([n] * B), q.repeat(B, 1, 1).cuda(), heads, codes,
                              starts=ints([count * b for b in range(B + 1)]), max_new=count, lse=lse)
    assert torch.equal(out.unflatten(0, (B, count)), out[:count].expand(B, -1, -1, -1))
    check_far_apart(c, out[:count], lse[:count], q, group, n)


# ---- attend: grids past one axis --------------------------------------------

def few_seen(ac, c, n, q, group, counts, places, weight, max_new):
    """Attention of sequences that all hold the same n tokens and bring `counts` new ones, most of which see
    nothing; checks the rows that see something, and that the others are empty."""
    B, heads, dim = len(counts), c.H, c.D
    w = torch.full((B, heads, places), 0.5, device="cuda") if weight else None
    lse = torch.empty(q.shape[:2], device="cuda")
    starts = [0]
    for t in counts:
        starts.append(starts[-1] + t)
    stride = -(-places // PAGE) if weight else c.pages.shape[1]
    pages = torch.full((B, stride), -1, dtype=torch.int64)
    pages[:, : c.pages.shape[1]] = c.pages
    out = ac.defrag_kv_attend(c.arena.cuda(), pages.cuda(), ints([n] * B), q, heads, c.codes, starts=ints(starts),
                              max_new=max_new, max_len=places if weight else None, lse=lse, weight=w)
    for b in sorted({0, B // 2, B - 1}):
        see = min(n, counts[b])
        rows = slice(starts[b + 1] - see, starts[b + 1])
        want, bound, lse_, lbound, add, wbound = attend(c, [n], q[rows].cpu(), group, [see], dim ** -0.5)
        got = out[rows].double().cpu()
        assert ((got - want).abs() <= bound * (1 + HALF[q.dtype]) + want.abs() * HALF[q.dtype] + 2.0 ** -25).all(), b
        assert ((lse[rows].double().cpu() - lse_).abs() <= lbound + 2.0 ** -22).all(), b
        if weight:
            got = w[b].double().cpu()
            assert ((got[:, :n] - 0.5 - add[0]).abs() <= wbound[0] + (add[0] + 0.5) * 2.0 ** -23).all(), b
            assert (got[:, n:] == 0.5).all(), b
        blind = slice(starts[b], starts[b + 1] - see)
        assert not out[blind].any() and (lse[blind] == -math.inf).all(), b


@pytest.mark.parametrize("weight", [False, True])
def test_attend_long_prompt_of_many_heads(ac, weight):
    """131,072 tokens of 128 query heads: 2^24 rows of a call, 2^21 of a head."""
    c = Cache([2], 8, 64, INT8)
    c.fill_random([100], 91)
    gen = torch.Generator(device="cuda").manual_seed(92)
    q = torch.randn(131072, 128, 64, device="cuda", generator=gen, dtype=torch.bfloat16)
    few_seen(ac, c, 100, q, 16, [131072], 128, weight, 131072)


@pytest.mark.parametrize("dim,codes", [(64, E4M3), (192, INT8)])
def test_attend_prompts_past_one_grid_axis(ac, dim, codes):
    """64 prompts, max_new left at all their tokens: 2,098,176 workgroups, more than one row of the grid."""
    c = Cache([2], 8, dim, codes, fill=0x7F)
    c.fill_random([70], 93)
    counts = [4097 + (b % 2) for b in range(64)]
    gen = torch.Generator(device="cuda").manual_seed(94)
    q = torch.randn(sum(counts), 16, dim, device="cuda", generator=gen, dtype=torch.float16)
    assert -(-sum(counts) * 2 // 128) * 8 * 64 > 1 << 21
    few_seen(ac, c, 70, q, 2, counts, 128, False, None)


@pytest.mark.parametrize("dim,codes", [(64, E4M3), (128, INT8)])
def test_attend_weights_past_one_grid_axis(ac, dim, codes):
    """64 x 32 x 1026 workgroups over the pages of a table for 65,664 tokens."""
    c = Cache([2], 32, dim, codes, fill=0x7F)
    c.fill_random([70], 95)
    gen = torch.Generator(device="cuda").manual_seed(96)
    counts = [8 - b % 3 for b in range(64)]
    q = torch.randn(sum(counts), 128, dim, device="cuda", generator=gen, dtype=torch.bfloat16)
    few_seen(ac, c, 70, q, 4, counts, 1026 * PAGE, True, 8)


# ---- append -------------------------------------------------------------------

@pytest.mark.parametrize("stride", [0, 1, 2])
def test_append_to_tables_of_few_pages(ac, stride):
    """More new tokens than a row of the table holds: refused and counted, the others written."""
    c = Cache([stride], 2, 64, INT8, stride=max(stride, 1))
    pages = c.pages[:, :stride].repeat(2, 1)
    x = queries(64 * stride + 200, 2, 64, torch.float16, 97)
    arena, n = c.arena.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda")
    count = 64 * stride
    ac.defrag_kv_append(arena, pages.cuda(), ints([0, 0]), x.cuda(), x.cuda(), INT8, starts=ints([0, count, count + 200]), n_invalid=n)
    assert int(n) == 1
    c.append(0, 0, x[:count], x[:count])
    same_pages(c, arena)


# ---- evict: weights and positions in place ------------------------------------

@pytest.mark.parametrize("n", [300, 17000])
def test_evict_in_place(ac, n):
    """Weights and positions replaced where they are equal those written elsewhere; lengths may not be."""
    lens = [n, 100, 128, n - 77]
    gen = torch.Generator().manual_seed(98)
    c = Cache([-(-x // PAGE) for x in lens], 2, 64, INT8)
    for off in c.pages[c.pages >= 0].tolist():
        for h in range(2):
            k, v, sc = c.head(off, h)
            for x in (k, v):
                x.copy_(torch.randint(-127, 128, x.shape, generator=gen).to(torch.int8))
            sc.copy_(2.0 ** torch.randint(-3, 3, (2,), generator=gen))
    w = torch.rand(4, 2, n + 3, generator=gen).cuda()
    pos = torch.rand(4, 2, n + 3, generator=gen).argsort(-1).int().cuda()
    kw = dict(sink=4, recent=32)
    results = []
    for in_place in (False, True):
        arena, wi, pi = c.arena.cuda(), w.clone(), pos.clone()
        wo, po = (wi, pi) if in_place else (torch.zeros_like(wi), torch.zeros_like(pi))
        lo, held = ints([-1] * 4), ints(lens)
        ac.defrag_kv_evict(arena, c.pages.cuda(), held, 128, wi, pi, wo, po, lo, 64, INT8, **kw)
        results.append([arena, lo, wo[:, :, :100], po[:, :, :100], wo[0, :, :128], po[0, :, :128], wo[3, :, :128], po[3, :, :128]])
        with pytest.raises(ac.DefragError):
            ac.defrag_kv_evict(arena, c.pages.cuda(), held, 128, wi, pi, wo, po, held, 64, INT8, **kw)
    assert results[0][1].tolist() == [128, 100, 128, 128]
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_numbers_past_their_fields(ac):
    """What ctypes would cut to 32 bits is refused: max_len 2^32 would make every sequence one that holds nothing."""
    c = Cache([2], 1, 64, INT8)
    c.fill_random([100], 99)
    q = queries(1, 2, 64, torch.float16, 100).cuda()
    arena, pages, lens = c.arena.cuda(), c.pages.cuda(), ints([100])
    w, pos = torch.zeros(1, 1, 128, device="cuda"), torch.zeros(1, 1, 128, dtype=torch.int32, device="cuda")
    wo, po, lo = torch.zeros_like(w), torch.zeros_like(pos), ints([0])
    for bad in (1 << 32, -1):
        with pytest.raises(ac.DefragError, match="max_len = "):
            ac.defrag_kv_attend(arena, pages, lens, q, 1, INT8, max_len=bad)
    with pytest.raises(ac.DefragError, match="max_new = "):
        ac.defrag_kv_attend(arena, pages, lens, q, 1, INT8, starts=ints([0, 1]), max_new=-1)
    for what, bad in (("budget", (1 << 32) + 64), ("max_len", 1 << 32), ("sink", 1 << 31), ("recent", 1 << 32)):
        kw = {"budget": 64, what: bad}
        with pytest.raises(ac.DefragError, match=what + " = "):
            ac.defrag_kv_evict(arena, pages, lens, kw.pop("budget"), w, pos, wo, po, lo, 64, INT8, **kw)


def test_entries_that_no_call_reads_are_not_counted(ac):
    """A bad entry counts where its page would be read: behind the last token, of a sequence that brings nothing,
    or of one that evict leaves as it is, it does not."""
    c = Cache([3, 3], 1, 64, INT8)
    c.fill_random([100, 100], 101)
    c.pages[0, 2] = -1                  # behind the tokens
    c.pages[1, 0] = 7                   # a sequence of no new tokens, within its budget
    arena, pages, lens, n = c.arena.cuda(), c.pages.cuda(), ints([100, 100]), torch.full((1,), 5, dtype=torch.int64, device="cuda")
    x = queries(3, 1, 64, torch.float16, 102).cuda()
    ac.defrag_kv_append(arena, pages, ints([97, 100]), x, x, INT8, starts=ints([0, 3, 3]), n_invalid=n)
    assert int(n) == 0
    w, pos = torch.rand(2, 1, 192, device="cuda"), torch.arange(192, dtype=torch.int32, device="cuda").expand(2, 1, 192).contiguous()
    before = w.clone()
    ac.defrag_kv_attend(arena, pages, lens, x, 1, INT8, starts=ints([0, 3, 3]), weight=w, n_invalid=n)
    assert int(n) == 0 and torch.equal(w[1], before[1])
    wo, po, lo = torch.zeros(2, 1, 128, device="cuda"), torch.zeros(2, 1, 128, dtype=torch.int32, device="cuda"), ints([0, 0])
    ac.defrag_kv_evict(arena, pages, lens, 128, w, pos, wo, po, lo, 64, INT8, n_invalid=n)
    assert int(n) == 0 and lo.tolist() == [100, 100] and torch.equal(wo[:, :, :100], w[:, :, :100])
    ac.defrag_kv_evict(arena, pages, lens, 64, w, pos, wo, po, lo, 64, INT8, n_invalid=n)
    assert int(n) == 1 and lo.tolist() == [64, 100]
    ac.defrag_kv_attend(arena, pages, lens, x, 1, INT8, starts=ints([0, 1, 3]), n_invalid=n)
    assert int(n) == 1
