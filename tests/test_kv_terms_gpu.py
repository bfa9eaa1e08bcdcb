"""Attention with terms over the 8-bit cache against plain 64-bit arithmetic,
within the bounds that kv_more_plain.attend derives, plus half a step of the
output's type (bf16 2^-8, fp16 2^-11 of the value)."""
import math

import pytest
import torch

from kv_more_plain import PAGE, Cache, attend, tree, words_of
from test_kv_gpu import HALF, ints, on_gpu, queries, starts_of

pytestmark = pytest.mark.gpu
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ac():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import arena_compaction_amd
    return arena_compaction_amd


def masks(counts, kind, seed):
    """Truth values [count, count] by sequence."""
    gen = torch.Generator().manual_seed(seed)
    out = []
    for t in counts:
        line = torch.arange(t)
        if kind == "tree":
            out.append(tree(t, 3, gen)[1])
        elif kind == "documents":
            of = (line * 3 // max(1, t)) if t else line
            out.append((of[:, None] == of[None, :]) & (line[None, :] <= line[:, None]))
        elif kind == "random":           # any order, rows that see nothing of the new tokens
            out.append(torch.rand(t, t, generator=gen) < 0.3)
        else:
            out.append((line[None, :] <= line[:, None]) | (line[None, :] < t // 2))
    return out


def pack(seen, counts, words, n):
    out = torch.full((n, words), -1, dtype=torch.int64)   # tokens of no sequence, and bits of no token: set
    at = 0
    for s, t in zip(seen, counts):
        w = words_of(s, words) if t else torch.zeros(0, words, dtype=torch.int64)
        junk = words_of(torch.cat([torch.zeros(t, t, dtype=torch.bool), torch.ones(t, words * 64 - t, dtype=torch.bool)], 1), words) \
            if t else w
        out[at: at + t] = w | junk
        at += t
    return out


def planes(lens, counts, heads, places, seed):
    """Positions as evictions leave them: gaps, other ones for each head, out of order at first; depths at the end."""
    gen = torch.Generator().manual_seed(seed)
    pos = torch.full((len(lens), heads, places), 1 << 30, dtype=torch.int32)
    for b, n in enumerate(lens):
        for h in range(heads):
            p = torch.randperm(2 * n + 1, generator=gen)[:n].sort()[0]
            half = n // 2
            p[:half] = p[torch.randperm(half, generator=gen)]
            pos[b, h, :n] = p.to(torch.int32)
    return pos


def check(ac, c, lens, q, group, counts, kind=None, cap=0.0, slopes=None, pos=None, weight=True, words=None, seed=1, **kw):
    scale = 2.0 * c.D ** -0.5
    mask = masks(counts, kind, seed) if kind else None
    want, bound, lse, lbound, add, wbound = attend(c, lens, q, group, counts, scale, mask, cap, slopes, pos)
    got_lse = torch.full((q.shape[0], q.shape[1]), 7.0, device="cuda")
    places = c.pages.shape[1] * PAGE + 3
    gen = torch.Generator().manual_seed(5)
    before = torch.rand(len(lens), c.H, places, generator=gen)
    w = before.cuda() if weight else None
    words = words or -(-max(counts + [1]) // 64)
    bad = torch.full((1,), 9, dtype=torch.int64, device="cuda")
    out = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
    ac.defrag_kv_attend_terms(c.arena.cuda(), c.pages.cuda(), ints(lens),
                              on_gpu(q) if not q.is_contiguous() else q.cuda(), c.H, c.codes,
                              mask=pack(mask, counts, words, q.shape[0]).cuda() if kind else None, cap=cap or None,
                              slopes=None if slopes is None else slopes.cuda(), pos=None if pos is None else pos.cuda(),
                              starts=starts_of(counts), max_new=max(counts), scale=scale, out=out, lse=got_lse, weight=w,
                              n_invalid=bad, **kw)
    torch.cuda.synchronize()
    n = sum(counts)
    got = out.double().cpu()
    assert (got[n:] == 3.0).all() and (got_lse[n:] == 7.0).all()     # rows behind the last sequence
    got, want, bound = got[:n], want[:n], bound[:n]
    tol = bound * (1 + HALF[q.dtype]) + want.abs() * HALF[q.dtype] + 2.0 ** -25
    # a result outside the type's range is its infinity (fp16: pages scaled by 2^20 give some above 65504)
    past = torch.isinf(got) & (want * got.sign() + bound >= torch.finfo(q.dtype).max)
    err = torch.where(past, 0.0, got - want).abs()
    assert (err <= tol).all(), f"out: {(err / tol).max()} of the bound"
    got, lse, lbound = got_lse.double().cpu()[:n], lse[:n], lbound[:n]
    assert torch.equal(torch.isinf(got), torch.isinf(lse))
    assert ((got - lse).abs().nan_to_num() <= lbound + 2.0 ** -22).all(), "lse"
    if weight:
        m = add.shape[2]
        after, exp = w.double().cpu(), before.double()
        exp[:, :, :m] += add
        tol = torch.zeros_like(exp)
        tol[:, :, :m] = wbound + exp[:, :, :m] * 2.0 ** -23
        assert ((after - exp).abs() <= tol).all(), "weight"
    return out, int(bad)


def slopes_of(heads):
    return torch.exp2(-8.0 * (torch.arange(heads) + 1) / heads).float()


SHAPES = [  # heads, group, dim, codes, dtype
    (1, 1, 64, E4M3, BF16), (2, 4, 64, INT8, FP16), (3, 3, 96, INT8, BF16), (2, 7, 96, E4M3, FP16), (2, 16, 128, E4M3, BF16),
    (1, 17, 128, INT8, FP16), (4, 2, 192, E4M3, FP16), (1, 8, 192, INT8, BF16), (1, 6, 256, E4M3, BF16), (2, 24, 256, INT8, FP16)]
TERMS = [("tree", 0.0, False, False), ("random", 0.0, False, False), (None, 4.0, False, False), (None, 0.0, True, False),
         (None, 30.0, True, True), ("prefix", 1.5, True, True), ("documents", 0.0, True, False)]


@pytest.mark.parametrize("kind,cap,bias,plane", TERMS)
@pytest.mark.parametrize("heads,group,dim,codes,dtype", SHAPES)
def test_few_rows(ac, heads, group, dim, codes, dtype, kind, cap, bias, plane):
    """One and a few new tokens, at the ends of pages; weights from kept scores and from scores made again."""
    for counts in ([1] * 7, [3, 1, 2, 0, 5, 4, 1]):
        lens = [a + t for a, t in zip([0, 62, 63, 64, 126, 300, 517], counts)]
        c = Cache([-(-n // PAGE) for n in lens], heads, dim, codes, fill=0x7F)
        c.fill_random(lens, 1, spread=6)
        q = queries(sum(counts) + 2, heads * group, dim, dtype, 2, "slice")
        pos = planes(lens, counts, heads, c.pages.shape[1] * PAGE, 3) if plane else None
        assert check(ac, c, lens, q, group, counts, kind, cap, slopes_of(heads * group) if bias else None, pos)[1] == 0


@pytest.mark.parametrize("kind,cap,bias,plane", TERMS)
@pytest.mark.parametrize("heads,group,dim,codes,dtype", SHAPES)
def test_many_rows(ac, heads, group, dim, codes, dtype, kind, cap, bias, plane):
    lens, counts = [5, 200, 64, 130, 0, 77, 3], [5, 37, 0, 66, 0, 77, 1]
    c = Cache([-(-n // PAGE) for n in lens], heads, dim, codes, fill=0x7F)
    c.fill_random(lens, 3, spread=3)
    q = queries(sum(counts), heads * group, dim, dtype, 4, "heads first")
    pos = planes(lens, counts, heads, c.pages.shape[1] * PAGE, 3) if plane else None
    assert check(ac, c, lens, q, group, counts, kind, cap, slopes_of(heads * group) if bias else None, pos, words=3)[1] == 0


@pytest.mark.parametrize("dtype,codes", [(BF16, E4M3), (FP16, INT8)])
@pytest.mark.parametrize("count", [1, 5, 40, 150])
@pytest.mark.parametrize("kind,cap,bias", [("tree", 0.0, False), ("prefix", 20.0, True)])
def test_split_cache(ac, dtype, codes, count, kind, cap, bias):
    """A long cache, cut into pieces; pages whose scales lie far apart."""
    lens, counts = [4999, 1], [count, 1]
    c = Cache([-(-n // PAGE) for n in lens], 2, 64, codes, fill=0x7F)
    c.fill_random(lens, 5, spread=20)
    q = queries(count + 1, 8, 64, dtype, 6, "unaligned")
    pos = planes(lens, counts, 2, c.pages.shape[1] * PAGE, 7) if bias else None
    assert check(ac, c, lens, q, 4, counts, kind, cap, slopes_of(8) if bias else None, pos)[1] == 0


@pytest.mark.parametrize("had", [0, 1, 15, 48, 63, 64, 100])
@pytest.mark.parametrize("group,count", [(1, 200), (2, 9), (1, 70), (4, 130)])
def test_masks_across_words_and_pages(ac, had, group, count):
    """Bits that cross 64-bit words, at every place in a page; more words than are needed, with bits of no token set."""
    lens, counts = [had + count, had + 3], [count, 3]
    c = Cache([-(-n // PAGE) for n in lens], 1, 64, E4M3, fill=0x7F)
    c.fill_random(lens, 8)
    q = queries(count + 3, group, 64, BF16, 9)
    for words in (-(-count // 64), 5):
        assert check(ac, c, lens, q, group, counts, "random", words=words, seed=had + words)[1] == 0


@pytest.mark.parametrize("dim,codes,dtype", [(64, E4M3, BF16), (64, INT8, FP16), (96, INT8, BF16), (96, E4M3, FP16), (128, E4M3, BF16),
                                             (128, INT8, FP16), (192, E4M3, BF16)])
@pytest.mark.parametrize("group,count", [(4, 16), (8, 5), (1, 64), (3, 11), (2, 33)])
def test_small_trees(ac, group, count, dim, codes, dtype):
    """33 to 66 rows a head; prefixes that are cut into pieces, and a sequence of its drafts alone."""
    counts = [count, count, max(1, count - 3)]
    lens = [2000 + count, count, 61 + counts[2]]
    c = Cache([-(-n // PAGE) for n in lens], 2, dim, codes, fill=0x7F)
    c.fill_random(lens, 6, spread=9)
    c.pages[0, 3] = -1
    q = queries(sum(counts) + 1, 2 * group, dim, dtype, 9, "slice")
    for kind in ("tree", "random"):
        assert check(ac, c, lens, q, group, counts, kind, seed=count)[1] == 1


@pytest.mark.parametrize("count,group", [(6, 2), (50, 3)])
@pytest.mark.parametrize("bias", [False, True])
def test_rows_that_see_nothing(ac, count, group, bias):
    c = Cache([2], 2, 64, E4M3, fill=0x7F)
    c.fill_random([count], 1)
    q = queries(count, 2 * group, 64, FP16, 2)
    mask = torch.eye(count, dtype=torch.bool)
    mask[1] = mask[count - 1] = False
    lse = torch.zeros(count, 2 * group, device="cuda")
    weight = torch.zeros(1, 2, 128, device="cuda")
    out = ac.defrag_kv_attend_terms(c.arena.cuda(), c.pages.cuda(), ints([count]), q.cuda(), 2, E4M3, mask=words_of(mask).cuda(),
                                    slopes=slopes_of(2 * group).cuda() if bias else None, starts=starts_of([count]), max_new=count,
                                    lse=lse, weight=weight)
    for r in (1, count - 1):
        assert (out[r] == 0).all() and (lse[r] == -math.inf).all()
    seen = torch.tensor([i for i in range(count) if i not in (1, count - 1)])
    assert (weight.cpu()[0, :, seen] - group).abs().max() <= group * 2.0 ** -20      # each sees itself alone
    assert (weight.cpu()[0, :, [1, count - 1]] == 0).all() and (weight.cpu()[0, :, count:] == 0).all()
    v = torch.stack([c.numbers(0, count, h)[1] for h in (0, 1)], 1)                  # [tokens, heads, D]
    want = v.repeat_interleave(group, 1)[seen]
    assert ((out.cpu().double()[seen] - want).abs() <= want.abs() * (2.0 ** -11 + 2.0 ** -20) + 2.0 ** -25).all()


@pytest.mark.parametrize("count,group", [(1, 2), (9, 3), (60, 2)])
def test_what_is_hidden_does_not_count(ac, count, group):
    """NaN in keys, values and positions of hidden tokens reaches no row; of seen ones the rows that see it."""
    had, heads, dim = 70, 2, 64
    n = had + count + 3
    lens, counts = [n], [count + 3]
    c = Cache([-(-n // PAGE)], heads, dim, E4M3, fill=0x7F)
    c.fill_random(lens, 1)
    mask = torch.eye(count + 3, dtype=torch.bool)
    mask[:, 0] = True
    mask[1, 2] = True
    spoiled = had + 2                                        # seen by rows 1 and 2
    kc, vc, _ = c.head(int(c.pages[0, spoiled // PAGE]), 1)
    raw = vc.view(torch.uint8) if vc.is_contiguous() else None
    assert raw is None
    at = int(c.pages[0, spoiled // PAGE]) + 2 * PAGE * dim   # head 1's strip
    c.arena[at + spoiled % PAGE * dim + 5] = 0x7F            # a key
    c.arena[at + PAGE * dim + 7 * PAGE + spoiled % PAGE] = 0xFF
    q = queries(count + 3, heads * group, dim, BF16, 2)
    out = ac.defrag_kv_attend_terms(c.arena.cuda(), c.pages.cuda(), ints(lens), q.cuda(), heads, E4M3, mask=words_of(mask).cuda(),
                                    cap=20.0, slopes=slopes_of(heads * group).cuda(), starts=starts_of(counts),
                                    max_new=count + 3).cpu()
    nan = torch.isnan(out).any(-1)
    assert not nan[:, :group].any() and nan[1:3, group:].all() and not nan[3:, group:].any() and not nan[0].any()
    c.arena[at + spoiled % PAGE * dim + 5] = 0               # the value alone: one dimension
    for cap in (None, 20.0):
        out = ac.defrag_kv_attend_terms(c.arena.cuda(), c.pages.cuda(), ints(lens), q.cuda(), heads, E4M3,
                                        mask=words_of(mask).cuda(), cap=cap, starts=starts_of(counts), max_new=count + 3).cpu()
        nan = torch.isnan(out)
        assert nan[1:3, group:, 7].all() and int(nan.sum()) == 2 * group


def test_no_terms_is_attend(ac):
    """Without terms, with a mask that is causal, and with a cap far above the scores: attend's own results."""
    lens, counts = [200, 90, 64], [9, 1, 64]
    c = Cache([4, 2, 1], 2, 128, E4M3, fill=0x7F)
    c.fill_random(lens, 1)
    q = queries(sum(counts), 8, 128, BF16, 2).cuda()
    args = (c.arena.cuda(), c.pages.cuda(), ints(lens), q, 2, E4M3)
    more = dict(starts=starts_of(counts), max_new=64)
    want = ac.defrag_kv_attend(*args, **more)
    assert torch.equal(ac.defrag_kv_attend_terms(*args, **more), want)
    causal = torch.cat([words_of(torch.ones(t, t, dtype=torch.bool).tril(), 1) for t in counts])
    assert torch.equal(ac.defrag_kv_attend_terms(*args, mask=causal.cuda(), **more), want)
    far = ac.defrag_kv_attend_terms(*args, cap=2.0 ** 40, **more)
    # scores of other roundings: each weight is rounded to float16 in both calls, by 2^-11 of it, so that results differ by
    # 2^-10 of sum p |v|, at most that of the largest |v|, and then by a step of bf16
    most = max(c.numbers(b, n, h)[1].abs().max() for b, n in enumerate(lens) for h in (0, 1))
    assert ((far.double() - want.double()).abs() <= want.double().abs() * 2.0 ** -7 + most * 2.0 ** -10 * 1.01).all()


@pytest.mark.parametrize("cap", [2.0 ** -64, 2.0 ** -10, 0.3, 2.0 ** 64])
def test_caps_at_their_limits(ac, cap):
    lens, counts = [130, 40], [1, 40]
    c = Cache([3, 1], 2, 64, INT8, fill=0)
    c.fill_random(lens, 1, size=8.0)
    q = queries(41, 6, 64, FP16, 2)
    assert check(ac, c, lens, q, 3, counts, None, cap)[1] == 0


def test_large_slopes_and_positions(ac):
    """Slopes of both signs, a bias of thousands, positions in the millions, several tokens at one."""
    lens, counts = [300, 150], [2, 70]
    c = Cache([5, 3], 2, 64, E4M3, fill=0x7F)
    c.fill_random(lens, 1)
    q = queries(72, 4, 64, BF16, 2)
    pos = planes(lens, counts, 2, 320, 4) // 3 + 5_000_000
    slopes = torch.tensor([16.0, -0.01, 0.0, 0.7])
    assert check(ac, c, lens, q, 2, counts, "tree", 0.0, slopes, pos)[1] == 0


def test_what_is_passed_over(ac):
    """Pages that are none, lengths out of range and shorter than the new tokens."""
    lens, counts = [200, 100, 130], [3, 2, 40]
    c = Cache([4, 2, 3], 1, 64, E4M3, fill=0x7F)
    c.fill_random(lens, 1)
    c.pages[0, 1], c.pages[2, 2] = -1, 33
    q = queries(45, 2, 64, BF16, 2)
    for kind in ("tree", "random"):
        assert check(ac, c, lens, q, 2, counts, kind, 9.0, slopes_of(2))[1] == 2
    # 30 of the 40 new tokens have no place: they see nothing, and nothing sees them
    lens = [200, 100, 10]
    c.pages[2, 2] = -1
    assert check(ac, c, lens, q, 2, counts, "prefix", 0.0, slopes_of(2))[1] == 1
    assert check(ac, c, lens, q, 2, counts, "random")[1] == 1
    out = ac.defrag_kv_attend_terms(c.arena.cuda(), c.pages.cuda(), ints([-3, 1000, 0]), q.cuda(), 1, E4M3, cap=5.0,
                                    starts=starts_of(counts), max_new=40)
    assert (out == 0).all()


def test_max_new_is_what_the_words_hold(ac):
    """Without max_new; a sequence that brings more than the words hold counts as invalid and brings nothing."""
    lens, counts = [100, 90], [70, 20]
    c = Cache([2, 2], 1, 64, E4M3, fill=0x7F)
    c.fill_random(lens, 1)
    q = queries(90, 2, 64, BF16, 2).cuda()
    mask = pack(masks(counts, "tree", 3), counts, 2, 90).cuda()
    args = (c.arena.cuda(), c.pages.cuda(), ints(lens), q, 1, E4M3)
    want = ac.defrag_kv_attend_terms(*args, mask=mask, starts=starts_of(counts), max_new=70)
    assert torch.equal(ac.defrag_kv_attend_terms(*args, mask=mask, starts=starts_of(counts)), want)
    bad, out = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.full_like(q, 3.0)
    ac.defrag_kv_attend_terms(*args, mask=mask[:, :1].contiguous(), starts=starts_of(counts), out=out, n_invalid=bad)
    # the cache may be cut elsewhere: weights rounded to float16 once more (2^-10 of the largest |v|), then a step of bf16
    most, got = c.numbers(1, 90, 0)[1].abs().max(), out[70:].double()
    assert int(bad) == 1 and (out[:70] == 3.0).all()
    assert ((got - want[70:].double()).abs() <= want[70:].double().abs() * 2.0 ** -7 + most * 2.0 ** -10 * 1.01).all()
    with pytest.raises(ac.DefragError):
        ac.defrag_kv_attend_terms(*args, mask=mask[:, :1].contiguous(), starts=starts_of(counts), max_new=70)
    with pytest.raises(ValueError):
        ac.defrag_kv_attend_terms(*args, mask=mask[:5], starts=starts_of(counts), max_new=70)


def test_stream_and_graph(ac):
    """Two calls of different kinds that share a workspace, captured and replayed with other inputs."""
    lens, counts = [1000, 700], [5, 4]
    c = Cache([16, 11], 2, 64, E4M3, fill=0x7F)
    c.fill_random(lens, 1)
    arena, pages, n, starts = c.arena.cuda(), c.pages.cuda(), ints(lens), starts_of(counts)
    q = torch.empty(9, 8, 64, dtype=BF16, device="cuda")
    mask = torch.empty(9, 1, dtype=torch.int64, device="cuda")
    slopes = torch.empty(8, device="cuda")
    one, two = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    weight = torch.zeros(2, 2, 1024, device="cuda")

    def step():
        weight.zero_()
        ac.defrag_kv_attend_terms(arena, pages, n, q, 2, E4M3, mask=mask, starts=starts, max_new=5, max_len=1024, out=one, ws=ws)
        ac.defrag_kv_attend_terms(arena, pages, n, q, 2, E4M3, mask=mask, cap=7.0, slopes=slopes, starts=starts, max_new=5,
                                  max_len=1024, out=two, weight=weight, ws=ws)

    def fill(i):
        gen = torch.Generator(device="cuda").manual_seed(i)
        q.normal_(generator=gen)
        mask.random_(0, 32, generator=gen)
        slopes.uniform_(generator=gen)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fill(9)
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.synchronize()
    for i in range(4):
        fill(i)
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (one, two, weight)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (one, two, weight)))
