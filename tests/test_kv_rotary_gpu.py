"""Appending with rotation on the GPU against plain 64-bit arithmetic.

Codes, scales, positions and weights are compared exactly.  Queries are the
result of 32-bit products with 64-bit angles, rounded once to their type (half
a step: bf16 2^-8, fp16 2^-11 of the value, 2^-25 below fp16's normal numbers).
Sine and cosine are rounded to 32 bits, 2^-24, and so are a product and a sum:
together at most 2^-22 of the pair's larger number; far positions add the
64-bit angle's own rounding, 2^-52 of it."""
import itertools

import pytest
import torch

from kv_more_plain import PAGE, Cache, rotate
from kv_same import assert_same_arena

pytestmark = pytest.mark.gpu
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
BF16, FP16 = torch.bfloat16, torch.float16


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


def freqs(rotary, base=10000.0):
    return base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)


def projection(n, q_heads, heads, dim, dtype, seed, layout="slice", size=1.0):
    """q, k, v as views of one tensor."""
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(n, q_heads + 2 * heads, dim, generator=gen) * size).to(dtype)
    if layout == "heads first":
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    if layout == "unaligned":
        x = torch.nn.functional.pad(x, (1, 2))[:, :, 1: 1 + dim]
    return x, x[:, :q_heads], x[:, q_heads: q_heads + heads], x[:, q_heads + heads:]


def on_gpu(x):
    y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
    return y.copy_(x)


def views(x, q_heads, heads):
    return x[:, :q_heads], x[:, q_heads: q_heads + heads], x[:, q_heads + heads:]


def check_q(got, q, pos, freq, interleaved):
    want = rotate(q, pos, freq, interleaved)
    got = got.double().cpu()
    half = torch.finfo(q.dtype).eps / 2
    # both numbers of a pair, times the angle's rounding
    R = 2 * len(freq)
    size = torch.zeros_like(want)
    size[..., :R] = q.double()[..., :R].abs().amax(-1, keepdim=True) * 2
    angle = float(pos.double().abs().max()) * float(freq.abs().max()) if len(pos) else 0.0
    near = size * (angle * 2.0 ** -52 + 2.0 ** -23)      # size is twice the larger number
    tol = (want.abs() + near) * half + near + 2.0 ** -25 * (q.dtype == FP16)
    assert torch.equal(torch.isfinite(got), torch.isfinite(want))
    fine = torch.isfinite(want)
    assert ((got - want).abs()[fine] <= tol[fine]).all()


def run(ac, lens, counts, heads, group, dim, rotary, interleaved, codes, dtype, seed, layout="slice", pos=None, inplace=False,
        size=1.0, first=None, edit=None, spread=4, base=10000.0):
    n = sum(counts)
    c = Cache([-(-(a + t) // PAGE) + 1 for a, t in zip(lens, counts)], heads, dim, codes, fill=0x55, seed=seed)
    c.fill_random(lens, seed + 1, spread=spread)
    x, q, k, v = projection(n, heads * group, heads, dim, dtype, seed + 2, layout, size)
    if edit:
        edit(q, k, v)
    first = [a + 3 for a in lens] if first is None else first
    at = torch.tensor([f + i for f, t in zip(first, counts) for i in range(t)], dtype=torch.int64) if pos is None else pos
    freq = freqs(rotary, base)
    arena = c.arena.cuda()
    places = c.pages.shape[1] * PAGE + 1
    weight, plane = torch.ones(len(lens), heads, places), torch.full((len(lens), heads, places), -5, dtype=torch.int32)
    wg, pg, bad = weight.cuda(), plane.cuda(), torch.full((1,), 9, dtype=torch.int64, device="cuda")
    xg = on_gpu(x)
    qg, kg, vg = views(xg, heads * group, heads)
    out = ac.defrag_kv_append_rotary(arena, c.pages.cuda(), ints(lens), kg, vg, codes, freq.cuda(), q=qg,
                                     q_out=qg if inplace else None, interleaved=interleaved, starts=starts_of(counts),
                                     max_new=max(counts + [1]) if n else 0, token_pos=None if pos is None else ints(pos.tolist()),
                                     weight=wg, pos=pg, first_pos=ints(first), n_invalid=bad)
    torch.cuda.synchronize()
    keys = rotate(k, at, freq, interleaved)
    s = 0
    for b, (a, t) in enumerate(zip(lens, counts)):
        c.append(b, a, keys[s: s + t], v[s: s + t].double())
        weight[b, :, a: a + t] = 0
        plane[b, :, a: a + t] = at[s: s + t].to(torch.int32)
        s += t
    assert int(bad) == 0
    assert_same_arena(c, arena)
    assert torch.equal(wg.cpu(), weight) and torch.equal(pg.cpu(), plane)
    if inplace:
        assert out is qg
        kk, vv = views(xg.cpu(), heads * group, heads)[1:]
        assert torch.equal(kk, k) and torch.equal(vv, v)
    check_q(out, q, at, freq, interleaved)


SHAPES = [  # heads, group, dim, rotated, interleaved, codes, dtype
    (1, 1, 64, 64, False, E4M3, BF16), (2, 4, 64, 32, True, INT8, FP16), (3, 3, 96, 96, False, INT8, BF16),
    (2, 7, 96, 40, True, E4M3, FP16), (2, 16, 128, 128, False, E4M3, BF16), (1, 17, 128, 128, True, INT8, FP16),
    (4, 2, 192, 64, False, E4M3, FP16), (1, 8, 192, 192, True, INT8, BF16), (1, 6, 256, 256, False, E4M3, BF16),
    (2, 9, 256, 8, False, INT8, FP16)]


@pytest.mark.parametrize("heads,group,dim,rotary,interleaved,codes,dtype", SHAPES)
def test_one_token(ac, heads, group, dim, rotary, interleaved, codes, dtype):
    lens = [0, 1, 3, 62, 63, 64, 65, 200]
    run(ac, lens, [1] * len(lens), heads, group, dim, rotary, interleaved, codes, dtype, 1)


@pytest.mark.parametrize("most", [2, 3, 4, 5, 17])
@pytest.mark.parametrize("heads,group,dim,rotary,interleaved,codes,dtype", SHAPES)
def test_few_tokens(ac, heads, group, dim, rotary, interleaved, codes, dtype, most):
    """Up to 4 a sequence a wave takes a head, above a workgroup; at every place in four, and over a page's end."""
    lens = [0, 1, 2, 3, 60, 61, 62, 63, 7, 130]
    run(ac, lens, [most, most, most, most, most, most, most, most, 1, 2], heads, group, dim, rotary, interleaved, codes, dtype, most)


@pytest.mark.parametrize("heads,group,dim,rotary,interleaved,codes,dtype", SHAPES)
def test_ragged(ac, heads, group, dim, rotary, interleaved, codes, dtype):
    run(ac, [0, 5, 64, 100, 7, 63], [64, 7, 0, 133, 17, 2], heads, group, dim, rotary, interleaved, codes, dtype, 2,
        layout="heads first")


@pytest.mark.parametrize("codes,dtype", [(E4M3, BF16), (INT8, FP16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_unaligned(ac, codes, dtype, interleaved):
    run(ac, [10, 70], [30, 16], 2, 3, 128, 64, interleaved, codes, dtype, 3, layout="unaligned", inplace=True)


@pytest.mark.parametrize("tokens", [1, 5])
def test_in_place_between_other_heads(ac, tokens):
    """A projection whose heads hold query, key and value side by side."""
    heads, dim = 3, 64
    gen = torch.Generator().manual_seed(11)
    x = torch.randn(tokens, heads, 3, dim, generator=gen).to(BF16)
    xg = x.cuda()
    c = Cache([1], heads, dim, E4M3)
    arena, freq, pos = c.arena.cuda(), freqs(dim), torch.arange(tokens) + 7
    out = ac.defrag_kv_append_rotary(arena, c.pages.cuda(), ints([0]), xg[:, :, 1], xg[:, :, 2], E4M3, freq.cuda(), q=xg[:, :, 0],
                                     q_out=xg[:, :, 0], starts=ints([0, tokens]), first_pos=ints([7]))
    check_q(out, x[:, :, 0], pos, freq, False)
    assert torch.equal(xg[:, :, 1:].cpu(), x[:, :, 1:])
    c.append(0, 0, rotate(x[:, :, 1], pos, freq, False), x[:, :, 2].double())
    assert_same_arena(c, arena)
    for q, to in ((xg[:, :, 0], xg[:, :, 1]), (xg[:, :2, 0], xg[:, 1:, 0])):   # over the keys, over other queries
        with pytest.raises(ac.DefragError):
            ac.defrag_kv_append_rotary(arena, c.pages.cuda(), ints([0]), xg[:, :, 1], xg[:, :, 2], E4M3, freq.cuda(), q=q, q_out=to,
                                       starts=ints([0, tokens]))


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_by_token(ac, interleaved):
    """Depths of trees, one position for several tokens, far and negative ones."""
    pos = torch.tensor([5, 6, 6, 7, 7, 7, 8, 0, 1, 1, 131071, 131071, 1000000, -1, -70000, 0], dtype=torch.int64)
    run(ac, [40, 0], [9, 7], 2, 2, 64, 64, interleaved, E4M3, BF16, 4, pos=pos)


def test_farthest_positions(ac):
    """Queries at the ends of the positions' range (no codes beside a border at this seed would need the last bits)."""
    n = 4
    x, q, k, v = projection(n, 2, 1, 64, FP16, 5)
    c = Cache([1], 1, 64, INT8)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 12345678], dtype=torch.int64)
    freq = freqs(64)
    q, k, v = (y.cuda() for y in (q, k, v))
    out = ac.defrag_kv_append_rotary(c.arena.cuda(), c.pages.cuda(), ints([0]), k, v, INT8, freq.cuda(), q=q,
                                     starts=ints([0, n]), token_pos=ints(pos.tolist()))
    check_q(out, q.cpu(), pos, freq, False)


@pytest.mark.parametrize("dtype,size", [(BF16, 2.0 ** 126), (BF16, 2.0 ** -130), (FP16, 2.0 ** 13), (FP16, 2.0 ** -18)])
@pytest.mark.parametrize("codes", [E4M3, INT8])
def test_ends_of_the_types_range(ac, dtype, size, codes):
    """A rotated key may lie outside the type's range, and outside float32's, and is a number still; a query becomes an
    infinity there."""
    gen = torch.Generator().manual_seed(6)
    c = Cache([2], 1, 64, codes)
    x = (torch.randn(70, 4, 64, generator=gen).clamp(-1.9, 1.9) * size).to(dtype)
    x[3, :, 5] = x[3, :, 37] = torch.finfo(dtype).max if size > 1 else torch.finfo(dtype).smallest_normal
    q, k, v = views(x, 2, 1)
    freq, pos = freqs(64), torch.arange(70)
    arena = c.arena.cuda()
    out = ac.defrag_kv_append_rotary(arena, c.pages.cuda(), ints([0]), k.cuda(), v.cuda(), codes, freq.cuda(), q=q.cuda(),
                                     starts=ints([0, 70]))
    c.append(0, 0, rotate(k, pos, freq, False), v.double())
    assert_same_arena(c, arena)
    want, got = rotate(q, pos, freq, False), out.double().cpu()
    top = torch.finfo(dtype).max
    inside = want.abs() <= top
    step = torch.finfo(dtype).eps / 2
    pair = torch.maximum(q.double().abs(), torch.cat([q.double()[..., 32:], q.double()[..., :32]], -1).abs()) * 2.0 ** -22
    assert torch.isinf(got[want.abs() - pair > top * (1 + step)]).all()
    fine = inside & ~(torch.isinf(got) & (want.abs() + pair >= top))
    err = (got - want).abs()[fine]
    least = torch.finfo(dtype).smallest_normal * step      # half a step of the numbers below the normal ones
    assert (err <= (want.abs() * step + pair * (1 + step) + least)[fine]).all()


@pytest.mark.parametrize("codes", [E4M3, INT8])
@pytest.mark.parametrize("interleaved", [False, True])
def test_not_finite(ac, codes, interleaved):
    """Infinities and NaN go by the formula: to both numbers of a pair, and no farther."""
    def edit(q, k, v):
        for x in (q, k, v):
            x[4, :, 3] = float("inf")
            x[9, :, 10] = float("nan")
            x[12, :, 60] = float("-inf")
    lens, counts = [20], [20]
    n, heads = 20, 2
    c = Cache([2], heads, 64, codes)
    c.fill_random(lens, 1)
    x, q, k, v = projection(n, 4, heads, 64, BF16, 7)
    edit(q, k, v)
    freq, pos = freqs(48), torch.arange(n) + 20
    arena = c.arena.cuda()
    q, k, v = views(x, 4, heads)
    out = ac.defrag_kv_append_rotary(arena, c.pages.cuda(), ints(lens), k.cuda(), v.cuda(), codes, freq.cuda(), q=q.cuda(),
                                     interleaved=interleaved, starts=starts_of(counts))
    keys = rotate(k, pos, freq, interleaved)
    c.append(0, 20, keys, v.double())
    assert_same_arena(c, arena)
    want = rotate(q, pos, freq, interleaved)
    got = out.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))
    assert torch.equal(got[torch.isinf(got)], want[torch.isinf(want)])


def test_without_queries_and_planes(ac):
    c = Cache([1, 2], 2, 64, E4M3)
    _, _, k, v = projection(60, 0, 2, 64, FP16, 8)
    arena, freq = c.arena.cuda(), freqs(64)
    got = ac.defrag_kv_append_rotary(arena, c.pages.cuda(), ints([0, 0]), k.cuda(), v.cuda(), E4M3, freq.cuda(),
                                     starts=starts_of([20, 40]))
    assert got is None
    for b, (s, t) in enumerate(((0, 20), (20, 40))):   # a token's position is its place
        c.append(b, 0, rotate(k[s: s + t], torch.arange(t), freq, False), v[s: s + t].double())
    assert_same_arena(c, arena)


def test_what_is_passed_over(ac):
    """Pages that are none, sequences out of range, tokens of no sequence: counted, their pages and queries as they were
    (queries of a page that is none are rotated)."""
    lens, counts = [60, 10, 10, -1, 500], [10, 4, 3, 2, 1]
    n = sum(counts) + 5
    c = Cache([2, 1, 1, 1, 1], 1, 64, E4M3, fill=0x33)
    c.fill_random([60, 10, 10], 3)
    c.pages[1, 0] = 17                         # not on the grid
    before = c.arena.clone()
    _, q, k, v = projection(n, 2, 1, 64, BF16, 9)
    arena, freq = c.arena.cuda(), freqs(64)
    bad = torch.zeros(1, dtype=torch.int64, device="cuda")
    q_out = torch.full((n, 2, 64), 7.0, dtype=BF16, device="cuda")
    ac.defrag_kv_append_rotary(arena, c.pages.cuda(), ints(lens), k.cuda(), v.cuda(), E4M3, freq.cuda(), q=q.cuda(), q_out=q_out,
                               starts=starts_of(counts), max_new=10, n_invalid=bad)
    assert int(bad) == 3                       # the entry, and two lengths
    c.arena = before
    c.append(0, 60, rotate(k[:10], torch.arange(60, 70), freq, False), v[:10].double())
    c.append(2, 10, rotate(k[14:17], torch.arange(10, 13), freq, False), v[14:17].double())
    assert_same_arena(c, arena)
    pos = torch.cat([torch.arange(60, 70), torch.arange(10, 14), torch.arange(10, 13)])
    check_q(q_out[:17], q[:17], pos, freq, False)
    assert (q_out[17:] == 7.0).all()


def test_agrees_with_append_at_position_zero(ac):
    """A rotation by nothing: the bytes that defrag_kv_append writes, and the queries as they were."""
    c = Cache([3], 3, 96, INT8)
    x, q, k, v = projection(150, 6, 3, 96, FP16, 10)
    one, two = c.arena.cuda(), c.arena.cuda()
    xg = on_gpu(x)
    q, k, v = views(xg, 6, 3)
    starts = starts_of([150])
    ac.defrag_kv_append(one, c.pages.cuda(), ints([0]), k, v, INT8, starts=starts)
    out = ac.defrag_kv_append_rotary(two, c.pages.cuda(), ints([0]), k, v, INT8, freqs(96).cuda(), q=q, starts=starts,
                                     token_pos=ints([0] * 150))
    assert torch.equal(one, two) and torch.equal(out, q)


def test_stream_and_graph(ac):
    """On a stream of its own, captured with an attention behind it and replayed with other inputs."""
    lens, heads, dim = [70, 3], 2, 64
    c = Cache([3, 2], heads, dim, E4M3)
    c.fill_random(lens, 1)
    start = c.arena.cuda()
    arena, pages, n = start.clone(), c.pages.cuda(), ints(lens)
    more = n + 1
    x = torch.empty(2, 12, dim, dtype=BF16, device="cuda")
    q, k, v = views(x, 8, heads)
    freq, first = freqs(dim).cuda(), ints([70, 3])
    q_out = torch.empty(2, 8, dim, dtype=BF16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q_out)

    def step():
        ac.defrag_kv_append_rotary(arena, pages, n, k, v, E4M3, freq, q=q, q_out=q_out, first_pos=first)
        ac.defrag_kv_attend(arena, pages, more, q_out, heads, E4M3, max_len=128, out=out, ws=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x.normal_()
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.synchronize()
    for i in range(4):
        gen = torch.Generator(device="cuda").manual_seed(i)
        x.copy_(torch.randn(x.shape, device="cuda", generator=gen))
        first += 1000
        arena.copy_(start)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), q_out.clone(), arena.clone()
        arena.copy_(start)
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, q_out, arena)))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (128, 96), (256, 256)])
def test_queries_by_their_pairs(ac, dim, rotary, interleaved, dtype):
    """Each query's error beside its own pair's larger number M, among pairs of sizes that lie far apart and some whose
    products cancel: sine and cosine rounded to 32 bits, (|cos| + |sin|) 2^-24 M <= 1.42 * 2^-24 M; a product, 2^-24 M; their
    sum, 1.42 * 2^-24 M; together below 2^-22 M.  The angle p f is off by 3 * 2^-53 of itself in the kernel's turns and 2^-53
    here, which moves a number by that times at most 1.42 M.  Then half a step of the type."""
    n, heads = 200, 6
    gen = torch.Generator().manual_seed(dim + interleaved)
    pos = torch.randint(0, 200_000, (n,), generator=gen)
    freq = freqs(rotary)
    q = torch.randn(n, heads, dim, generator=gen, dtype=torch.float64)
    first, second = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, rotary // 2), slice(rotary // 2, rotary))
    size = torch.exp2(torch.randint(-6, 7, (n, heads, rotary // 2), generator=gen).double())
    angle = pos.double()[:, None] * freq
    near = torch.rand(n, heads, rotary // 2, generator=gen) < 0.5       # these lie where the first number comes to almost 0
    x, y = q[..., first] * size, q[..., second] * size
    x = torch.where(near, (size * torch.sin(angle)[:, None]), x)
    y = torch.where(near, (size * torch.cos(angle)[:, None]), y)
    q[..., first], q[..., second] = x, y
    q = q.to(dtype)
    k = torch.zeros(n, 1, dim, dtype=dtype)
    c = Cache([-(-n // PAGE)], 1, dim, INT8)
    out = ac.defrag_kv_append_rotary(c.arena.cuda(), c.pages.cuda(), ints([0]), k.cuda(), k.cuda(), INT8, freq.cuda(), q=q.cuda(),
                                     interleaved=interleaved, starts=ints([0, n]), token_pos=ints(pos.tolist()))
    got, want = out.double().cpu(), rotate(q, pos, freq, interleaved)
    half = torch.finfo(dtype).eps / 2
    for at in (first, second):
        most = torch.maximum(q[..., first].double().abs(), q[..., second].double().abs())
        near = most * (2.0 ** -22 + 1.42 * 2.0 ** -51 * angle[:, None])
        tol = near + (want[..., at].abs() + near) * half + 2.0 ** -25 * (dtype == FP16)
        assert ((got[..., at] - want[..., at]).abs() <= tol).all()
    assert torch.equal(got[..., rotary:], q.double()[..., rotary:])
