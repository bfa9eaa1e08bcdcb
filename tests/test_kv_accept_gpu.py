"""Keeping an accepted path on the GPU against plain 64-bit arithmetic: every
byte of the arena, the planes and the lengths are compared exactly."""
import pytest
import torch

from kv_more_plain import PAGE, Cache, accept, attend, rotate, tree, walk, words_of
from kv_same import assert_same_arena
from test_kv_gpu import HALF, ints, starts_of

pytestmark = pytest.mark.gpu
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ac():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import arena_compaction_amd
    return arena_compaction_amd


def run(ac, c, lens, counts, paths, planes=True, bad=0, left=()):
    """left: sequences that the call leaves alone."""
    B, places = len(lens), c.pages.shape[1] * PAGE + 3
    gen = torch.Generator().manual_seed(4)
    weight = torch.rand(B, c.H, places, generator=gen)
    pos = torch.randint(0, 1 << 30, (B, c.H, places), generator=gen, dtype=torch.int32)
    most = max([len(p) for p in paths] + [1]) + 2
    table = torch.full((B, most), 12345, dtype=torch.int32)
    for b, p in enumerate(paths):
        table[b, : len(p)] = torch.tensor(p, dtype=torch.int32)
    arena = c.arena.cuda()
    wg, pg = (weight.cuda(), pos.cuda()) if planes else (None, None)
    lens_out, n_bad = ints([-7] * B), torch.full((1,), 9, dtype=torch.int64, device="cuda")
    ac.defrag_kv_accept(arena, c.pages.cuda(), ints(lens), table.cuda(), ints([len(p) for p in paths]), lens_out, c.H, c.D, c.codes,
                        starts=starts_of(counts), max_new=max(counts), weight=wg, pos=pg, n_invalid=n_bad)
    torch.cuda.synchronize()
    sane = [[] if b in left else p for b, p in enumerate(paths)]
    want = accept(c, [0 if b in left else n for b, n in enumerate(lens)], [0 if b in left else t for b, t in enumerate(counts)],
                  sane, weight if planes else None, pos if planes else None)
    want = [lens[b] if b in left else w for b, w in enumerate(want)]
    assert lens_out.tolist() == want and int(n_bad) == bad
    assert_same_arena(c, arena)
    if planes:
        assert torch.equal(wg.cpu(), weight) and torch.equal(pg.cpu(), pos)


def pages_of(lens):
    return [-(-n // PAGE) for n in lens]


@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 96), (2, 128), (4, 192), (1, 256)])
@pytest.mark.parametrize("codes", [E4M3, INT8])
@pytest.mark.parametrize("spread", [0, 6])
def test_trees(ac, heads, dim, codes, spread):
    """Drafts within a page and over the border of two, whose scales differ."""
    gen = torch.Generator().manual_seed(dim + spread)
    had, counts = [0, 5, 50, 60, 63, 64, 120, 127, 200], [7, 20, 25, 33, 2, 64, 10, 1, 90]
    lens = [a + t for a, t in zip(had, counts)]
    c = Cache(pages_of(lens), heads, dim, codes, fill=0x11)
    c.fill_random(lens, 1, spread=spread)
    paths = []
    for t in counts:
        up = tree(t, 4, gen)[0]
        paths.append(walk(up, gen))
    run(ac, c, lens, counts, paths)


@pytest.mark.parametrize("codes", [E4M3, INT8])
def test_ends(ac, codes):
    """All kept, none kept, the first, the last alone, one from the page behind, a whole page from the page behind."""
    had = [70, 70, 70, 70, 60, 64, 0, 128]
    counts = [10, 10, 10, 10, 70, 128, 64, 64]
    paths = [list(range(10)), [], [0], [9], [69], list(range(64, 128)), list(range(64)), [63]]
    lens = [a + t for a, t in zip(had, counts)]
    c = Cache(pages_of(lens), 2, 64, codes, fill=0x11)
    c.fill_random(lens, 2, spread=8)
    run(ac, c, lens, counts, paths)


@pytest.mark.parametrize("codes", [E4M3, INT8])
def test_over_many_pages(ac, codes):
    """Paths through drafts of many pages; a page that takes from several others."""
    gen = torch.Generator().manual_seed(3)
    had, counts = [30, 0, 64], [700, 1000, 400]
    lens = [a + t for a, t in zip(had, counts)]
    paths = [sorted(torch.randperm(t, generator=gen)[: t * k // 8].tolist()) for t, k in zip(counts, (1, 6, 4))]
    c = Cache(pages_of(lens), 2, 96, codes, fill=0x11)
    c.fill_random(lens, 2, spread=10)
    run(ac, c, lens, counts, paths)
    run(ac, c, lens, counts, paths, planes=False)


def test_codes_that_are_no_numbers(ac):
    """NaN of a token that changes its page stays one and does not count for the scale."""
    lens, counts, paths = [100], [50], [[10, 20, 21, 49]]
    c = Cache([2], 1, 64, E4M3, fill=0x11)
    c.fill_random(lens, 1, spread=3)
    page = int(c.pages[0, 1])
    c.arena[page + 7 * 64 + 3] = 0x7F              # key of place 71, the path's third
    c.arena[page + 64 * 64 + 9 * 64 + 35] = 0xFF   # a value of place 99
    run(ac, c, lens, counts, paths)
    assert torch.isnan(c.head(int(c.pages[0, 0]), 0)[0].float()).sum() == 1


def test_scales_at_the_ends_of_their_range(ac):
    """Pages of zeros, of the least scale and of the largest numbers that append stores."""
    for codes in (E4M3, INT8):
        for e_from, e_to in ((-64, 100), (120, -64), (120, 119), (-64, -64)):
            lens, counts, paths = [100, 100], [50, 36], [[20, 30, 49], [5, 35]]
            c = Cache([2, 2], 1, 64, codes, fill=0)
            c.fill_random(lens, 1)
            for b in (0, 1):
                for j, e in ((0, e_to), (1, e_from)):
                    c.head(int(c.pages[b, j]), 0)[2][:] = 2.0 ** e
            run(ac, c, lens, counts, paths)
        c = Cache([2], 1, 64, codes, fill=0)
        for j in (0, 1):
            c.head(int(c.pages[0, j]), 0)[2][:] = 2.0 ** -3
        run(ac, c, [100], [50], [[20, 49]])


def test_what_is_left_alone(ac):
    """Paths that do not ascend, numbers and lengths out of range, pages that are none: counted, left as they were."""
    had, t = 50, 20
    paths = [[3, 3], [5, 4], [20], [-1, 2], [0, 5], [1, 15], [0, 1], [2], [0, 1]]
    lens = [had + t] * 9
    lens[4], lens[7] = -1, 5000
    c = Cache([2] * 9, 2, 64, INT8, fill=0x11)
    c.fill_random([70] * 9, 1)
    c.pages[5, 1] = 1          # read: place 65 goes to 51
    c.pages[6, 0] = -1         # not read: nothing moves
    keep = c.pages.clone()
    run(ac, c, lens, [t] * 9, paths, bad=7, left=(0, 1, 2, 3, 4, 5, 7))
    assert torch.equal(c.pages, keep)
    # ranges of starts that are none: longer than max_new, descending
    c = Cache([2, 2], 1, 64, INT8, fill=0x11)
    c.fill_random([70, 70], 1)
    arena, bad, out = c.arena.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"), ints([0, 0])
    ac.defrag_kv_accept(arena, c.pages.cuda(), ints([70, 70]), ints([[3], [3]]), ints([1, 1]), out, 1, 64, INT8,
                        starts=ints([0, 20, 10]), max_new=10, n_invalid=bad)
    assert out.tolist() == [70, 70] and int(bad) == 2 and torch.equal(arena.cpu(), c.arena)
    # more kept than path has room for
    ac.defrag_kv_accept(arena, c.pages.cuda(), ints([70, 70]), ints([[3], [3]]), ints([2, 1]), out, 1, 64, INT8,
                        starts=ints([0, 10, 20]), max_new=10, n_invalid=bad)
    assert out.tolist() == [70, 61] and int(bad) == 1


def test_one_token_each_and_graph(ac):
    """Without starts a sequence has one drafted token; captured and replayed."""
    c = Cache([2, 2, 1], 2, 64, E4M3, fill=0x11)
    c.fill_random([70, 65, 1], 1)
    arena, pages, lens, out = c.arena.cuda(), c.pages.cuda(), ints([70, 65, 1]), ints([0, 0, 0])
    path, kept = ints([[0], [0], [0]]), ints([1, 0, 0])

    def step():
        ac.defrag_kv_accept(arena, pages, lens, path, kept, out, 2, 64, E4M3)

    step()
    assert out.tolist() == [70, 64, 0] and torch.equal(arena.cpu(), c.arena)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in ([0, 0, 1], [1, 1, 1], [0, 1, 0]):
        kept.copy_(ints(k))
        g.replay()
        torch.cuda.synchronize()
        assert out.tolist() == [69 + k[0], 64 + k[1], k[2]]


@pytest.mark.parametrize("codes", [E4M3, INT8])
def test_drafting_cycle(ac, codes):
    """Drafts are appended at their depths, verified under the tree's mask, and the accepted path is kept, several times
    over; the cache is then that of a cache to which the accepted tokens alone were given, up to what a larger scale of
    the rejected ones has cost, and attention over it is attention over what it holds."""
    B, H, G, D, T, R = 3, 2, 3, 64, 12, 64
    gen = torch.Generator().manual_seed(1)
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    c = Cache([3] * B, H, D, codes, fill=0)
    arena, pages = c.arena.cuda(), c.pages.cuda()
    lens, pos = ints([0] * B), torch.zeros(B, H, 3 * PAGE, dtype=torch.int32, device="cuda")
    weight = torch.zeros(B, H, 3 * PAGE, device="cuda")
    lens_out, held, tokens = torch.zeros_like(lens), [0] * B, [[] for _ in range(B)]
    starts = starts_of([T] * B)
    for step in range(50):
        trees = [tree(T, 3, gen) for _ in range(B)]
        x = torch.randn(B * T, (G + 2) * H, D, generator=gen).to(BF16)
        q, k, v = x[:, : G * H], x[:, G * H: (G + 1) * H], x[:, (G + 1) * H:]
        at = torch.tensor([held[b] + d for b in range(B) for d in trees[b][2]])
        xg = x.cuda()
        turned = ac.defrag_kv_append_rotary(arena, pages, lens, xg[:, G * H: (G + 1) * H], xg[:, (G + 1) * H:], codes, freq.cuda(),
                                            q=xg[:, : G * H], starts=starts, max_new=T, token_pos=ints(at.tolist()), weight=weight,
                                            pos=pos)
        lens += T
        mask = torch.cat([words_of(t[1]) for t in trees])
        out = ac.defrag_kv_attend_terms(arena, pages, lens, turned, H, codes, mask=mask.cuda(), starts=starts, max_new=T)
        if step % 8 == 7:
            c.arena = arena.cpu()
            n = [h + T for h in held]
            want, bound, *_ = attend(c, n, turned.cpu(), G, [T] * B, D ** -0.5, [t[1] for t in trees])
            err = (out.double().cpu() - want).abs()
            assert (err <= bound * (1 + HALF[BF16]) + want.abs() * HALF[BF16] + 2.0 ** -25).all()
        paths = [walk(t[0], gen)[: int(torch.randint(0, 6, (1,), generator=gen))] for t in trees]
        table = torch.zeros(B, T, dtype=torch.int32)
        keys = rotate(k, at, freq, False)
        for b, p in enumerate(paths):
            table[b, : len(p)] = torch.tensor(p, dtype=torch.int32)
            tokens[b] += [(keys[b * T + i], v[b * T + i].double(), int(at[b * T + i])) for i in p]
            held[b] += len(p)
        ac.defrag_kv_accept(arena, pages, lens, table.cuda(), ints([len(p) for p in paths]), lens_out, H, D, codes, starts=starts,
                            max_new=T, weight=weight, pos=pos)
        lens, lens_out = lens_out, lens
        assert lens.tolist() == held
    assert max(held) > PAGE, "no page's border was crossed"
    c.arena = arena.cpu()
    for b in range(B):
        assert pos[b, :, : held[b]].cpu().tolist() == [[t[2] for t in tokens[b]]] * H
        assert [t[2] for t in tokens[b]] == list(range(held[b]))
        for h in range(H):
            ks, vs, ok = c.numbers(b, held[b], h)
            assert ok.all()
            for got, i in ((ks, 0), (vs, 1)):
                want = torch.stack([t[i][h] for t in tokens[b]])
                # numbers below 127 * 2^-4: scales are at most 2^-4 (int8) and 2^-5 (e4m3).  int8 rounds by half a scale,
                # and by half of each smaller one before: 2^-5 + 2^-6 + ...; e4m3 by 2^-4 of the number once, and below
                # its normal numbers by half of 2^-9 scales at each scale: 2^-15 + 2^-16 + ...
                assert want.abs().max() < 127 * 2.0 ** -4
                tol = 2.0 ** -4 if codes == INT8 else want.abs() * 2.0 ** -4 + 2.0 ** -14
                assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("codes", [E4M3, INT8])
@pytest.mark.parametrize("e_from", [63, 64, 100, 120])
def test_zeros_out_of_a_page_of_large_numbers(ac, codes, e_from):
    """Tokens of zeros stay zeros, whatever their page's scale was: into a page of zeros, alone and beside small numbers
    out of a third page, and into a page that they fill."""
    lens, counts = [128 + 40, 128 + 40, 64 + 128], [128 + 20, 128 + 20, 128]
    paths = [[50, 55, 60], [50, 110, 112, 115], list(range(64, 128))]
    c = Cache(pages_of(lens), 2, 64, codes, fill=0)
    c.fill_random(lens, 1)
    for b in (0, 1, 2):
        for h in (0, 1):
            for w in (0, 1):
                first, second = (c.head(int(c.pages[b, j]), h) for j in (0, 1))
                if b < 2:                                    # the first page: zeros
                    first[w].view(torch.uint8)[:] = 0
                    first[2][w] = 2.0 ** -64
                second[2][w] = 2.0 ** e_from
                second[w].view(torch.uint8)[:] = 0
                second[w].view(torch.uint8)[0] = 0x38        # its large numbers, which go
                third = c.head(int(c.pages[b, 2]), h)
                third[2][w] = 2.0 ** (e_from if b == 2 else -10)
                if b == 2:                                   # its path takes zeros alone
                    third[w].view(torch.uint8)[:] = 0
    run(ac, c, lens, counts, paths)
    assert not any(torch.isnan(x).any() for x in c.numbers(0, 23, 0)[:2])


def test_missing_pages_are_counted_once_each(ac):
    """A path over more pages than a wave has lanes, of which some are none: each is counted, by one head."""
    t = 150 * PAGE
    lens, counts, paths = [t + 5, 40], [t, 10], [list(range(1, t, 97)) + [t - 1], [4, 7]]
    c = Cache(pages_of(lens), 3, 64, INT8, fill=0x11)
    c.fill_random([70, 40], 1)
    none = [1, 60, 63, 64, 65, 100, 130, 149]
    for j in none:
        c.pages[0, j] = -1
    run(ac, c, lens, counts, paths, bad=len(none), left=(0,))
