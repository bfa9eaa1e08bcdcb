"""Attention under a mask where a workgroup goes over more than 64 pages, as
batches of so many (sequence, head, rows) that no cache is cut do: against the
plain 64-bit arithmetic and its bounds.  Most sequences are short, so that the
batch is large and the plain side small."""
import pytest
import torch

from kv_more_plain import PAGE, Cache
from test_kv_gpu import queries
from test_kv_terms_gpu import BF16, E4M3, FP16, INT8, check, planes, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ac():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import arena_compaction_amd
    return arena_compaction_amd


def cache(lens, heads, dim, codes, spread):
    c = Cache([-(-n // PAGE) for n in lens], heads, dim, codes, fill=0x7F)
    c.fill_random(lens, 1, spread=spread)
    return c


@pytest.mark.parametrize("kind,dim,codes,dtype,cap,bias,count", [
    ("tree", 64, E4M3, BF16, 0.0, False, 50),       # 64 rows a workgroup
    ("random", 64, INT8, FP16, 0.0, False, 90),     # 128
    ("documents", 128, E4M3, FP16, 20.0, False, 70),
    ("tree", 96, INT8, BF16, 0.0, True, 66),
    ("random", 256, E4M3, BF16, 0.0, False, 40),
    ("documents", 192, INT8, FP16, 300.0, True, 70)])
def test_behind_long_prefixes(ac, kind, dim, codes, dtype, cap, bias, count):
    """512 (sequence, head)s, prefixes of 64 pages less a few tokens, whose mask begins inside the first turn of 64 pages and
    ends in the second, and of more, whose mask lies in the second alone; scales several bands apart; pages that are none."""
    batch, heads = 64, 8
    had = [64 * PAGE - 30, 70 * PAGE + 13] + [3 + b % 9 for b in range(batch - 2)]
    counts = [count, count - 3] + [1 + b % 2 for b in range(batch - 2)]
    lens = [a + t for a, t in zip(had, counts)]
    c = cache(lens, heads, dim, codes, 24)
    c.pages[0, 5] = c.pages[1, 69] = -1
    q = queries(sum(counts) + 1, heads, dim, dtype, 2, "slice")
    pos = planes(lens, counts, heads, c.pages.shape[1] * PAGE, 3) if bias else None
    assert check(ac, c, lens, q, 1, counts, kind, cap, slopes_of(heads) if bias else None, pos, weight=dim < 192)[1] == 2


@pytest.mark.parametrize("had", [0, 40, 64, 100])
@pytest.mark.parametrize("kind,codes,dtype,bias", [("random", E4M3, BF16, False), ("documents", INT8, FP16, False),
                                                   ("prefix", E4M3, FP16, True)])
def test_over_many_new_tokens(ac, had, kind, codes, dtype, bias):
    """4300 new tokens, whose rows see from a part to all of 68 pages, behind no prefix, one of less than a page and of more:
    544 workgroups' rows over one head."""
    counts = [4300] + [1] * 15
    lens = [had + 4300] + [5 + b for b in range(15)]
    c = cache(lens, 1, 64, codes, 24)
    q = queries(sum(counts), 1, 64, dtype, 3)
    assert check(ac, c, lens, q, 1, counts, kind, 0.0, slopes_of(1) * 2.0 ** -8 if bias else None, seed=4)[1] == 0


@pytest.mark.parametrize("batch,group,count,dim,codes,dtype,cap,bias", [
    (34, 4, 1, 128, E4M3, BF16, 0.0, True), (48, 2, 3, 96, INT8, FP16, 30.0, False), (40, 16, 1, 128, INT8, BF16, 200.0, True)])
def test_two_pieces(ac, batch, group, count, dim, codes, dtype, cap, bias):
    """272 to 384 (sequence, head)s with a cap or a bias, the longest of 70 pages: cut in two."""
    heads = 8
    lens = [70 * PAGE - 11, 35 * PAGE, 36 * PAGE + 1] + [3 + 5 * b for b in range(batch - 3)]
    counts = [count] * batch
    c = cache(lens, heads, dim, codes, 9)
    q = queries(batch * count, heads * group, dim, dtype, 5)
    pos = planes(lens, counts, heads, c.pages.shape[1] * PAGE, 3) if bias else None
    slopes = slopes_of(heads * group) if bias else None
    assert check(ac, c, lens, q, group, counts, None, cap, slopes, pos)[1] == 0
    assert check(ac, c, lens, q, group, counts, "tree", cap, slopes, pos, weight=False)[1] == 0
