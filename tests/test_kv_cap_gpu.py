"""Capped scores over the 8-bit cache: a row's results are its own, bit for bit
whatever the other rows and the tokens that it does not see hold, and a capped
score is as close as its own size allows beside much larger ones."""
import math

import pytest
import torch

from kv_more_plain import PAGE, Cache, words_of
from test_kv_gpu import HALF, ints, queries, starts_of

pytestmark = pytest.mark.gpu
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ac():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import arena_compaction_amd
    return arena_compaction_amd


SIZES = [(1, 5, 2, 64, E4M3, FP16), (2, 7, 4, 128, INT8, FP16), (1, 3, 3, 256, E4M3, BF16), (2, 60, 2, 64, INT8, BF16),
         (1, 40, 5, 128, E4M3, FP16), (1, 50, 4, 256, INT8, FP16)]   # heads, new tokens, group, dimensions


def capped(ac, c, lens, q, mask, cap, bias):
    """out, lse and weight of one sequence whose last mask.shape[0] tokens are new."""
    n, heads = mask.shape[0], q.shape[1]
    lse, weight = torch.zeros(n, heads, device="cuda"), torch.zeros(1, c.H, c.pages.shape[1] * PAGE, device="cuda")
    slopes = torch.exp2(-1.0 - torch.arange(heads) % 4).float().cuda() if bias else None
    out = ac.defrag_kv_attend_terms(c.arena.cuda(), c.pages.cuda(), ints(lens), q.cuda(), c.H, c.codes, mask=words_of(mask).cuda(),
                                    cap=cap, slopes=slopes, starts=starts_of([n]), max_new=n, scale=0.25, lse=lse, weight=weight)
    return out.cpu(), lse.cpu(), weight.cpu()


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("heads,count,group,dim,codes,dtype", SIZES)
def test_what_a_row_does_not_see_changes_no_bit(ac, heads, count, group, dim, codes, dtype, bias):
    """Scores are below an eighth of the cap; that of a token which one row sees is above it, and so are those of codes
    behind the last token."""
    had = 70
    n = had + count
    c = Cache([-(-n // PAGE)], heads, dim, codes, fill=0)
    c.fill_random([n], 1, size=0.2)
    q = queries(count, heads * group, dim, dtype, 2)
    mask = torch.eye(count, dtype=torch.bool)
    spoiled = count // 2
    cap = 60.0 * dim / 64
    want = capped(ac, c, [n], q, mask, cap, bias)
    place = had + spoiled
    for h in range(heads):
        kc, vc, sc = c.head(int(c.pages[0, place // PAGE]), h)
        sign = torch.sign(q[spoiled, h * group].float())
        top = 448 if codes == E4M3 else 127
        assert top * float(sc[0]) * float(q[spoiled, h * group].float().abs().sum()) * 0.25 > cap / 8
        kc[place % PAGE] = (sign * top).to(codes)
        vc[place % PAGE] = (-sign * top).to(codes)
        if n % PAGE:
            kc, vc, _ = c.head(int(c.pages[0, n // PAGE]), h)
            kc[n % PAGE:] = (sign * top).to(codes)
            vc[n % PAGE:] = top
    got = capped(ac, c, [n], q, mask, cap, bias)
    others = torch.arange(count) != spoiled
    tokens = torch.arange(want[2].shape[2]) != place
    assert torch.equal(got[0][others], want[0][others]) and torch.equal(got[1][others], want[1][others])
    assert not torch.equal(got[1][spoiled], want[1][spoiled])
    # new tokens are seen by their own row alone
    assert torch.equal(got[2][:, :, had:][..., tokens[had:]], want[2][:, :, had:][..., tokens[had:]])


@pytest.mark.parametrize("cap", [30.0, 2.0 ** 14])
@pytest.mark.parametrize("heads,count,group,dim,codes,dtype", SIZES)
def test_another_rows_query_changes_no_bit(ac, heads, count, group, dim, codes, dtype, cap):
    """One query so large that its scores pass an eighth of the cap, beside rows whose scores are far below."""
    n = 70 + count
    c = Cache([-(-n // PAGE)], heads, dim, codes, fill=0)
    c.fill_random([n], 1, size=0.2)
    q = queries(count, heads * group, dim, dtype, 2) * 0.5
    mask = torch.ones(count, count, dtype=torch.bool).tril()
    want = capped(ac, c, [n], q, mask, cap, False)
    q[count // 2, 0] = q[count // 2, 0] * 2.0 ** (3 if cap < 100 else 14)
    got = capped(ac, c, [n], q, mask, cap, False)
    rows = torch.ones(count, heads * group, dtype=torch.bool)
    rows[count // 2, 0] = False
    assert torch.equal(got[0][rows], want[0][rows]) and torch.equal(got[1][rows], want[1][rows])


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("group", [16, 40, 200])
def test_scores_of_many_sizes_in_one_tile(ac, group, bias):
    """One token, seen by rows whose scores go from below 1 to far above the cap: the logarithm of a row's sum is its score.

    Whole numbers make q.k exact.  A capped score is off by 2^-19 of itself at the most, by the form that its own size
    asks for.  The sum's logarithm is that of one weight 2^(t - m), 13 < t - m <= 15: the shift rounds t by 2^-21 of its
    size, and beside it stand 2^-20 of t - m for the exponent and the logarithm and their product with ln 2."""
    cap, dim = 2.0 ** 20, 64
    c = Cache([1], 1, dim, INT8, fill=0)
    kc, vc, sc = c.head(int(c.pages[0, 0]), 0)
    kc[0], vc[0] = 1, 1
    sc[:] = 1.0
    size = torch.logspace(0, 17, group, base=2, dtype=torch.float64).round()
    q = torch.zeros(1, group, dim, dtype=BF16)
    q[0, :, 0] = size.to(BF16)
    s = q[0, :, 0].double() * 64                                # 2^6 to 2^23: far below, beside and far above the cap
    lse = torch.zeros(1, group, device="cuda")
    out = ac.defrag_kv_attend_terms(c.arena.cuda(), c.pages.cuda(), ints([1]), q.cuda(), 1, INT8, cap=cap, scale=64.0, lse=lse,
                                    slopes=torch.ones(group, device="cuda") if bias else None)
    want = cap * torch.tanh(s / cap)
    err = (lse[0].double().cpu() - want).abs()
    assert (err <= want * 2.0 ** -19 + want * 2.0 ** -21 + 15 * 2.0 ** -20).all()
    assert (out == 1.0).all()


@pytest.mark.parametrize("cap", [2.0 ** -64, 2.0 ** -30, 2.0 ** 64])
@pytest.mark.parametrize("count", [1, 50])
def test_scores_of_zero_under_any_cap(ac, cap, count):
    """Queries of zeros over keys of the largest scale: every score is 0, and every token counts alike."""
    n = 90
    c = Cache([2], 1, 64, INT8, fill=0)
    c.fill_random([n], 1)
    for j in (0, 1):
        c.head(int(c.pages[0, j]), 0)[2][0] = 2.0 ** 120
    q = torch.zeros(count, 2, 64, dtype=BF16)
    lse = torch.full((count, 2), 7.0, device="cuda")
    out = ac.defrag_kv_attend_terms(c.arena.cuda(), c.pages.cuda(), ints([n]), q.cuda(), 1, INT8, cap=cap, starts=starts_of([count]),
                                    max_new=count, lse=lse).double().cpu()
    v = c.numbers(0, n, 0)[1]
    for t in range(count):
        see = n - count + t + 1
        want = v[:see].mean(0)
        assert abs(float(lse[t, 0]) - math.log(see)) <= 2.0 ** -19
        # each weight is rounded to float16 alike, and the sum to 32 bits
        assert ((out[t] - want).abs() <= want.abs() * HALF[BF16] + v[:see].abs().mean(0) * 2.0 ** -10 + 2.0 ** -25).all()
