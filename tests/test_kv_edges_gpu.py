"""The 8-bit key/value cache on the GPU at the ends of its ranges: scales far
apart, scores without numbers, grids past one axis, lengths past one part.

Codes, scales, positions and lengths are compared exactly; attention within
the bounds that kv_plain.attend derives, plus half a step of the output's type
(bf16 2^-8, fp16 2^-11 of the value)."""
import math

import pytest
import torch

from kv_plain import PAGE, Cache, evict

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
