"""What the comparison of two arenas sees."""
import pytest
import torch

from kv_plain import Cache
from kv_same import assert_same_arena

E4M3, INT8 = torch.float8_e4m3fn, torch.int8


@pytest.mark.parametrize("codes", [E4M3, INT8])
def test_a_changed_byte_is_seen(codes):
    c = Cache([2, 1], 2, 64, codes)
    c.fill_random([100, 30], 1)
    assert_same_arena(c, c.arena.clone())
    strips = 2 * 2 * 64 * 64
    for off in c.pages[c.pages >= 0].tolist():
        for h in range(2):
            for side in range(2):
                for bit in (22, 23, 24, 31):    # of a scale: its mantissa, its exponent's lowest bits, its sign
                    other = c.arena.clone()
                    scale = other[off + strips + 8 * h + 4 * side:][:4].view(torch.int32)
                    scale ^= 1 << bit if bit < 31 else -(1 << 31)
                    with pytest.raises(AssertionError, match="no codes"):
                        assert_same_arena(c, other)
        other = c.arena.clone()
        other[off + strips + 16] ^= 0x80        # behind the page
        with pytest.raises(AssertionError, match="no codes"):
            assert_same_arena(c, other)
        other = c.arena.clone()
        other[off + 5] += 1
        with pytest.raises(AssertionError, match="codes"):
            assert_same_arena(c, other)


def test_codes_are_numbers():
    c = Cache([1], 1, 64, E4M3)
    off = int(c.pages[0, 0])
    c.arena[off: off + 3] = torch.tensor([0x00, 0x7F, 0x80], dtype=torch.uint8)
    other = c.arena.clone()
    other[off: off + 3] = torch.tensor([0x80, 0xFF, 0x00], dtype=torch.uint8)
    assert_same_arena(c, other)
