"""Comparison of two arenas of cache pages."""
import torch

from kv_plain import PAGE


def code_bytes(c):
    """Truth value of every byte of the arena: it is a code of a page in the table."""
    codes = torch.zeros(c.arena.numel(), dtype=torch.bool)
    for off in c.pages.flatten().tolist():
        if c.usable(off):
            codes[off: off + c.H * 2 * PAGE * c.D] = True
    return codes


def assert_same_arena(c, arena):
    """Codes as the numbers they stand for (-0 is +0, every NaN alike); all
    other bytes, the scales among them, bit for bit."""
    got = arena.cpu()
    differ, codes = got != c.arena, code_bytes(c)
    assert not (differ & ~codes).any(), f"bytes that are no codes: {(differ & ~codes).nonzero()[:8, 0].tolist()}"
    at = (differ & codes).nonzero()[:, 0]
    x, y = got[at].view(c.codes).float(), c.arena[at].view(c.codes).float()
    assert ((x == y) | (torch.isnan(x) & torch.isnan(y))).all(), f"codes: {at[:8].tolist()}"
