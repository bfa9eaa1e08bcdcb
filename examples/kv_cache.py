"""A key/value cache that lives in an arena and is compacted with it.

Sequences generate tokens into cache pages, which are blocks of the arena next
to others.  Every step appends the new tokens' keys and values, attends over
the cache and adds up the weight each cached token receives.  When a sequence
outgrows its budget, the tokens of least weight are evicted and the pages
behind the budget are freed; the holes this leaves are closed by a compaction
of the arena, which remaps the page table like any other handles.

    python examples/kv_cache.py [--steps 800] [--batch 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import arena_compaction_amd as ac  # noqa: E402

PAGE = ac.KV_PAGE_TOKENS


class Arena:
    """Blocks of a device arena in address order; allocation is first fit."""

    def __init__(self, nbytes):
        self.bytes = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        self.blocks = {}  # offset -> size

    def alloc(self, size):
        size = (size + 31) // 32 * 32
        at = 0
        for off in sorted(self.blocks):
            if off - at >= size:
                break
            at = off + self.blocks[off]
        if at + size > self.bytes.numel():
            return None
        self.blocks[at] = size
        return at

    def free(self, off):
        del self.blocks[off]

    def compact(self, handles):
        """Slides every block down; returns the handles' new offsets and the
        fragmentation before and after."""
        table = sorted(self.blocks.items())
        off, size = (torch.tensor(x, dtype=torch.int64, device="cuda") for x in zip(*table))
        n, total = len(table), self.bytes.numel()
        ws = ac.workspace(n, total)
        new = torch.empty(n, dtype=torch.int64, device="cuda")
        off_out, size_out = torch.empty_like(off), torch.empty_like(size)
        out = torch.empty_like(handles)
        plan, after = ac.defrag_compact(off, size, None, total, self.bytes, ws, new_offset=new, handles=handles,
                                        h_out=out, offset_out=off_out, size_out=size_out)
        self.blocks = {int(o): s for o, (_, s) in zip(new.tolist(), table)}
        return out, plan.stats.frag_free_over_largest_minus_1, after.frag_free_over_largest_minus_1


def main(argv=None):
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=800)
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--heads", type=int, default=4)
    p.add_argument("--group", type=int, default=4)
    p.add_argument("--dim", type=int, default=128)
    p.add_argument("--budget", type=int, default=256)
    p.add_argument("--slack", type=int, default=128, help="tokens over the budget before an eviction")
    a = p.parse_args(argv)
    B, H, G, D, codes = a.batch, a.heads, a.group, a.dim, torch.float8_e4m3fn
    per = (a.budget + a.slack) // PAGE + 1
    size = ac.defrag_kv_page_bytes(H, D)
    gen = torch.Generator(device="cuda").manual_seed(0)
    arena = Arena(B * per * size * 2)
    pages = torch.full((B, per), -1, dtype=torch.int64, device="cuda")
    table = [[-1] * per for _ in range(B)]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    next_pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    places = per * PAGE
    weight, pos = torch.zeros(B, H, places, device="cuda"), torch.zeros(B, H, places, dtype=torch.int32, device="cuda")
    weight_out, pos_out = torch.zeros_like(weight), torch.zeros_like(pos)
    lens_out = torch.zeros_like(lens)
    held, others, report = [0] * B, [], []

    for step in range(a.steps):
        for b in range(B):  # a page for the new token, and other tenants between the pages
            if table[b][held[b] // PAGE] < 0:
                table[b][held[b] // PAGE] = arena.alloc(size)
                others.append(arena.alloc(4096 + 32 * step))
                pages.copy_(torch.tensor(table))
        qkv = torch.randn(B, (G + 2) * H, D, device="cuda", generator=gen).to(torch.bfloat16)
        q, k, v = qkv[:, : G * H], qkv[:, G * H: (G + 1) * H], qkv[:, (G + 1) * H:]
        ac.defrag_kv_append(arena.bytes, pages, lens, k, v, codes, weight=weight, pos=pos, first_pos=next_pos)
        lens += 1
        next_pos += 1
        held = [n + 1 for n in held]
        ac.defrag_kv_attend(arena.bytes, pages, lens, q, H, codes, weight=weight)
        if max(held) < a.budget + a.slack:
            continue
        ac.defrag_kv_evict(arena.bytes, pages, lens, a.budget, weight, pos, weight_out, pos_out, lens_out, D, codes,
                           sink=4, recent=32, next_pos=next_pos)
        weight, weight_out, pos, pos_out, lens, lens_out = weight_out, weight, pos_out, pos, lens_out, lens
        held = [min(n, a.budget) for n in held]
        for b in range(B):  # the pages behind the budget are free
            for j in range(-(-held[b] // PAGE), per):
                if table[b][j] >= 0:
                    arena.free(table[b][j])
                    table[b][j] = -1
        for off in others[::2]:
            arena.free(off)
        others = others[1::2]
        pages.copy_(torch.tensor(table))
        before = ac.defrag_kv_attend(arena.bytes, pages, lens, q, H, codes)
        live = pages >= 0
        handles = torch.cat([pages[live], torch.tensor(others, dtype=torch.int64, device="cuda")])
        moved, frag, frag_after = arena.compact(handles)
        n = int(live.sum())
        pages[live] = moved[:n]
        table, others = pages.tolist(), moved[n:].tolist()
        after = ac.defrag_kv_attend(arena.bytes, pages, lens, q, H, codes)
        assert torch.equal(before, after), "attention changed with the pages' place"
        report.append((step, frag, frag_after))
        print(f"step {step}: kept {held[0]} tokens a head, fragmentation {frag:.3f} -> {frag_after:.3f}", flush=True)
    print(f"{a.steps} steps of {B} sequences, {len(report)} evictions and compactions", flush=True)
    return report


if __name__ == "__main__":
    main()
