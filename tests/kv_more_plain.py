"""Rotation, attention with terms and the keeping of an accepted path in plain
64-bit arithmetic on the CPU, written from their definitions: what the tests
compare the kernels with."""
import math

import torch

from kv_plain import PAGE, Cache, finite_max, least_exp, nearest


def rotate(x, pos, freq, interleaved):
    """x [tokens, heads, D], pos [tokens], freq [pairs], all float64 inside."""
    x, R = x.double(), 2 * len(freq)
    out = x.clone()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        angle = (pos.double() * float(freq[i]))[:, None]
        c, s = torch.cos(angle), torch.sin(angle)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., a] * s + x[..., b] * c
    return out


def words_of(seen, words=None):
    """Truth values [tokens, n] as int64 words [tokens, words]."""
    n = seen.shape[1]
    words = words or -(-n // 64)
    full = torch.zeros(seen.shape[0], words * 64, dtype=torch.bool)
    full[:, :n] = seen
    return (full.view(-1, words, 64).long() << torch.arange(64)).sum(-1)


def attend(cache, lens, q, group, counts, scale, mask=None, cap=0.0, slopes=None, pos=None):
    """As kv_plain.attend, with the terms: mask is a list of truth values
    [count, count] by sequence, pos an int tensor [B, H, places] or None.

    The bounds, beyond those of kv_plain.attend for a score s and its products'
    magnitudes: the cap changes no error for the worse (its slope is at most 1)
    and adds 2^-21 of its result where that comes from a series, and some 2^-22
    of the cap where it comes from exponents (a power of at most 2^-23, of an
    exponent rounded by 2^-23 of itself, a sum and a quotient by 2^-23, times at
    most one cap), with the shift by the running maximum 2^-21 of it; the bias has a slope
    rounded twice and a product, 2^-21 of it; the sum and the running maximum's
    subtraction round by 2^-22 of the score and of the largest.  With d_j the
    error of s_j, that of a weight p_j is d_j + sum_k p_k d_k, to first order;
    a tenth more covers the rest, d being far below 1."""
    N, HG, D = q.shape
    H = cache.H
    out, bound = torch.zeros(2, N, HG, D, dtype=torch.float64).unbind()
    lse, lbound = torch.full((N, HG), -math.inf, dtype=torch.float64), torch.zeros(N, HG, dtype=torch.float64)
    most = max(list(lens) + [1])
    weight, wbound = torch.zeros(2, len(lens), H, most, dtype=torch.float64).unbind()
    at = 0
    for b, n in enumerate(lens):
        t = counts[b]
        had = n - t
        for h in range(H):
            k, v, ok = cache.numbers(b, n, h)
            # whether any score of these rows is high; all others may then go by exponents too
            raw = torch.einsum("tgd,nd->tgn", q[at: at + t, h * group: (h + 1) * group].double(), k) * scale
            high = bool(cap) and bool((raw.abs() >= 0.12 * cap).any())
            for g in range(group):
                hg = h * group + g
                if n == 0 or t == 0:
                    continue
                x = q[at: at + t, hg].double()
                s = x @ k.t() * scale
                mag = x.abs() @ k.abs().t() * abs(scale)
                place = torch.arange(n)[None, :]
                row = torch.arange(t)[:, None]
                if mask is None:
                    see = place <= had + row
                else:
                    see = (place < had).expand(t, n).clone()
                    for j in range(max(0, -had), t):
                        see[:, had + j] = mask[b][:, j]
                see = see & ok[None, :]
                d = mag * ((D + 4) * 2.0 ** -24) + mag * 2.0 ** -22 + 2.0 ** -22
                if cap:
                    s = cap * torch.tanh(s / cap)
                    d = d + s.abs() * 2.0 ** -21 + cap * 2.0 ** -21 * high
                if slopes is not None:
                    where = pos[b, h, :n].double() if pos is not None else torch.arange(n).double()
                    mine = had + torch.arange(t)
                    own = torch.where(mine >= 0, where[mine.clamp(min=0)], mine.double())
                    bias = float(slopes[hg]) * (where[None, :] - own[:, None])
                    s = s + bias
                    d = d + bias.abs() * 2.0 ** -21
                s = s.masked_fill(~see, -math.inf)
                top = s.amax(-1, keepdim=True)
                ts = torch.where(torch.isinf(top), 0.0, top)
                d = (d + (s.masked_fill(~see, 0.0).abs() + ts.abs()) * 2.0 ** -22).masked_fill(~see, 0.0)
                e = torch.exp(s - ts)
                total = e.sum(-1, keepdim=True)
                p = e / torch.where(total == 0, 1.0, total)
                mean = (p * d).sum(-1, keepdim=True)
                err = 1.1 * (d + mean) + 2.0 ** -22 + n * 2.0 ** -24
                out[at: at + t, hg] = p @ v
                bound[at: at + t, hg] = (p * (err + 2.0 ** -11 + (n + 4) * 2.0 ** -24) + see * 2.0 ** -38) @ v.abs()
                lse[at: at + t, hg] = (top + torch.log(total))[:, 0]
                lbound[at: at + t, hg] = (1.1 * mean + n * 2.0 ** -24 + 2.0 ** -22)[:, 0] + \
                    lse[at: at + t, hg].abs().nan_to_num(posinf=0.0) * 2.0 ** -22
                weight[b, h, :n] += p.sum(0)
                wbound[b, h, :n] += (p * (err + t * 2.0 ** -24)).sum(0)
        at += t
    return out, bound, lse, lbound, weight, wbound


def accept(cache, lens, counts, paths, weight=None, pos=None):
    """Keeps the paths in place (arena, weight and pos [B, H, places]); the new lengths."""
    out = []
    for b, n in enumerate(lens):
        had, path = n - counts[b], paths[b]
        out.append(had + len(path))
        take = [had + i for i in path]
        for h in range(cache.H):
            for j in range(had // PAGE, -(-(had + len(path)) // PAGE)):
                lo, hi = max(had, j * PAGE), min(had + len(path), (j + 1) * PAGE)
                mine = take[lo - had: hi - had]
                if mine == list(range(lo, hi)):
                    continue
                dst = cache.head(int(cache.pages[b, j]), h)
                come = [cache.head(int(cache.pages[b, i // PAGE]), h) for i in mine]
                far = [i // PAGE != j for i in mine]
                for w in (0, 1):
                    rows = [c[w][i % PAGE].clone() for c, i in zip(come, mine)]
                    exps = [round(math.log2(float(c[2][w]))) for c in come]
                    was = e = round(math.log2(float(dst[2][w])))
                    if any(far):
                        e = max(least_exp(finite_max(r.double() * 2.0 ** x), cache.codes) for r, x, f in zip(rows, exps, far) if f)
                        if lo > j * PAGE or not all(far):
                            e = max(e, was)
                    c, old = dst[w], lo - j * PAGE
                    if e != was:
                        c[:old] = nearest(c[:old].double() * 2.0 ** (was - e), cache.codes)
                    for i, (r, x) in enumerate(zip(rows, exps)):
                        c[old + i] = r if x == e else nearest(r.double() * 2.0 ** (x - e), cache.codes)
                    dst[2][w] = 2.0 ** e
            for plane in (weight, pos):
                if plane is not None:
                    moved = [plane[b, h, i].clone() for i in take]
                    for i, x in enumerate(moved):
                        plane[b, h, had + i] = x
    return out


def tree(t, width, gen):
    """Parents of t drafted tokens (-1: the last cached one) and who sees whom."""
    up = [max(-1, i - 1 - int(torch.randint(0, width, (1,), generator=gen))) for i in range(t)]
    seen, depth = torch.zeros(t, t, dtype=torch.bool), []
    for i, p in enumerate(up):
        if p >= 0:
            seen[i] = seen[p]
        seen[i, i] = True
        depth.append(0 if p < 0 else depth[p] + 1)
    return up, seen, depth


def walk(up, gen):
    """A path down the tree until there is no child."""
    at, path = -1, []
    while True:
        below = [i for i, p in enumerate(up) if p == at]
        if not below:
            return path
        at = below[int(torch.randint(0, len(below), (1,), generator=gen))]
        path.append(at)


__all__ = ["Cache", "PAGE", "accept", "attend", "rotate", "tree", "walk", "words_of"]
