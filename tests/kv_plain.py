"""The 8-bit key/value cache in plain 64-bit arithmetic on the CPU, written
from its definition: what the tests compare the kernels with."""
import math

import torch

PAGE = 64
TOP = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def least_exp(amax, codes):
    """Least e >= -64 with amax <= top * 2^e."""
    e = -64
    if amax > 0:
        e = max(-64, math.floor(math.log2(amax / TOP[codes])) - 1)
        while amax > TOP[codes] * 2.0 ** e:
            e += 1
    return e


def nearest(x, codes):
    """float64 numbers in units of their scale -> codes (ties to even)."""
    if codes == torch.int8:
        return torch.nan_to_num(x, nan=0.0, posinf=127.0, neginf=-127.0).round().clamp(-127, 127).to(torch.int8)
    nan = torch.isnan(x)
    a = torch.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0).clamp(-448, 448)
    power = torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -6)))
    power = torch.where(torch.exp2(power) > a.abs().clamp(min=2.0 ** -6), power - 1, power)
    step = torch.exp2(power - 3)
    y = (a / step).round() * step
    return torch.where(nan, math.nan, y).float().to(torch.float8_e4m3fn)


def finite_max(x):
    x = x.abs()
    x = x[torch.isfinite(x)]
    return float(x.max()) if x.numel() else 0.0


class Cache:
    """Pages of H heads and D dimensions in an arena of bytes on the CPU."""

    def __init__(self, per, heads, dim, codes, stride=None, gap=96, fill=0, seed=0, base=0):
        self.H, self.D, self.codes = heads, dim, codes
        need = heads * 2 * PAGE * dim + 8 * heads
        self.pitch = (need + 31) // 32 * 32 + gap
        slots = sum(per) + 1
        gen = torch.Generator().manual_seed(seed)
        order = torch.randperm(slots, generator=gen).tolist()
        self.arena = torch.full((base + slots * self.pitch,), fill, dtype=torch.uint8)
        self.pages = torch.full((len(per), stride or max(per + [1])), -1, dtype=torch.int64)
        for b, n in enumerate(per):
            for j in range(n):
                self.pages[b, j] = base + order.pop() * self.pitch

    def head(self, off, h):
        """Views: key codes [64, D], value codes [64, D], scales [2]."""
        strip = 2 * PAGE * self.D
        c = self.arena[off + h * strip: off + (h + 1) * strip].view(self.codes)
        at = off + self.H * strip + 8 * h
        return c[: PAGE * self.D].view(PAGE, self.D), c[PAGE * self.D:].view(self.D, PAGE).t(), \
            self.arena[at: at + 8].view(torch.float32)

    def usable(self, off):
        off = int(off)
        return off >= 0 and off % 32 == 0 and off + self.H * (2 * PAGE * self.D + 8) <= self.arena.numel()

    def numbers(self, b, n, h):
        """Keys, values [n, D] in float64 and whether each token's page is usable."""
        k, v = torch.zeros(2, n, self.D, dtype=torch.float64).unbind()
        ok = torch.zeros(n, dtype=torch.bool)
        for j in range(-(-n // PAGE)):
            if not self.usable(self.pages[b, j]):
                continue
            kc, vc, sc = self.head(int(self.pages[b, j]), h)
            m = min(PAGE, n - j * PAGE)
            k[j * PAGE: j * PAGE + m] = kc[:m].double() * float(sc[0])
            v[j * PAGE: j * PAGE + m] = vc[:m].double() * float(sc[1])
            ok[j * PAGE: j * PAGE + m] = True
        return k, v, ok

    def append(self, b, n, k, v):
        """k, v: [t, H, D] behind the first n tokens of sequence b."""
        t = k.shape[0]
        for j in range(n // PAGE, -(-(n + t) // PAGE)):
            lo, hi = max(n, j * PAGE), min(n + t, (j + 1) * PAGE)
            old = lo - j * PAGE
            for h in range(self.H):
                kc, vc, sc = self.head(int(self.pages[b, j]), h)
                for i, (c, x) in enumerate(((kc, k), (vc, v))):
                    x = x[lo - n: hi - n, h].double()
                    e = least_exp(finite_max(x), self.codes)
                    if old:
                        was = round(math.log2(float(sc[i])))
                        if was > e:
                            e = was
                        c[:old] = nearest(c[:old].double() * 2.0 ** (was - e), self.codes)
                    c[old: hi - j * PAGE] = nearest(x * 2.0 ** -e, self.codes)
                    sc[i] = 2.0 ** e

    def fill_random(self, lens, seed, size=1.0, spread=0):
        """Random tokens; `spread`: page scales differ by up to 2^spread."""
        gen = torch.Generator().manual_seed(seed)
        for b, n in enumerate(lens):
            for j in range(-(-n // PAGE)):
                m = min(PAGE, n - j * PAGE)
                f = 2.0 ** int(torch.randint(0, spread + 1, (1,), generator=gen))
                x = torch.randn(2, m, self.H, self.D, generator=gen) * size
                self.append_page(b, j, x[0], x[1] * f)

    def append_page(self, b, j, k, v):
        for h in range(self.H):
            kc, vc, sc = self.head(int(self.pages[b, j]), h)
            for i, (c, x) in enumerate(((kc, k), (vc, v))):
                e = least_exp(finite_max(x[:, h]), self.codes)
                c[: x.shape[0]] = nearest(x[:, h].double() * 2.0 ** -e, self.codes)
                sc[i] = 2.0 ** e


def attend(cache, lens, q, group, counts, scale):
    """out, lse [N, H * G, ..], the weight [B, H, max len] and bounds on each
    of a 32-bit computation with float16 weights, all float64.

    The bounds: a score is a sum of D products rounded to 32 bits at each
    step (in any order), then scaled and shifted: D + 4 steps of 2^-24 of the
    sum of magnitudes, and the running maximum's exponent, |s| 2^-22; twice
    that (numerator and sum) is the relative error d of a weight.  float16
    rounds a weight by 2^-11.  The value product adds n + 4 steps of 2^-24."""
    N, HG, D = q.shape
    H = cache.H
    out, bound = torch.zeros(2, N, HG, D, dtype=torch.float64).unbind()
    lse, lbound = torch.full((N, HG), -math.inf, dtype=torch.float64), torch.zeros(N, HG, dtype=torch.float64)
    most = max(list(lens) + [1])
    weight, wbound = torch.zeros(2, len(lens), H, most, dtype=torch.float64).unbind()
    at = 0
    for b, n in enumerate(lens):
        t = counts[b]
        for h in range(H):
            k, v, ok = cache.numbers(b, n, h)
            for g in range(group):
                x = q[at: at + t, h * group + g].double()
                s = x @ k.t() * scale
                mag = x.abs() @ k.abs().t() * abs(scale)
                see = torch.arange(n)[None, :] <= (n - t + torch.arange(t))[:, None]
                see &= ok[None, :]
                s = s.masked_fill(~see, -math.inf)
                d = (mag * ((D + 4) * 2.0 ** -24) + mag * 2.0 ** -22 + 2.0 ** -22).masked_fill(~see, 0.0)
                if n == 0:
                    continue
                top = s.amax(-1, keepdim=True)
                e = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
                total = e.sum(-1, keepdim=True)
                p = e / torch.where(total == 0, 1.0, total)
                worst = d.amax(-1, keepdim=True)
                err = 2 * worst + 2.0 ** -22 + n * 2.0 ** -24
                hg = h * group + g
                out[at: at + t, hg] = p @ v
                bound[at: at + t, hg] = (p * (err + 2.0 ** -11 + (n + 4) * 2.0 ** -24) + see * 2.0 ** -38) @ v.abs()
                lse[at: at + t, hg] = (top + torch.log(total))[:, 0]
                lbound[at: at + t, hg] = (worst + n * 2.0 ** -24 + 2.0 ** -22)[:, 0] + lse[at: at + t, hg].abs().nan_to_num(posinf=0.0) * 2.0 ** -22
                weight[b, h, :n] += p.sum(0)
                wbound[b, h, :n] += (p * (err + t * 2.0 ** -24)).sum(0)
        at += t
    return out, bound, lse, lbound, weight, wbound


def evict(cache, lens, budget, weight, pos, sink, recent, next_pos):
    """Folds the cache in place; (weight, pos, lens) of what is kept, as lists."""
    old = cache.arena.clone()
    kept_w, kept_p = {}, {}
    for b, n in enumerate(lens):
        for h in range(cache.H):
            src = list(range(min(n, budget)))
            w, p = weight[b, h, :n].tolist(), pos[b, h, :n].tolist()
            if n > budget:
                border = int(next_pos[b]) - recent
                key = [math.inf if math.isnan(x) else x for x in w]
                best = sorted(range(n), key=lambda i: (0 if p[i] < sink or p[i] >= border else 1, -key[i], i))[:budget]
                kept = set(best)
                behind = iter(sorted(i for i in best if i >= budget))
                src = [i if i in kept else next(behind) for i in range(budget)]
                for j in range(budget // PAGE):
                    mine = src[j * PAGE: (j + 1) * PAGE]
                    if mine == list(range(j * PAGE, (j + 1) * PAGE)):
                        continue
                    was = Cache.__new__(Cache)
                    was.__dict__.update(cache.__dict__)
                    was.arena = old
                    x = torch.zeros(2, PAGE, cache.D, dtype=torch.float64)
                    for c, i in enumerate(mine):
                        kc, vc, sc = was.head(int(cache.pages[b, i // PAGE]), h)
                        x[0, c] = kc[i % PAGE].double() * float(sc[0])
                        x[1, c] = vc[i % PAGE].double() * float(sc[1])
                    kc, vc, sc = cache.head(int(cache.pages[b, j]), h)
                    for i, c in ((0, kc), (1, vc)):
                        e = least_exp(finite_max(x[i]), cache.codes)
                        c.copy_(nearest(x[i] * 2.0 ** -e, cache.codes))
                        sc[i] = 2.0 ** e
            kept_w[b, h], kept_p[b, h] = [w[i] for i in src], [p[i] for i in src]
    return kept_w, kept_p, [min(n, budget) for n in lens]
