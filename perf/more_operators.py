"""More operators of the 8-bit key/value cache in the arena, as cases to measure.

What a server does with the cache's pages (64 tokens of every head in 8 bits,
one power-of-two scale for the keys and one for the values of each (page,
head), blocks of the arena) beside plain appending and causal attention:

  rotary  appends new keys, rotated by their positions on the way, and values;
          the queries of the same tokens are rotated in the same call;
  attend  attention whose new tokens see one another by a bit mask (drafted
          trees, packed documents, prefixes read both ways), whose scores are
          capped by a tanh, or get a bias that grows with the distance;
  accept  keeps the accepted path of a tree of drafted tokens and closes the
          holes that the rejected ones leave.

Layout of a page of H heads and D dimensions: for every head a strip of
64 x D key codes (token by token) and then D x 64 value codes (dimension by
dimension); behind the strips H pairs of float32 scales (key, value).

`run` computes each operator in elementary torch operations, or calls the
framework where `own` is true.  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

PAGE = 64          # tokens of a page
EMIN = -64         # least exponent of a scale
BASE = 10000.0     # of the rotation's frequencies
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    def rotary(name, **c):
        return {"name": name, "op": "rotary", "tlo": 1.0, "lo": 1.0, "tree": 0, **c}

    def attend(name, **c):
        return {"name": name, "op": "attend", "tlo": 1.0, "lo": 1.0, "mask": "", "tree": 0, "cap": 0.0, "slopes": False,
                "pos": False, "scored": False, **c}

    def accept(name, **c):
        return {"name": name, "op": "accept", "tlo": 1.0, "lo": 1.0, **c}

    return [
        # a serving step: one new token of every sequence of a batch
        rotary("rotary step", B=128, past=4000, lo=0.2, T=1, H=8, G=4, D=128, R=128, pairs="half", codes="e4m3", dtype="bf16"),
        # prompts into the cache
        rotary("rotary prompt", B=4, past=100, T=4097, tlo=0.6, H=8, G=4, D=128, R=128, pairs="half", codes="int8", dtype="fp16"),
        # trees of drafted tokens, whose positions are their depths; a part of the dimensions is rotated
        rotary("rotary drafts", B=48, past=8000, lo=0.3, T=24, tree=4, H=4, G=7, D=96, R=64, pairs="next", codes="e4m3", dtype="bf16"),
        # one short conversation, a small tree: launches and latency
        attend("tree one", B=1, past=300, T=7, mask="tree", tree=3, H=2, G=4, D=64, codes="e4m3", dtype="bf16"),
        # trees verified over a ragged batch
        attend("tree batch", B=16, past=10000, lo=0.5, T=25, tlo=0.6, mask="tree", tree=5, H=8, G=4, D=128, codes="e4m3", dtype="bf16"),
        # two long documents, a tree each
        attend("tree long", B=2, past=131000, lo=0.9, T=12, mask="tree", tree=4, H=8, G=8, D=128, codes="int8", dtype="fp16"),
        # a serving step of a model with capped scores and wide heads
        attend("cap step", B=64, past=4096, lo=0.1, T=1, cap=50.0, H=4, G=2, D=256, codes="e4m3", dtype="bf16"),
        # a serving step with a distance bias over a cache that has been evicted from, whose weights are added up
        attend("distance scored", B=48, past=8000, lo=0.3, T=1, slopes=True, pos=True, scored=True, H=8, G=4, D=128, codes="e4m3", dtype="bf16"),
        # chunks of prompts behind a cached prefix, capped scores
        attend("cap chunk", B=3, past=2048, lo=0.3, T=2000, tlo=0.5, cap=30.0, H=8, G=4, D=128, codes="e4m3", dtype="bf16"),
        # several documents packed into one prompt, with a distance bias
        attend("distance documents", B=1, past=0, T=8200, mask="documents", slopes=True, H=4, G=8, D=64, codes="int8", dtype="fp16"),
        # the path of one small tree: launches and latency
        accept("accept one", B=1, past=300, T=7, tree=3, H=2, D=64, codes="e4m3"),
        # trees of a large batch after their verification
        accept("accept batch", B=256, past=4000, lo=0.2, T=40, tlo=0.5, tree=2, H=8, D=128, codes="int8"),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["rotary", "attend", "attend", "attend", "accept"])
    H, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 96, 128, 192, 256])
    c = {"op": op, "H": H, "D": D, "codes": rng.choice(["e4m3", "int8"]), "lo": rng.choice([1.0, 0.7, 0.2]), "tlo": rng.choice([1.0, 0.5]),
         "tree": rng.choice([1, 2, 4, 9])}
    if op == "accept":
        c["T"], c["past"] = log(1, 200), rng.choice([0, log(1, 8192)])
        c["B"] = log(1, max(1, min(256, (1 << 27) // ((c["past"] + 256) * H * D))))
        return c
    c["dtype"], c["G"] = rng.choice(["bf16", "fp16"]), rng.choice([1, 2, 3, 4, 6, 8, 16])
    if op == "rotary":
        c["T"], c["past"] = rng.choice([1, log(2, 64), log(65, 4097)]), rng.choice([0, log(1, 4097)])
        c["tree"] = c["tree"] if c["T"] <= 64 and rng.random() < 0.5 else 0
        c["R"], c["pairs"] = rng.choice([D, D, D // 2, 32]), rng.choice(["half", "next"])
        c["B"] = log(1, max(1, min(128, (1 << 26) // ((c["T"] + c["past"]) * H * D), (1 << 28) // (c["T"] * H * c["G"] * D))))
        return c
    c["mask"] = rng.choice(["", "tree", "tree", "documents", "prefix"])
    c["cap"] = rng.choice([0.0, 5.0, 30.0, 50.0])
    c["slopes"] = rng.random() < (0.4 if c["mask"] or c["cap"] else 1.0)
    c["pos"], c["scored"] = c["slopes"] and rng.random() < 0.5, rng.random() < 0.3
    if rng.random() < 0.6:  # few new tokens over a cache
        c["T"], c["past"] = rng.choice([1, 3, 7, 16, 33]), log(1, 65536)
        c["B"] = log(1, max(1, min(128, (1 << 27) // ((c["past"] + 64) * H * D), int(5e10 / (c["T"] * (c["past"] + c["T"]) * H * c["G"] * D)))))
    else:                   # many of them
        c["T"], c["past"] = log(34, 2049), rng.choice([0, log(1, 8192)])
        c["T"] = max(34, min(c["T"], int(5e10 / ((c["T"] + c["past"]) * H * c["G"] * D))))
        pairs = c["T"] * (c["T"] + c["past"]) * H * c["G"]
        c["B"] = log(1, max(1, min(8, int(5e10 / (pairs * D)))))
    return c


def spread(top, lo, n, least):
    """n lengths from top down to lo * top."""
    return [max(least, round(top * (1 - (1 - lo) * i / max(1, n - 1)))) for i in range(n)]


def lengths(case):
    """(tokens cached before the call, new tokens) of every sequence, before the seed deals them out."""
    return spread(case["past"], case["lo"], case["B"], 0), spread(case["T"], case["tlo"], case["B"], 1)


def documents(n):
    """Lengths of the documents that n new tokens hold: about five, no two alike."""
    cuts = sorted({n * i * (i + 1) // 30 for i in range(1, 5)} | {0, n})
    return [b - a for a, b in zip(cuts, cuts[1:])]


def seen_pairs(case, p, t):
    """(new token, cached token) pairs that a sequence's mask leaves; of a tree, itself and the one before at least."""
    m = case["mask"]
    if m == "tree":
        return t * p + 2 * t - 1
    if m == "documents":
        return t * p + sum(n * (n + 1) // 2 for n in documents(t))
    return t * p + t * (t + 1) // 2 + (t // 3 * (t // 3 - 1) // 2 if m == "prefix" else 0)


def work(case):
    H, D = case["H"], case["D"]
    past, new = lengths(case)
    N = sum(new)
    if case["op"] == "rotary":  # keys, values and queries in 16 bits in, codes and queries out
        return {"bytes": N * H * D * 2 * (2 + 1) + N * H * case["G"] * D * 4, "flops": 3 * N * H * (1 + case["G"]) * case["R"] + 2 * N * H * D}
    if case["op"] == "accept":  # a path is about as long as the tree is deep; half of it moves
        moved = sum(min(t, 1 + round(math.log2(t) * 2 / case["tree"])) for t in new) * H / 2
        return {"bytes": moved * (2 * D + 8) * 2 + case["B"] * 8, "flops": 2 * moved * D}
    rows = N * H * case["G"]
    held = sum(p + t for p, t in zip(past, new)) * H
    seen = sum(seen_pairs(case, p, t) for p, t in zip(past, new)) * H * case["G"]
    plane = held * (4 * case["pos"] + 8 * case["scored"])
    return {"bytes": held * 2 * D + rows * D * 2 * 2 + rows * 4 + plane, "flops": 4 * D * seen}


def limits(codes):
    """(largest code value, its exponent k with value = m * 2^k and m in [0.5, 1), that m)."""
    return (448.0, 9, 0.875) if codes == "e4m3" else (127.0, 7, 127 / 128)


def exponent(amax, codes):
    """Least e with amax <= largest code * 2^e, at least EMIN."""
    _, k, top = limits(codes)
    m, e = torch.frexp(amax)
    e = e - k + (m > top).to(e.dtype)
    return torch.where(amax > 0, e, EMIN).clamp(min=EMIN)


def to_codes(x, codes):
    """Values in units of their scale, to the nearest code (ties to even)."""
    top = limits(codes)[0]
    if codes == "int8":
        return torch.nan_to_num(x, nan=0.0, posinf=top, neginf=-top).round().clamp(-top, top).to(torch.int8)
    step = torch.exp2(torch.frexp(x.abs().clamp(min=2.0**-6))[1].to(x.dtype) - 4)
    return ((x / step).round() * step).clamp(-top, top).to(torch.float8_e4m3fn)


def finite_max(x, dim):
    return torch.nan_to_num(x.abs(), nan=0.0, posinf=0.0).amax(dim)


def strips(state, rows):
    """Views of pages: key codes [.., H, 64, D], value codes [.., H, D, 64], scales [.., H, 2]."""
    H, D = state["case"]["H"], state["case"]["D"]
    codes = rows[..., : H * 2 * PAGE * D].view(CODES[state["case"]["codes"]]).unflatten(-1, (H, 2, PAGE * D))
    scales = rows[..., H * 2 * PAGE * D : H * 2 * PAGE * D + 8 * H].view(torch.float32).unflatten(-1, (H, 2))
    return codes[..., 0, :].unflatten(-1, (PAGE, D)), codes[..., 1, :].unflatten(-1, (D, PAGE)), scales


def parents(t, width, rng):
    """A tree of t drafted tokens: each hangs from one of the `width` before it (1: a chain); -1 stands for the last cached token."""
    return [max(-1, i - 1 - int(torch.randint(0, width, (1,), generator=rng))) for i in range(t)]


def words_of(seen):
    """Truth values [n, t] as bits of 64-bit words [n, ceil(t / 64)]."""
    n, t = seen.shape
    full = torch.nn.functional.pad(seen, (0, -t % 64)).unflatten(1, (-1, 64))
    return (full.long() << torch.arange(64, device=seen.device)).sum(-1)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    B, H, D, codes, op = case["B"], case["H"], case["D"], case["codes"], case["op"]
    past, new = lengths(case)
    deal = torch.randperm(B, generator=host).tolist()
    past, new = [past[i] for i in deal], [new[i] for i in deal]
    total = [p + n for p, n in zip(past, new)]
    held = past if op == "rotary" else total
    per = [-(-n // PAGE) for n in total]
    stride = max(per) + 1
    pitch = H * 2 * PAGE * D + (8 * H + 31) // 32 * 32 + 32 * 3  # other small blocks lie between the pages
    slots = sum(per) + 3
    # the pages lie in the arena in no order
    order = torch.randperm(slots, generator=host)[: sum(per)]
    pages = torch.full((B, stride), -1, dtype=torch.int64)
    pages[torch.arange(stride)[None, :] < torch.tensor(per)[:, None]] = order * pitch
    arena = torch.zeros(slots, pitch, dtype=torch.uint8, device=dev)
    if op == "attend":
        arena.fill_(0x7F)  # what is not the cache's own is no number
    state = {"case": dict(case), "arena": arena, "pages": pages.to(dev), "past": past, "new": new}

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    state["lens"], state["max_len"], state["max_new"] = ints(held), max(held), max(new)
    # every dimension has its own size, as keys and values of a model have
    size = [torch.exp(0.7 * torch.randn(H, 1, D, device=dev, generator=gen)) for _ in range(2)]
    at, count = order.to(dev), torch.cat([(torch.tensor(n) - torch.arange(k) * PAGE).clamp(0, PAGE) for n, k in zip(held, per)]).to(dev)
    group = max(1, (1 << 27) // (H * PAGE * D))
    for i in range(0, len(at), group):
        rows = torch.zeros(len(at[i : i + group]), pitch, dtype=torch.uint8, device=dev)
        kc, vc, sc = strips(state, rows)
        there = torch.arange(PAGE, device=dev) < count[i : i + group, None]
        for w, c in ((0, kc), (1, vc)):
            x = torch.randn(len(rows), H, PAGE, D, device=dev, generator=gen) * size[w] * there[:, None, :, None]
            e = exponent(x.abs().amax((-1, -2)), codes)
            sc[..., w] = torch.exp2(e.float())
            y = to_codes(x * torch.exp2(-e.float())[..., None, None], codes)
            c.copy_(y if w == 0 else y.transpose(-1, -2))
        if op == "attend" and codes == "e4m3":  # tokens behind the last one: left over, no numbers
            kc.view(torch.uint8).masked_fill_(~there[:, None, :, None], 0x7F)
            vc.view(torch.uint8).masked_fill_(~there[:, None, None, :], 0x7F)
        arena[at[i : i + group]] = rows
    starts = torch.tensor([0] + new).cumsum(0)
    state["starts"] = starts.to(torch.int32).to(dev)
    N = int(starts[-1])
    state["of"] = torch.repeat_interleave(torch.arange(B), torch.tensor(new)).to(dev)
    state["nth"] = torch.arange(N, device=dev) - starts.to(dev)[state["of"]]
    hang = [parents(t, case["tree"], host) for t in new] if case["tree"] and (op != "attend" or case["mask"] == "tree") else None
    depth = None
    if hang:
        depth = []
        for up in hang:
            d = []
            for p in up:
                d.append(0 if p < 0 else d[p] + 1)
            depth += d
        depth = torch.tensor(depth)
    places = -(-max(total) // PAGE) * PAGE
    next_pos = [p + 7 for p in past]  # the cache has lost some tokens
    if op == "rotary":
        # queries, keys and values as slices of one fused projection
        G, R = case["G"], case["R"]
        qkv = torch.randn(N, (G + 2) * H, D, device=dev, generator=gen).to(FLOATS[case["dtype"]])
        qkv[:, G * H :].unflatten(1, (2, H)).mul_(torch.stack([s[:, 0] for s in size]).to(qkv.dtype))
        state["q"], state["k"], state["v"] = qkv[:, : G * H], qkv[:, G * H : (G + 1) * H], qkv[:, (G + 1) * H :]
        state["freq"] = BASE ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)
        state["weight"] = torch.ones(B, H, places, device=dev)
        state["pos"] = torch.full((B, H, places), -1, dtype=torch.int32, device=dev)
        far = 1 + (1 << 17) * (case["T"] == 1)  # steps also come late in long documents
        state["first_pos"] = ints([p + i * far // B for i, p in enumerate(next_pos)])
        if hang:
            state["token_pos"] = state["first_pos"][state["of"]] + depth.to(dev, torch.int32)
    elif op == "attend":
        G = case["G"]
        qkv = (2 * torch.randn(N, (G + 2) * H * D, device=dev, generator=gen)).to(FLOATS[case["dtype"]])
        state["q"] = qkv.view(N, (G + 2) * H, D)[:, : G * H]
        state["scale"] = D**-0.5
        state["lse"] = torch.empty(N, G * H, device=dev)
        t = max(new)
        line, nth = torch.arange(t, device=dev), state["nth"]
        count_of = torch.tensor(new, device=dev)[state["of"]]
        if hang:
            seen = torch.zeros(N, t, dtype=torch.bool)
            for s, up in zip(starts.tolist(), hang):
                for i, p in enumerate(up):
                    if p >= 0:
                        seen[s + i] = seen[s + p]
                    seen[s + i, i] = True
            state["mask"] = words_of(seen.to(dev))
        elif case["mask"] == "documents":
            first = torch.zeros(N, dtype=torch.long)
            for s, n in zip(starts.tolist(), new):
                lens = documents(n)
                lens = [lens[i] for i in torch.randperm(len(lens), generator=host).tolist()]
                first[s : s + n] = torch.repeat_interleave(torch.tensor([0] + lens[:-1]).cumsum(0), torch.tensor(lens))
            state["mask"] = words_of((line <= nth[:, None]) & (line >= first.to(dev)[:, None]))
        elif case["mask"] == "prefix":
            state["mask"] = words_of((line <= nth[:, None]) | ((line < (count_of // 3)[:, None]) & (nth < count_of // 3)[:, None]))
        if case["slopes"]:
            state["slopes"] = torch.exp2(-8.0 * (torch.arange(G * H, device=dev) + 1) / (G * H)).float()
        if case["pos"]:
            # earlier evictions have left gaps, other ones for each head, and put the first half out of order
            line = torch.arange(places, device=dev)
            key = torch.rand(B, H, places, device=dev, generator=gen)
            mixed = torch.where(line < min(past) // 2, key, 1.0 + line).argsort(-1)
            pos = (mixed * 2 + (key < 0.5)).to(torch.int32)
            fresh = (line - ints(past)[:, None]).clamp(min=0, max=t - 1)
            nums = torch.arange(N, device=dev) - starts.to(dev)[state["of"]] if depth is None else depth.to(dev)
            all_new = nums[(starts.to(dev)[:-1, None] + fresh).clamp(max=N - 1)]
            mine = (line >= ints(past)[:, None])[:, None, :]
            state["pos"] = torch.where(mine, (2 * ints(past)[:, None] + all_new).to(torch.int32)[:, None, :], pos).contiguous()
        if case["scored"]:
            state["weight"] = torch.rand(B, H, places, device=dev, generator=gen)
    else:
        # the path that verification took: down the tree until no child is right
        path, kept = torch.zeros(B, max(new), dtype=torch.int32), []
        for b, up in enumerate(hang):
            at_, k = -1, 0
            while True:
                below = [i for i, p in enumerate(up) if p == at_]
                if not below or float(torch.rand(1, generator=host)) < 0.1:
                    break
                at_ = below[int(torch.randint(0, len(below), (1,), generator=host))]
                path[b, k] = at_
                k += 1
            kept.append(k)
        state["path"], state["kept"] = path.to(dev), ints(kept)
        state["weight"] = torch.rand(B, H, places, device=dev, generator=gen)
        state["pos"] = torch.arange(places, dtype=torch.int32, device=dev).expand(B, H, places).contiguous()
        for b in range(B):
            d = depth[int(starts[b]) : int(starts[b + 1])].to(dev, torch.int32)
            state["pos"][b, :, past[b] : total[b]] = past[b] + d
        state["lens_out"] = torch.zeros(B, dtype=torch.int32, device=dev)
    return state


def numbers(state, last):
    """Keys and values [B, H, tokens, D] of the first `last` pages as float32, nothing in place of what is not there."""
    pages = state["pages"][:, :last]
    k, v, s = strips(state, state["arena"][pages.clamp(min=0) // state["arena"].shape[1]])
    k, v = k.float() * s[..., 0, None, None], v.float().transpose(-1, -2) * s[..., 1, None, None]
    live = torch.arange(k.shape[1] * PAGE, device=k.device) < state["lens"][:, None]
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))
    return (torch.where(live[:, None, :, None], x, 0.0) for x in (k, v))


def run_attend(state):
    c = state["case"]
    H, G, D, B = c["H"], c["G"], c["D"], c["B"]
    k, v = numbers(state, -(-state["max_len"] // PAGE))
    T, L, dev = state["max_new"], k.shape[2], k.device
    q = torch.zeros(B, T, H, G, D, device=dev)
    q[state["of"], state["nth"]] = state["q"].float().unflatten(1, (H, G))
    s = (q.permute(0, 2, 3, 1, 4).reshape(B, H, G * T, D) @ k.transpose(-1, -2).contiguous() * state["scale"]).view(B, H, G, T, L)
    if c["cap"]:
        s = torch.tanh(s / c["cap"]) * c["cap"]
    had = (state["lens"] - (state["starts"][1:] - state["starts"][:-1])).long()
    line, row = torch.arange(L, device=dev), torch.arange(T, device=dev)
    if c["slopes"]:
        at = (had[:, None] + row).clamp(max=L - 1)
        if c["pos"]:
            pos = state["pos"][:, :, :L].long()
            far = pos[:, :, None, :] - pos.gather(-1, at[:, None].expand(B, H, T))[..., None]
        else:
            far = (line - at[..., None])[:, None]
        s += state["slopes"].view(H, G, 1, 1) * far.float()[:, :, None]
    nth = line - had[:, None]  # of each place among the new tokens
    if c["mask"]:
        words = torch.zeros(B, T, state["mask"].shape[1], dtype=torch.int64, device=dev)
        words[state["of"], state["nth"]] = state["mask"]
        at = nth.clamp(0, T - 1)[:, None].expand(B, T, L)
        seen = (nth < 0)[:, None] | ((words.gather(-1, at // 64) >> at % 64) & 1).bool()
    else:
        seen = nth[:, None] <= row[:, None]
    seen = seen & (line < state["lens"][:, None])[:, None]
    real = row < (state["lens"] - had)[:, None]
    s = s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total == 0, 1.0, total)
    o = (p.view(B, H, G * T, L) @ v).view(B, H, G, T, D).permute(0, 3, 1, 2, 4)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2)
    out = {"out": o[state["of"], state["nth"]].flatten(1, 2).to(state["q"].dtype), "lse": lse[state["of"], state["nth"]].flatten(1, 2)}
    if c["scored"]:
        n = min(L, state["weight"].shape[2])
        state["weight"][:, :, :n] += (p * real[:, None, None, :, None]).sum((2, 3))[:, :, :n]
        out["weight"] = state["weight"]
    return out


def whole(state):
    """Codes and scales of all pages, as the values they stand for: views of the arena."""
    H, D = state["case"]["H"], state["case"]["D"]
    n = H * 2 * PAGE * D
    return {"codes": state["arena"][:, :n].view(CODES[state["case"]["codes"]]), "scales": state["arena"][:, n : n + 8 * H].view(torch.float32)}


def put(state, rows, there, keys, values, scales):
    """Writes pages back: [B, pages, H, 64, D] codes of both and [B, pages, H, 2] scales."""
    at = rows[there]
    page = state["arena"][at]
    k, v, s = strips(state, page)
    k.copy_(keys[there])
    v.copy_(values[there].transpose(-1, -2))
    s.copy_(scales[there])
    state["arena"][at] = page


def touched(state, had):
    """Rows of the arena [B, pages] of the pages from the one that holds place `had` on, and the number of each place [B, pages, 64] among the new tokens."""
    dev = had.device
    nth = (had // PAGE)[:, None] + torch.arange(-(-(state["max_new"] + PAGE - 1) // PAGE), device=dev)
    rows = state["pages"].gather(1, nth.clamp(max=state["pages"].shape[1] - 1)).clamp(min=0) // state["arena"].shape[1]
    return rows, nth[..., None] * PAGE + torch.arange(PAGE, device=dev) - had[:, None, None]


def rotated(x, angle, pairs):
    """[tokens, heads, D] in 64 bits (angles of far positions, numbers next to a code's border)."""
    x, half = x.double(), angle.shape[-1]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = (x[..., :half], x[..., half : 2 * half]) if pairs == "half" else (x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2])
    y = (a * c - b * s, a * s + b * c)
    y = torch.cat(y, -1) if pairs == "half" else torch.stack(y, -1).flatten(-2)
    return torch.cat((y, x[..., 2 * half :]), -1)


def run_rotary(state):
    c = state["case"]
    codes = c["codes"]
    lens, N = state["lens"].long(), len(state["of"])
    pos = state.get("token_pos")
    if pos is None:
        pos = state["first_pos"][state["of"]] + state["nth"].int()
    angle = pos.double()[:, None] * state["freq"]
    q = rotated(state["q"], angle, c["pairs"]).to(state["q"].dtype)
    keys = rotated(state["k"], angle, c["pairs"])
    rows, token = touched(state, lens)
    count = (state["starts"][1:] - state["starts"][:-1]).long()[:, None, None]
    fresh, old = (token >= 0) & (token < count), token < 0
    src = (state["starts"][:-1].long()[:, None, None] + token).clamp(0, N - 1)
    k, v, s = strips(state, state["arena"][rows])
    sides, scales = [], []
    for was, x, w in ((k, keys, 0), (v.transpose(-1, -2), state["v"].double(), 1)):
        x = x[src].permute(0, 1, 3, 2, 4)
        e = exponent(finite_max(torch.where(fresh[:, :, None, :, None], x, 0.0), (-1, -2)), codes)
        before = torch.frexp(s[..., w])[1] - 1
        e = torch.where(old[..., :1], torch.maximum(e, before), e)
        again = to_codes(was.float() * torch.exp2((before - e).float())[..., None, None], codes)
        fine = to_codes(x * torch.exp2(-e.double())[..., None, None], codes)
        both = torch.where(fresh[:, :, None, :, None], fine.float(), torch.where(old[:, :, None, :, None], again.float(), was.float()))
        sides.append(both.to(CODES[codes]))
        scales.append(torch.exp2(e.float()))
    put(state, rows, fresh.any(-1), sides[0], sides[1], torch.stack(scales, -1))
    at = lens[state["of"]] + state["nth"]
    state["weight"][state["of"], :, at] = 0.0
    state["pos"][state["of"], :, at] = pos[:, None]
    return {**whole(state), "q": q, "weight": state["weight"], "pos": state["pos"]}


def run_accept(state):
    c = state["case"]
    codes, D, dev = c["codes"], c["D"], state["pages"].device
    count = (state["starts"][1:] - state["starts"][:-1]).long()
    had, kept = state["lens"].long() - count, state["kept"].long()
    rows, token = touched(state, had)
    B, P = rows.shape
    mine = (token >= 0) & (token < kept[:, None, None])
    # the place, counted from the first of these pages, that each place takes its token from
    here = torch.arange(P * PAGE, device=dev).view(P, PAGE)
    take = state["path"].long().gather(1, token.clamp(0, state["path"].shape[1] - 1).flatten(1)).view_as(token) + (had % PAGE)[:, None, None]
    src = torch.where(mine, take, here)
    far = mine & (src // PAGE != here // PAGE)
    k, v, s = strips(state, state["arena"][rows])
    own_tokens = ((token < 0) | (mine & ~far)).any(-1)[..., None]
    sides, scales = [], []
    for was, w in ((k, 0), (v.transpose(-1, -2), 1)):
        flat = was.transpose(2, 3).flatten(1, 2)                                # [B, places, H, D]
        moved = flat.float().gather(1, src.flatten(1)[..., None, None].expand(-1, -1, c["H"], D)).unflatten(1, (P, PAGE)).transpose(2, 3)
        e0 = torch.frexp(s[..., w])[1] - 1                                      # [B, P, H]
        e_src = e0.transpose(1, 2).gather(2, (src // PAGE).flatten(1)[:, None].expand(-1, c["H"], -1)).unflatten(2, (P, PAGE)).transpose(1, 2)
        value = moved * torch.exp2(e_src.float())[..., None]
        e = exponent(finite_max(torch.where(far[:, :, None, :, None], value, 0.0), (-1, -2)), codes)
        e = torch.where(own_tokens, torch.maximum(e, e0), e)
        e = torch.where(far.any(-1)[..., None], e, e0)
        fit = to_codes(moved * torch.exp2((e_src - e[..., None]).float())[..., None], codes)
        same = e_src == e[..., None]                                            # as they are: no rounding, and a NaN stays
        fit = torch.where(same[..., None], moved, fit.float())
        holds = (token < 0) | mine
        sides.append(torch.where(holds[:, :, None, :, None], fit, was.float()).to(CODES[codes]))
        scales.append(torch.exp2(e.float()))
    put(state, rows, (mine & (src != here)).any(-1), sides[0], sides[1], torch.stack(scales, -1))
    T = state["path"].shape[1]
    line = torch.arange(T, device=dev)
    at, from_ = had[:, None] + line, had[:, None] + state["path"].long()
    on = line < kept[:, None]
    for name in ("weight", "pos"):
        plane = state[name]
        last = plane.shape[2] - 1
        old = plane.clone()
        i, j = (x.clamp(max=last)[:, None].expand(B, c["H"], T) for x in (at, from_))
        line_ = torch.zeros_like(plane, dtype=torch.bool).scatter_(-1, i, on[:, None].expand(B, c["H"], T))
        plane.copy_(torch.where(line_, old.scatter(-1, i, old.gather(-1, j)), old))
    state["lens_out"].copy_(had + kept)
    return {**whole(state), "weight": state["weight"], "pos": state["pos"], "lens": state["lens_out"]}


def run(state):
    c = state["case"]
    if not own:
        return {"rotary": run_rotary, "attend": run_attend, "accept": run_accept}[c["op"]](state)
    import arena_compaction_amd as ac
    arena, codes = state["arena"].view(-1), CODES[c["codes"]]
    if c["op"] == "rotary":
        q = ac.defrag_kv_append_rotary(arena, state["pages"], state["lens"], state["k"], state["v"], codes, state["freq"], q=state["q"],
                                       interleaved=c["pairs"] == "next", starts=state["starts"], max_new=state["max_new"],
                                       token_pos=state.get("token_pos"), first_pos=state["first_pos"], weight=state["weight"], pos=state["pos"])
        return {**whole(state), "q": q, "weight": state["weight"], "pos": state["pos"]}
    if c["op"] == "attend":
        out = ac.defrag_kv_attend_terms(arena, state["pages"], state["lens"], state["q"], c["H"], codes, mask=state.get("mask"),
                                        cap=c["cap"] or None, slopes=state.get("slopes"), pos=state.get("pos"), starts=state["starts"],
                                        max_new=state["max_new"], max_len=state["max_len"], scale=state["scale"], lse=state["lse"],
                                        weight=state.get("weight"))
        got = {"out": out, "lse": state["lse"]}
        return {**got, "weight": state["weight"]} if c["scored"] else got
    ac.defrag_kv_accept(arena, state["pages"], state["lens"], state["path"], state["kept"], state["lens_out"], c["H"], c["D"], codes,
                        starts=state["starts"], max_new=state["max_new"], weight=state["weight"], pos=state["pos"])
    return {**whole(state), "weight": state["weight"], "pos": state["pos"], "lens": state["lens_out"]}


def nearest(x, codes):
    """float64 values in units of their scale -> the nearest code's value, by the number system's own steps."""
    if codes == "int8":
        return torch.clamp(torch.round(x), -127, 127)
    a = x.abs().clamp(max=448.0)
    power = torch.floor(torch.log2(a.clamp(min=2.0**-6)))
    power = torch.where(torch.exp2(power) > a.clamp(min=2.0**-6), power - 1, power)
    step = torch.exp2(power - 3)
    return torch.sign(x) * torch.round(a / step) * step


def least_scale(x, codes):
    """Smallest power of two 2^e, e >= -64, that brings all of x within the code's range."""
    top = {"e4m3": 448.0, "int8": 127.0}[codes]
    a = float(x.abs().max()) if x.numel() else 0.0
    e = -64
    if a > 0:
        e = max(-64, math.floor(math.log2(a / top)) - 1)
        while a > top * 2.0**e:
            e += 1
    return 2.0**e


def turned(x, pos, freq, pairs):
    """The rotation as a product of complex numbers."""
    x, R = x.double(), 2 * len(freq)
    y = x[..., :R].unflatten(-1, (2, -1)).transpose(-1, -2) if pairs == "half" else x[..., :R].unflatten(-1, (-1, 2))
    angle = pos.double()[:, None] * freq
    z = torch.view_as_complex(y.contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None]
    z = torch.view_as_real(z)
    out = x.clone()
    out[..., :R] = (z.transpose(-1, -2) if pairs == "half" else z).flatten(-2)
    return out


def exact(case, seed):
    state = prepare(case, seed)
    H, D, codes, B = case["H"], case["D"], case["codes"], case["B"]
    pitch, strip = state["arena"].shape[1], 2 * PAGE * D
    lens, new = state["lens"].tolist(), state["new"]
    pages = (state["pages"] // pitch).tolist()

    def page(b, j, h):
        """One head's keys and values [64, D] of a page (views of codes) and its two scales (a view)."""
        row = state["arena"][pages[b][j]]
        code = row[h * strip : (h + 1) * strip].view(CODES[codes])
        return code[: PAGE * D].view(PAGE, D), code[PAGE * D :].view(D, PAGE).t(), row[H * strip : H * strip + 8 * H].view(torch.float32)[2 * h : 2 * h + 2]

    if case["op"] == "attend":
        G = case["G"]
        pairs = sum(l * n for l, n in zip(lens, new)) * H * G
        if pairs * D > 6e12 or sum(lens) * H > 6e6:
            return None
        q = state["q"].double()
        out, lse, at = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device), 0
        weight = state["weight"].double() if case["scored"] else None
        for b in range(B):
            n, t = lens[b], new[b]
            rows = state["arena"][torch.tensor(pages[b][: -(-n // PAGE)], device=q.device)]
            if case["mask"]:
                bit = torch.arange(t, device=q.device)
                hides = (state["mask"][at : at + t][:, bit // 64] >> (bit % 64)) & 1 == 0
            else:
                hides = torch.ones(t, t, dtype=torch.bool, device=q.device).triu(1)
            for h in range(H):
                code = rows[:, h * strip : (h + 1) * strip].view(CODES[codes]).double()
                sc = rows[:, H * strip + 8 * h : H * strip + 8 * h + 8].contiguous().view(torch.float32).double()
                k = (code[:, : PAGE * D] * sc[:, :1]).reshape(-1, D)[:n]
                v = (code[:, PAGE * D :] * sc[:, 1:]).view(-1, D, PAGE).transpose(1, 2).reshape(-1, D)[:n]
                where = state["pos"][b, h, :n].double() if case["pos"] else torch.arange(n, device=q.device).double()
                for g in range(G):
                    s = (q[at : at + t, h * G + g] @ k.t()) * state["scale"]
                    if case["cap"]:
                        s = case["cap"] * (1 - 2 / (torch.exp(2 * s / case["cap"]) + 1))
                    if case["slopes"]:
                        s = s - float(state["slopes"][h * G + g]) * (where[n - t :, None] - where[None, :])
                    s[:, n - t :].masked_fill_(hides, -math.inf)
                    lse[at : at + t, h * G + g] = torch.logsumexp(s, -1)
                    p = torch.softmax(s, -1)
                    out[at : at + t, h * G + g] = p @ v
                    if weight is not None:
                        weight[b, h, :n] += p.sum(0)
            at += t
        return {"out": out, "lse": lse, **({"weight": weight} if weight is not None else {})}

    if case["op"] == "rotary":
        if sum(-(-(n + t) // PAGE) - n // PAGE for n, t in zip(lens, new)) * H > 12000:
            return None
        first = state["first_pos"].tolist()
        pos = state.get("token_pos")
        if pos is None:
            pos = torch.tensor([f + i for f, t in zip(first, new) for i in range(t)], dtype=torch.int32, device=state["k"].device)
        keys, at = turned(state["k"], pos, state["freq"], case["pairs"]), 0
        for b in range(B):
            n, t = lens[b], new[b]
            for j in range(n // PAGE, -(-(n + t) // PAGE)):
                lo, hi = max(n, j * PAGE), min(n + t, (j + 1) * PAGE)
                for h in range(H):
                    kc, vc, sc = page(b, j, h)
                    for i, (c, x) in enumerate(((kc, keys), (vc, state["v"]))):
                        x = x[at + lo - n : at + hi - n, h].double()
                        scale, old = least_scale(x, codes), lo - j * PAGE
                        if old:
                            was = float(sc[i])
                            scale = max(scale, was)
                            if scale > was:
                                c[:old] = nearest(c[:old].double() * (was / scale), codes).to(c.dtype)
                        c[old : hi - j * PAGE] = nearest(x / scale, codes).to(c.dtype)
                        sc[i] = scale
            state["weight"][b, :, n : n + t] = 0
            state["pos"][b, :, n : n + t] = pos[at : at + t]
            at += t
        return {**whole(state), "q": turned(state["q"], pos, state["freq"], case["pairs"]), "weight": state["weight"].double(), "pos": state["pos"]}

    path, kept = state["path"].tolist(), state["kept"].tolist()
    if sum(-(-k // PAGE) + 1 for k in kept) * H > 8000:
        return None
    for b in range(B):
        had = lens[b] - new[b]
        take = [had + i for i in path[b][: kept[b]]]  # the place that place had + i takes its token from
        state["lens_out"][b] = had + kept[b]
        if kept[b] and take != list(range(had, had + kept[b])):
            idx = torch.tensor(take, device=state["pos"].device)
            for name in ("weight", "pos"):
                state[name][b, :, had : had + kept[b]] = state[name][b][:, idx]
        for h in range(H):
            for j in range(had // PAGE, -(-(had + kept[b]) // PAGE)):
                lo, hi = max(had, j * PAGE), min(had + kept[b], (j + 1) * PAGE)
                mine = take[lo - had : hi - had]
                if mine == list(range(lo, hi)):
                    continue
                dst = page(b, j, h)
                come = [page(b, i // PAGE, h) for i in mine]
                far = [i // PAGE != j for i in mine]
                for w in (0, 1):
                    was = float(dst[2][w])
                    codes_of = [s[w][i % PAGE].double() for s, i in zip(come, mine)]
                    steps = [float(s[2][w]) for s in come]
                    scale = was
                    if any(far):
                        scale = least_scale(torch.stack([x * s for x, s, f in zip(codes_of, steps, far) if f]), codes)
                        if lo > j * PAGE or not all(far):
                            scale = max(scale, was)
                    c = dst[w]
                    if scale != was and lo > j * PAGE:
                        c[: lo - j * PAGE] = nearest(c[: lo - j * PAGE].double() * (was / scale), codes).to(c.dtype)
                    c[lo - j * PAGE : hi - j * PAGE] = torch.stack([nearest(x * (s / scale), codes) for x, s in zip(codes_of, steps)]).to(c.dtype)
                    dst[2][w] = scale
    return {**whole(state), "weight": state["weight"].double(), "pos": state["pos"], "lens": state["lens_out"]}
