"""The operators of the 8-bit key/value cache in the arena, as cases to measure.

A cache page is one block of the arena: 64 tokens of every head, held in 8
bits with one power-of-two scale for the keys and one for the values of each
(page, head).  The page table holds the pages' byte offsets in the arena, so a
compaction of the arena remaps it like any other handles.  Three operators:

  append  quantises new tokens into the pages;
  attend  softmax attention of the newest tokens' queries over the cache,
          optionally adding up the weight that every cached token receives;
  evict   keeps `budget` tokens of every (sequence, head) by that weight and
          folds the kept ones into the first pages, so that the rest are free.

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
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    def attend(name, **c):
        return {"name": name, "op": "attend", "tlo": 1.0, "lo": 1.0, "scored": False, **c}

    def append(name, **c):
        return {"name": name, "op": "append", "tlo": 1.0, "lo": 1.0, **c}

    def evict(name, **c):
        return {"name": name, "op": "evict", "lo": 1.0, **c}

    return [
        # one short conversation, one token: launches and latency
        attend("attend one short", B=1, past=64, T=1, H=2, G=4, D=64, codes="e4m3", dtype="bf16"),
        # a serving step over a ragged batch
        attend("attend batch", B=64, past=4096, lo=0.1, T=1, H=8, G=4, D=128, codes="e4m3", dtype="bf16"),
        # two long documents, one token each: the work is split along the cache
        attend("attend long", B=2, past=131000, lo=0.9, T=1, H=8, G=8, D=128, codes="int8", dtype="fp16"),
        # a serving step that also adds up the weights an eviction goes by
        attend("attend scored", B=48, past=8000, lo=0.3, T=1, H=4, G=7, D=128, codes="e4m3", dtype="bf16", scored=True),
        # five drafted tokens verified at once
        attend("attend draft", B=16, past=10000, lo=0.5, T=5, H=8, G=4, D=96, codes="int8", dtype="bf16"),
        # chunks of prompts behind a cached prefix
        attend("attend chunk", B=3, past=2048, lo=0.3, T=2000, tlo=0.5, H=8, G=4, D=128, codes="e4m3", dtype="bf16"),
        # a whole prompt, with its weights
        attend("attend prompt scored", B=1, past=0, T=8200, H=4, G=8, D=64, codes="int8", dtype="fp16", scored=True),
        # one new token of every sequence of a batch
        append("append step", B=128, past=4000, lo=0.2, T=1, H=8, D=128, codes="e4m3", dtype="bf16"),
        # prompts into the cache
        append("append prompt", B=4, past=100, T=4097, tlo=0.6, H=8, D=128, codes="int8", dtype="fp16"),
        # one short sequence halved: launches and latency
        evict("evict one", B=1, L=1000, budget=512, sink=4, recent=64, H=2, D=64, codes="e4m3"),
        # a batch under memory pressure halved
        evict("evict batch", B=32, L=8190, lo=0.4, budget=4096, sink=4, recent=256, H=8, D=128, codes="e4m3"),
        # two long documents cut to a quarter
        evict("evict long", B=2, L=131000, lo=0.9, budget=32768, sink=16, recent=1024, H=8, D=128, codes="int8"),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["attend", "attend", "attend", "append", "evict"])
    H, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 96, 128, 192, 256])
    c = {"op": op, "H": H, "D": D, "codes": rng.choice(["e4m3", "int8"]), "lo": rng.choice([1.0, 0.7, 0.2])}
    if op == "evict":
        c["budget"] = PAGE * log(1, 256)
        c["L"] = c["budget"] + log(1, 3 * c["budget"])
        c["sink"], c["recent"] = rng.choice([0, 1, 4]), rng.randint(0, c["budget"] // 2)
        c["B"] = log(1, max(1, min(64, (1 << 28) // (c["L"] * H * D))))
        return c
    c["dtype"], c["tlo"] = rng.choice(["bf16", "fp16"]), rng.choice([1.0, 0.5])
    if op == "append":
        c["T"] = rng.choice([1, log(2, 4097)])
        c["past"] = rng.choice([0, log(1, 4097)])
        c["B"] = log(1, max(1, min(128, (1 << 26) // ((c["T"] + c["past"]) * H * D))))
        return c
    c["scored"], c["G"] = rng.random() < 0.4, rng.choice([1, 2, 3, 4, 6, 8, 16])
    if rng.random() < 0.6:  # few new tokens over a cache
        c["T"], c["past"] = rng.choice([1, 1, 2, 7]), log(1, 65536)
        c["B"] = log(1, max(1, min(128, (1 << 27) // ((c["past"] + 64) * H * D))))
    else:                   # many of them
        c["T"], c["past"] = log(9, 2049), rng.choice([0, log(1, 8192)])
        c["T"] = max(9, min(c["T"], int(5e10 / ((c["T"] + c["past"]) * H * c["G"] * D))))
        pairs = c["T"] * (c["T"] + c["past"]) * H * c["G"]
        c["B"] = log(1, max(1, min(8, int(5e10 / (pairs * D)))))
    return c


def spread(top, lo, n, least):
    """n lengths from top down to lo * top."""
    return [max(least, round(top * (1 - (1 - lo) * i / max(1, n - 1)))) for i in range(n)]


def lengths(case):
    """(tokens cached before the call, new tokens) of every sequence, before the seed deals them out."""
    if case["op"] == "evict":
        return spread(case["L"], case["lo"], case["B"], 1), [0] * case["B"]
    past = spread(case["past"], case["lo"], case["B"], 0)
    return past, spread(case["T"], case["tlo"], case["B"], 1)


def work(case):
    B, H, D = case["B"], case["H"], case["D"]
    past, new = lengths(case)
    if case["op"] == "append":  # keys and values in 16 bits in, codes out
        return {"bytes": sum(new) * H * D * 2 * (2 + 1), "flops": 2 * sum(new) * H * D}
    if case["op"] == "evict":   # weights and positions of all, codes of the kept tokens behind the budget
        K = case["budget"]
        moved = sum(K * (n - K) / n for n in past if n > K) * H
        return {"bytes": sum(past) * H * 8 + B * H * K * 8 + moved * 2 * D * 2, "flops": 2 * moved * D}
    G, rows = case["G"], sum(new) * H * case["G"]
    seen = sum(t * p + t * (t + 1) // 2 for p, t in zip(past, new)) * H * G
    held = sum(p + t for p, t in zip(past, new)) * H
    return {"bytes": held * 2 * D + rows * D * 2 * 2 + rows * 4 + (held * 8 if case["scored"] else 0), "flops": 4 * D * seen}


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
    step = torch.exp2(torch.frexp(x.abs().clamp(min=2.0**-6))[1].float() - 4)
    return ((x / step).round() * step).clamp(-top, top).to(torch.float8_e4m3fn)


def finite_max(x, dim):
    return torch.nan_to_num(x.abs(), nan=0.0, posinf=0.0).amax(dim)


def strips(state, rows):
    """Views of pages: key codes [.., H, 64, D], value codes [.., H, D, 64], scales [.., H, 2]."""
    H, D = state["case"]["H"], state["case"]["D"]
    codes = rows[..., : H * 2 * PAGE * D].view(CODES[state["case"]["codes"]]).unflatten(-1, (H, 2, PAGE * D))
    scales = rows[..., H * 2 * PAGE * D : H * 2 * PAGE * D + 8 * H].view(torch.float32).unflatten(-1, (H, 2))
    return codes[..., 0, :].unflatten(-1, (PAGE, D)), codes[..., 1, :].unflatten(-1, (D, PAGE)), scales


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    B, H, D, codes = case["B"], case["H"], case["D"], case["codes"]
    past, new = lengths(case)
    deal = torch.randperm(B, generator=host).tolist()
    past, new = [past[i] for i in deal], [new[i] for i in deal]
    total = [p + n for p, n in zip(past, new)]
    attend = case["op"] == "attend"
    per = [-(-n // PAGE) for n in total]
    stride = max(per) + 1
    pitch = H * 2 * PAGE * D + (8 * H + 31) // 32 * 32 + 32 * 3  # other small blocks lie between the pages
    slots = sum(per) + 3
    # the pages lie in the arena in no order
    order = torch.randperm(slots, generator=host)[: sum(per)]
    pages = torch.full((B, stride), -1, dtype=torch.int64)
    pages[torch.arange(stride)[None, :] < torch.tensor(per)[:, None]] = order * pitch
    arena = torch.zeros(slots, pitch, dtype=torch.uint8, device=dev)
    if attend:
        arena.fill_(0x7F)  # what is not the cache's own is no number
    state = {"case": dict(case), "arena": arena, "pages": pages.to(dev), "past": past, "new": new}

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    held = total if attend else past
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
        if attend and codes == "e4m3":  # tokens behind the last one: left over, no numbers
            kc.view(torch.uint8).masked_fill_(~there[:, None, :, None], 0x7F)
            vc.view(torch.uint8).masked_fill_(~there[:, None, None, :], 0x7F)
        arena[at[i : i + group]] = rows
    starts = torch.tensor([0] + new).cumsum(0)
    state["starts"] = starts.to(torch.int32).to(dev)
    N = int(starts[-1])
    state["of"] = torch.repeat_interleave(torch.arange(B), torch.tensor(new)).to(dev)
    state["nth"] = torch.arange(N, device=dev) - starts.to(dev)[state["of"]]
    if case["op"] == "append":
        # keys and values as slices of one fused projection
        qkv = torch.randn(N, 6 * H * D, device=dev, generator=gen).to(FLOATS[case["dtype"]])
        qkv.view(N, 6, H, D)[:, 4:] *= torch.stack([s[:, 0] for s in size]).to(qkv.dtype)
        state["k"], state["v"] = (qkv.view(N, 6 * H, D)[:, (4 + w) * H : (5 + w) * H] for w in (0, 1))
        state["weight"] = torch.ones(B, H, max(total) + 5, device=dev)
        state["pos"] = torch.full((B, H, max(total) + 5), -1, dtype=torch.int32, device=dev)
        state["first_pos"] = ints([p + 7 for p in past])
    elif attend:
        G = case["G"]
        qkv = (2 * torch.randn(N, (G + 2) * H * D, device=dev, generator=gen)).to(FLOATS[case["dtype"]])
        state["q"] = qkv.view(N, (G + 2) * H, D)[:, : G * H]
        state["scale"] = D**-0.5
        state["lse"] = torch.empty(N, G * H, device=dev)
        if case["scored"]:
            state["weight"] = torch.rand(B, H, max(total) + 5, device=dev, generator=gen)
    else:
        cap = max(past) + 5
        w = torch.exp(2 * torch.randn(B, H, cap, device=dev, generator=gen))
        # many tokens have not been looked at: ties
        state["weight"] = w * (torch.rand(B, H, cap, device=dev, generator=gen) < 0.9)
        # earlier evictions have put the first half out of order
        key = torch.rand(B, H, cap, device=dev, generator=gen)
        line = torch.arange(cap, device=dev)
        key = torch.where(line < min(past) // 2, key, 1.0 + line)
        state["pos"] = key.argsort(-1).to(torch.int32)
        state["next_pos"] = ints(past)
        state["weight_out"] = torch.zeros(B, H, case["budget"], device=dev)
        state["pos_out"] = torch.full((B, H, case["budget"]), -1, dtype=torch.int32, device=dev)
        state["lens_out"] = torch.zeros(B, dtype=torch.int32, device=dev)
    return state


def held_pages(state, first=0, last=None):
    """(row of the arena for every page, truth value: there is one)."""
    pages = state["pages"][:, first:last]
    return pages.clamp(min=0) // state["arena"].shape[1], pages >= 0


def numbers(state, last):
    """Keys and values [B, H, tokens, D] of the first `last` pages as float32, nothing in place of what is not there."""
    rows, there = held_pages(state, 0, last)
    k, v, s = strips(state, state["arena"][rows])
    k, v = k.float() * s[..., 0, None, None], v.float().transpose(-1, -2) * s[..., 1, None, None]
    live = torch.arange(k.shape[1] * PAGE, device=k.device) < state["lens"][:, None]
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))
    return (torch.where(live[:, None, :, None], x, 0.0) for x in (k, v))


def run_attend(state):
    c = state["case"]
    H, G, D, B = c["H"], c["G"], c["D"], c["B"]
    k, v = numbers(state, -(-state["max_len"] // PAGE))
    T, L = state["max_new"], k.shape[2]
    q = torch.zeros(B, T, H, G, D, device=k.device)
    q[state["of"], state["nth"]] = state["q"].float().unflatten(1, (H, G))
    s = q.permute(0, 2, 3, 1, 4).reshape(B, H, G * T, D) @ k.transpose(-1, -2).contiguous() * state["scale"]
    had = state["lens"] - (state["starts"][1:] - state["starts"][:-1])
    seen = torch.arange(L, device=k.device) <= had[:, None, None] + torch.arange(T, device=k.device)[:, None]
    seen &= torch.arange(L, device=k.device) < state["lens"][:, None, None]
    real = torch.arange(T, device=k.device) < (state["lens"] - had)[:, None]
    s = s.view(B, H, G, T, L).masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total == 0, 1.0, total)
    o = (p.view(B, H, G * T, L) @ v).view(B, H, G, T, D).permute(0, 3, 1, 2, 4)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2)
    out = {"out": o[state["of"], state["nth"]].flatten(1, 2).to(state["q"].dtype), "lse": lse[state["of"], state["nth"]].flatten(1, 2)}
    if c["scored"]:
        state["weight"][:, :, :L] += (p * real[:, None, None, :, None]).sum((2, 3))[:, :, : state["weight"].shape[2]]
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


def run_append(state):
    c = state["case"]
    H, D, B, codes = c["H"], c["D"], c["B"], c["codes"]
    dev, lens, N = state["pages"].device, state["lens"].long(), len(state["of"])
    touched = -(-(state["max_new"] + PAGE - 1) // PAGE)
    nth = (lens // PAGE)[:, None] + torch.arange(touched, device=dev)
    rows = state["pages"].gather(1, nth.clamp(max=state["pages"].shape[1] - 1)).clamp(min=0) // state["arena"].shape[1]
    token = nth[..., None] * PAGE + torch.arange(PAGE, device=dev) - lens[:, None, None]  # among the new ones
    count = (state["starts"][1:] - state["starts"][:-1]).long()[:, None, None]
    fresh, old = (token >= 0) & (token < count), token < 0
    src = (state["starts"][:-1].long()[:, None, None] + token).clamp(0, N - 1)
    k, v, s = strips(state, state["arena"][rows])
    sides, scales = [], []
    for was, x, w in ((k, state["k"], 0), (v.transpose(-1, -2), state["v"], 1)):
        x = x.float()[src].permute(0, 1, 3, 2, 4)
        e = exponent(finite_max(torch.where(fresh[:, :, None, :, None], x, 0.0), (-1, -2)), codes)
        before = torch.frexp(s[..., w])[1] - 1
        e = torch.where(old[..., :1], torch.maximum(e, before), e)
        again = to_codes(was.float() * torch.exp2((before - e).float())[..., None, None], codes)
        new = to_codes(x * torch.exp2(-e.float())[..., None, None], codes)
        both = torch.where(fresh[:, :, None, :, None], new.float(), torch.where(old[:, :, None, :, None], again.float(), was.float()))
        sides.append(both.to(CODES[codes]))
        scales.append(torch.exp2(e.float()))
    put(state, rows, fresh.any(-1), sides[0], sides[1], torch.stack(scales, -1))
    at = lens[state["of"]] + state["nth"]
    state["weight"][state["of"], :, at] = 0.0
    state["pos"][state["of"], :, at] = (state["first_pos"][state["of"]] + state["nth"].int())[:, None]
    return {**whole(state), "weight": state["weight"], "pos": state["pos"]}


def run_evict(state):
    c = state["case"]
    H, D, B, K, codes = c["H"], c["D"], c["B"], c["budget"], c["codes"]
    L = state["max_len"]
    w, pos, lens = state["weight"][:, :, :L], state["pos"][:, :, :L], state["lens"][:, None, None]
    line = torch.arange(L, device=w.device)
    live = line < lens
    safe = (pos < c["sink"]) | (pos >= state["next_pos"][:, None, None] - c["recent"])
    rank = torch.where(live, torch.where(safe, 2, 1), 0)
    by = torch.where(torch.isnan(w), math.inf, w).sort(dim=-1, descending=True, stable=True)[1]
    by = by.gather(-1, rank.gather(-1, by).sort(dim=-1, descending=True, stable=True)[1])
    keep = torch.zeros_like(live.expand(B, H, L)).scatter_(-1, by[..., :K], True) & live
    # the first hole takes the first kept token behind the budget, and so on
    kept_behind = keep & (line >= K)
    tail = torch.where(kept_behind, line, L).sort(-1)[0]
    holes = ~keep[..., :K] & live[..., :K]
    src = torch.where(holes, tail.gather(-1, (holes.cumsum(-1) - 1).clamp(min=0)), line[:K]).clamp(max=L - 1)
    there = live[..., :K]
    state["weight_out"][:, :, :K] = torch.where(there, w.gather(-1, src), state["weight_out"][:, :, :K])
    state["pos_out"][:, :, :K] = torch.where(there, pos.gather(-1, src), state["pos_out"][:, :, :K])
    state["lens_out"].copy_(state["lens"].clamp(max=K))
    # codes: only pages with a hole change
    rows, has = held_pages(state, 0, K // PAGE)
    k, v = numbers(state, -(-L // PAGE))
    kc, vc, s = strips(state, state["arena"][rows])
    P = rows.shape[1]
    change = holes[..., : P * PAGE].unflatten(-1, (P, PAGE)).any(-1).transpose(1, 2)
    sides, scales = [], []
    for x, was, i in ((k, kc, 0), (v, vc.transpose(-1, -2), 1)):
        y = x.gather(2, src[..., : P * PAGE, None].expand(-1, -1, -1, D)).unflatten(2, (P, PAGE)).transpose(1, 2)
        e = exponent(finite_max(y, (-1, -2)), codes)
        new = to_codes(y * torch.exp2(-e.float())[..., None, None], codes)
        sides.append(torch.where(change[..., None, None], new.float(), was.float()).to(CODES[codes]))
        scales.append(torch.where(change, torch.exp2(e.float()), s[..., i]))
    put(state, rows, has, sides[0], sides[1], torch.stack(scales, -1))
    return {**whole(state), "weight": state["weight_out"], "pos": state["pos_out"], "lens": state["lens_out"]}


def run(state):
    c = state["case"]
    if not own:
        return {"attend": run_attend, "append": run_append, "evict": run_evict}[c["op"]](state)
    import arena_compaction_amd as ac
    arena, codes = state["arena"].view(-1), CODES[c["codes"]]
    if c["op"] == "attend":
        out = ac.defrag_kv_attend(arena, state["pages"], state["lens"], state["q"], c["H"], codes, starts=state["starts"],
                                  max_new=state["max_new"], max_len=state["max_len"], scale=state["scale"],
                                  lse=state["lse"], weight=state.get("weight"))
        got = {"out": out, "lse": state["lse"]}
        return {**got, "weight": state["weight"]} if c["scored"] else got
    if c["op"] == "append":
        ac.defrag_kv_append(arena, state["pages"], state["lens"], state["k"], state["v"], codes, starts=state["starts"],
                            max_new=state["max_new"], weight=state["weight"], pos=state["pos"], first_pos=state["first_pos"])
        return {**whole(state), "weight": state["weight"], "pos": state["pos"]}
    ac.defrag_kv_evict(arena, state["pages"], state["lens"], c["budget"], state["weight"], state["pos"], state["weight_out"],
                       state["pos_out"], state["lens_out"], c["D"], codes, sink=c["sink"], recent=c["recent"],
                       next_pos=state["next_pos"], max_len=state["max_len"])
    return {**whole(state), "weight": state["weight_out"], "pos": state["pos_out"], "lens": state["lens_out"]}


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
            for h in range(H):
                code = rows[:, h * strip : (h + 1) * strip].view(CODES[codes]).double()
                sc = rows[:, H * strip + 8 * h : H * strip + 8 * h + 8].contiguous().view(torch.float32).double()
                k = (code[:, : PAGE * D] * sc[:, :1]).reshape(-1, D)[:n]
                v = (code[:, PAGE * D :] * sc[:, 1:]).view(-1, D, PAGE).transpose(1, 2).reshape(-1, D)[:n]
                for g in range(G):
                    s = (q[at : at + t, h * G + g] @ k.t()) * state["scale"]
                    ahead = torch.arange(n, device=q.device)[None, :] > (n - t + torch.arange(t, device=q.device))[:, None]
                    s.masked_fill_(ahead, -math.inf)
                    lse[at : at + t, h * G + g] = torch.logsumexp(s, -1)
                    p = torch.softmax(s, -1)
                    out[at : at + t, h * G + g] = p @ v
                    if weight is not None:
                        weight[b, h, :n] += p.sum(0)
            at += t
        return {"out": out, "lse": lse, **({"weight": weight} if weight is not None else {})}

    if case["op"] == "append":
        if sum(-(-(n + t) // PAGE) - n // PAGE for n, t in zip(lens, new)) * H > 12000:
            return None
        at = 0
        for b in range(B):
            n, t = lens[b], new[b]
            for j in range(n // PAGE, -(-(n + t) // PAGE)):
                lo, hi = max(n, j * PAGE), min(n + t, (j + 1) * PAGE)
                for h in range(H):
                    kc, vc, sc = page(b, j, h)
                    for i, (c, x) in enumerate(((kc, state["k"]), (vc, state["v"]))):
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
            state["pos"][b, :, n : n + t] = int(state["first_pos"][b]) + torch.arange(t, dtype=torch.int32, device=kc.device)
            at += t
        return {**whole(state), "weight": state["weight"].double(), "pos": state["pos"]}

    K = case["budget"]
    if sum(min(n, K) for n in lens) * H // PAGE > 20000:
        return None
    weight, pos = state["weight"].cpu().double(), state["pos"].cpu()
    for b in range(B):
        n = lens[b]
        state["lens_out"][b] = min(n, K)
        for h in range(H):
            src = list(range(min(n, K)))
            if n > K:
                p, w = pos[b, h, :n].tolist(), weight[b, h, :n].tolist()
                border = int(state["next_pos"][b]) - case["recent"]
                best = sorted(range(n), key=lambda i: (0 if p[i] < case["sink"] or p[i] >= border else 1, -w[i], i))[:K]
                kept = set(best)
                behind = iter(sorted(i for i in best if i >= K))
                src = [i if i in kept else next(behind) for i in range(K)]
                old = {}
                for j in range(K // PAGE):
                    mine = src[j * PAGE : (j + 1) * PAGE]
                    if mine == list(range(j * PAGE, (j + 1) * PAGE)):
                        continue
                    for f in sorted({i // PAGE for i in mine} - old.keys()):
                        kc, vc, sc = page(b, f, h)
                        old[f] = (kc.double() * float(sc[0]), vc.double() * float(sc[1]))
                    kc, vc, sc = page(b, j, h)
                    from_ = sorted({i // PAGE for i in mine})
                    pick = torch.tensor([from_.index(i // PAGE) * PAGE + i % PAGE for i in mine], device=kc.device)
                    for i, c in ((0, kc), (1, vc)):
                        x = torch.cat([old[f][i] for f in from_])[pick]
                        scale = least_scale(x, codes)
                        c.copy_(nearest(x / scale, codes).to(c.dtype))
                        sc[i] = scale
            state["weight_out"][b, h, : len(src)] = weight[b, h][src].to(state["weight_out"])
            state["pos_out"][b, h, : len(src)] = pos[b, h][src].to(state["pos_out"])
    return {**whole(state), "weight": state["weight_out"].double(), "pos": state["pos_out"], "lens": state["lens_out"]}
