"""Operators on the paged e4m3 cache of a serving step, beside its writing, reading and attention, as measured cases.

  shared  attention of a batch whose sequences begin with the same long prefix: the prefix's keys and values are read once
          for all rows that see it, each sequence's own tokens as ever
  weigh   the attention weight that every cached token received from the step's new tokens, summed over them and over the
          query heads of a kv head, added to the token's running sum
  evict   a sequence shortened to a budget: every kv head keeps its first, its most recent and its heaviest tokens, which
          move in order to the pages that the sequence goes on with

`own` false: the plain forms below, elementary torch operations in 32 bits.  `own` true: the library's calls.
"""
import math

import torch

own = False

FP8_MAX = 448.0
DEV = "cuda"


# ------------------------------------------------------------------- cases ---

def listed():
    """Heads are those of the repository's Qwen3-32B-sized layers (64 query and 8 key heads of 128); narrow heads in
    groups of three with small pages and odd lengths stand for the rest of what the cache holds."""
    shared = dict(op="shared", heads=64, kv_heads=8, dim=128, page=64, groups=1)
    weigh = dict(op="weigh", heads=64, kv_heads=8, dim=128, page=64, window=0, add=True)
    evict = dict(op="evict", heads=64, kv_heads=8, dim=128, page=64, first=4, coarse=False)
    return [
        # a few samples of one short prompt: latency
        dict(shared, name="shared b4 p500 decode", mode="decode", B=4, q_max=1, kv_max=40, prefix=500),
        # a decode batch behind a long system prompt
        dict(shared, name="shared b64 p8192 decode", mode="decode", B=64, q_max=1, kv_max=1000, prefix=8192),
        # three prompts of odd lengths, some sequences with a draft of several tokens, narrow heads
        dict(shared, name="shared b30 g3 d64 mixed", mode="mixed", B=30, q_max=7, kv_max=777, prefix=3001, groups=3, heads=24,
             dim=64, page=16),
        # new questions of hundreds of tokens about one long document
        dict(shared, name="shared b8 q512 p16384", mode="chunk", B=8, q_max=512, kv_max=700, prefix=16384),
        # one token of a single stream: latency
        dict(weigh, name="weigh b1 8k decode", mode="decode", B=1, q_max=1, kv_max=8192),
        # a decode batch of ragged contexts
        dict(weigh, name="weigh b64 8k decode", mode="decode", B=64, q_max=1, kv_max=8000),
        # the last tokens of prompts weigh the whole of them, narrow heads, a window, sums that begin here
        dict(weigh, name="weigh b8 q33 d64 window", mode="chunk", B=8, q_max=33, kv_max=2500, heads=24, dim=64, page=16,
             window=1777, add=False),
        # a long prompt's chunk over what came before it
        dict(weigh, name="weigh q4096 16k", mode="chunk", B=1, q_max=4096, kv_max=16384),
        # a single sequence cut to half: latency
        dict(evict, name="evict b1 2000", B=1, kv_max=2000, budget=1000, recent=64),
        # short and long sequences, narrow heads, sums with many ties, some sequences within the budget
        dict(evict, name="evict b16 d64 ties", B=16, kv_max=3333, budget=999, recent=100, dim=64, page=16, coarse=True),
        # one very long sequence
        dict(evict, name="evict b1 60000", B=1, kv_max=60000, budget=8192, recent=1024),
        # a batch at its memory's limit
        dict(evict, name="evict b64 8k", B=64, kv_max=8000, budget=2048, recent=256),
    ]


MAX_SCORES = 4096 * 14336 * 64


def draw(rng):
    def logint(lo, hi):
        return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    op = rng.choice(["shared", "weigh", "evict"])
    heads, kv_heads = rng.choice([(64, 8), (40, 8), (24, 8), (8, 8), (16, 1), (32, 4)])
    case = dict(op=op, heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]))
    if op == "evict":
        B = logint(1, 64)
        kv_max = logint(16, 60000 if B == 1 else 16000 if B < 8 else 8000)
        budget = max(1, int(kv_max * rng.uniform(0.05, 0.9)))
        recent = int(budget * rng.uniform(0, 0.5))
        return dict(case, B=B, kv_max=kv_max, budget=budget, recent=recent, first=min(budget - recent, rng.choice([0, 1, 4])),
                    coarse=rng.random() < 0.3)
    mode = rng.choice(["decode", "mixed", "chunk"])
    B = logint(1, 64) if mode == "decode" else logint(1, 16)
    q_max = 1 if mode == "decode" else logint(2, 600 if op == "shared" else 2048)
    if op == "shared":
        kv_max = logint(max(2, q_max), 2000)
        prefix = logint(16, 16384)
        while B * q_max * (prefix + kv_max) * heads > MAX_SCORES // 2:
            q_max = max(1, q_max // 2)
        return dict(case, mode=mode, B=B, q_max=q_max, kv_max=kv_max, prefix=prefix, groups=min(B, rng.choice([1, 1, 2, 5])))
    kv_max = logint(max(16, q_max), 32768 if B < 8 else 8192)
    while B * q_max * kv_max * heads > MAX_SCORES // 2:
        q_max = max(1, q_max // 2)
    return dict(case, mode=mode, B=B, q_max=q_max, kv_max=kv_max, window=rng.choice([0, 0, 0, 128, 1000]), add=rng.random() < 0.7)


def spread(i, most, step):
    """Sizes from 1 to `most`, the first one the largest."""
    return most if i == 0 else 1 + int((most - 1) * ((i * step) % 1.0))


def lengths(case):
    """New tokens and context (which holds them; of the shared form: the sequence's own) of every sequence."""
    q, kv = [], []
    for i in range(case["B"]):
        n = spread(i, case["kv_max"], 0.6180339887)
        if case["op"] == "evict":
            m = 0
        elif case["mode"] == "decode" or (case["mode"] == "mixed" and i % 2 == 1):
            m = 1
        else:
            m = spread(i, case["q_max"], 0.4142135624)
        q.append(min(m, n))
        kv.append(n)
    return q, kv


def prefixes(case):
    """Of every prefix: its first sequence (one more for the end), and its tokens."""
    G, B = case["groups"], case["B"]
    return [g * B // G for g in range(G + 1)], [spread(g, case["prefix"], 0.7320508076) for g in range(G)]


def visible(case):
    """(new token, key) pairs that the mask leaves, and the keys that some new token sees."""
    pairs = keys = 0
    w = case.get("window", 0)
    for m, n in zip(*lengths(case)):
        pairs += sum(min(p + 1, w) for p in range(n - m, n)) if w else m * (n - m) + m * (m + 1) // 2
        keys += min(n, m - 1 + w) if w else n
    return pairs, keys


def work(case):
    Hq, H, D = case["heads"], case["kv_heads"], case["dim"]
    q_lens, kv_lens = lengths(case)
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in kv_lens)
        sums = sum(n for n in kv_lens if n > case["budget"])
        return {"bytes": 4 * sums * H + 2 * kept * H * (2 * D + 12), "flops": 0}
    pairs, keys = visible(case)
    T = sum(q_lens)
    if case["op"] == "weigh":
        return {"bytes": keys * H * (D + 4 + (8 if case["add"] else 4)) + T * Hq * (2 * D + 4), "flops": 2 * pairs * Hq * D}
    at, P = prefixes(case)
    pairs += sum(P[g] * sum(q_lens[at[g]:at[g + 1]]) for g in range(case["groups"]))
    return {"bytes": (keys + sum(P)) * H * (2 * D + 8) + T * Hq * (4 * D + 4), "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs ---

def quantised(x):
    """e4m3 codes and fp32 scales of rows of x (its last axis)."""
    s = x.abs().amax(-1).clamp(min=1e-10) / FP8_MAX
    return (x / s.unsqueeze(-1)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn), s


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    H, D, page = case["kv_heads"], case["dim"], case["page"]
    q_lens, kv_lens = lengths(case)
    runs = list(kv_lens)                                    # stretches of tokens that have pages of their own
    if case["op"] == "shared":
        first, prefix_lens = prefixes(case)
        runs += prefix_lens
    if case["op"] == "evict":
        new_lens = [min(n, case["budget"]) for n in kv_lens]
        runs += new_lens
    need = [(n + page - 1) // page for n in runs]
    pages = sum(need) + 3
    # keys with a common part and values of differing size a token
    k = randn(pages, H, page, D) + 0.5 * randn(1, H, 1, D)
    v = randn(pages, H, page, D) * torch.exp(0.5 * randn(pages, 1, page, 1))
    (kq, ks), (vq, vs) = quantised(k.to(torch.bfloat16).float()), quantised(v.to(torch.bfloat16).float())
    del k, v
    s = dict(case=case, k=kq, v=vq, ks=ks, vs=vs, kv_max=max(kv_lens), kv_lens=ints(kv_lens))
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    starts = [sum(need[:i]) for i in range(len(need))]

    def table_of(lo, hi):
        t = torch.zeros(hi - lo, max(need[lo:hi]), dtype=torch.int32, device=DEV)
        for i in range(lo, hi):
            t[i - lo, :need[i]] = order[starts[i]:starts[i] + need[i]]
        return t

    B = case["B"]
    s["table"] = table_of(0, B)
    if case["op"] != "shared":
        # sums as they stand after some steps: a few tokens hold most of the weight, some none
        s["weights"] = torch.exp(2 * randn(pages, H, page)) * (torch.rand(pages, H, page, generator=g, device=DEV) < 0.95)
    if case["op"] == "evict":
        if case["coarse"]:
            s["weights"] = (s["weights"] * 4).floor() / 4
        s["out_table"] = table_of(B, 2 * B)
        # (sequence, position) of every token that stays, as the host knows them
        s["stay_b"] = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(new_lens, device=DEV))
        s["stay_i"] = torch.cat([torch.arange(n, device=DEV) for n in new_lens])
        return s
    cu = [0]
    for m in q_lens:
        cu.append(cu[-1] + m)
    s["cu_q"], s["q_max"], s["scale"] = ints(cu), max(q_lens), 1.0 / math.sqrt(D)
    s["q"] = (randn(cu[-1], case["heads"], D) * 2).to(torch.bfloat16)
    if case["op"] == "shared":
        rows = [cu[b] for b in first]
        s["prefix_table"] = table_of(B, len(need))
        s["prefix_cu_q"], s["prefix_lens"] = ints(rows), ints(prefix_lens)
        s["prefix_q_max"] = max(b - a for a, b in zip(rows, rows[1:]))
        s["prefix_max"] = max(prefix_lens)
    else:
        # (sequence, position) of every cached token, as the host knows them
        s["tok_b"] = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(kv_lens, device=DEV))
        s["tok_j"] = torch.cat([torch.arange(n, device=DEV) for n in kv_lens])
        # what the step's attention returned beside its output
        S = masked_scores(s, s["table"], s["cu_q"], s["kv_lens"], s["q_max"], s["kv_max"], True)
        top = S.amax(-1)
        s["lse"] = to_rows(top + S.sub_(top.unsqueeze(-1)).exp_().sum(-1).log(), s["cu_q"], cu[-1]).contiguous()
    return s


# -------------------------------------------------------------------- runs ---

def run(s):
    op = s["case"]["op"]
    if own:
        return {"shared": own_shared, "weigh": own_weigh, "evict": own_evict}[op](s)
    return {"shared": plain_shared, "weigh": plain_weigh, "evict": plain_evict}[op](s)


def cache_of(s):
    import block_scaled_fp8_02_gb300 as bf
    return bf.KVCache(s["k"], s["v"], s["ks"], s["vs"])


def own_shared(s):
    import block_scaled_fp8_02_gb300 as bf
    out, lse = bf.bfp8_shared_prefix_attention(s["q"], cache_of(s), s["prefix_table"], s["prefix_cu_q"], s["prefix_lens"],
                                               s["prefix_q_max"], s["prefix_max"], s["table"], s["cu_q"], s["kv_lens"],
                                               s["q_max"], s["kv_max"], scale=s["scale"], return_lse=True)
    return {"out": out, "lse": lse}


def own_weigh(s):
    import block_scaled_fp8_02_gb300 as bf
    bf.bfp8_kv_cache_weigh(s["q"], s["lse"], cache_of(s), s["weights"], s["table"], s["cu_q"], s["kv_lens"], s["q_max"],
                           s["kv_max"], scale=s["scale"], window=s["case"]["window"], accumulate=s["case"]["add"])
    return {"weights": s["weights"]}


def own_evict(s):
    import block_scaled_fp8_02_gb300 as bf
    c = s["case"]
    lens = bf.bfp8_kv_cache_evict(cache_of(s), s["weights"], s["table"], s["kv_lens"], s["kv_max"], c["budget"],
                                  recent=c["recent"], first=c["first"], out_table=s["out_table"])
    return {"k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"], "weights": s["weights"], "lens": lens}


def context(q, sc, table, n):
    """[B, H, n, D] fp32 keys or values of the first n tokens of every row of the table (past its end: whatever is there)."""
    x = q.view(torch.uint8)[table.long()].view(torch.float8_e4m3fn).float() * sc[table.long()].unsqueeze(-1)
    B, P, H, page, D = x.shape
    return x.transpose(1, 2).reshape(B, H, P * page, D)[:, :, :n]


def from_rows(x, cu, m):
    """[B, m, ...] rows of every sequence (past its end: some other row)."""
    at = cu[:-1].long()[:, None] + torch.arange(m, device=x.device)
    return x[at.clamp(max=x.shape[0] - 1)]


def to_rows(x, cu, T):
    """[T, H * g, ...] of x [B, H, g, m, ...]."""
    t = torch.arange(T, device=x.device)
    b = torch.searchsorted(cu.long(), t, right=True) - 1
    y = x.movedim(3, 1)[b, t - cu.long()[b]]
    return y.reshape(T, y.shape[1] * y.shape[2], *y.shape[3:])


def masked_scores(s, table, cu, lens, m, n, causal):
    """[B, H, g, m, n] fp32 scores, -inf where the row does not see the token."""
    c = s["case"]
    H, D, B = c["kv_heads"], c["dim"], table.shape[0]
    g = c["heads"] // H
    K = context(s["k"], s["ks"], table, n)
    Q = from_rows(s["q"], cu, m).float().view(B, m, H, g, D).permute(0, 2, 3, 1, 4).reshape(B, H, g * m, D)
    S = torch.matmul(Q, K.transpose(-1, -2)).mul_(s["scale"]).view(B, H, g, m, n)
    j, i, q_len = torch.arange(n, device=K.device), torch.arange(m, device=K.device), (cu[1:] - cu[:-1]).long()
    if causal:
        pos = ((lens.long() - q_len)[:, None] + i)[..., None]
        seen = j <= pos
        if c.get("window", 0):
            seen &= j > pos - c["window"]
    else:
        seen = (j < lens.long()[:, None, None]).expand(B, m, n)
    return S.masked_fill_(~seen[:, None, None], -math.inf)


def part(s, table, cu, lens, m, n, causal):
    """Of every row: the largest score over one part of its context, the sum of the weights by it, the weighted values."""
    T = s["q"].shape[0]
    S = masked_scores(s, table, cu, lens, m, n, causal)
    top = S.amax(-1)
    S.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top).unsqueeze(-1)).exp_()
    B, H, g, _, _ = S.shape
    O = torch.matmul(S.view(B, H, g * m, n), context(s["v"], s["vs"], table, n)).view(B, H, g, m, -1)
    return to_rows(top, cu, T), to_rows(S.sum(-1), cu, T), to_rows(O, cu, T)


def plain_shared(s):
    t1, l1, o1 = part(s, s["prefix_table"], s["prefix_cu_q"], s["prefix_lens"], s["prefix_q_max"], s["prefix_max"], False)
    t2, l2, o2 = part(s, s["table"], s["cu_q"], s["kv_lens"], s["q_max"], s["kv_max"], True)
    top = torch.maximum(t1, t2)
    f1, f2 = torch.exp(t1 - top), torch.exp(t2 - top)
    total = l1 * f1 + l2 * f2
    out = (o1 * f1.unsqueeze(-1) + o2 * f2.unsqueeze(-1)) / total.unsqueeze(-1)
    return {"out": out.to(torch.bfloat16), "lse": top + total.log()}


def plain_weigh(s):
    c = s["case"]
    B, H = s["table"].shape[0], c["kv_heads"]
    g, m, n, page = c["heads"] // H, s["q_max"], s["kv_max"], c["page"]
    S = masked_scores(s, s["table"], s["cu_q"], s["kv_lens"], m, n, True)
    lse = from_rows(s["lse"], s["cu_q"], m).view(B, m, H, g).permute(0, 2, 3, 1)
    live = torch.arange(m, device=S.device) < (s["cu_q"][1:] - s["cu_q"][:-1])[:, None]
    S.sub_(lse.unsqueeze(-1)).exp_().mul_(live[:, None, None, :, None])
    got = S.view(B, H, g * m, n).sum(2)
    b, j = s["tok_b"], s["tok_j"]
    w, at, off = s["weights"].transpose(1, 2), s["table"][b, j // page].long(), j % page
    got = got[b, :, j]
    if c["add"]:
        new = j >= (s["kv_lens"].long() - (s["cu_q"][1:] - s["cu_q"][:-1]).long())[b]       # their sums begin here
        got = got + torch.where(new[:, None], torch.zeros_like(got), w[at, off])
    w[at, off] = got
    return {"weights": s["weights"]}


def plain_evict(s):
    c = s["case"]
    page, n, budget = c["page"], s["kv_max"], c["budget"]
    t = s["table"].long()
    B, P = t.shape
    W = s["weights"][t].transpose(1, 2).reshape(B, c["kv_heads"], P * page)[:, :, :n]
    lens, j = s["kv_lens"].long()[:, None], torch.arange(n, device=t.device)
    always = (j < c["first"]) | (j >= lens - c["recent"]) | (lens <= budget)
    W = torch.where(always[:, None], torch.full_like(W, math.inf), W)
    W = torch.where((j < lens)[:, None], W, torch.full_like(W, -math.inf))
    keep = torch.sort(W, dim=-1, descending=True, stable=True).indices[:, :, :budget]
    last = torch.arange(keep.shape[-1], device=t.device) >= lens
    keep = torch.where(last[:, None], n, keep).sort(-1).values
    b, i = s["stay_b"], s["stay_i"]
    src = keep[b, :, i]                                                                      # [N, H]
    at, h = t[b[:, None], src // page], torch.arange(c["kv_heads"], device=t.device)
    to, off = s["out_table"].long()[b, i // page], i % page
    for x in (s["k"].view(torch.uint8), s["v"].view(torch.uint8), s["ks"], s["vs"], s["weights"]):
        x[to, :, off] = x[at, h, src % page]
    return {"k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"], "weights": s["weights"],
            "lens": s["kv_lens"].clamp(max=budget)}


# ------------------------------------------------------------------- exact ---

def exact(case, seed):
    """The definition in 64 bits."""
    s = prepare(case, seed)
    q_lens, kv_lens = lengths(case)
    page, H, D = case["page"], case["kv_heads"], case["dim"]
    if case["op"] == "evict":
        got = {"k": s["k"].double(), "v": s["v"].double(), "k_scale": s["ks"].double(), "v_scale": s["vs"].double(),
               "weights": s["weights"].double(), "lens": s["kv_lens"].clone()}
        for b, n in enumerate(kv_lens):
            m = min(n, case["budget"])
            got["lens"][b] = m
            j, i = torch.arange(n, device=DEV), torch.arange(m, device=DEV)
            src, dst = s["table"][b].long()[j // page] * page + j % page, s["out_table"][b].long()[i // page] * page + i % page
            for h in range(H):
                flat = [x[:, h].reshape(-1, *x.shape[3:]) for x in (s["k"].view(torch.uint8), s["v"].view(torch.uint8), s["ks"],
                                                                    s["vs"], s["weights"])]
                keep = j
                if n > m:
                    lo, hi = case["first"], n - case["recent"]
                    mid = flat[4][src[lo:hi]]
                    need = m - lo - case["recent"]
                    border = mid.sort(descending=True).values[need - 1] if need else math.inf
                    over, ties = (mid > border).nonzero().flatten(), (mid == border).nonzero().flatten()
                    mid = torch.cat([over, ties[:need - len(over)]]).sort().values + lo
                    keep = torch.cat([j[:lo], mid, j[hi:]])
                for x, name in zip(flat, ("k", "v", "k_scale", "v_scale", "weights")):
                    row = x[src[keep]]
                    row = row.view(torch.float8_e4m3fn).double() if row.dtype == torch.uint8 else row.double()
                    got[name][dst // page, h, dst % page] = row
        return got
    g = case["heads"] // H
    T = s["q"].shape[0]
    w = s["weights"].double() if case["op"] == "weigh" else None
    out = torch.zeros(T, case["heads"], D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(T, case["heads"], dtype=torch.float64, device=DEV)

    def rows_of(x, sc, pages, n, h):
        return (x.view(torch.uint8)[pages, h].view(torch.float8_e4m3fn).double() * sc[pages, h].double()[..., None]).reshape(-1, D)[:n]

    at = 0
    for b, (m, n) in enumerate(zip(q_lens, kv_lens)):
        pages = s["table"][b].long()
        j, pos = torch.arange(n, device=DEV), torch.arange(n - m, n, device=DEV)[:, None]
        hide = j > pos
        if case.get("window", 0):
            hide |= j <= pos - case["window"]
        for h in range(H):
            k = rows_of(s["k"], s["ks"], pages, n, h)
            if case["op"] == "weigh":
                total = torch.zeros(n, dtype=torch.float64, device=DEV)
                for r in range(h * g, (h + 1) * g):
                    x = (s["q"][at:at + m, r].double() @ k.T * s["scale"]).masked_fill(hide, -math.inf)
                    total += torch.exp(x - s["lse"][at:at + m, r].double()[:, None]).sum(0)
                if case["add"]:
                    total[:n - m] += s["weights"][pages, h].reshape(-1)[:n - m].double()
                w[pages[j // page], h, j % page] = total
                continue
            f = max(i for i in range(case["groups"]) if prefixes(case)[0][i] <= b)
            ahead, P = s["prefix_table"][f].long(), prefixes(case)[1][f]
            k = torch.cat([rows_of(s["k"], s["ks"], ahead, P, h), k])
            v = torch.cat([rows_of(s["v"], s["vs"], ahead, P, h), rows_of(s["v"], s["vs"], pages, n, h)])
            both = torch.cat([torch.zeros(m, P, dtype=torch.bool, device=DEV), hide], 1)
            for r in range(h * g, (h + 1) * g):
                x = (s["q"][at:at + m, r].double() @ k.T * s["scale"]).masked_fill(both, -math.inf)
                lse[at:at + m, r] = torch.logsumexp(x, 1)
                out[at:at + m, r] = torch.softmax(x, 1) @ v
        at += m
    return {"weights": w} if case["op"] == "weigh" else {"out": out, "lse": lse}
