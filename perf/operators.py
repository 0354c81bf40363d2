"""The operators around the linear layers of a W8A8 decoder block, as measured cases.

  norm    residual addition + root-mean-square norm, output as e4m3 codes with fp32 scales per 128 elements
  write   new keys and values quantised into a paged e4m3 cache, one fp32 scale per (token, head)
  read    rows of that cache back as bf16
  attend  attention of new tokens (one to thousands a sequence) over the paged cache, grouped heads

`own` false: the plain forms below, elementary torch operations in 32 bits.  `own` true: the library's calls.
"""
import math

import torch

own = False

FP8_MAX = 448.0
DEV = "cuda"


# ------------------------------------------------------------------- cases ---

def listed():
    """Widths and heads are those of the repository's Qwen3-32B-sized layers (hidden 5120, 64 query and 8 key
    heads of 128) and of its ragged workloads (K = 7168 and 1000, M = 1000)."""
    norm = dict(op="norm", f32=False, ue8m0=False, col_major=True)
    attend = dict(op="attend", heads=64, kv_heads=8, dim=128, page=64, window=0)
    return [
        # one token of a single stream before its qkv projection: latency
        dict(norm, name="norm m1 k5120", M=1, K=5120),
        # a ragged batch, fp32 activations, power-of-two scales, row-major scales
        dict(norm, name="norm m1000 k7168 f32", M=1000, K=7168, f32=True, ue8m0=True, col_major=False),
        # a prefill chunk
        dict(norm, name="norm m8192 k5120", M=8192, K=5120),
        # the new tokens of a decode batch
        dict(op="write", name="write t64", T=64, kv_heads=8, heads=64, dim=128, page=64, ue8m0=False),
        # the new tokens of a prefill chunk
        dict(op="write", name="write t8192", T=8192, kv_heads=8, heads=64, dim=128, page=64, ue8m0=False),
        # a short prefix handed to another worker, small pages, narrow heads
        dict(op="read", name="read t1000 d64", T=1000, kv_heads=8, dim=64, page=16),
        # a long prefix
        dict(op="read", name="read t65536", T=65536, kv_heads=8, dim=128, page=64),
        # single-stream decoding at a long context
        dict(attend, name="decode b1 32k", mode="decode", B=1, q_max=1, kv_max=32768),
        # a decode batch of ragged contexts
        dict(attend, name="decode b64 8k", mode="decode", B=64, q_max=1, kv_max=8000),
        # chunked prefill and decoding in one batch
        dict(attend, name="mixed b16 q512 8k", mode="mixed", B=16, q_max=512, kv_max=8192),
        # a long prompt's chunk over what came before it
        dict(attend, name="chunk q4096 16k", mode="chunk", B=1, q_max=4096, kv_max=16384),
        # narrow heads in groups of three, odd lengths, small pages, a sliding window
        dict(attend, name="chunk d64 window", mode="chunk", B=8, q_max=333, kv_max=2500, heads=24, kv_heads=8, dim=64,
             page=16, window=777),
    ]


MAX_SCORES = 4096 * 16384 * 64


def draw(rng):
    def logint(lo, hi):
        return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    op = rng.choice(["norm", "write", "read", "attend", "attend", "attend"])
    if op == "norm":
        K = logint(256, 8192)
        if rng.random() < 0.7:
            K = max(256, K // 128 * 128)
        return dict(op=op, M=logint(1, 8192), K=K if K != 3072 else 2944, f32=rng.random() < 0.3, ue8m0=rng.random() < 0.3,
                    col_major=rng.random() < 0.7)
    heads, kv_heads = rng.choice([(64, 8), (40, 8), (24, 8), (8, 8), (16, 1), (32, 4)])
    dim, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if op == "write":
        return dict(op=op, T=logint(1, 8192), heads=heads, kv_heads=kv_heads, dim=dim, page=page, ue8m0=rng.random() < 0.3)
    if op == "read":
        return dict(op=op, T=logint(1, 65536), kv_heads=kv_heads, dim=dim, page=page)
    mode = rng.choice(["decode", "mixed", "chunk"])
    B = logint(1, 64) if mode == "decode" else logint(1, 16)
    kv_max = logint(16, 32768 if B < 8 else 8192)
    q_max = 1 if mode == "decode" else min(kv_max, logint(2, 2048))
    while B * q_max * kv_max * heads > MAX_SCORES // 2:
        q_max = max(1, q_max // 2)
    return dict(op=op, mode=mode, B=B, q_max=q_max, kv_max=kv_max, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                window=rng.choice([0, 0, 0, 128, 1000]))


def lengths(case):
    """New tokens and context (which holds them) of every sequence: spread over the range, the first one longest."""
    q, kv = [], []
    for i in range(case["B"]):
        n = case["kv_max"] if i == 0 else 1 + int((case["kv_max"] - 1) * ((i * 0.6180339887) % 1.0))
        if case["mode"] == "decode" or (case["mode"] == "mixed" and i % 2 == 1):
            m = 1
        else:
            m = case["q_max"] if i == 0 else 1 + int((case["q_max"] - 1) * ((i * 0.4142135624) % 1.0))
        q.append(min(m, n))
        kv.append(n)
    return q, kv


def visible(case):
    """(query, key) pairs that the mask leaves, and the keys that some query sees."""
    pairs = keys = 0
    w = case["window"]
    for m, n in zip(*lengths(case)):
        full = sum(min(p + 1, w) for p in range(n - m, n)) if w else m * (n - m) + m * (m + 1) // 2
        pairs += full
        keys += min(n, m - 1 + w) if w else n
    return pairs, keys


def work(case):
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        b = 4 if case["f32"] else 2
        return {"bytes": M * K * (3 * b + 1) + 4 * M * ((K + 127) // 128) + 2 * K, "flops": 10 * M * K}
    H, D = case["kv_heads"], case["dim"]
    if case["op"] in ("write", "read"):
        T = case["T"]
        return {"bytes": T * (2 * H * (3 * D + 4) + 8), "flops": 4 * T * H * D}
    pairs, keys = visible(case)
    T = sum(lengths(case)[0])
    Hq = case["heads"]
    return {"bytes": keys * H * (2 * D + 8) + T * Hq * (4 * D + 4), "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs ---

def quantised(x):
    """e4m3 codes and fp32 scales of rows of x (its last axis)."""
    s = x.abs().amax(-1).clamp(min=1e-10) / FP8_MAX
    return (x / s.unsqueeze(-1)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        t = torch.float32 if case["f32"] else torch.bfloat16
        # a layer's output beside a residual stream that has grown over the layers, with a few large channels
        big = 1.0 + 20.0 * (torch.rand(K, generator=g, device=DEV) < 0.004).float()
        x, r = randn(M, K).to(t), (randn(M, K) * 4 * big).to(t)
        w = (1 + 0.2 * randn(K)).to(torch.bfloat16)
        return dict(case=case, x=x, r=r, r_out=torch.empty_like(r), w=w)
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "attend":
        q_lens, kv_lens = lengths(case)
        need = [(n + page - 1) // page for n in kv_lens]
    else:
        need = [(case["T"] + case["T"] // 4 + page) // page]
    pages = sum(need) + 3
    # keys with a common part and a token that every query attends to, values of differing size a token
    k = randn(pages, H, page, D) + 0.5 * randn(1, H, 1, D)
    v = randn(pages, H, page, D) * torch.exp(0.5 * randn(pages, 1, page, 1))
    (kq, ks), (vq, vs) = quantised(k.to(torch.bfloat16).float()), quantised(v.to(torch.bfloat16).float())
    del k, v
    s = dict(case=case, k=kq, v=vq, ks=ks, vs=vs)
    order = torch.randperm(pages, generator=g, device=DEV)
    if case["op"] in ("write", "read"):
        T = case["T"]
        at = torch.arange(T, device=DEV) + torch.randint(0, page, (1,), generator=g, device=DEV)
        s["slots"] = (order[at // page] * page + at % page).to(torch.int64)
        if case["op"] == "write":
            # the keys' and values' columns of a fused projection's output
            qkv = randn(T, (case["heads"] + 2 * H) * D).to(torch.bfloat16)
            s["new_k"] = qkv[:, case["heads"] * D:(case["heads"] + H) * D].view(T, H, D)
            s["new_v"] = qkv[:, (case["heads"] + H) * D:].view(T, H, D)
    else:
        width = max(need)
        table = torch.zeros(len(need), width, dtype=torch.int32, device=DEV)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n].to(torch.int32)
            at += n
        cu = [0]
        for m in q_lens:
            cu.append(cu[-1] + m)
        s["table"] = table
        s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["kv_lens"] = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
        s["q"] = (randn(cu[-1], case["heads"], D) * 2).to(torch.bfloat16)
        s["q_max"], s["kv_max"] = max(q_lens), max(kv_lens)
        s["scale"] = 1.0 / math.sqrt(D)
    return s


# -------------------------------------------------------------------- runs ---

def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm": own_norm, "write": own_write, "read": own_read, "attend": own_attend}[op](s)
    return {"norm": plain_norm, "write": plain_write, "read": plain_read, "attend": plain_attend}[op](s)


def cache_of(s):
    import block_scaled_fp8_02_gb300 as bf
    return bf.KVCache(s["k"], s["v"], s["ks"], s["vs"])


def own_norm(s):
    import block_scaled_fp8_02_gb300 as bf
    c = s["case"]
    q, sc = bf.bfp8_rmsnorm_quant(s["x"], s["w"], residual=s["r"], residual_out=s["r_out"], eps=1e-6,
                                  col_major=c["col_major"], ue8m0=c["ue8m0"])
    return {"q": q, "s": sc, "residual": s["r_out"]}


def own_write(s):
    import block_scaled_fp8_02_gb300 as bf
    bf.bfp8_kv_cache_write(s["new_k"], s["new_v"], cache_of(s), s["slots"], ue8m0=s["case"]["ue8m0"])
    return {"k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"]}


def own_read(s):
    import block_scaled_fp8_02_gb300 as bf
    k, v = bf.bfp8_kv_cache_read(cache_of(s), s["slots"])
    return {"k": k, "v": v}


def own_attend(s):
    import block_scaled_fp8_02_gb300 as bf
    out, lse = bf.bfp8_paged_attention(s["q"], cache_of(s), s["table"], s["cu_q"], s["kv_lens"], s["q_max"], s["kv_max"],
                                       scale=s["scale"], window=s["case"]["window"], return_lse=True)
    return {"out": out, "lse": lse}


def ceil_pow2(x):
    """Positive fp32 values rounded up to powers of two."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.ones_like(x), torch.where(m == 0.5, e - 1, e))


def scale_of(amax, ue8m0):
    s = amax.clamp(min=1e-10) / FP8_MAX
    return ceil_pow2(s) if ue8m0 else s


def codes(x, s):
    return (x / s).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def plain_norm(s):
    c = s["case"]
    M, K = s["x"].shape
    G = (K + 127) // 128
    h = s["x"].float() + s["r"].float()
    s["r_out"].copy_(h)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["w"].float()
    y = torch.nn.functional.pad(y, (0, G * 128 - K)).view(M, G, 128)
    sc = scale_of(y.abs().amax(-1), c["ue8m0"])
    q = codes(y, sc.unsqueeze(-1)).view(M, G * 128)[:, :K]
    return {"q": q, "s": sc, "residual": s["r_out"]}


def plain_write(s):
    page = s["case"]["page"]
    at, off = s["slots"] // page, s["slots"] % page
    for x, q, sc in ((s["new_k"], s["k"], s["ks"]), (s["new_v"], s["v"], s["vs"])):
        x = x.float()
        ns = scale_of(x.abs().amax(-1), s["case"]["ue8m0"])
        q.view(torch.uint8)[at, :, off] = codes(x, ns.unsqueeze(-1)).view(torch.uint8)
        sc[at, :, off] = ns
    return {"k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"]}


def rows(q, sc, at, off):
    return q.view(torch.uint8)[at, :, off].view(torch.float8_e4m3fn).float() * sc[at, :, off].unsqueeze(-1)


def plain_read(s):
    page = s["case"]["page"]
    at, off = s["slots"] // page, s["slots"] % page
    return {"k": rows(s["k"], s["ks"], at, off).to(torch.bfloat16), "v": rows(s["v"], s["vs"], at, off).to(torch.bfloat16)}


def context(q, sc, table, n):
    """[B, H, n, D] fp32 keys or values of the first n tokens of every sequence (past its end: whatever is there)."""
    x = q.view(torch.uint8)[table.long()].view(torch.float8_e4m3fn).float() * sc[table.long()].unsqueeze(-1)
    B, P, H, page, D = x.shape
    return x.transpose(1, 2).reshape(B, H, P * page, D)[:, :, :n]


def plain_attend(s):
    c = s["case"]
    B, Hq, H, D = s["table"].shape[0], c["heads"], c["kv_heads"], c["dim"]
    g, m, n = Hq // H, s["q_max"], s["kv_max"]
    T = s["q"].shape[0]
    start, q_len = s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    K, V = context(s["k"], s["ks"], s["table"], n), context(s["v"], s["vs"], s["table"], n)
    i, j = torch.arange(m, device=DEV), torch.arange(n, device=DEV)
    Q = s["q"][(start[:, None] + i).clamp(max=T - 1)].float()                      # [B, m, Hq, D]
    Q = Q.view(B, m, H, g, D).permute(0, 2, 3, 1, 4).reshape(B, H, g * m, D)
    S = torch.matmul(Q, K.transpose(-1, -2)).mul_(s["scale"]).view(B, H, g, m, n)
    pos = (s["kv_lens"].long() - q_len)[:, None] + i                               # [B, m]
    seen = j <= pos[..., None]
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    S.masked_fill_(~seen[:, None, None], -math.inf)
    top = S.amax(-1, keepdim=True)
    S.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = S.sum(-1, keepdim=True)
    O = torch.matmul(S.view(B, H, g * m, n), V).view(B, H, g, m, D) / total.clamp(min=1e-38)
    lse = (top + total.log()).squeeze(-1)                                          # [B, H, g, m]
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(s["cu_q"].long(), t, right=True) - 1
    i = t - start[b]
    out = O.permute(0, 3, 1, 2, 4)[b, i].reshape(T, Hq, D).to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2)[b, i].reshape(T, Hq).contiguous()}


# ------------------------------------------------------------------- exact ---

def exact(case, seed):
    """The definition in 64 bits.  Codes come as the quotients that they round."""
    s = prepare(case, seed)

    def scale64(a):
        a = torch.maximum(a, torch.full_like(a, 1e-10)) / FP8_MAX
        return torch.exp2(torch.ceil(torch.log2(a.float().double()))) if case.get("ue8m0") else a

    if case["op"] == "norm":
        h = s["x"].double() + s["r"].double()
        y = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * s["w"].double()
        q, sc = torch.empty_like(y), []
        for k in range(0, y.shape[1], 128):
            part = y[:, k:k + 128]
            sc.append(scale64(part.abs().amax(1)))
            q[:, k:k + 128] = part / sc[-1][:, None]
        return {"q": q, "s": torch.stack(sc, 1), "residual": h}
    page = case["page"]
    if case["op"] == "write":
        got = {"k": s["k"].double(), "v": s["v"].double(), "k_scale": s["ks"].double(), "v_scale": s["vs"].double()}
        for name in ("k", "v"):
            x = s["new_" + name].double()
            a = scale64(x.abs().amax(-1))
            got[name].transpose(1, 2)[s["slots"] // page, s["slots"] % page] = x / a[..., None]
            got[name + "_scale"].transpose(1, 2)[s["slots"] // page, s["slots"] % page] = a
        return got
    K, V = ((q.double() * sc.double()[..., None]).transpose(1, 2) for q, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])))
    if case["op"] == "read":                                                       # K, V: [pages, page, H, D]
        at = s["slots"]
        return {"k": K[at // page, at % page], "v": V[at // page, at % page]}
    g = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (m, n) in enumerate(zip(*lengths(case))):
        pages = s["table"][b].long()
        seen_by = torch.arange(n - m, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)
        hide = j > seen_by
        if case["window"]:
            hide |= j <= seen_by - case["window"]
        for h in range(case["heads"]):
            k = K[pages, :, h // g].reshape(-1, case["dim"])[:n]
            v = V[pages, :, h // g].reshape(-1, case["dim"])[:n]
            x = (s["q"][at:at + m, h].double() @ k.T * s["scale"]).masked_fill(hide, -math.inf)
            lse[at:at + m, h] = torch.logsumexp(x, 1)
            out[at:at + m, h] = torch.softmax(x, 1) @ v
        at += m
    return {"out": out, "lse": lse}
