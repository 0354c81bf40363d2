"""64-bit references of the attention-block operators (numpy-free torch on the CPU) and the error bounds that
their arithmetic allows."""
import math

import torch

FP8_MAX = 448.0


def quant_rows(x, ue8m0=False):
    """Codes (float8_e4m3fn) and fp32 scales of fp32 rows x (last axis one group): IEEE fp32 divisions."""
    x = x.float()
    s = x.abs().amax(-1).clamp(min=1e-10) / FP8_MAX
    if ue8m0:
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    return (x / s.unsqueeze(-1)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn), s


def attention_ref(q, k, v, ks, vs, table, cu_q, kv_lens, scale, causal=True, window=0):
    """out, lse, and per element A = sum_j w_j |v_j| and per row B = scale * max|q| * max_j sum_d |k_j| -- what the
    bounds below are relative to.  q [T, Hq, D]; k, v [P, H, page, D] codes; lists of lengths."""
    T, Hq, D = q.shape
    H, page = k.shape[1], k.shape[2]
    g = Hq // H
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    A = torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    B = torch.zeros(T, Hq, dtype=torch.float64)
    K = k.double() * ks.double()[..., None]
    V = v.double() * vs.double()[..., None]
    for b, n in enumerate(kv_lens):
        r0, r1 = cu_q[b], cu_q[b + 1]
        m = r1 - r0
        if m == 0 or n == 0:
            continue
        pages = table[b].long()[: (n + page - 1) // page]
        kb = K[pages].transpose(1, 2).reshape(-1, H, D)[:n]
        vb = V[pages].transpose(1, 2).reshape(-1, H, D)[:n]
        pos = torch.arange(n - m, n)[:, None]
        j = torch.arange(n)[None]
        seen = (j <= pos) if causal else (j < n).expand(m, n)
        if window:
            seen = seen & (j > pos - window)
        for h in range(Hq):
            x = (q[r0:r1, h].double() @ kb[:, h // g].T) * scale
            x = x.masked_fill(~seen, -math.inf)
            lse[r0:r1, h] = torch.logsumexp(x, 1)
            w = torch.exp(x - torch.where(lse[r0:r1, h] == -math.inf, 0.0, lse[r0:r1, h])[:, None])
            out[r0:r1, h] = w @ vb[:, h // g]
            A[r0:r1, h] = w @ vb[:, h // g].abs()
            B[r0:r1, h] = abs(scale) * q[r0:r1, h].double().abs().amax(1) * kb[:, h // g].abs().sum(1).max()
    return out, lse, A, B


def check_attention(out, lse, ref):
    """Scores are within d = 2^-17 B of the exact ones (queries held to 2^-17.8 of their largest element at
    worst, fp32 sums of exact products otherwise), so weights within a factor exp(2 d); weights and scaled values are
    rounded to 11 bits (2^-11 each), the output to 8 (2^-8)."""
    want, want_lse, A, B = ref
    d = 2.0 ** -17 * B
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -10 + 2.0 ** -16 + torch.expm1(2 * d)[..., None]) * 1.01 * A + 1e-37
    bad = (got - want).abs() > tol
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} elements, worst "
                           f"{float(((got - want).abs() / tol).max()):.2f} x bound, first {bad.nonzero()[0].tolist()}")
    if lse is not None:
        g = lse.double().cpu()
        empty = torch.isinf(want_lse)
        assert torch.equal(torch.isinf(g) & (g < 0), empty)
        ok = (g - want_lse).abs()[~empty] <= (d + 2.0 ** -19 * (1 + want_lse.abs()))[~empty]
        assert ok.all(), float((g - want_lse).abs()[~empty].max())


def make_cache(pages, H, page, D, g, spread=0.5, device="cpu"):
    """Random codes and scales as a cache holds them: keys N(0,1), values of sizes spread over the tokens."""
    k = torch.randn(pages, H, page, D, generator=g)
    v = torch.randn(pages, H, page, D, generator=g) * torch.exp(spread * torch.randn(pages, H, page, 1, generator=g))
    return (*quant_rows(k.bfloat16()), *quant_rows(v.bfloat16()))


def make_table(kv_lens, page, pages, g):
    width = max(1, max((n + page - 1) // page for n in kv_lens))
    order = torch.randperm(pages, generator=g)
    table = torch.zeros(len(kv_lens), width, dtype=torch.int32)
    at = 0
    for b, n in enumerate(kv_lens):
        c = (n + page - 1) // page
        table[b, :c] = order[at:at + c].int()
        at += c
    return table
