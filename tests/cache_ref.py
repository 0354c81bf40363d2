"""64-bit references, on the CPU, of the operators that share, weigh and shorten a paged cache, and the error bounds that
their arithmetic allows."""
import math

import torch


def rows_of(x, sc, table, n):
    """[n, H, D] fp64 keys or values of the first n tokens on the pages of `table`."""
    page = x.shape[2]
    pages = table.long()[: (n + page - 1) // page]
    v = x.view(torch.uint8)[pages].view(x.dtype).double() * sc[pages].double()[..., None]
    return v.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:n]


def seen_by(m, n, causal, window):
    """[m, n]: which of n tokens each of the m newest sees."""
    pos, j = torch.arange(n - m, n)[:, None], torch.arange(n)[None]
    seen = (j <= pos) if causal else torch.ones(m, n, dtype=torch.bool)
    return seen & (j > pos - window) if window else seen


def shared_ref(q, k, v, ks, vs, ptable, pcu, plens, table, cu_q, kv_lens, scale, causal=True):
    """out, lse and the quantities that check_attention's bounds are relative to (as attention_ref returns them)."""
    T, Hq, D = q.shape
    g = Hq // k.shape[1]
    out, A = (torch.zeros(T, Hq, D, dtype=torch.float64) for _ in range(2))
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    B = torch.zeros(T, Hq, dtype=torch.float64)
    own = [(rows_of(k, ks, table[b], n), rows_of(v, vs, table[b], n)) for b, n in enumerate(kv_lens)]
    ahead = [(rows_of(k, ks, ptable[f], n), rows_of(v, vs, ptable[f], n)) for f, n in enumerate(plens)]
    for b, n in enumerate(kv_lens):
        m = cu_q[b + 1] - cu_q[b]
        seen = seen_by(m, n, causal, 0)
        for i in range(m):
            t = cu_q[b] + i
            parts = [(own[b][0][seen[i]], own[b][1][seen[i]])]
            parts += [ahead[f] for f in range(len(plens)) if pcu[f] <= t < pcu[f + 1]]
            K, V = (torch.cat([p[e] for p in parts]) for e in (0, 1))
            if len(K) == 0:
                continue
            K, V = K.repeat_interleave(g, 1), V.repeat_interleave(g, 1)
            x = torch.einsum("hd,jhd->hj", q[t].double(), K) * scale
            lse[t] = torch.logsumexp(x, 1)
            w = torch.exp(x - lse[t][:, None])
            out[t] = torch.einsum("hj,jhd->hd", w, V)
            A[t] = torch.einsum("hj,jhd->hd", w, V.abs())
            B[t] = abs(scale) * q[t].double().abs().amax(1) * K.abs().sum(2).amax(0)
    return out, lse, A, B


def weigh_ref(q, lse, k, ks, weights, table, cu_q, kv_lens, scale, causal=True, window=0, accumulate=True):
    """The weights after the call, and how far each may be off: scores are sums of D products in fp32 (within D 2^-24
    of the terms' sum, at most B as in attention_ref), x = score - lse is rounded a few times at the size of either (and
    the exponential by 2^-21), and R terms are added one by one (R 2^-24)."""
    T, Hq, D = q.shape
    H, page = k.shape[1], k.shape[2]
    g = Hq // H
    want, tol = weights.double().clone(), torch.zeros_like(weights, dtype=torch.float64)
    for b, n in enumerate(kv_lens):
        r0, m = cu_q[b], cu_q[b + 1] - cu_q[b]
        if m == 0 or n == 0:
            continue
        K = rows_of(k, ks, table[b], n)
        seen = seen_by(m, n, causal, window)
        total, off = (torch.zeros(n, H, dtype=torch.float64) for _ in range(2))
        for h in range(Hq):
            x = q[r0:r0 + m, h].double() @ K[:, h // g].T * scale
            ls = lse[r0:r0 + m, h].double()[:, None]
            w = torch.where(seen, torch.exp(x - ls), 0.0)
            terms = abs(scale) * (q[r0:r0 + m, h].double().abs() @ K[:, h // g].abs().T)
            d = D * 2.0 ** -24 * terms + 2.0 ** -21 * (1 + x.abs() + torch.where(seen, ls.abs(), 0.0))
            total[:, h // g] += w.sum(0)
            off[:, h // g] += (w * torch.expm1(torch.where(seen, d, 0.0))).sum(0)
        off += total * (m * g * 2.0 ** -24)
        j = torch.arange(n)
        at, o = table[b].long()[j // page], j % page
        old = want[at, :, o].clone()
        if not accumulate:
            old.zero_()
        elif causal:
            old[max(0, n - m):] = 0
        want[at, :, o] = old + total
        tol[at, :, o] = 1.01 * off + 2.0 ** -23 * (old.abs() + total) + 1e-37
    return want, tol


def check_weights(got, before, ref):
    """Places of no sequence keep their bits."""
    want, tol = ref
    got = got.cpu()
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(),
                           float(((got.double() - want).abs() / tol.clamp(min=1e-300))[bad].max()))
    rest = tol == 0
    assert torch.equal(got[rest].view(torch.int32), before.cpu()[rest].view(torch.int32))


def kept_positions(w, budget, recent, first):
    """Positions of one head's n weights that stay."""
    n = len(w)
    if n <= budget:
        return list(range(n))
    always = [j for j in range(n) if j < first or j >= n - recent]
    rest = [j for j in range(n) if first <= j < n - recent]

    def heavy(j):
        v = float(w[j])
        return (0, 0.0, j) if math.isnan(v) else (1, -v, j)
    return sorted(always + sorted(rest, key=heavy)[: budget - len(always)])


def evict_ref(parts, weights, table, kv_lens, budget, recent, first, out_table=None):
    """parts: tensors [pages, H, page, ...] that move (the weights last); copies of them after the call, and the lengths."""
    H, page = weights.shape[1], weights.shape[2]
    got = [x.clone() for x in parts]
    dst = table if out_table is None else out_table
    for b, n in enumerate(kv_lens):
        for h in range(H):
            j = torch.arange(n)
            w = weights[table[b].long()[j // page], h, j % page]
            for i, p in enumerate(kept_positions(w, budget, recent, first)):
                for x, y in zip(parts, got):
                    y[dst[b, i // page], h, i % page] = x[table[b, p // page], h, p % page]
    return got, [min(n, budget) for n in kv_lens]
