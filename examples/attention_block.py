"""The attention half of a W8A8 decoder block on libbfp8: norm, fused qkv projection, paged 8-bit cache, attention
and output projection, as a serving step runs them.

    python examples/attention_block.py            # a prompt in chunks, then single tokens, checked against one pass

Everything between the two projections stays on the device in the library's kernels:

    q8, s = bfp8_rmsnorm_quant(x, w, residual=r)       # r += x; e4m3 codes + scales for the GEMM
    qkv   = bfp8_gemm(q8, Wqkv, s, Sqkv)
    bfp8_kv_cache_write(k, v, cache, slots)            # k, v are columns of qkv
    o     = bfp8_paged_attention(q, cache, ...)        # so is q
    y     = bfp8_linear(o, Wo, So)

(A rotary position encoding, which the library does not provide, would be applied to q and k before the write.)
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_02_gb300 as bf  # noqa: E402


def quantise_weight(w: torch.Tensor):
    """e4m3 codes and one fp32 scale per 128 x 128 tile of w [N, K] (N and K multiples of 128)."""
    N, K = w.shape
    t = w.view(N // 128, 128, K // 128, 128)
    s = t.abs().amax((1, 3)).clamp(min=1e-10) / 448.0
    q = (t / s[:, None, :, None]).clamp(-448, 448).view(N, K).to(torch.float8_e4m3fn)
    return q, s.contiguous()


class AttentionBlock:
    def __init__(self, hidden: int, heads: int, kv_heads: int, dim: int, device, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.norm = (1 + 0.1 * torch.randn(hidden, generator=g)).bfloat16().to(device)
        width = (heads + 2 * kv_heads) * dim
        self.qkv = quantise_weight((torch.randn(width, hidden, generator=g) / hidden ** 0.5).to(device))
        self.out = quantise_weight((torch.randn(hidden, heads * dim, generator=g) / (heads * dim) ** 0.5).to(device))

    def __call__(self, x, residual, cache, slots, table, cu_q, kv_lens, max_q_len, max_kv_len):
        """x [T, hidden] bf16: the new tokens of all sequences; residual is updated in place.  Returns the block's
        output, to be added to the residual by the next norm."""
        T = x.shape[0]
        hq, hk, d = self.heads, self.kv_heads, self.dim
        q8, s = bf.bfp8_rmsnorm_quant(x, self.norm, residual=residual)
        qkv = bf.bfp8_gemm(q8, self.qkv[0], s, self.qkv[1], options={"prefetch_weights": 1})
        q = qkv[:, :hq * d].view(T, hq, d)
        k = qkv[:, hq * d:(hq + hk) * d].view(T, hk, d)
        v = qkv[:, (hq + hk) * d:].view(T, hk, d)
        bf.bfp8_kv_cache_write(k, v, cache, slots)
        o = bf.bfp8_paged_attention(q, cache, table, cu_q, kv_lens, max_q_len, max_kv_len)
        return bf.bfp8_linear(o.view(T, hq * d), *self.out)


class Sequences:
    """The host's side of a paged cache: which pages each sequence owns and how long it is."""

    def __init__(self, batch: int, max_len: int, page: int, device):
        self.page, self.max_len, self.dev = page, max_len, device
        per = (max_len + page - 1) // page
        order = torch.randperm(batch * per, generator=torch.Generator().manual_seed(1))
        self.table_cpu = order.view(batch, per)
        self.table = self.table_cpu.int().to(device)
        self.lens = [0] * batch

    def append(self, counts):
        """Takes counts[b] new tokens of each sequence; the arguments of the step that computes them."""
        slots = []
        for b, n in enumerate(counts):
            at = torch.arange(self.lens[b], self.lens[b] + n)
            slots.append(self.table_cpu[b, at // self.page] * self.page + at % self.page)
            self.lens[b] += n
        cu = torch.tensor([0] + counts).cumsum(0).int().to(self.dev)
        kv = torch.tensor(self.lens, dtype=torch.int32, device=self.dev)
        return (torch.cat(slots).to(self.dev), self.table, cu, kv, max(counts), max(self.lens))


def run(block, x, batch, steps, page=64, cache=None):
    """Feeds x [batch, length, hidden] through the block in the given steps (tokens a sequence); returns the
    outputs [batch, length, hidden], the cache and the sequences."""
    _, length, hidden = x.shape
    seqs = Sequences(batch, length, page, x.device)
    if cache is None:
        cache = bf.KVCache.empty(seqs.table.numel(), block.kv_heads, page, block.dim, x.device)
    outs, at = [], 0
    for n in steps:
        xs = x[:, at:at + n].reshape(batch * n, hidden).contiguous()
        residual = torch.zeros_like(xs)
        outs.append(block(xs, residual, cache, *seqs.append([n] * batch)).view(batch, n, hidden))
        at += n
    return torch.cat(outs, 1), cache, seqs


def main(hidden=1024, heads=16, kv_heads=2, dim=128, batch=3, length=700, device="cuda"):
    dev = torch.device(device)
    block = AttentionBlock(hidden, heads, kv_heads, dim, dev)
    x = torch.randn(batch, length, hidden, generator=torch.Generator().manual_seed(2)).bfloat16().to(dev)
    whole, cache, seqs = run(block, x, batch, [length])
    # the same prompt in chunks, its last tokens one by one
    chunks = [256, 256, length - 512 - 4] + [1] * 4
    parts, _, _ = run(block, x, batch, chunks)
    err = float((parts.float() - whole.float()).norm() / whole.float().norm())
    print(f"chunks and single tokens against one pass: relative difference {err:.1e}")
    # sequence 0's prefix handed to another cache: read back, written again, the same values
    at = torch.arange(length)
    slots = (seqs.table_cpu[0, at // 64] * 64 + at % 64).to(dev)
    k, v = bf.bfp8_kv_cache_read(cache, slots, dtype=torch.float32)
    other = bf.KVCache.empty(seqs.table.shape[1], kv_heads, 64, dim, dev)
    bf.bfp8_kv_cache_write(k, v, other, torch.arange(length, device=dev))
    k2, v2 = bf.bfp8_kv_cache_read(other, torch.arange(length, device=dev), dtype=torch.float32)
    drift = max(float((a - b).abs().max() / a.abs().max()) for a, b in ((k, k2), (v, v2)))
    print(f"prefix of {length} tokens handed over: largest change {drift:.1e}")
    torch.cuda.synchronize()
    assert bf.bfp8_device_status() == 0
    return err, drift


if __name__ == "__main__":
    main()
