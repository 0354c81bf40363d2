"""The example's attention block on the GPU: norm, projections, cache and attention together."""
import importlib.util
import os

import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from block_scaled_fp8_02_gb300 import build as bfbuild

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.fixture(scope="module")
def ex():
    bfbuild.build()
    assert torch.cuda.is_available()
    return _example()


def test_chunks_and_single_tokens_agree_with_one_pass(ex):
    """The same numbers up to the projections' tile shapes: a bf16 rounding of q, k and v here and there (2^-8 each),
    and with it now and then a neighbouring e4m3 code (2^-4 of one element)."""
    err, drift = ex.main(hidden=512, heads=8, kv_heads=2, dim=128, batch=2, length=600)
    assert err < 2 ** -6
    # a stored value is code * scale with the largest code 448: quantising it again gives the same code, but
    # for the scale's own rounding (2^-23), and so the same value up to that
    assert drift < 2 ** -20


def test_block_against_fp32(ex):
    """One pass of a small block against the same steps in fp32 torch on the dequantised operands."""
    dev = torch.device("cuda")
    blk = ex.AttentionBlock(512, 8, 2, 64, dev)
    x = torch.randn(1, 300, 512, generator=torch.Generator().manual_seed(3)).bfloat16().to(dev)
    got, cache, seqs = ex.run(blk, x, 1, [300], page=32)

    def deq(w):
        q, s = w
        N, K = q.shape
        return (q.float().view(N // 128, 128, K // 128, 128) * s[:, None, :, None]).view(N, K)

    h = x[0].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * blk.norm.float()
    qkv = y @ deq(blk.qkv).T
    q, k, v = qkv[:, :512].view(300, 8, 64), qkv[:, 512:640].view(300, 2, 64), qkv[:, 640:].view(300, 2, 64)
    s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(4, 1)) * 64 ** -0.5
    s = s.masked_fill(torch.ones(300, 300, device=dev).triu(1).bool(), float("-inf"))
    o = torch.einsum("hij,jhd->ihd", s.softmax(-1), v.repeat_interleave(4, 1)).reshape(300, 512)
    want = o @ deq(blk.out).T
    err = float((got[0].float() - want).norm() / want.norm())
    # four 8-bit roundings (inputs of two projections, keys, values), each with a relative error of about 2^-5 / sqrt(3) a
    # element; keys act on the weights through scores of order one
    assert err < 2 * 2 ** -5
    assert bf.bfp8_device_status() == 0
