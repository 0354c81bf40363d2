"""bfp8_rmsnorm_quant on the GPU against a 64-bit reference."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from block_scaled_fp8_02_gb300 import build as bfbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    bfbuild.build()
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def _reference(x, r, w, eps):
    h = x.double() + (r.double() if r is not None else 0.0)
    y = h / (h.square().mean(1, keepdim=True) + eps).sqrt()
    return h, y * w.double() if w is not None else y


def _check(x, r, w, eps, q, s, ro, y_out, ue8m0):
    h, y = _reference(x.cpu(), r.cpu() if r is not None else None, w.cpu() if w is not None else None, eps)
    M, K = h.shape
    G = (K + 127) // 128
    if ro is not None:
        # one fp32 addition, one rounding
        want = h.float().to(x.dtype)
        unit = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
        assert ((ro.cpu().double() - h).abs() <= unit * 1.001 * h.abs() + 2.0 ** -24 * h.abs()).all()
        assert (ro.cpu() == want).float().mean() > 0.999
    # fp32: the sum of squares within K 2^-24 (halved by the root), two products, the root
    e = (K / 2 + 8) * 2.0 ** -24
    if y_out is not None:
        assert ((y_out.cpu().double() - y).abs() <= (2.0 ** -8 * 1.001 + e) * y.abs() + 1e-38).all()
    if q is None:
        return
    yp = torch.nn.functional.pad(y, (0, G * 128 - K)).view(M, G, 128)
    amax = yp.abs().amax(-1).clamp(min=1e-10)
    want_s = amax / 448.0
    s = s.cpu().double()
    if ue8m0:
        lo, hi = (torch.exp2(torch.ceil(torch.log2(want_s * f))) for f in (1 - 2 * e, 1 + 2 * e))
        assert ((s == lo) | (s == hi)).all()
    else:
        assert ((s - want_s).abs() <= (2.0 ** -23 + 2 * e) * want_s).all()
    # a code stands for a value within half an e4m3 step of y / s: 2^-4 relative, 2^-10 absolute where subnormal
    codes = torch.nn.functional.pad(q.cpu().float().double(), (0, G * 128 - K)).view(M, G, 128)
    ratio = yp / s[..., None]
    assert ((codes - ratio).abs() <= (2.0 ** -4 + 4 * e) * ratio.abs().clamp(min=2.0 ** -6)).all()
    # and it is the code of some quotient within the arithmetic's error of the exact one
    def encode(t):
        return t.float().clamp(-448, 448).to(torch.float8_e4m3fn).float().double()
    d = 4 * e + 2.0 ** -23
    assert ((codes == encode(ratio * (1 - d))) | (codes == encode(ratio * (1 + d)))).all()


CASES = [(1, 5120), (1, 1), (3, 127), (5, 128), (2, 129), (83, 7168), (1000, 1000), (7, 8192), (400, 264), (33, 12288),
         (2, 20000), (2, 40960), (1, 70001), (700, 5120), (0, 256)]


@pytest.mark.parametrize("M,K", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ue8m0,col_major", [(False, True), (True, False)])
def test_norm_against_64_bits(dev, M, K, dtype, ue8m0, col_major):
    g = torch.Generator().manual_seed(M * 131 + K)
    x = torch.randn(M, K, generator=g).to(dtype).to(dev)
    r = (3 * torch.randn(M, K, generator=g)).to(dtype).to(dev)
    w = (1 + 0.2 * torch.randn(K, generator=g)).to(torch.bfloat16 if K % 2 else torch.float32).to(dev)
    ro = torch.empty_like(r)
    q, s, y = bf.bfp8_rmsnorm_quant(x, w, residual=r, residual_out=ro, eps=1e-6, col_major=col_major, ue8m0=ue8m0,
                                    want_y=True)
    torch.cuda.synchronize()
    assert q.shape == (M, K) and s.shape == (M, (K + 127) // 128)
    if M:
        _check(x, r, w, 1e-6, q, s, ro, y, ue8m0)


@pytest.mark.parametrize("M,K", [(5, 512), (300, 1000), (2, 40960)])
def test_norm_in_place_equals_out_of_place(dev, M, K):
    x = torch.randn(M, K, device=dev).bfloat16()
    r = torch.randn(M, K, device=dev).bfloat16()
    w = torch.rand(K, device=dev).bfloat16()
    ro = torch.empty_like(r)
    q0, s0 = bf.bfp8_rmsnorm_quant(x, w, residual=r, residual_out=ro)
    r1 = r.clone()
    q1, s1 = bf.bfp8_rmsnorm_quant(x, w, residual=r1)
    x1 = x.clone()
    q2, s2 = bf.bfp8_rmsnorm_quant(x1, w, residual=r, residual_out=x1)
    for a, b in ((q0, q1), (q0, q2)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(s0, s1) and torch.equal(s0, s2) and torch.equal(ro, r1) and torch.equal(ro, x1)


@pytest.mark.parametrize("K", [256, 1000])
def test_norm_strided_rows_and_plain_forms(dev, K):
    """Rows of a wider buffer at an odd column (the element-wise path), no residual, no weight, no quantisation."""
    M = 37
    wide = torch.randn(M, K + 77, generator=torch.Generator().manual_seed(K)).bfloat16().to(dev)
    for first in (0, 8, 5):
        x = wide[:, first:first + K]
        q, s, y = bf.bfp8_rmsnorm_quant(x, None, eps=1e-5, want_y=True)
        _check(x, None, None, 1e-5, q, s, None, y, False)
        q, s, y = bf.bfp8_rmsnorm_quant(x, None, eps=1e-5, want_y=True, quantise=False)
        assert q is None and s is None
        _check(x, None, None, 1e-5, None, None, None, y, False)


def test_norm_zero_rows_and_one_hot(dev):
    x = torch.zeros(3, 512, device=dev).bfloat16()
    x[1, 300] = 5.0
    q, s, y = bf.bfp8_rmsnorm_quant(x, torch.ones(512, device=dev), eps=1e-6, want_y=True)
    assert (y[0] == 0).all() and (q[0].float() == 0).all()
    assert (s[0].cpu().numpy() == np.float32(1e-10) / np.float32(448)).all()
    assert abs(float(y[1, 300]) - 512 ** 0.5) < 0.1 and float(q[1].float()[300]) == 448.0


def test_norm_feeds_the_gemm(dev):
    """Its codes and scales are what bfp8_gemm takes: the same as quantising y in fp32 with bfp8_group_quant."""
    M, K, N = 64, 5120, 512
    g = torch.Generator().manual_seed(5)
    x, r = (torch.randn(M, K, generator=g).bfloat16().to(dev) for _ in range(2))
    w = torch.rand(K, generator=g).to(dev)
    q, s = bf.bfp8_rmsnorm_quant(x, w, residual=r.clone())
    h = x.float() + r.float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * w
    q2, s2 = bf.bfp8_group_quant(y)
    B = torch.randn(N, K, generator=g).to(dev).clamp(-448, 448).to(torch.float8_e4m3fn)
    Bs = torch.rand((N + 127) // 128, K // 128, generator=g).to(dev)
    a, b = bf.bfp8_gemm(q, B, s, Bs).float(), bf.bfp8_gemm(q2, B, s2, Bs).float()
    assert float((a - b).norm() / b.norm()) < 2e-3
