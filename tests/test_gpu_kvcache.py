"""The paged e4m3 cache on the GPU: codes, scales and values bit for bit."""
import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from attn_ref import quant_rows
from block_scaled_fp8_02_gb300 import build as bfbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    bfbuild.build()
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def _layout(order, P, H, page, D, dev):
    """A cache filled with 0x55 codes and scale 7, as [page, head, token], [page, token, head] or with keys and
    values interleaved by page."""
    if order == "phtd":
        k, v = (torch.full((P, H, page, D), 0x55, dtype=torch.uint8, device=dev) for _ in range(2))
    elif order == "pthd":
        k, v = (torch.full((P, page, H, D), 0x55, dtype=torch.uint8, device=dev).transpose(1, 2) for _ in range(2))
    else:
        kv = torch.full((P, 2, H, page, D), 0x55, dtype=torch.uint8, device=dev)
        k, v = kv[:, 0], kv[:, 1]
    ks, vs = (torch.full((P, H, page), 7.0, device=dev) for _ in range(2))
    return bf.KVCache(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs)


@pytest.mark.parametrize("order", ["phtd", "pthd", "kv"])
@pytest.mark.parametrize("T,H,D,page", [(1, 8, 128, 64), (77, 1, 64, 16), (500, 3, 128, 32), (1000, 8, 64, 128),
                                        (33, 5, 128, 256)])
@pytest.mark.parametrize("dtype,ue8m0", [(torch.bfloat16, False), (torch.float32, False), (torch.bfloat16, True)])
def test_write_then_read(dev, order, T, H, D, page, dtype, ue8m0):
    g = torch.Generator().manual_seed(T * 7 + D)
    P = (T + page - 1) // page + 3
    cache = _layout(order, P, H, page, D, dev)
    # keys and values as columns of a projection's output, one row of zeros and one tiny one
    qkv = torch.randn(T, (2 + 2 * H) * D, generator=g).to(dtype)
    qkv[T // 2] = 0
    qkv[T - 1] *= 1e-12
    qkv = qkv.to(dev)
    k = qkv[:, 2 * D:(2 + H) * D].view(T, H, D)
    v = qkv[:, (2 + H) * D:].view(T, H, D)
    slots = torch.randperm(P * page, generator=g)[:T]
    skipped = slots.clone()
    skipped[::5] = -1
    bf.bfp8_kv_cache_write(k, v, cache, skipped.to(dev), ue8m0=ue8m0)
    torch.cuda.synchronize()
    for x, codes, scales in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        want_q, want_s = quant_rows(x.cpu(), ue8m0)
        got_q = codes.view(torch.uint8).cpu().transpose(1, 2).reshape(P * page, H, D)
        got_s = scales.cpu().transpose(1, 2).reshape(P * page, H)
        put = skipped >= 0
        assert torch.equal(got_q[slots[put]], want_q.view(torch.uint8)[put])
        assert torch.equal(got_s[slots[put]], want_s[put])
        rest = torch.ones(P * page, dtype=torch.bool)
        rest[slots[put]] = False
        assert (got_q[rest] == 0x55).all() and (got_s[rest] == 7.0).all()      # nothing else is touched
    for out in (torch.bfloat16, torch.float32):
        rk, rv = bf.bfp8_kv_cache_read(cache, skipped.to(dev), dtype=out)
        for got, codes, scales in ((rk, cache.k, cache.k_scale), (rv, cache.v, cache.v_scale)):
            q = codes.view(torch.uint8).cpu().transpose(1, 2).reshape(P * page, H, D)[slots].view(torch.float8_e4m3fn)
            s = scales.cpu().transpose(1, 2).reshape(P * page, H)[slots]
            want = (q.float() * s[..., None]).to(out)
            want[skipped < 0] = 0
            assert torch.equal(got.cpu(), want)
    assert bf.bfp8_device_status(clear=True) == 0


def test_slots_outside_the_cache_are_recorded_and_harmless(dev):
    cache = _layout("phtd", 2, 2, 16, 64, dev)
    k = torch.randn(3, 2, 64, device=dev).bfloat16()
    slots = torch.tensor([5, 32, 1 << 40], device=dev)
    bf.bfp8_kv_cache_write(k, k, cache, slots)
    assert bf.bfp8_device_status(clear=True) == 6            # BFP8_DEV_BAD_CACHE_INDEX
    assert int((cache.k.view(torch.uint8) != 0x55).any(-1).sum()) <= 2          # slot 5's two heads at most
    rk, _ = bf.bfp8_kv_cache_read(cache, slots)
    assert bf.bfp8_device_status(clear=True) == 6
    assert (rk[1:] == 0).all() and rk[0].any()


def test_empty_calls_and_another_stream(dev):
    cache = _layout("phtd", 4, 2, 16, 128, dev)
    none = torch.empty(0, dtype=torch.int64, device=dev)
    e = torch.empty(0, 2, 128, device=dev).bfloat16()
    bf.bfp8_kv_cache_write(e, e, cache, none)
    assert bf.bfp8_kv_cache_read(cache, none)[0].shape == (0, 2, 128)
    s = torch.cuda.Stream()
    k = torch.randn(20, 2, 128, device=dev).bfloat16()
    slots = torch.arange(20, device=dev)
    s.wait_stream(torch.cuda.current_stream())
    bf.bfp8_kv_cache_write(k, k, cache, slots, stream=s)
    s.synchronize()
    q, sc = quant_rows(k.cpu())
    got = cache.k.view(torch.uint8).cpu().transpose(1, 2).reshape(64, 2, 128)[:20]
    assert torch.equal(got, q.view(torch.uint8))


def test_offsets_past_32_bits(dev):
    """A cache whose last page starts beyond 2^32 bytes."""
    P, H, page, D = 5, 2, 16, 128
    big = torch.zeros((P - 1) * (1 << 30) + 2 * H * page * D, dtype=torch.uint8, device=dev)
    kc = torch.as_strided(big, (P, H, page, D), (1 << 30, page * D, D, 1))
    vc = torch.as_strided(big, (P, H, page, D), (1 << 30, page * D, D, 1), H * page * D)
    sc = [torch.zeros(P, H, page, device=dev) for _ in range(2)]
    cache = bf.KVCache(kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), *sc)
    k, v = (torch.randn(P * page, H, D, device=dev).bfloat16() for _ in range(2))
    slots = torch.arange(P * page, device=dev)
    bf.bfp8_kv_cache_write(k, v, cache, slots)
    rk, rv = bf.bfp8_kv_cache_read(cache, slots, dtype=torch.float32)
    for x, got in ((k, rk), (v, rv)):
        q, s = quant_rows(x.cpu())
        assert torch.equal(got.cpu(), q.float() * s[..., None])
