"""Forms of the cache's calls beside the ordinary ones: more places a token than a block has threads, rows that are not
aligned, keys or values alone."""
import ctypes

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


def _cache(P, H, page, D, dev):
    k, v = (torch.full((P, H, page, D), 0x55, dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.full((P, H, page), 7.0, device=dev) for _ in range(2))
    return bf.KVCache(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs)


def _rows(cache, slots):
    """(codes, scales) of slots, keys then values, on the CPU."""
    P, H, page, D = cache.shape
    out = []
    for q, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        out.append((q.view(torch.uint8).cpu().transpose(1, 2).reshape(P * page, H, D)[slots],
                    s.cpu().transpose(1, 2).reshape(P * page, H)[slots]))
    return out


@pytest.mark.parametrize("H,D", [(16, 128), (17, 128), (40, 64), (64, 128), (33, 64)])
@pytest.mark.parametrize("T", [1, 3, 700])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype,ue8m0", [(torch.bfloat16, False), (torch.float32, True)])
def test_many_heads_and_unaligned_rows(dev, H, D, T, shift, dtype, ue8m0):
    """shift: the columns of keys and values begin one element off a 16-byte boundary, in rows of an odd width."""
    g = torch.Generator().manual_seed(T + H)
    page = 16
    P = T // page + 2
    cache = _cache(P, H, page, D, dev)
    wide = torch.randn(T, 2 * H * D + shift, generator=g).to(dtype)
    wide[T // 2, shift:] = 0
    w = wide.to(dev)
    k, v = w[:, shift:shift + H * D].view(T, H, D), w[:, shift + H * D:].view(T, H, D)
    slots = torch.randperm(P * page, generator=g)[:T]
    bf.bfp8_kv_cache_write(k, v, cache, slots.to(dev), ue8m0=ue8m0)
    rest = torch.ones(P * page, dtype=torch.bool)
    rest[slots] = False
    for x, (q, s) in zip((k, v), _rows(cache, slots)):
        want_q, want_s = quant_rows(x.cpu(), ue8m0)
        assert torch.equal(q, want_q.view(torch.uint8)) and torch.equal(s, want_s)
    for q, s in _rows(cache, rest):
        assert (q == 0x55).all() and (s == 7.0).all()
    rk, rv = bf.bfp8_kv_cache_read(cache, slots.to(dev), dtype=dtype)
    for got, (q, s) in zip((rk, rv), _rows(cache, slots)):
        assert torch.equal(got.cpu(), (q.view(torch.float8_e4m3fn).float() * s[..., None]).to(dtype))
    assert bf.bfp8_device_status(clear=True) == 0


@pytest.mark.parametrize("H,D", [(2, 64), (8, 128), (40, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", ["k", "v", "kv"])
@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 0), (0, 3), (8, 16)])
def test_keys_or_values_alone_into_strided_rows(dev, H, D, dtype, which, shift, pad):
    T, page = 131, 32
    g = torch.Generator().manual_seed(H)
    P = T // page + 2
    cache = _cache(P, H, page, D, dev)
    x = torch.randn(2, P * page, H, D, generator=g).bfloat16().to(dev)
    bf.bfp8_kv_cache_write(x[0], x[1], cache, torch.arange(P * page, device=dev))
    slots = torch.randperm(P * page, generator=g)[:T]
    asked = slots.clone()
    asked[::9] = -1
    ld = H * D + pad
    outs = {n: torch.full((T * ld + shift,), 5.0, dtype=dtype, device=dev) for n in which}
    ptr = {n: o.data_ptr() + shift * o.element_size() for n, o in outs.items()}
    dt = 0 if dtype == torch.bfloat16 else 1
    dev_slots = asked.to(dev)
    rc = bf.lib().bfp8_kv_cache_read(cache._desc, dev_slots.data_ptr(), T, dt, ptr.get("k"), ld, ptr.get("v"), ld,
                                     ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0, bf.bfp8_last_error()
    torch.cuda.synchronize()
    for n, (q, s) in zip("kv", _rows(cache, slots)):
        if n not in outs:
            continue
        want = (q.view(torch.float8_e4m3fn).float() * s[..., None]).to(dtype)
        want[asked < 0] = 0
        got = outs[n].cpu()
        assert (got[:shift] == 5).all()
        rows = got[shift:].view(T, ld)
        assert torch.equal(rows[:, :H * D].view(T, H, D), want) and (rows[:, H * D:] == 5).all()
    assert bf.bfp8_device_status(clear=True) == 0
