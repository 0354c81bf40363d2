"""The attention-block entry points reject bad arguments on the host, before any device is touched."""
import ctypes

import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from block_scaled_fp8_02_gb300 import _binding as B
from block_scaled_fp8_02_gb300 import build as bfbuild


@pytest.fixture(scope="module")
def L():
    bfbuild.build()
    return bf.lib()


P = 256        # a fake, aligned device address: nothing is dereferenced on the host
OK_STATUS = (0, 3)      # 3: the device check, without a GPU


def _norm(L, **kw):
    a = dict(x=P, dt=0, ld_x=256, r=P, ld_r=256, ro=P, ld_ro=256, w=P, wd=0, eps=1e-6, M=0, K=256, y=None, ld_y=256,
             col=1, fmt=0, q=P, ld_q=256, s=P, ld_s=4)
    a.update(kw)
    return L.bfp8_rmsnorm_quant(*a.values(), None)


def test_norm(L):
    assert _norm(L) == 0                                          # M == 0
    for bad in (dict(dt=2), dict(wd=-1), dict(fmt=2), dict(col=2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(M=-1), dict(K=0), dict(K=(1 << 20) + 1)):
        assert _norm(L, **bad) == 1, bad
    for bad in (dict(x=None), dict(s=None), dict(q=None), dict(ro=None, q=None, s=None), dict(ld_x=255), dict(ld_r=255),
                dict(r=512, ro=1024, ld_ro=255), dict(ro=P, ld_ro=512, r=P), dict(y=P, ld_y=255), dict(ld_q=255),
                dict(ld_s=3), dict(col=0, ld_s=1)):
        assert _norm(L, M=4, **bad) == 1, bad
    for bad in (dict(x=257), dict(r=257, ro=512), dict(w=257), dict(w=258, wd=1), dict(y=257), dict(s=258),
                dict(x=258, dt=1, r=None)):
        assert _norm(L, M=4, **bad) == 2, bad
    if not torch.cuda.is_available():
        assert _norm(L, M=4) == 3


def _cache(**kw):
    a = dict(k=P, v=P, ks=P, vs=P, pages=4, page=64, heads=2, dim=128, res=0, sp=2 * 64 * 128, sh=64 * 128, st=128,
             ssp=128, ssh=64)
    a.update(kw)
    return B.KVCacheDesc(*a.values())


BAD_CACHE = [(dict(k=None), 1), (dict(vs=None), 1), (dict(page=48), 1), (dict(page=8), 1), (dict(page=512), 1),
             (dict(dim=96), 1), (dict(heads=0), 1), (dict(pages=0), 1), (dict(pages=1 << 31), 1), (dict(st=64), 1),
             (dict(ssh=63), 1), (dict(sp=1 << 40), 1), (dict(st=136), 2), (dict(ssh=66), 2), (dict(k=264), 2),
             (dict(ks=260), 2)]


def _write(L, c=None, **kw):
    a = dict(k=P, v=P, dt=0, kt=256, kh=128, vt=256, vh=128, slots=P, T=3, fmt=0)
    a.update(kw)
    return L.bfp8_kv_cache_write(*a.values(), ctypes.byref(c or _cache()), None)


def _read(L, c=None, **kw):
    a = dict(slots=P, T=3, dt=0, k=P, kt=256, v=P, vt=256)
    a.update(kw)
    return L.bfp8_kv_cache_read(ctypes.byref(c or _cache()), *a.values(), None)


def test_cache_calls(L):
    for kw, want in BAD_CACHE:
        assert _write(L, _cache(**kw)) == want and _read(L, _cache(**kw)) == want, kw
    assert L.bfp8_kv_cache_write(P, P, 0, 256, 128, 256, 128, P, 3, 0, None, None) == 1
    assert _write(L, T=0) == 0 and _read(L, T=0) == 0
    for bad in (dict(k=None), dict(slots=None), dict(dt=2), dict(fmt=3), dict(T=-1), dict(kt=-1)):
        assert _write(L, **bad) == 1, bad
    for bad in (dict(k=None, v=None), dict(slots=None), dict(dt=2), dict(T=-1), dict(kt=255), dict(vt=1)):
        assert _read(L, **bad) == 1, bad
    assert _write(L, k=257) == 2 and _write(L, slots=260) == 2 and _read(L, v=257) == 2
    assert _write(L, T=1 << 30) == 3 and _read(L, T=1 << 30) == 3         # too large for one launch


def _attend(L, c=None, ws=P, wsb=1 << 30, **kw):
    a = dict(q=P, out=P, lse=P, T=10, heads=8, batch=2, qt=1024, qh=128, ot=1024, oh=128, table=P, ld=8, mp=8, mq=5,
             mkv=500, cu=P, kv=P, scale=0.1, causal=1, window=0, res=0)
    a.update(kw)
    return L.bfp8_paged_attention(ctypes.byref(B.AttentionArgs(*a.values())), ctypes.byref(c or _cache()), ws, wsb, None)


def test_attention(L):
    for kw, want in BAD_CACHE:
        assert _attend(L, _cache(**kw)) == want, kw
    for bad in (dict(heads=7), dict(heads=1), dict(heads=2 * 129), dict(batch=-1), dict(T=-1), dict(mp=0), dict(ld=7),
                dict(mkv=513), dict(mkv=-1), dict(mq=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(causal=2),
                dict(window=-1), dict(q=None), dict(out=None), dict(table=None), dict(cu=None), dict(kv=None),
                dict(qt=-8), dict(oh=120), dict(ot=64)):
        assert _attend(L, **bad) == 1, bad
    for bad in (dict(q=264), dict(out=258), dict(lse=258), dict(table=258), dict(cu=257), dict(kv=258), dict(qt=1025),
                dict(oh=132)):
        assert _attend(L, **bad) == 2, bad
    assert _attend(L, wsb=16) == 5 and _attend(L, ws=None) == 5 and _attend(L, ws=128) == 5
    assert "workspace" in bf.bfp8_last_error()
    assert _attend(L, batch=0) == 0 and _attend(L, T=0) == 0
    n = ctypes.c_size_t(0)
    size = L.bfp8_paged_attention_workspace_size
    assert size(7, 2, 128, 1, ctypes.byref(n)) == 1 and size(8, 2, 80, 1, ctypes.byref(n)) == 1
    assert size(8, 2, 128, 0, ctypes.byref(n)) == 1 and size(8, 2, 128, 1, None) == 1
    if not torch.cuda.is_available():
        assert _attend(L) == 3


def test_binding_refuses_mismatched_tensors():
    f8, f32 = torch.float8_e4m3fn, torch.float32
    k = torch.zeros(2, 2, 16, 64, dtype=torch.uint8).view(f8)
    s = torch.zeros(2, 2, 16)
    c = bf.KVCache(k, k, s, s)
    for bad in ((k, k, s[:1], s), (k, k.view(torch.uint8), s, s), (k, k, s, s.double()),
                (k, k.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(f8), s, s)):
        with pytest.raises(ValueError):
            bf.KVCache(*bad)
    x = torch.zeros(3, 2, 64).bfloat16()
    slots = torch.zeros(3, dtype=torch.int64)
    for args in ((x[:, :1], x, c, slots), (x, x.float(), c, slots), (x.half(), x.half(), c, slots), (x, x, c, slots[:2]),
                 (x, x, c, slots.int())):
        with pytest.raises(ValueError):
            bf.bfp8_kv_cache_write(*args)
    with pytest.raises(ValueError):
        bf.bfp8_kv_cache_read(c, slots, dtype=torch.float16)
    q = torch.zeros(3, 4, 64).bfloat16()
    t, cu, kv = torch.zeros(1, 2, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32), torch.tensor([20], dtype=torch.int32)
    for args in ((q.float(), c, t, cu, kv), (q[..., :32], c, t, cu, kv), (q, c, t.long(), cu, kv), (q, c, t, cu[:1], kv),
                 (q, c, t[:0], cu, kv)):
        with pytest.raises(ValueError):
            bf.bfp8_paged_attention(*args, 3, 20)
    w = torch.ones(8)
    for args, kw in (((torch.zeros(3, 8).half(), w), {}), ((torch.zeros(3, 8), w[:7]), {}),
                     ((torch.zeros(3, 8), w), dict(residual=torch.zeros(3, 8).bfloat16())),
                     ((torch.zeros(3, 16)[:, ::2], w), {})):
        with pytest.raises(ValueError):
            bf.bfp8_rmsnorm_quant(*args, **kw)
