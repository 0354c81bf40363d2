"""The calls that share, weigh and shorten a paged cache reject bad arguments on the host, before any device is touched."""
import ctypes
from types import SimpleNamespace

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
BIG = 1 << 40


def _cache(**kw):
    a = dict(k=P, v=P, ks=P, vs=P, pages=40, page=64, heads=2, dim=128, res=0, sp=2 * 64 * 128, sh=64 * 128, st=128,
             ssp=128, ssh=64)
    a.update(kw)
    return B.KVCacheDesc(*a.values())


def _attention(**kw):
    a = dict(q=P, out=P, lse=P, total_q=6, heads=8, batch=3, qt=1024, qh=128, ot=1024, oh=128, table=P, ld=4, pages=4, max_q=4,
             max_kv=256, cu=P, kv=P, scale=0.1, causal=1, window=0, res=0)
    a.update(kw)
    return B.AttentionArgs(*a.values())


def _prefix(**kw):
    a = dict(table=P, ld=3, pages=3, prefixes=2, cu=P, lens=P, max_q=6, res=0, max_len=192)
    a.update(kw)
    return B.PrefixArgs(*a.values())


BAD_ATTENTION = [(dict(q=None), 1), (dict(table=None), 1), (dict(cu=None), 1), (dict(kv=None), 1), (dict(heads=7), 1),
                 (dict(heads=512), 1), (dict(batch=-1), 1), (dict(batch=70000), 1), (dict(total_q=-1), 1), (dict(pages=0), 1), (dict(ld=3), 1),
                 (dict(max_kv=257), 1), (dict(max_kv=-1), 1), (dict(max_q=0), 1), (dict(max_q=(1 << 24) + 1), 1),
                 (dict(scale=float("nan")), 1), (dict(causal=2), 1), (dict(window=-1), 1), (dict(qt=-8), 1), (dict(qh=132), 2),
                 (dict(q=264), 2), (dict(table=258), 2)]


@pytest.mark.parametrize("kw,status", BAD_ATTENTION + [(dict(out=None), 1), (dict(oh=64), 1), (dict(window=5), 1), (dict(out=264), 2)])
def test_shared_prefix_attention_arguments(L, kw, status):
    assert L.bfp8_shared_prefix_attention(ctypes.byref(_attention(**kw)), ctypes.byref(_prefix()), ctypes.byref(_cache()), P, BIG,
                                          None) == status, kw


@pytest.mark.parametrize("kw,status", [(dict(table=None), 1), (dict(cu=None), 1), (dict(lens=None), 1), (dict(prefixes=-1), 1),
                                       (dict(prefixes=70000), 1), (dict(pages=0), 1), (dict(ld=2), 1), (dict(max_len=193), 1),
                                       (dict(max_len=-1), 1), (dict(max_q=0), 1), (dict(max_q=(1 << 24) + 1), 1), (dict(cu=257), 2),
                                       (dict(lens=258), 2)])
def test_shared_prefix_attention_prefixes(L, kw, status):
    assert L.bfp8_shared_prefix_attention(ctypes.byref(_attention()), ctypes.byref(_prefix(**kw)), ctypes.byref(_cache()), P, BIG,
                                          None) == status, kw


def test_shared_prefix_attention_rest(L):
    f = L.bfp8_shared_prefix_attention
    a, p, c = ctypes.byref(_attention()), ctypes.byref(_prefix()), ctypes.byref(_cache())
    assert f(None, p, c, P, BIG, None) == 1 and f(a, None, c, P, BIG, None) == 1 and f(a, p, None, P, BIG, None) == 1
    assert f(a, p, c, None, BIG, None) == 5 and f(a, p, c, P, 100, None) == 5 and f(a, p, c, P + 16, BIG, None) == 5
    assert b"workspace" in L.bfp8_last_error()
    for empty in (dict(batch=0), dict(total_q=0), dict(batch=0, max_q=0, pages=0, ld=0, max_kv=0)):
        assert f(ctypes.byref(_attention(**empty)), p, c, None, 0, None) == 0
    n = ctypes.c_size_t()
    g = L.bfp8_shared_prefix_attention_workspace_size
    assert g(8, 2, 128, 4, 4, -1, ctypes.byref(n)) == 1 and g(8, 3, 128, 4, 4, 1, ctypes.byref(n)) == 1
    assert g(8, 2, 96, 4, 4, 1, ctypes.byref(n)) == 1 and g(8, 2, 128, 0, 4, 1, ctypes.byref(n)) == 1 and g(8, 2, 128, 4, 4, 1, None) == 1


def _weigh(L, a=None, c=None, w=P, sp=128, sh=64, acc=1, ws=P, ws_bytes=BIG):
    return L.bfp8_kv_cache_weigh(ctypes.byref(_attention(**(a or {}))), ctypes.byref(_cache(**(c or {}))), w, sp, sh, acc, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", BAD_ATTENTION + [(dict(lse=None), 1), (dict(qt=120), 1), (dict(qh=0), 1), (dict(lse=258), 2)])
def test_weigh_arguments(L, kw, status):
    assert _weigh(L, kw) == status, kw


def test_weigh_rest(L):
    for bad in (dict(w=None), dict(sp=63), dict(sh=63), dict(sp=1 << 39), dict(acc=2), dict(acc=-1)):
        assert _weigh(L, **bad) == 1, bad
    assert _weigh(L, w=P + 2) == 2
    assert _weigh(L, c=dict(page=48)) == 1 and _weigh(L, c=dict(st=136)) == 2
    assert _weigh(L, ws=None) == 5 and _weigh(L, ws_bytes=16) == 5 and _weigh(L, ws=P + 32) == 5
    # the output that an attention call would write is neither looked at nor needed
    if not torch.cuda.is_available():
        assert _weigh(L, dict(out=None, ot=0, oh=0)) == 3 and _weigh(L, dict(out=3, ot=-5, oh=1)) == 3
    for empty in (dict(batch=0), dict(total_q=0)):
        assert _weigh(L, empty, ws=None, w=None) == 0
    n = ctypes.c_size_t()
    g = L.bfp8_kv_cache_weigh_workspace_size
    assert g(8, 3, 128, 4, ctypes.byref(n)) == 1 and g(8, 2, 100, 4, ctypes.byref(n)) == 1 and g(8, 2, 128, 4, None) == 1


def _evict(L, c=None, ws=P, ws_bytes=BIG, **kw):
    a = dict(w=P, sp=128, sh=64, table=P, ld=8, out=P, ld_out=2, pages=8, out_pages=2, kv=P, new=2 * P, max_kv=512, budget=100,
             recent=10, first=4, batch=3, res=0)
    a.update(kw)
    return L.bfp8_kv_cache_evict(ctypes.byref(B.EvictArgs(*a.values())), ctypes.byref(_cache(**(c or {}))), ws, ws_bytes, None)


def test_evict_arguments(L):
    for bad in (dict(w=None), dict(table=None), dict(kv=None), dict(new=None), dict(new=P), dict(new=P + 8), dict(kv=2 * P + 8),
                dict(batch=-1), dict(batch=70000), dict(max_kv=-1), dict(max_kv=513), dict(max_kv=(1 << 30) + 1), dict(ld=7), dict(pages=-1),
                dict(budget=0), dict(budget=-5), dict(recent=-1), dict(first=-1), dict(recent=97), dict(first=91), dict(recent=101),
                dict(recent=1 << 62, first=1 << 62), dict(ld_out=1), dict(out_pages=1), dict(out_pages=1, ld_out=1), dict(sp=63), dict(sh=0)):
        assert _evict(L, **bad) == 1, bad
    for bad in (dict(w=P + 1), dict(table=P + 2), dict(out=P + 2), dict(kv=P + 1), dict(new=3 * P + 2)):
        assert _evict(L, **bad) == 2, bad
    assert _evict(L, batch=40000) == 3                                               # batch x kv heads
    assert _evict(L, c=dict(heads=0)) == 1 and _evict(L, c=dict(k=264)) == 2
    assert _evict(L, ws=None) == 5 and _evict(L, ws_bytes=16384) == 5 and _evict(L, ws=P + 8) == 5
    assert _evict(L, batch=0, kv=None, new=None, w=None, table=None, ws=None) == 0
    assert L.bfp8_kv_cache_evict(None, ctypes.byref(_cache()), P, BIG, None) == 1
    n = ctypes.c_size_t()
    g = L.bfp8_kv_cache_evict_workspace_size
    assert g(3, 2, 512, 100, ctypes.byref(n)) == 0 and n.value >= 3 * 2 * 100 * 4
    short = n.value - 4
    assert _evict(L, ws_bytes=short) == 5
    assert g(-1, 2, 512, 100, ctypes.byref(n)) == 1 and g(3, 0, 512, 100, ctypes.byref(n)) == 1 and g(3, 2, -1, 100, ctypes.byref(n)) == 1
    assert g(3, 2, 512, 0, ctypes.byref(n)) == 1 and g(3, 2, 512, 100, None) == 1
    if not torch.cuda.is_available():
        assert _evict(L) == 3 and _evict(L, out=None, ld_out=0, out_pages=0) == 3
        assert _evict(L, budget=1 << 40, max_kv=512, out_pages=8, ld_out=8) == 3      # nothing to evict


# ------------------------------------------------------------- the binding ---

def _tensors(T=3, Hq=4, H=2, D=64, pages=4, page=16):
    k = torch.zeros(pages, H, page, D, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(pages, H, page)
    return SimpleNamespace(q=torch.zeros(T, Hq, D).bfloat16(), lse=torch.zeros(T, Hq), cache=bf.KVCache(k, k, s, s), w=torch.zeros(pages, H, page),
                           table=torch.zeros(1, 2, dtype=torch.int32), cu=torch.tensor([0, T], dtype=torch.int32),
                           kv=torch.tensor([20], dtype=torch.int32))


@pytest.fixture
def fake(monkeypatch):
    calls = []

    def f(*args):
        calls.append(args)
        return 0
    monkeypatch.setattr(B, "_lib", SimpleNamespace(bfp8_shared_prefix_attention=f, bfp8_kv_cache_weigh=f, bfp8_kv_cache_evict=f))
    monkeypatch.setattr(B, "_stream_of", lambda stream: 0)
    return calls


def _shared(t, **kw):
    a = dict(q=t.q, cache=t.cache, prefix_table=t.table, prefix_cu_q=t.cu, prefix_lens=t.kv, max_prefix_q_len=3, max_prefix_len=20,
             block_table=t.table, cu_q=t.cu, kv_lens=t.kv, max_q_len=3, max_kv_len=20, workspace=torch.zeros(16))
    a.update(kw)
    return bf.bfp8_shared_prefix_attention(**a)


def test_shared_binding(fake):
    t = _tensors()
    out, lse = _shared(t, return_lse=True)
    assert out.shape == t.q.shape and lse.shape == (3, 4)
    a = dict(zip([f for f, _ in B.PrefixArgs._fields_], B._pack_prefix.unpack(fake[0][1])))
    assert (a["prefixes"], a["max_pages"], a["ld_table"], a["max_q_len"], a["max_len"]) == (1, 2, 2, 3, 20)
    for bad in (dict(q=t.q.float()), dict(q=t.q[0]), dict(prefix_table=t.table.long()), dict(prefix_cu_q=t.kv), dict(prefix_lens=t.cu),
                dict(prefix_table=torch.zeros(2, 2, dtype=torch.int32)), dict(prefix_lens=t.kv[None]), dict(cu_q=t.cu.long()),
                dict(block_table=t.table[0]), dict(out=torch.zeros(3, 4, 64)), dict(kv_lens=t.kv.to("meta")), dict(prefix_lens=t.kv.to("meta"))):
        with pytest.raises(ValueError):
            _shared(t, **bad)
    assert len(fake) == 1


def _weigh_call(t, **kw):
    a = dict(q=t.q, lse=t.lse, cache=t.cache, weights=t.w, block_table=t.table, cu_q=t.cu, kv_lens=t.kv, max_q_len=3, max_kv_len=20,
             workspace=torch.zeros(16))
    a.update(kw)
    return bf.bfp8_kv_cache_weigh(**a)


def test_weigh_binding(fake):
    t = _tensors()
    assert _weigh_call(t) is None
    assert fake[0][3:6] == (2 * 16, 16, 1)
    for bad in (dict(lse=t.lse.double()), dict(lse=t.lse[:2]), dict(lse=torch.zeros(4, 3).t()), dict(weights=t.w.double()), dict(weights=t.w[:3]),
                dict(weights=torch.zeros(4, 2, 32)[..., ::2]), dict(q=t.q[..., :32]), dict(kv_lens=t.kv.float()), dict(lse=t.lse.to("meta")),
                dict(weights=t.w.to("meta"))):
        with pytest.raises(ValueError):
            _weigh_call(t, **bad)
    assert len(fake) == 1


def _evict_call(t, **kw):
    a = dict(cache=t.cache, weights=t.w, block_table=t.table, kv_lens=t.kv, max_kv_len=20, budget=10, workspace=torch.zeros(16))
    a.update(kw)
    return bf.bfp8_kv_cache_evict(**a)


def test_evict_binding(fake):
    t = _tensors()
    lens = _evict_call(t, out_table=t.table)
    assert lens.shape == (1,) and lens.dtype == torch.int32
    a = dict(zip([f for f, _ in B.EvictArgs._fields_], B._pack_evict.unpack(fake[0][0])))
    assert (a["batch"], a["budget"], a["max_pages"], a["max_out_pages"], a["weights_stride_page"]) == (1, 10, 2, 2, 32)
    _evict_call(t)
    assert B._pack_evict.unpack(fake[1][0])[5] == 0                                  # in place
    for bad in (dict(block_table=t.table.long()), dict(block_table=t.table[0]), dict(out_table=torch.zeros(2, 1, dtype=torch.int32)),
                dict(kv_lens=t.kv.long()), dict(kv_lens=t.kv[None]), dict(new_lens=torch.zeros(2, dtype=torch.int32)),
                dict(new_lens=torch.zeros(1)), dict(weights=t.w[:, :1]), dict(out_table=t.table.to("meta")), dict(kv_lens=t.kv.to("meta"))):
        with pytest.raises(ValueError):
            _evict_call(t, **bad)
    assert len(fake) == 2


def test_one_workspace_size_for_every_length(monkeypatch):
    """The remembered sizes grow with what they go by, not with every length of a prompt or context."""
    asked = []

    def size(*key):
        asked.append(key)
        raise LookupError
    t = _tensors()
    monkeypatch.setattr(B, "_stream_of", lambda stream: 0)
    for name in ("_shared_workspace", "_weigh_workspace", "_evict_workspace"):
        monkeypatch.setattr(B, name, size)
    for n in (33, 34, 1000, 1 << 20):
        for call in (lambda: _shared(t, workspace=None, max_q_len=n, max_prefix_q_len=n), lambda: _weigh_call(t, workspace=None, max_q_len=n),
                     lambda: _evict_call(t, workspace=None, max_kv_len=n)):
            with pytest.raises(LookupError):
                call()
    assert len(set(asked)) == 3
