"""The attention call's host side, without a device."""
from types import SimpleNamespace

import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from block_scaled_fp8_02_gb300 import _binding as B
from block_scaled_fp8_02_gb300 import build as bfbuild


def _args(T=3, Hq=4, H=2, D=64, pages=2, page=16):
    k = torch.zeros(pages, H, page, D, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(pages, H, page)
    return (torch.zeros(T, Hq, D).bfloat16(), bf.KVCache(k, k, s, s), torch.zeros(1, pages, dtype=torch.int32),
            torch.tensor([0, T], dtype=torch.int32), torch.tensor([20], dtype=torch.int32))


def test_long_prompts_share_a_workspace_size(monkeypatch):
    """One remembered size for all of them, not one for every length."""
    asked = []

    def size(*key):
        asked.append(key[1:])
        raise LookupError

    monkeypatch.setattr(B, "_attention_workspace", size)
    monkeypatch.setattr(B, "_stream_of", lambda stream: 0)
    for n in (1, 8, 33, 34, 1000, 1 << 20):
        with pytest.raises(LookupError):
            bf.bfp8_paged_attention(*_args(), n, 20)
    assert len(set(asked)) == 3


@pytest.fixture
def packed(monkeypatch):
    """The calls' argument structures, instead of the calls."""
    calls = []

    def attention(args, desc, ws, ws_bytes, stream):
        calls.append(dict(zip([f for f, _ in B.AttentionArgs._fields_], B._pack_attention.unpack(args))))
        return 0

    monkeypatch.setattr(B, "_lib", SimpleNamespace(bfp8_paged_attention=attention))
    monkeypatch.setattr(B, "_stream_of", lambda stream: 0)
    return calls


@pytest.mark.parametrize("T,Hq", [(1, 4), (3, 1), (1, 1)])
def test_strides_of_single_tokens_and_heads_are_free(packed, T, Hq):
    """A slice of one has whatever stride its parent had; the library wants multiples of 8 elements, at least head_dim."""
    D = 64
    _, cache, table, cu, kv = _args(T=T, H=1)
    q = torch.zeros(10 * 10 * D).bfloat16()
    token = 3 if T == 1 else Hq * D
    head = 5 if Hq == 1 else D
    q, out = (torch.as_strided(q, (T, Hq, D), (token, head, 1)) for _ in range(2))
    bf.bfp8_paged_attention(q, cache, table, cu, kv, T, 20, out=out, workspace=torch.zeros(16))
    a = packed[0]
    for n in ("q_stride_token", "q_stride_head", "out_stride_token", "out_stride_head"):
        assert a[n] % 8 == 0 and a[n] >= D
    assert T == 1 or a["q_stride_token"] == token
    assert Hq == 1 or a["q_stride_head"] == head


def test_a_table_of_one_page_may_be_a_column(packed):
    q, cache, _, cu, kv = _args()
    wide = torch.zeros(1, 4, dtype=torch.int32)
    bf.bfp8_paged_attention(q, cache, torch.as_strided(wide, (1, 1), (4, 4)), cu, kv, 3, 16, workspace=torch.zeros(16))
    assert packed[0]["max_pages"] == 1 and packed[0]["ld_table"] == 1


@pytest.mark.parametrize("T,batch", [(0, 1), (0, 0), (0, 3), (5, 0)])
def test_empty_calls_with_bounds_of_zero(T, batch):
    """The natural bounds of a batch without new tokens are zero; nothing is launched, so no device is needed."""
    bfbuild.build()
    q, cache, _, _, _ = _args(T=T)
    table = torch.zeros(batch, 0, dtype=torch.int32)
    cu, kv = torch.zeros(batch + 1, dtype=torch.int32), torch.zeros(batch, dtype=torch.int32)
    out, lse = bf.bfp8_paged_attention(q, cache, table, cu, kv, 0, 0, return_lse=True, workspace=torch.zeros(256), stream=0)
    assert out.shape == q.shape and lse.shape == (T, 4)
    with pytest.raises(bf.BFP8Error):
        bf.bfp8_paged_attention(q, cache, table, cu, kv, -1, 0, workspace=torch.zeros(256), stream=0)


def test_tensors_of_another_device_are_refused(packed):
    q, cache, table, cu, kv = _args()
    ws = torch.zeros(16)
    bf.bfp8_paged_attention(q, cache, table, cu, kv, 3, 20, workspace=ws)
    for i, t in ((1, table), (2, cu), (3, kv)):
        args = [cache, table, cu, kv]
        args[i] = t.to("meta")
        with pytest.raises(ValueError):
            bf.bfp8_paged_attention(q, *args, 3, 20, workspace=ws)
    for kw in (dict(out=q.to("meta"), workspace=ws), dict(workspace=ws.to("meta"))):
        with pytest.raises(ValueError):
            bf.bfp8_paged_attention(q, cache, table, cu, kv, 3, 20, **kw)
    assert len(packed) == 1
    k, s, slots = q[:, :2].contiguous(), torch.zeros(2, 2, 16), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        bf.KVCache(cache.k, cache.v, s, s.to("meta"))
    for args in ((k, k.to("meta"), cache, slots), (k, k, cache, slots.to("meta"))):
        with pytest.raises(ValueError):
            bf.bfp8_kv_cache_write(*args)
    with pytest.raises(ValueError):
        bf.bfp8_kv_cache_read(cache, slots.to("meta"))
    x = torch.zeros(3, 8)
    for kw in (dict(weight=torch.ones(8, device="meta")), dict(weight=None, residual=x.to("meta"))):
        with pytest.raises(ValueError):
            bf.bfp8_rmsnorm_quant(x, **kw)
