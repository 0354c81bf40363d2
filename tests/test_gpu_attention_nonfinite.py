"""What is not finite stays with the rows that see it: NaN and infinities among the keys, values, scales and queries."""
import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from attn_ref import attention_ref, check_attention, make_cache, make_table
from block_scaled_fp8_02_gb300 import build as bfbuild

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def dev():
    bfbuild.build()
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def _inputs(q_lens, kv_lens, Hq, H, D, page, seed):
    g = torch.Generator().manual_seed(seed)
    pages = sum((n + page - 1) // page for n in kv_lens) + 1
    kq, ks, vq, vs = make_cache(pages, H, page, D, g)
    table = make_table(kv_lens, page, pages, g)
    cu = [0]
    for m in q_lens:
        cu.append(cu[-1] + m)
    q = torch.randn(cu[-1], Hq, D, generator=g).bfloat16()
    return q, kq, ks, vq, vs, table, cu


def _attend(dev, q, kq, ks, vq, vs, table, cu, q_lens, kv_lens, causal=True, window=0):
    cache = bf.KVCache(*(t.to(dev) for t in (kq, vq, ks, vs)))
    out, lse = bf.bfp8_paged_attention(q.to(dev), cache, table.to(dev), torch.tensor(cu, dtype=torch.int32, device=dev),
                                       torch.tensor(kv_lens, dtype=torch.int32, device=dev), max(q_lens), max(kv_lens),
                                       causal=causal, window=window, return_lse=True)
    torch.cuda.synchronize()
    assert bf.bfp8_device_status(clear=True) == 0
    return out.cpu(), lse.cpu()


def _rows(ref, keep):
    return tuple(t[keep] for t in ref)


KINDS = ["value code", "value scale inf", "value scale nan", "key code", "key scale nan", "key scale inf"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", [(4, 200), (6, 131), (8, 300), (40, 333), (200, 700)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 50), (False, 60)])
@pytest.mark.parametrize("D", [64, 128])
def test_one_bad_token(dev, kind, m, n, causal, window, D):
    """Token j of the second sequence, kv head 0, is spoilt: among the new tokens, which earlier rows do not see, and
    just before them, which a window hides from later rows.  Rows that see it get no finite output (all elements but
    those of a finite part of the value), rows that do not, other heads and the other sequence their usual one."""
    Hq, H, page = 8, 2, 16
    g4 = Hq // H
    q_lens, kv_lens = [3, m], [150, n]
    for j in (n - (m + 1) // 2, n - m - 20):
        q, kq, ks, vq, vs, table, cu = _inputs(q_lens, kv_lens, Hq, H, D, page, 1000 * m + j)
        ref = attention_ref(q, kq, vq, ks, vs, table, cu, kv_lens, D ** -0.5, causal, window)
        pg, o = int(table[1, j // page]), j % page
        bad = [t.clone() for t in (kq.view(torch.uint8), ks, vq.view(torch.uint8), vs)]
        if kind.endswith("code"):
            bad[0 if kind[0] == "k" else 2][pg, 0, o, 17] = 0x7F
        else:
            bad[1 if kind[0] == "k" else 3][pg, 0, o] = INF if kind.endswith("inf") else NAN
        f8 = torch.float8_e4m3fn
        out, lse = _attend(dev, q, bad[0].view(f8), bad[1], bad[2].view(f8), bad[3], table, cu, q_lens, kv_lens, causal, window)
        p = torch.arange(n - m, n)
        sees = ((j <= p) if causal else torch.ones(m, dtype=torch.bool)) & ((j > p - window) if window else True)
        clean = torch.ones(cu[-1], Hq, dtype=torch.bool)
        clean[cu[1]:, :g4] = ~sees[:, None]
        check_attention(out[clean], lse[clean], _rows(ref, clean))
        if kind == "key scale inf":               # a score of minus infinity is a weight of zero
            continue
        spoilt = out[~clean]
        assert torch.isnan(spoilt[:, 17]).all()
        if kind != "value code":
            assert not torch.isfinite(spoilt).any()
        if kind.startswith("key"):
            assert torch.isnan(lse[~clean]).all()
        else:
            got, want = lse[~clean].double(), ref[1][~clean]
            assert ((got - want).abs() <= 2.0 ** -17 * ref[3][~clean] + 2.0 ** -19 * (1 + want.abs())).all()


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [700, 33]), ([4, 1], [129, 5]), ([8, 2], [300, 257]), ([150], [201])])
@pytest.mark.parametrize("D", [64, 128])
def test_unused_places_leave_no_trace(dev, q_lens, kv_lens, D):
    """Whatever the places past a context's end hold, the bits are the same."""
    page = 32
    args = _inputs(q_lens, kv_lens, 8, 2, D, page, 7)
    q, kq, ks, vq, vs, table, cu = args
    outs = [_attend(dev, *args, q_lens, kv_lens)]
    for code, scale in ((0x7F, NAN), (0xFF, INF), (0x7F, -INF)):
        bad = [t.clone() for t in (kq.view(torch.uint8), ks, vq.view(torch.uint8), vs)]
        for b, n in enumerate(kv_lens):
            pg, o = int(table[b, (n - 1) // page]), (n - 1) % page + 1
            for t, x in zip(bad, (code, scale, code, scale)):
                t[pg, :, o:] = x
        f8 = torch.float8_e4m3fn
        outs.append(_attend(dev, q, bad[0].view(f8), bad[1], bad[2].view(f8), bad[3], table, cu, q_lens, kv_lens))
        assert torch.equal(outs[-1][0], outs[0][0]) and torch.equal(outs[-1][1], outs[0][1])


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [700, 33]), ([4, 3], [129, 2]), ([8], [4000]), ([150], [120]),
                                            ([300], [900])])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("D", [64, 128])
def test_queries_that_are_not_finite(dev, q_lens, kv_lens, value, D):
    """They spoil their own row and head, and not even that where the row sees no token."""
    Hq, H = 8, 2
    q, kq, ks, vq, vs, table, cu = _inputs(q_lens, kv_lens, Hq, H, D, 32, 11)
    ref = attention_ref(q, kq, vq, ks, vs, table, cu, kv_lens, D ** -0.5)
    hit = torch.zeros(cu[-1], Hq, dtype=torch.bool)
    hit[0, 3] = hit[cu[1] // 2, 0] = hit[-1, 7] = True
    bad = q.clone()
    bad[..., 5] = torch.where(hit, torch.tensor(value, dtype=q.dtype), q[..., 5])
    out, lse = _attend(dev, bad, kq, ks, vq, vs, table, cu, q_lens, kv_lens)
    clean = ~hit | torch.isinf(ref[1])
    check_attention(out[clean], lse[clean], _rows(ref, clean))
    assert torch.isnan(out[~clean]).all() and torch.isnan(lse[~clean]).all()
