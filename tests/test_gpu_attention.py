"""bfp8_paged_attention on the GPU against a 64-bit reference, within bounds derived from its arithmetic."""
import math

import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from attn_ref import attention_ref, check_attention, make_cache, make_table, quant_rows
from block_scaled_fp8_02_gb300 import build as bfbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    bfbuild.build()
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def _run(dev, q_lens, kv_lens, Hq=8, H=2, D=128, page=64, causal=True, window=0, scale=None, seed=0, qmul=2.0,
         codes=None, max_q=None, max_kv=None, spread=0.5, layout="phtd", check=True):
    g = torch.Generator().manual_seed(seed + 17 * sum(kv_lens) + sum(q_lens))
    pages = sum((n + page - 1) // page for n in kv_lens) + 2
    kq, ks, vq, vs = codes(pages, H, page, D, g) if codes else make_cache(pages, H, page, D, g, spread)
    table = make_table(kv_lens, page, pages, g)
    cu = [0]
    for m in q_lens:
        cu.append(cu[-1] + m)
    T = cu[-1]
    wide = (qmul * torch.randn(T, (Hq + 2 * H) * D, generator=g)).bfloat16()
    q = wide[:, :Hq * D].view(T, Hq, D)
    scale = D ** -0.5 if scale is None else scale
    if layout == "pthd":
        dk, dv = (t.view(torch.uint8).transpose(1, 2).contiguous().to(dev).transpose(1, 2).view(torch.float8_e4m3fn)
                  for t in (kq, vq))
    else:
        dk, dv = kq.to(dev), vq.to(dev)
    cache = bf.KVCache(dk, dv, ks.to(dev), vs.to(dev))
    dq = wide.to(dev)[:, :Hq * D].view(T, Hq, D)
    args = (dq, cache, table.to(dev), torch.tensor(cu, dtype=torch.int32, device=dev),
            torch.tensor(kv_lens, dtype=torch.int32, device=dev), max_q or max(q_lens + [1]),
            max(kv_lens) if max_kv is None else max_kv)
    kw = dict(scale=scale, causal=causal, window=window, return_lse=True)
    out, lse = bf.bfp8_paged_attention(*args, **kw)
    torch.cuda.synchronize()
    assert bf.bfp8_device_status(clear=True) == 0
    if check:
        check_attention(out, lse, attention_ref(q, kq, vq, ks, vs, table, cu, kv_lens, scale, causal, window))
    again, lse2 = bf.bfp8_paged_attention(*args, **kw)
    assert torch.equal(out, again) and torch.equal(lse, lse2)          # the same bits every time
    return out, lse


DECODE = [([1], [1]), ([1], [2]), ([1], [64]), ([1], [65]), ([1], [5000]), ([1] * 5, [0, 1, 17, 333, 1024]),
          ([1] * 3, [4097, 15, 128]), ([1] * 40, [40 * i + 1 for i in range(40)])]


@pytest.mark.parametrize("q_lens,kv_lens", DECODE)
@pytest.mark.parametrize("Hq,H,D,page", [(8, 1, 128, 64), (8, 8, 64, 16), (10, 2, 128, 32), (32, 2, 128, 256),
                                         (6, 2, 64, 128)])
def test_single_tokens(dev, q_lens, kv_lens, Hq, H, D, page):
    _run(dev, q_lens, kv_lens, Hq, H, D, page)


CHUNKS = [([5], [5]), ([7], [100]), ([128], [128]), ([33, 1, 0, 64], [500, 70, 30, 64]), ([300], [301]),
          ([256], [1000]), ([129, 2, 1], [129, 700, 1]), ([17] * 6, [17, 18, 64, 129, 255, 400]), ([700], [700])]


@pytest.mark.parametrize("q_lens,kv_lens", CHUNKS)
@pytest.mark.parametrize("Hq,H,D,page", [(8, 1, 128, 64), (3, 3, 64, 16), (10, 2, 128, 128), (6, 2, 64, 32)])
def test_chunks(dev, q_lens, kv_lens, Hq, H, D, page):
    _run(dev, q_lens, kv_lens, Hq, H, D, page)


@pytest.mark.parametrize("causal,window", [(True, 1), (True, 5), (True, 64), (True, 200), (False, 0), (False, 50),
                                           (True, 100000)])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [1, 300, 777]), ([9, 40], [9, 333]), ([200, 130], [450, 131])])
@pytest.mark.parametrize("D", [64, 128])
def test_masks(dev, causal, window, q_lens, kv_lens, D):
    _run(dev, q_lens, kv_lens, 8, 2, D, 32, causal=causal, window=window)


@pytest.mark.parametrize("q_lens,kv_lens", [([4], [0]), ([4, 3], [2, 1]), ([200], [90]), ([300, 1], [0, 0])])
def test_rows_that_see_nothing(dev, q_lens, kv_lens):
    """More new tokens than context: the first rows have no position; an empty context leaves all rows empty."""
    out, lse = _run(dev, q_lens, kv_lens, 8, 2, 128, 64, max_kv=max(max(kv_lens), 0))
    empty = q_lens[0] - kv_lens[0]
    assert (out[:empty] == 0).all() and torch.isinf(lse[:empty]).all()


def _zero_values(pages, H, page, D, g):
    """Every third token's value and every fifth token's key all zero (scales 1e-10 / 448)."""
    k = torch.randn(pages, H, page, D, generator=g)
    v = torch.randn(pages, H, page, D, generator=g)
    v[:, :, ::3] = 0
    k[:, :, ::5] = 0
    return (*quant_rows(k.bfloat16()), *quant_rows(v.bfloat16()))


def _spread_scales(pages, H, page, D, g):
    """Keys and values whose sizes differ by many orders of magnitude from token to token."""
    k = torch.randn(pages, H, page, D, generator=g) * torch.exp(torch.randn(pages, H, page, 1, generator=g))
    v = torch.randn(pages, H, page, D, generator=g) * torch.exp2(
        torch.randint(-30, 30, (pages, H, page, 1), generator=g).float())
    return (*quant_rows(k.bfloat16()), *quant_rows(v.bfloat16()))


def _large(pages, H, page, D, g):
    k = torch.randn(pages, H, page, D, generator=g) * 10
    v = torch.randn(pages, H, page, D, generator=g) * 1e30
    return (*quant_rows(k.bfloat16()), *quant_rows(v.bfloat16()))


@pytest.mark.parametrize("codes", [_zero_values, _spread_scales, _large])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [700, 33]), ([3], [200]), ([150], [600])])
def test_scales_of_all_sizes(dev, codes, q_lens, kv_lens):
    _run(dev, q_lens, kv_lens, 8, 2, 128, 64, codes=codes)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [900, 33]), ([140], [600])])
@pytest.mark.parametrize("qmul,scale", [(0.0, None), (1e-20, None), (30.0, None), (2.0, -0.1), (2.0, 0.0), (1e15, 1e-15)])
def test_queries_of_all_sizes(dev, q_lens, kv_lens, qmul, scale):
    """Zero, tiny and huge queries, softmax scales of zero and below."""
    _run(dev, q_lens, kv_lens, 4, 1, 128, 64, qmul=qmul, scale=scale)


def test_queries_with_one_large_element(dev):
    """A channel a thousand times the others must not drown them."""
    g = torch.Generator().manual_seed(3)
    for m in (1, 150):
        n, Hq, H, D, page = 400, 4, 1, 128, 64
        kq, ks, vq, vs = make_cache(9, H, page, D, g)
        kf = kq.float() * ks[..., None]
        kf[..., 5] = 0                                # the large channel multiplies zeros: the rest decides
        kq, ks = quant_rows(kf)
        table = make_table([n], page, 9, g)
        q = torch.randn(m, Hq, D, generator=g)
        q[..., 5] = 3000.0
        q = q.bfloat16()
        cache = bf.KVCache(*(t.to(dev) for t in (kq, vq, ks, vs)))
        out, lse = bf.bfp8_paged_attention(q.to(dev), cache, table.to(dev),
                                           torch.tensor([0, m], dtype=torch.int32, device=dev),
                                           torch.tensor([n], dtype=torch.int32, device=dev), m, n, return_lse=True)
        check_attention(out, lse, attention_ref(q, kq, vq, ks, vs, table, [0, m], [n], D ** -0.5))


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [100, 900, 2000]), ([20, 150], [120, 160])])
def test_token_major_cache(dev, q_lens, kv_lens):
    _run(dev, q_lens, kv_lens, 16, 4, 128, 64, layout="pthd")


def test_bounds_above_the_lengths(dev):
    """Host bounds larger than any length (a captured graph's) give the same rows."""
    for q_lens, kv_lens in (([1, 1], [300, 20]), ([130, 3], [300, 20])):
        a = _run(dev, q_lens, kv_lens, max_kv=max(kv_lens))
        b = _run(dev, q_lens, kv_lens, max_kv=320, max_q=max(q_lens) + 700)
        ref = torch.linalg.vector_norm(a[0].double())
        assert float(torch.linalg.vector_norm(a[0].double() - b[0].double()) / ref) < 2 ** -7


def test_rows_outside_every_sequence_are_not_written(dev):
    g = torch.Generator().manual_seed(1)
    for m in (2, 140):
        kq, ks, vq, vs = make_cache(8, 2, 64, 128, g)
        cache = bf.KVCache(*(t.to(dev) for t in (kq, vq, ks, vs)))
        q = torch.randn(m + 9, 4, 128, generator=g).bfloat16().to(dev)
        out = torch.full_like(q, 5.0)
        bf.bfp8_paged_attention(q, cache, torch.arange(8, dtype=torch.int32, device=dev)[None],
                                torch.tensor([4, 4 + m], dtype=torch.int32, device=dev),
                                torch.tensor([300], dtype=torch.int32, device=dev), m, 300, out=out)
        assert (out[:4] == 5).all() and (out[4 + m:] == 5).all() and (out[4:4 + m] != 5).any(-1).all()


def test_strided_output_and_out_of_range_pages(dev):
    g = torch.Generator().manual_seed(2)
    kq, ks, vq, vs = make_cache(8, 2, 64, 128, g)
    cache = bf.KVCache(*(t.to(dev) for t in (kq, vq, ks, vs)))
    for m in (1, 140):
        q = torch.randn(m, 4, 128, generator=g).bfloat16().to(dev)
        cu = torch.tensor([0, m], dtype=torch.int32, device=dev)
        lens = torch.tensor([300], dtype=torch.int32, device=dev)
        table = torch.arange(8, dtype=torch.int32, device=dev)[None]
        want = bf.bfp8_paged_attention(q, cache, table, cu, lens, m, 300)
        wide = torch.zeros(m, 6, 256, dtype=torch.bfloat16, device=dev)
        got = bf.bfp8_paged_attention(q, cache, table, cu, lens, m, 300, out=wide[:, 1:5, 64:192])
        assert torch.equal(got, want) and (wide[:, 0] == 0).all() and (wide[:, 1:5, :64] == 0).all()
        for wrong in (8, -1, 1 << 30):
            bad = table.clone()
            bad[0, 2] = wrong
            bf.bfp8_paged_attention(q, cache, bad, cu, lens, m, 300)
            assert bf.bfp8_device_status(clear=True) == 6            # BFP8_DEV_BAD_CACHE_INDEX
        assert torch.equal(bf.bfp8_paged_attention(q, cache, table, cu, lens, m, 300), want)


def test_captured_graph_serves_other_lengths(dev):
    g = torch.Generator().manual_seed(4)
    Hq, H, D, page, B = 16, 2, 128, 64, 4
    kq, ks, vq, vs = make_cache(60, H, page, D, g)
    cache = bf.KVCache(*(t.to(dev) for t in (kq, vq, ks, vs)))
    table = torch.randperm(60, generator=g)[:B * 15].view(B, 15).int()
    q = torch.randn(B, Hq, D, generator=g).bfloat16()
    dq, dt = q.to(dev), table.to(dev)
    cu = torch.arange(B + 1, dtype=torch.int32, device=dev)
    lens = torch.ones(B, dtype=torch.int32, device=dev)
    out = torch.empty_like(dq)
    ws = torch.zeros(bf.bfp8_paged_attention_workspace_size(Hq, H, D, 1), dtype=torch.uint8, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bf.bfp8_paged_attention(dq, cache, dt, cu, lens, 1, 15 * page, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bf.bfp8_paged_attention(dq, cache, dt, cu, lens, 1, 15 * page, out=out, workspace=ws)
    for kv in ([1, 1, 1, 1], [960, 3, 500, 77], [0, 960, 960, 960]):
        lens.copy_(torch.tensor(kv, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check_attention(out, None, attention_ref(q, kq, vq, ks, vs, table, list(range(B + 1)), kv, D ** -0.5))


def test_shares_a_workspace_with_the_gemm(dev):
    """One buffer serves the GEMM and the attention in turn: both leave its counters zero."""
    from block_scaled_fp8_02_gb300 import workloads as wl
    c = wl.linear_case(256, 512, 4096, seed=3)
    A, s = bf.bfp8_group_quant(c["x"].to(dev))
    opt = {"k_split": 1, "schedule": 2}
    first = bf.bfp8_gemm(A, c["B"].to(dev), s, c["Bs"].to(dev), options=opt)
    _run(dev, [1, 1, 1], [3000, 5, 700], 16, 2)
    _run(dev, [150], [900], 16, 2)
    assert torch.equal(first, bf.bfp8_gemm(A, c["B"].to(dev), s, c["Bs"].to(dev), options=opt))


def test_cache_offsets_past_32_bits(dev):
    P, H, page, D = 5, 2, 64, 128
    g = torch.Generator().manual_seed(8)
    kq, ks, vq, vs = make_cache(P, H, page, D, g)
    n = H * page * D
    big = torch.zeros((P - 1) * (1 << 30) + 2 * n, dtype=torch.uint8, device=dev)
    kc = torch.as_strided(big, (P, H, page, D), (1 << 30, page * D, D, 1))
    vc = torch.as_strided(big, (P, H, page, D), (1 << 30, page * D, D, 1), n)
    kc.copy_(kq.view(torch.uint8))
    vc.copy_(vq.view(torch.uint8))
    cache = bf.KVCache(kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), ks.to(dev), vs.to(dev))
    table = torch.tensor([[4, 0, 3, 1, 2]], dtype=torch.int32)
    for m in (1, 200):
        q = torch.randn(m, 4, D, generator=g).bfloat16()
        out, lse = bf.bfp8_paged_attention(q.to(dev), cache, table.to(dev),
                                           torch.tensor([0, m], dtype=torch.int32, device=dev),
                                           torch.tensor([310], dtype=torch.int32, device=dev), m, 310, return_lse=True)
        check_attention(out, lse, attention_ref(q, kq, vq, ks, vs, table, [0, m], [310], D ** -0.5))


def test_one_weight_beside_a_long_tail(dev):
    """One token far above 20000 equal others, whose small weights add up: none of their mass may be lost."""
    n, H, D, page = 20000, 1, 128, 64
    P = (n + page - 1) // page
    k = torch.zeros(P, H, page, D)
    k[0, 0, 0, 0] = 1.0                               # score log(2^16) for the first token, zero for the rest
    v = torch.ones(P, H, page, D)
    v[0, 0, 0] = -1.0
    kq, ks = quant_rows(k)
    vq, vs = quant_rows(v)
    table = torch.arange(P, dtype=torch.int32)[None]
    for m in (1, 140):
        q = torch.zeros(m, 2, D)
        q[..., 0] = 16 * math.log(2) / D ** -0.5
        q = q.bfloat16()
        cache = bf.KVCache(*(t.to(dev) for t in (kq, vq, ks, vs)))
        out, lse = bf.bfp8_paged_attention(q.to(dev), cache, table.to(dev),
                                           torch.tensor([0, m], dtype=torch.int32, device=dev),
                                           torch.tensor([n], dtype=torch.int32, device=dev), m, n, return_lse=True)
        check_attention(out, lse, attention_ref(q, kq, vq, ks, vs, table, [0, m], [n], D ** -0.5))


@pytest.mark.parametrize("q_lens,kv_lens,max_q", [([40, 40], [90, 300], None), ([40, 39, 1], [300, 90, 77], None),
                                                  ([40], [300], 64), ([1, 40, 0], [500, 41, 9], 200), ([2, 5], [9, 300], None)])
@pytest.mark.parametrize("Hq,H", [(8, 1), (6, 2), (33, 1)])
def test_batches_that_may_or_may_not_hold_short_sequences(dev, q_lens, kv_lens, max_q, Hq, H):
    """From batches whose token count leaves no room for a short sequence to ones with nothing else."""
    _run(dev, q_lens, kv_lens, Hq, H, 64, 16, max_q=max_q)


@pytest.mark.parametrize("q_lens,kv_lens,window", [([1200], [1300], 0), ([1, 1100, 60], [400, 1100, 700], 0),
                                                   ([1150, 1, 1], [1500, 900, 2], 300)])
def test_more_blocks_than_lanes(dev, q_lens, kv_lens, window):
    """A head's blocks of 256 rows pass 32: shares begin anywhere among them."""
    _run(dev, q_lens, kv_lens, 8, 1, 64, 32, window=window)


def test_more_sequences_than_are_counted_at_once(dev):
    n = 2060
    _run(dev, [2] * n, [2 + i % 5 for i in range(n)], 17, 1, 64, 16)


@pytest.mark.parametrize("D", [64, 128])
def test_other_sequences_nans_leave_no_trace(dev, D):
    """Every other sequence's keys are NaN: the rest come out bit for bit as beside ordinary ones, although their last
    tiles are not full and their row blocks have rows to spare, which see what the tiles before left there."""
    n, page, g = 600, 16, torch.Generator().manual_seed(5)      # (pages end inside a tile's halves)
    kv_lens = [256 if i % 2 == 0 else 168 for i in range(n)]
    pages = sum((m + page - 1) // page for m in kv_lens)
    kq, ks, vq, vs = make_cache(pages, 1, page, D, g, 0.5)
    table = torch.zeros(n, 16, dtype=torch.int32)
    at = 0
    spoilt = kq.view(torch.uint8).clone()
    for i, m in enumerate(kv_lens):
        c = (m + page - 1) // page
        table[i, :c] = torch.arange(at, at + c)
        if i % 2 == 0:
            spoilt[at:at + c] = 0x7F
        at += c
    q = torch.randn(n * 5, 8, D, generator=g).bfloat16().to(dev)
    cu = (torch.arange(n + 1) * 5).int().to(dev)
    outs = []
    for codes in (kq, spoilt.view(torch.float8_e4m3fn)):
        cache = bf.KVCache(codes.to(dev), vq.to(dev), ks.to(dev), vs.to(dev))
        out, lse = bf.bfp8_paged_attention(q, cache, table.to(dev), cu, torch.tensor(kv_lens, dtype=torch.int32, device=dev),
                                           5, 256, return_lse=True)
        outs.append((out.view(n, 5, 8, D)[1::2], lse.view(n, 5, 8)[1::2]))
    assert torch.isfinite(outs[0][0].float()).all()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
