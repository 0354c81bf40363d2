"""bfp8_kv_cache_weigh on the GPU against a 64-bit reference, within bounds derived from its arithmetic."""
import math

import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from attn_ref import attention_ref, make_cache, make_table
from block_scaled_fp8_02_gb300 import build as bfbuild
from cache_ref import check_weights, weigh_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    bfbuild.build()
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def make(q_lens, kv_lens, Hq=8, H=2, D=128, page=64, causal=True, window=0, seed=0, qmul=2.0, scale=None):
    g = torch.Generator().manual_seed(seed + 31 * sum(kv_lens) + sum(q_lens))
    pages = sum((n + page - 1) // page for n in kv_lens) + 2
    kq, ks, vq, vs = make_cache(pages, H, page, D, g)
    table = make_table(kv_lens, page, pages, g)
    cu = [0]
    for m in q_lens:
        cu.append(cu[-1] + m)
    q = (qmul * torch.randn(cu[-1], Hq, D, generator=g)).bfloat16()
    scale = D ** -0.5 if scale is None else scale
    lse = attention_ref(q, kq, vq, ks, vs, table, cu, kv_lens, scale, causal, window)[1].float()
    weights = torch.rand(pages, H, page, generator=g)
    return dict(q=q, lse=lse, k=kq, ks=ks, v=vq, vs=vs, w=weights, table=table, cu=cu, kv=kv_lens, scale=scale,
                mq=max(q_lens + [1]), mk=max(kv_lens), causal=causal, window=window)


def run(dev, c, accumulate=True, w=None, **kw):
    cache = bf.KVCache(*(c[n].to(dev) for n in ("k", "v", "ks", "vs")))
    w = c["w"].to(dev) if w is None else w
    bf.bfp8_kv_cache_weigh(c["q"].to(dev), c["lse"].to(dev), cache, w, c["table"].to(dev), ints(c["cu"], dev),
                           ints(c["kv"], dev), c["mq"], c["mk"], scale=c["scale"], causal=c["causal"], window=c["window"],
                           accumulate=accumulate, **kw)
    torch.cuda.synchronize()
    return w


def check(dev, c, accumulate=True):
    got = run(dev, c, accumulate)
    assert bf.bfp8_device_status(clear=True) == 0
    ref = weigh_ref(c["q"], c["lse"], c["k"], c["ks"], c["w"], c["table"], c["cu"], c["kv"], c["scale"], c["causal"],
                    c["window"], accumulate)
    check_weights(got, c["w"], ref)
    # the bound above is the worst case; as a whole the sums come much nearer
    new = ref[1] > 0
    if new.any():
        assert float((got.cpu().double() - ref[0])[new].norm() / ref[0][new].norm()) < 1e-5
    assert torch.equal(run(dev, c, accumulate).view(torch.int32), got.view(torch.int32))         # the same bits every time
    return got


LENGTHS = {
    "single tokens": ([1] * 7, [1, 2, 15, 64, 129, 400, 1000]),
    "drafts": ([2, 3, 4, 5], [2, 130, 517, 64]),
    "between the kernels": ([7, 8, 9, 16, 17], [7, 130, 300, 16, 200]),
    "a chunk": ([150], [700]),
    "a whole prompt": ([300], [300]),
    "mixed": ([1, 60, 1, 33, 1, 0, 128], [333, 60, 1, 500, 127, 90, 129]),
    "empty contexts": ([1, 3, 0, 40], [0, 2, 0, 10]),
}


@pytest.mark.parametrize("name", LENGTHS)
@pytest.mark.parametrize("Hq,H,D,page", [(16, 2, 128, 64), (6, 2, 64, 16), (4, 4, 128, 32), (64, 8, 64, 128)])
def test_against_reference(dev, name, Hq, H, D, page):
    check(dev, make(*LENGTHS[name], Hq=Hq, H=H, D=D, page=page))


@pytest.mark.parametrize("Hq,H,D,page", [(40, 1, 128, 256), (3, 1, 64, 16), (128, 1, 64, 64), (20, 4, 128, 128), (33, 1, 128, 64)])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [77, 300]), ([9, 70], [9, 400])])
def test_head_layouts(dev, Hq, H, D, page, q_lens, kv_lens):
    check(dev, make(q_lens, kv_lens, Hq=Hq, H=H, D=D, page=page))


@pytest.mark.parametrize("window", [1, 5, 64, 100, 1000])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2], [300, 77]), ([50, 130], [50, 400])])
@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("causal", [True, False])
def test_windows(dev, window, q_lens, kv_lens, accumulate, causal):
    check(dev, make(q_lens, kv_lens, window=window, causal=causal), accumulate)


@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("causal", [True, False])
def test_where_sums_begin(dev, accumulate, causal):
    check(dev, make([1, 3, 40, 100], [64, 3, 150, 300], causal=causal), accumulate)


def test_long_contexts(dev):
    check(dev, make([1, 5], [20000, 9000], Hq=4, H=1))
    check(dev, make([700], [3000], Hq=2, H=1))


def test_many_sequences(dev):
    check(dev, make([1] * 300, [i % 40 + 1 for i in range(300)], Hq=2, H=1, page=16, D=64))
    check(dev, make([20 + i % 3 for i in range(100)], [30 + i % 40 for i in range(100)], Hq=4, H=2, page=16, D=64))


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5])
@pytest.mark.parametrize("q_lens", [[1, 2], [60, 33]])
def test_scales(dev, scale, q_lens):
    check(dev, make(q_lens, [200, 90], scale=scale))


@pytest.mark.parametrize("q_lens", [[2], [100]])
def test_queries_of_any_size(dev, q_lens):
    """Elements far below and rows far above the others."""
    c = make(q_lens, [150], qmul=1.0)
    c["q"][:, :, ::3] *= 2.0 ** -20
    c["q"][0] *= 2.0 ** 60
    c["q"][-1] *= 2.0 ** -60
    c["k"], c["ks"] = c["k"], c["ks"] * 1e-3
    c["scale"] = 2.0 ** -50
    c["lse"] = attention_ref(c["q"], c["k"], c["v"], c["ks"], c["vs"], c["table"], c["cu"], c["kv"], c["scale"])[1].float()
    check(dev, c)


@pytest.mark.parametrize("q_lens,kv_lens", [([2, 2, 3], [70, 80, 90]), ([70, 40, 50], [70, 150, 90])])
@pytest.mark.parametrize("where", ["query", "infinite query", "lse", "key", "key scale"])
def test_not_a_number_stays_with_the_tokens_concerned(dev, q_lens, kv_lens, where):
    c = make(q_lens, kv_lens)
    want = run(dev, c).cpu()
    q0, i, n = c["cu"][1], 1, kv_lens[1]                  # row i of sequence 1, head 3 (kv head 0 of 2)
    seen = n - q_lens[1] + i + 1                          # its tokens
    hit = torch.zeros_like(want, dtype=torch.bool)
    j = torch.arange(n)
    at, off = c["table"][1].long()[j // 64], j % 64
    if where == "query":
        c["q"][q0 + i, 3, 7] = float("nan")
    elif where == "infinite query":
        c["q"][q0 + i, 3, 7] = float("inf")
    elif where == "lse":
        c["lse"][q0 + i, 3] = float("nan")
    elif where == "key":
        c["k"].view(torch.uint8)[at[20], 0, off[20], 9] = 0x7F
    else:
        c["ks"][at[20], 0, off[20]] = float("nan")
    if where.startswith("key"):
        hit[at[20], 0, off[20]] = True
    else:
        hit[at[:seen], 0, off[:seen]] = True
    got = run(dev, c).cpu()
    if where == "infinite query":                        # inf - lse: nothing, all or a NaN, by the sign of each score
        assert torch.equal(got[~hit], want[~hit])
    else:
        assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], want[~hit])


def test_rows_that_see_nothing(dev):
    """More new tokens than context: the first rows see no token, their lse is -infinity."""
    c = make([6, 80], [4, 50])
    assert torch.isinf(c["lse"]).any()
    check(dev, c)


def test_strides(dev):
    """Queries as columns of a projection, weights with strides of their own, a cache in [page, token, head] order."""
    c = make([1, 2, 50], [100, 64, 130], Hq=8, H=2, D=128)
    want = run(dev, c)
    T = c["q"].shape[0]
    wide = torch.zeros(T, 12 * 128, dtype=torch.bfloat16, device=dev)
    wide[:, 128:9 * 128] = c["q"].view(T, -1).to(dev)
    k, v = (c[n].view(torch.uint8).transpose(1, 2).contiguous().to(dev).transpose(1, 2).view(torch.float8_e4m3fn) for n in "kv")
    big = torch.full((c["w"].shape[0], 3, 71), 9.0, device=dev)
    w = big[:, :2, :64]
    w.copy_(c["w"])
    bf.bfp8_kv_cache_weigh(wide[:, 128:9 * 128].view(T, 8, 128), c["lse"].to(dev), bf.KVCache(k, v, c["ks"].to(dev), c["vs"].to(dev)),
                           w, c["table"].to(dev), ints(c["cu"], dev), ints(c["kv"], dev), c["mq"], c["mk"])
    assert torch.equal(w, want) and (big[:, 2] == 9.0).all() and (big[:, :, 64:] == 9.0).all()


def test_bounds_above_the_lengths(dev):
    """Larger bounds and wider tables change nothing (whatever stands behind the sequence's pages)."""
    for q_lens, kv in (([1, 2], [100, 30]), ([60, 1], [100, 30])):
        c = make(q_lens, kv)
        want = run(dev, c)
        c["table"] = torch.cat([c["table"], torch.full((2, 400), -5, dtype=torch.int32)], 1)
        c["mk"] = 400 * 64
        assert torch.equal(run(dev, c), want)
        c["mq"] = 500
        got = run(dev, c).cpu()
        check_weights(got, c["w"], weigh_ref(c["q"], c["lse"], c["k"], c["ks"], c["w"], c["table"], c["cu"], c["kv"], c["scale"]))
    assert bf.bfp8_device_status(clear=True) == 0


def test_pages_outside_the_cache(dev):
    for q_lens in ([1, 1], [50, 50]):
        c = make(q_lens, [200, 200])
        want = run(dev, c)
        bad = dict(c, table=c["table"].clone())
        bad["table"][0, 1] = 1 << 20
        got = run(dev, bad)
        assert bf.bfp8_device_status(clear=True) == 6
        other = c["table"][1].long()
        assert torch.equal(got[other], want[other])                                    # the other sequence
        lost = int(c["table"][0, 1])
        assert torch.equal(got[lost].cpu(), c["w"][lost])


def test_rows_add_up(dev):
    """Every row's weights sum to one: the sums of all tokens to rows x heads, where they all begin here."""
    c = make([1, 90], [500, 300])
    got = run(dev, c, accumulate=False)
    for b, m in enumerate((1, 90)):
        n = c["kv"][b]
        j = torch.arange(n)
        s = got.cpu().double()[c["table"][b].long()[j // 64], :, j % 64].sum(0)
        assert torch.allclose(s, torch.full((2,), 4.0 * m, dtype=torch.float64), rtol=1e-5)


def test_captured(dev):
    c = make([1] * 4 + [70], [50, 60, 70, 80, 200])
    cache = bf.KVCache(*(c[n].to(dev) for n in ("k", "v", "ks", "vs")))
    w, cu, kv = c["w"].to(dev), ints(c["cu"], dev), ints(c["kv"], dev)
    args = (c["q"].to(dev), c["lse"].to(dev), cache, w, c["table"].to(dev), cu, kv, 70, 200)
    bf.bfp8_kv_cache_weigh(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        bf.bfp8_kv_cache_weigh(*args)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            bf.bfp8_kv_cache_weigh(*args)
    for lens in (c["kv"], [1, 2, 3, 80, 71]):
        kv.copy_(ints(lens, dev))
        w.copy_(c["w"])
        graph.replay()
        torch.cuda.synchronize()
        check_weights(w, c["w"], weigh_ref(c["q"], c["lse"], c["k"], c["ks"], c["w"], c["table"], c["cu"], lens, c["scale"]))
    assert not math.isnan(float(w.sum()))
