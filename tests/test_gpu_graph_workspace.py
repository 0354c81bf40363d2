"""Captured calls on the library's own workspaces, beside eager calls that need larger ones."""
import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from attn_ref import make_cache
from block_scaled_fp8_02_gb300 import build as bfbuild
from block_scaled_fp8_02_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    bfbuild.build()
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def _attention(dev, m, out=None):
    """A call whose contexts are cut between SMs, so that it lives off the workspace: m new tokens, two sequences."""
    g = torch.Generator().manual_seed(m)
    Hq, H, D, page, P = 16, 2, 128, 64, 100
    kq, ks, vq, vs = make_cache(P, H, page, D, g)
    cache = bf.KVCache(*(t.to(dev) for t in (kq, vq, ks, vs)))
    table = torch.randperm(P, generator=g).int().view(2, 50).to(dev)
    q = torch.randn(2 * m, Hq, D, generator=g).bfloat16().to(dev)
    cu = torch.tensor([0, m, 2 * m], dtype=torch.int32, device=dev)
    lens = torch.tensor([3200, 1777], dtype=torch.int32, device=dev)
    return lambda: bf.bfp8_paged_attention(q, cache, table, cu, lens, m, 3200, out=out)


def _gemm(dev, M, N, K, out=None):
    c = wl.linear_case(M, N, K, seed=3)
    A, s = bf.bfp8_group_quant(c["x"].to(dev))
    B, Bs = c["B"].to(dev), c["Bs"].to(dev)
    return lambda: bf.bfp8_gemm(A, B, s, Bs, out=out, options={"k_split": 1, "schedule": 2})


@pytest.mark.parametrize("what", ["attention", "gemm"])
def test_a_larger_eager_call_leaves_the_graph_its_buffer(dev, what):
    if what == "attention":
        out = torch.empty(2, 16, 128, dtype=torch.bfloat16, device=dev)
        small, large = _attention(dev, 1, out), _attention(dev, 150)
    else:
        out = torch.empty(128, 512, dtype=torch.bfloat16, device=dev)
        small, large = _gemm(dev, 128, 512, 2048, out), _gemm(dev, 256, 4096, 4096)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        small()
        want = out.clone()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            small()
        large()
        # takes what the allocator has to give, the graph's buffer too if that was let go
        taken = [torch.full((n << 18,), 0xAB, dtype=torch.uint8, device=dev) for n in (1, 2, 4, 8, 16, 32) for _ in range(8)]
        for _ in range(3):
            out.zero_()
            graph.replay()
            s.synchronize()
            assert torch.equal(out, want)
        assert all(bool((t == 0xAB).all()) for t in taken)
    assert bf.bfp8_device_status(clear=True) == 0


def test_captures_on_a_cold_stream(dev):
    """No call warmed the stream up: each graph zeroes a buffer of its own, and runs in any order, eager calls between."""
    outs = [torch.empty(2, 16, 128, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    calls = [_attention(dev, 1, o) for o in outs]
    calls[0]()
    want = outs[0].clone()
    s = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    for call in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            call()
    eager = torch.empty_like(want)
    with torch.cuda.stream(s):
        for order in ((1,), (1, 0), (0, 1, 1)):
            for i in order:
                outs[i].zero_()
                graphs[i].replay()
                s.synchronize()
                assert torch.equal(outs[i], want)
            _attention(dev, 1, eager)()
            s.synchronize()
            assert torch.equal(eager, want)
    assert bf.bfp8_device_status(clear=True) == 0


@pytest.mark.parametrize("Hq,H,D", [(1, 1, 64), (8, 8, 128), (64, 8, 128), (24, 8, 64), (33, 1, 128), (128, 1, 128)])
def test_attention_workspaces_of_long_prompts_are_of_one_size(dev, Hq, H, D):
    sizes = {bf.bfp8_paged_attention_workspace_size(Hq, H, D, n) for n in (33, 34, 100, 4096, 1 << 24)}
    assert len(sizes) == 1
