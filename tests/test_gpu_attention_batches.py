"""Batches of more sequences than a CTA of the kernel for few rows has threads, and shares of more than it keeps."""
import pytest
import torch

from block_scaled_fp8_02_gb300 import build as bfbuild
from test_gpu_attention import _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    bfbuild.build()
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


@pytest.mark.parametrize("Hq,H,D", [(8, 1, 64), (16, 1, 64), (32, 1, 64), (6, 2, 128)])
@pytest.mark.parametrize("n", [385, 513, 1100])
def test_many_single_tokens(dev, Hq, H, D, n):
    """Ragged contexts, every seventh empty; a few long ones that shares cut."""
    kv = [0 if i % 7 == 3 else 1500 if i % 251 == 0 else 1 + (i * 37) % 60 for i in range(n)]
    _run(dev, [1] * n, kv, Hq, H, D, 16)


def test_sequences_without_tokens_among_many(dev):
    n = 900
    q = [0 if i % 3 == 0 or 100 < i < 400 else 1 for i in range(n)]
    _run(dev, q, [5 + i % 40 for i in range(n)], 8, 1, 64, 16)


def test_shares_of_more_sequences_than_are_kept(dev):
    n = 6000
    _run(dev, [1] * n, [i % 3 for i in range(n)], 4, 1, 64, 16)


@pytest.mark.parametrize("Hq,H", [(8, 1), (24, 1)])
def test_chunks_among_many_single_tokens(dev, Hq, H):
    """Both kernels beside each other, each with its own path for large batches."""
    n = 700
    q = [40 if i % 50 == 7 else 1 for i in range(n)]
    _run(dev, q, [m + (i * 13) % 70 for i, m in enumerate(q)], Hq, H, 64, 16)


def test_chunks_among_more_sequences_than_are_counted_at_once(dev):
    n = 2100
    q = [35 if i % 300 == 299 else 1 for i in range(n)]
    _run(dev, q, [m + i % 5 for i, m in enumerate(q)], 8, 1, 64, 16)


def test_one_token_in_a_row_of_odd_width(dev):
    """A single token's slice of a wider row, whose stride is no multiple of 8."""
    import block_scaled_fp8_02_gb300 as bf
    from attn_ref import make_cache
    g = torch.Generator().manual_seed(6)
    kq, ks, vq, vs = make_cache(3, 2, 16, 64, g)
    cache = bf.KVCache(*(t.to(dev) for t in (kq, vq, ks, vs)))
    args = (cache, torch.arange(3, dtype=torch.int32, device=dev)[None], torch.tensor([0, 1], dtype=torch.int32, device=dev),
            torch.tensor([40], dtype=torch.int32, device=dev), 1, 40)
    wide = torch.randn(4, 8 * 64 + 3, generator=g).bfloat16().to(dev)
    q = torch.as_strided(wide, (1, 8, 64), (515, 64, 1))
    assert torch.equal(bf.bfp8_paged_attention(q, *args), bf.bfp8_paged_attention(q.contiguous().clone(), *args))


def test_batches_without_new_tokens(dev):
    """Bounds of zero, the library's own workspace; and the next call finds everything in order."""
    import block_scaled_fp8_02_gb300 as bf
    cache = bf.KVCache.empty(2, 2, 16, 64, dev)
    for batch in (0, 2):
        cu, kv = torch.zeros(batch + 1, dtype=torch.int32, device=dev), torch.zeros(batch, dtype=torch.int32, device=dev)
        q = torch.zeros(0, 8, 64, dtype=torch.bfloat16, device=dev)
        out, lse = bf.bfp8_paged_attention(q, cache, torch.zeros(batch, 0, dtype=torch.int32, device=dev), cu, kv, 0, 0,
                                           return_lse=True)
        assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    _run(dev, [1, 3], [700, 9], 8, 2, 64, 16)
