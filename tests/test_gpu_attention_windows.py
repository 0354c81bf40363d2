"""Windows up to the largest that the entry point takes, with rows that stand before the context's first token."""
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


@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 8, 1 << 30, 4])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens", [([6], [2]), ([5, 1], [2, 300]), ([7, 3], [0, 1]), ([200], [90]),
                                            ([300, 2, 40], [290, 1, 3])])
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (3, 3, 64)])
def test_windows_wider_than_any_context(dev, window, causal, q_lens, kv_lens, Hq, H, D):
    _run(dev, q_lens, kv_lens, Hq, H, D, 32, causal=causal, window=window)
