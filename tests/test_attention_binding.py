"""The attention call's host side, without a device."""
import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from block_scaled_fp8_02_gb300 import _binding as B


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
