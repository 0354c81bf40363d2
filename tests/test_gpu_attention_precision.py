"""How small an element of a query may be beside its row's largest, in either kernel."""
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


def _case(dev, m, D, small, scale):
    """Queries of 1 in a channel where the keys are zero and elements up to `small` in the others, which alone decide."""
    g = torch.Generator().manual_seed(int(1e9 * small) + m)
    n, Hq, H, page = 300, 4, 1, 64
    kq, ks, vq, vs = make_cache(7, H, page, D, g)
    kf = kq.float() * ks[..., None]
    kf[..., 5] = 0
    kq, ks = quant_rows(kf)
    table = make_table([n], page, 7, g)
    q = small * (2 * torch.rand(m, Hq, D, generator=g) - 1)
    q[..., 5] = 1.0
    q = q.bfloat16()
    cache = bf.KVCache(*(t.to(dev) for t in (kq, vq, ks, vs)))
    out, lse = bf.bfp8_paged_attention(q.to(dev), cache, table.to(dev), torch.tensor([0, m], dtype=torch.int32, device=dev),
                                       torch.tensor([n], dtype=torch.int32, device=dev), m, n, scale=scale, return_lse=True)
    return out, lse.double().cpu(), attention_ref(q, kq, vq, ks, vs, table, [0, m], [n], scale)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e", [9, 14, 16, 17, 18, 25])
def test_many_rows_hold_elements_to_2_17_of_the_largest(dev, D, e):
    """Two e4m3 parts after scaling the largest into [2^7, 2^8): the smallest step is 2^-9, so an element is off by
    2^-17 of the largest at most; the scores by 2^-17 B with B = scale max|q| max_j sum |k_j|, a bound that
    check_attention holds weights and lse to.  The scale leaves it small enough to tell."""
    out, lse, ref = _case(dev, 150, D, 2.0 ** -e, 1.0)
    assert float(ref[3].max()) * 2.0 ** -17 < 2.0 ** -8
    check_attention(out, lse, ref)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e", [9, 14, 17, 22, 25])
def test_few_rows_hold_elements_to_2_38_of_the_largest(dev, D, e):
    """f16 after scaling the largest into [2^13, 2^14): the smallest step is 2^-24, so an element is off by 2^-38 of the
    largest at most.  With a softmax scale that makes the small elements' scores of ordinary size: off by 2^-38 B, and by
    the fp32 sums' 2^-17 of their own sum |q k| <= small / max|q| B."""
    small = 2.0 ** -e
    out, lse, ref = _case(dev, 1, D, small, 0.1 / small)
    bound = (2.0 ** -38 + 2.0 ** -17 * small) * ref[3]
    assert ((lse - ref[1]).abs() <= bound + 2.0 ** -19 * (1 + ref[1].abs())).all()
    assert torch.isfinite(out.float()).all()
