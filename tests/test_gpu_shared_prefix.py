"""bfp8_shared_prefix_attention on the GPU against a 64-bit reference, within bounds derived from its arithmetic."""
import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from attn_ref import check_attention, make_cache, make_table
from block_scaled_fp8_02_gb300 import build as bfbuild
from cache_ref import shared_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    bfbuild.build()
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def make(dev, plens, pcu, q_lens, kv_lens, Hq=8, H=2, D=128, page=64, seed=0, extra=0, edit=None):
    """A call's tensors here and on the device; extra rows of q behind the last sequence."""
    g = torch.Generator().manual_seed(seed + 17 * sum(kv_lens) + sum(plens))
    lens = list(kv_lens) + list(plens)
    pages = sum((n + page - 1) // page for n in lens) + 2
    kq, ks, vq, vs = make_cache(pages, H, page, D, g)
    both = make_table(lens, page, pages, g)
    B = len(kv_lens)
    table, ptable = both[:B].contiguous(), both[B:].contiguous()
    cu = [0]
    for m in q_lens:
        cu.append(cu[-1] + m)
    q = (2 * torch.randn(cu[-1] + extra, Hq, D, generator=g)).bfloat16()
    if edit:
        edit(kq, ks, vq, vs, q, table, ptable)
    cache = bf.KVCache(*(t.to(dev) for t in (kq, vq, ks, vs)))
    host = (q, kq, vq, ks, vs, ptable, pcu, plens, table, cu, kv_lens)
    mp = max([b - a for a, b in zip(pcu, pcu[1:])] + [1])
    args = [q.to(dev), cache, ptable.to(dev), ints(pcu, dev), ints(plens, dev), mp, max(plens + [0]), table.to(dev),
            ints(cu, dev), ints(kv_lens, dev), max(q_lens + [1]), max(kv_lens)]
    return host, args


def check(host, args, causal=True, **kw):
    T, D = host[9][-1], host[0].shape[2]
    out, lse = bf.bfp8_shared_prefix_attention(*args, causal=causal, return_lse=True, **kw)
    torch.cuda.synchronize()
    assert bf.bfp8_device_status(clear=True) == 0
    ref = shared_ref(host[0][:T], *host[1:], D ** -0.5, causal)
    check_attention(out[:T], lse[:T], ref)
    again, lse2 = bf.bfp8_shared_prefix_attention(*args, causal=causal, return_lse=True, **kw)
    assert torch.equal(out[:T], again[:T]) and torch.equal(lse[:T], lse2[:T])
    return out, lse


# prefixes' lengths, their bounds among the rows, new and own tokens of the sequences
CASES = {
    "one row": ([100], [0, 1], [1], [1]),
    "few rows, both parts by the kernel for few": ([333], [0, 3], [1] * 3, [5, 64, 129]),
    "a batch's prefix by the tile kernel": ([700], [0, 20], [1] * 20, [13 * i + 1 for i in range(20)]),
    "own parts of both kinds": ([515], [0, 88], [1, 40, 1, 45, 1], [300, 40, 1, 200, 77]),
    "chunks": ([260], [0, 300], [100, 150, 50], [100, 400, 60]),
    "prefixes of one and of many rows": ([129, 64, 1000], [0, 1, 3, 40], [1] * 40, [20 + i for i in range(40)]),
    "rows before and behind the prefixes": ([200, 65], [5, 9, 18], [1] * 25, [30 + 3 * i for i in range(25)]),
    "an empty prefix": ([0, 128], [0, 10, 20], [2] * 10, [40] * 10),
    "an empty own part": ([77], [0, 6], [1, 1, 2, 2], [0, 4, 0, 1]),
    "nothing at all": ([0], [0, 3], [1] * 3, [0, 0, 2]),
    "no prefix": ([], [0], [1, 1, 30], [50, 1, 300]),
    "sequences without new tokens": ([90], [0, 4], [0, 2, 0, 2, 0], [10, 12, 0, 300, 7]),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("Hq,H,D,page", [(16, 2, 128, 64), (6, 2, 64, 16), (8, 8, 128, 32)])
def test_against_reference(dev, name, Hq, H, D, page):
    check(*make(dev, *CASES[name], Hq=Hq, H=H, D=D, page=page))


@pytest.mark.parametrize("Hq,H,D,page", [(40, 1, 128, 128), (3, 1, 64, 256), (64, 8, 64, 64), (20, 4, 128, 16)])
def test_head_layouts(dev, Hq, H, D, page):
    check(*make(dev, [1030], [0, 11], [1, 4, 3, 3], [500, 4, 129, 77], Hq=Hq, H=H, D=D, page=page))


def test_not_causal(dev):
    check(*make(dev, [300], [0, 60], [50, 10], [70, 200]), causal=False)


def test_long_prefix_and_many_sequences(dev):
    check(*make(dev, [9000], [0, 70], [1] * 70, [3 * i + 1 for i in range(70)], Hq=4, H=1))


def test_rows_outside_every_sequence_are_left_alone(dev):
    for lens in (([1] * 5, [9] * 5), ([30, 40], [64, 100])):
        host, args = make(dev, [200], [0, sum(lens[0])], *lens, extra=3)
        out = torch.full(args[0].shape, 7.0, dtype=torch.bfloat16, device=dev)
        check(host, args, out=out)
        assert (out[-3:] == 7.0).all()


def test_strided_queries_and_output(dev):
    host, args = make(dev, [150], [0, 45], [40, 5], [60, 5])
    T, Hq, D = args[0].shape
    wide = torch.zeros(T, Hq + 4, D, dtype=torch.bfloat16, device=dev)
    wide[:, 2:2 + Hq] = args[0]
    args[0] = wide[:, 2:2 + Hq]
    out = torch.zeros(Hq, T, D, dtype=torch.bfloat16, device=dev).transpose(0, 1)
    check(host, args, out=out)


def test_one_softmax_over_pages_in_every_table(dev):
    """The same tokens given as a prefix and as part of every sequence's own context (prefix of whole pages)."""
    P, lens = 256, [5, 64, 130]
    host, args = make(dev, [P], [0, 3], [1] * 3, lens)
    out, lse = bf.bfp8_shared_prefix_attention(*args, return_lse=True)
    q, cache, ptable, _, _, _, _, table, cu, kv, mq, mk = args
    whole = torch.cat([ptable[:, : P // 64].expand(3, -1), table], 1)
    o2, l2 = bf.bfp8_paged_attention(q, cache, whole, cu, kv + P, mq, mk + P, return_lse=True)
    # each is within its own bound of the exact result (2^-8 of it, and less of the weighted values, for the output)
    assert (lse - l2).abs().max() < 2e-3
    assert ((out.float() - o2.float()).norm() / o2.float().norm()) < 2.0 ** -8


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("where", ["prefix value", "prefix key", "own value", "own key scale"])
def test_not_a_number_stays_with_the_rows_that_see_it(dev, many, where):
    """Sequence 1's rows, or prefix 0's, are NaN; the others are what they are without it."""
    q_lens, kv_lens = ([40, 50, 60], [60, 70, 80]) if many else ([1] * 3, [60, 70, 80])
    rows = [0]
    for m in q_lens:
        rows.append(rows[-1] + m)
    pcu, plens = [0, rows[1], rows[3]], [130, 140]

    def edit(kq, ks, vq, vs, q, table, ptable):
        if where == "prefix value":
            vq.view(torch.uint8)[int(ptable[0, 1]), :, 3, 5] = 0x7F
        elif where == "prefix key":
            kq.view(torch.uint8)[int(ptable[0, 0]), :, 63, 0] = 0xFF
        elif where == "own value":
            vq.view(torch.uint8)[int(table[1, 0]), :, 0, 1] = 0x7F
        else:
            ks[int(table[1, 0]), :, 0] = float("nan")
    host, args = make(dev, plens, pcu, q_lens, kv_lens, edit=edit)
    host0, args0 = make(dev, plens, pcu, q_lens, kv_lens)
    out, lse = bf.bfp8_shared_prefix_attention(*args, return_lse=True)
    want, want_lse = bf.bfp8_shared_prefix_attention(*args0, return_lse=True)
    lo, hi = (0, rows[1]) if where.startswith("prefix") else (rows[1], rows[2])
    hit = torch.zeros(rows[-1], dtype=torch.bool)
    hit[lo:hi] = True
    assert torch.equal(out[~hit.to(dev)], want[~hit.to(dev)]) and torch.equal(lse[~hit.to(dev)], want_lse[~hit.to(dev)])
    got = out[hit.to(dev)]
    if "value" in where:
        d = 5 if where == "prefix value" else 1
        assert torch.isnan(got[:, :, d]).all()
    else:
        assert torch.isnan(got).all()


def test_captured_with_other_lengths(dev):
    """A captured call serves other lengths within its bounds."""
    host, args = make(dev, [500, 300], [0, 20, 40], [1] * 40, [100] * 40)
    out = torch.empty_like(args[0])
    bf.bfp8_shared_prefix_attention(*args, out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        bf.bfp8_shared_prefix_attention(*args, out=out)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            bf.bfp8_shared_prefix_attention(*args, out=out)
    for plens, kv in (([500, 300], [100] * 40), ([1, 299], [2 * i + 1 for i in range(40)]), ([0, 17], [99] * 40)):
        args[4].copy_(ints(plens, dev))
        args[9].copy_(ints(kv, dev))
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        h = list(host)
        h[7], h[10] = plens, kv
        check_attention(out, None, shared_ref(*h, 128 ** -0.5))
    assert bf.bfp8_device_status() == 0


# bounds of the workspace (rows a prefix, new tokens a sequence), and prefixes, rows, new and own tokens of calls within them
WITHIN = [
    ((200, 100), ([700], [0, 200], [1] * 200, [3 * i % 90 + 1 for i in range(200)])),
    ((200, 100), ([700], [0, 200], [4] * 50, [3 * i + 4 for i in range(50)])),
    ((200, 100), ([300, 90], [0, 2, 200], [8] * 25, [3 * i + 8 for i in range(25)])),
    ((200, 100), ([300], [0, 8], [8], [100])),
    ((200, 100), ([300], [0, 190], [90, 100], [100, 300])),
    ((200, 1), ([300], [0, 7], [1] * 7, [40] * 7)),
    ((1, 8), ([], [0], [8, 1], [50, 300])),
    ((1, 100), ([], [0], [8, 7], [50, 300])),
    # (9.9 MB of rows: more than the size has over what this call's partial rows take, so that both parts' do not fit)
    ((2400, 100), ([130], [0, 2400], [4] * 600, [4 + i % 9 for i in range(600)])),
    ((2400, 100), ([130, 5], [0, 2396, 2400], [4] * 600, [4 + i % 9 for i in range(600)])),
]


@pytest.mark.parametrize("i", range(len(WITHIN)))
def test_a_workspace_for_larger_bounds(dev, i):
    """A workspace of the size for some bounds serves every call within them, and no byte behind it is touched."""
    (pq, mq), lens = WITHIN[i]
    Hq, H, D = 8, 2, 128
    host, args = make(dev, *lens, Hq=Hq, H=H, D=D)
    n = bf.bfp8_shared_prefix_attention_workspace_size(Hq, H, D, pq, mq, args[0].shape[0])
    assert n >= bf.bfp8_shared_prefix_attention_workspace_size(Hq, H, D, args[5], args[10], 0)
    buf = torch.zeros(n + 4096, dtype=torch.uint8, device=dev)
    buf[n:] = 0x5A
    check(host, args, workspace=buf[:n])
    assert (buf[n:] == 0x5A).all()


def test_pages_outside_the_cache(dev):
    host, args = make(dev, [300], [0, 12], [1] * 12, [40] * 12)
    bad = args[2].clone()
    bad[0, 2] = 1 << 20
    bf.bfp8_shared_prefix_attention(*args[:2], bad, *args[3:])
    assert bf.bfp8_device_status(clear=True) == 6
    check(host, args)
