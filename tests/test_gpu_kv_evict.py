"""bfp8_kv_cache_evict on the GPU: what stays and where it goes, bit for bit."""
import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from attn_ref import make_cache, make_table
from block_scaled_fp8_02_gb300 import build as bfbuild
from cache_ref import evict_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    bfbuild.build()
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def make(kv_lens, budget, H=2, D=128, page=64, seed=0, coarse=False):
    g = torch.Generator().manual_seed(seed + 13 * sum(kv_lens) + budget)
    new = [min(n, budget) for n in kv_lens]
    need = [(n + page - 1) // page for n in list(kv_lens) + new]
    pages = sum(need) + 2
    kq, ks, vq, vs = make_cache(pages, H, page, D, g)
    w = torch.exp(2 * torch.randn(pages, H, page, generator=g)) * (torch.rand(pages, H, page, generator=g) < 0.9)
    if coarse:
        w = w.floor()
    both = make_table(list(kv_lens) + new, page, pages, g)
    return dict(k=kq, v=vq, ks=ks, vs=vs, w=w, table=both[:len(kv_lens)].contiguous(), out=both[len(kv_lens):].contiguous(),
                kv=list(kv_lens), budget=budget)


def check(dev, c, recent=0, first=0, in_place=False, max_kv=None, order="phtd", **kw):
    parts = [c["k"].view(torch.uint8), c["v"].view(torch.uint8), c["ks"], c["vs"], c["w"]]
    want, lens = evict_ref(parts, c["w"], c["table"], c["kv"], c["budget"], recent, first, None if in_place else c["out"])
    d = [x.to(dev) for x in parts]
    if order == "pthd":
        d[0], d[1] = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in d[:2])
    cache = bf.KVCache(d[0].view(torch.float8_e4m3fn), d[1].view(torch.float8_e4m3fn), d[2], d[3])
    got = bf.bfp8_kv_cache_evict(cache, d[4], c["table"].to(dev), ints(c["kv"], dev), max_kv or max(c["kv"] + [0]), c["budget"],
                                 recent=recent, first=first, out_table=None if in_place else c["out"].to(dev), **kw)
    torch.cuda.synchronize()
    assert bf.bfp8_device_status(clear=True) == 0
    assert got.tolist() == lens
    for x, y in zip(d, want):
        x, y = (t.contiguous().cpu().view(torch.uint8 if t.element_size() == 1 else torch.int32) for t in (x, y))
        assert torch.equal(x, y)


LENGTHS = {
    "one sequence": ([300], 100),
    "within and beyond the budget": ([0, 1, 99, 100, 101, 250, 1000], 100),
    "one token stays": ([1, 2, 65, 500], 1),
    "almost all stay": ([700], 699),
    "long": ([5000, 70], 1100),
    "many": ([10 * i + 1 for i in range(20)], 64),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", LENGTHS)
@pytest.mark.parametrize("H,D,page", [(2, 128, 64), (3, 64, 16), (1, 128, 256)])
def test_against_reference(dev, name, H, D, page, in_place):
    lens, budget = LENGTHS[name]
    c = make(lens, budget, H, D, page)
    check(dev, c, in_place=in_place)
    check(dev, c, recent=budget // 3, first=min(4, budget // 2), in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("recent,first", [(100, 0), (0, 100), (60, 40), (99, 0), (1, 1)])
def test_first_and_recent(dev, recent, first, in_place):
    check(dev, make([100, 101, 150, 777], 100), recent, first, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_ties_go_to_the_lowest_position(dev, in_place):
    c = make([900, 5000], 333, coarse=True)
    check(dev, c, recent=11, in_place=in_place)
    c["w"] = torch.zeros_like(c["w"])
    c["w"][:, 0] = -0.0
    check(dev, c, recent=5, first=2, in_place=in_place)
    c["w"].view(torch.int32).bernoulli_(0.5).mul_(-2 ** 31)                         # zeros of both signs are equal
    check(dev, c, in_place=in_place)


def test_values_that_are_ordered_oddly(dev):
    """Negative weights, infinities, denormals and what is not a number (larger than any)."""
    c = make([600], 150, H=4)
    w = c["w"]
    w[:, 0] -= 2
    w[:, 1] *= 1e-42
    w[:, 2][torch.rand(w[:, 2].shape) < 0.1] = float("inf")
    w[:, 2][torch.rand(w[:, 2].shape) < 0.1] = float("-inf")
    w[:, 3][torch.rand(w[:, 3].shape) < 0.3] = float("nan")
    w[:, 3].neg_()
    check(dev, c, recent=3)


def test_longer_than_a_cluster_holds(dev):
    """Keys that its shared memory does not hold are read again."""
    c = make([50000], 700, H=1, D=64, page=256)
    check(dev, c, recent=10)
    g = torch.Generator().manual_seed(1)
    n, budget, page = 350000, 100, 256
    P = n // page + 2
    w = torch.rand(P, 1, page, generator=g)
    k = torch.zeros(P + 1, 1, page, 64, dtype=torch.uint8)
    k[..., :4] = torch.arange((P + 1) * page, dtype=torch.int32).view(P + 1, 1, page, 1).view(torch.uint8)
    sc = torch.ones(P + 1, 1, page)
    w = torch.cat([w, torch.zeros(1, 1, page)])
    table, out = torch.randperm(P, generator=g).int()[None], ints([[P]], "cpu")
    d = [x.to(dev) for x in (k, sc, w)]
    cache = bf.KVCache(d[0].view(torch.float8_e4m3fn), d[0].clone().view(torch.float8_e4m3fn), d[1], d[1].clone())
    lens = bf.bfp8_kv_cache_evict(cache, d[2], table.to(dev), ints([n], dev), n, budget, out_table=out.to(dev))
    j = torch.arange(n)
    flat = w[table[0].long()[j // page], 0, j % page]
    keep = torch.sort(flat, descending=True, stable=True).indices[:budget].sort().values
    assert lens.tolist() == [budget]
    assert torch.equal(cache.k.view(torch.uint8)[P, 0, :budget].cpu(), k[table[0].long()[keep // page], 0, keep % page])
    assert torch.equal(d[2][P, 0, :budget].cpu(), flat[keep])


@pytest.mark.parametrize("in_place", [False, True])
def test_many_sequences_longer_than_a_small_block_holds(dev, in_place):
    """More (sequence, head)s than SMs, so small blocks, some of whose keys do not fit them: those are read anew."""
    lens = [50 + i for i in range(200)]
    lens[3], lens[77], lens[199] = 8192, 8193, 21000
    c = make(lens, 300, H=1, D=64, page=256)
    check(dev, c, recent=20, first=3, in_place=in_place)
    check(dev, make(lens, 60, H=1, D=64, page=256, coarse=True), in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_orders_and_strides(dev, in_place):
    c = make([300, 80, 64], 64, H=3)
    check(dev, c, recent=9, in_place=in_place, order="pthd")
    big = torch.full((c["w"].shape[0], 4, 67), 3.0, device=dev)
    w = big[:, 1:, 2:66]
    w.copy_(c["w"])
    cache = bf.KVCache(*(c[n].to(dev) for n in ("k", "v", "ks", "vs")))
    bf.bfp8_kv_cache_evict(cache, w, c["table"].to(dev), ints(c["kv"], dev), 300, 64, recent=9,
                           out_table=None if in_place else c["out"].to(dev))
    parts = [c["k"].view(torch.uint8), c["w"]]
    want, _ = evict_ref(parts, c["w"], c["table"], c["kv"], 64, 9, 0, None if in_place else c["out"])
    assert torch.equal(cache.k.view(torch.uint8).cpu(), want[0]) and torch.equal(w.cpu(), want[1])
    assert (big[:, 0] == 3).all() and (big[:, :, :2] == 3).all() and (big[:, :, 66] == 3).all()


def test_bounds_above_the_lengths(dev):
    def wide(budget):
        c = make([300, 80], budget)
        for key in ("table", "out"):
            c[key] = torch.cat([c[key], torch.full((2, 700), -7, dtype=torch.int32)], 1)
        return c
    c = wide(64)
    for most in (300, 4000, 40000):
        check(dev, c, recent=9, max_kv=most)
        check(dev, c, recent=9, max_kv=most, in_place=True)
    c = wide(1 << 20)                                                               # nothing to do but to copy
    check(dev, c, max_kv=40000)
    check(dev, c, max_kv=40000, in_place=True)


def test_block_table_as_its_own_destination(dev):
    """The same as none: in place."""
    c = make([1300, 80], 600, H=1)
    want, lens = evict_ref([c["k"].view(torch.uint8), c["w"]], c["w"], c["table"], c["kv"], 600, 7, 0)
    for columns in (c["table"].shape[1], 10):
        d = {n: c[n].to(dev) for n in ("k", "v", "ks", "vs", "w")}
        table = c["table"].to(dev)
        got = bf.bfp8_kv_cache_evict(bf.KVCache(d["k"], d["v"], d["ks"], d["vs"]), d["w"], table, ints(c["kv"], dev), 1300, 600, recent=7,
                                     out_table=table[:, :columns])
        assert got.tolist() == lens
        assert torch.equal(d["k"].view(torch.uint8).cpu(), want[0]) and torch.equal(d["w"].cpu(), want[1])


@pytest.mark.parametrize("H,D,page", [(1, 128, 64), (8, 128, 16), (2, 64, 64)])
@pytest.mark.parametrize("n,budget", [(1300, 600), (9000, 2500)])
def test_one_sequence_onto_the_first_columns_of_its_table(dev, n, budget, H, D, page):
    """In place too, although a single row's stride says nothing: many more rows than a block moves at a time."""
    c = make([n], budget, H, D, page)
    parts = [c["k"].view(torch.uint8), c["v"].view(torch.uint8), c["ks"], c["vs"], c["w"]]
    want, lens = evict_ref(parts, c["w"], c["table"], c["kv"], budget, 7, 1)
    wide = torch.full((1, c["table"].shape[1] + 3), -9, dtype=torch.int32)
    wide[:, :-3] = c["table"]
    for columns in ((budget + page - 1) // page, (n + page - 1) // page, wide.shape[1]):
        d = [x.to(dev) for x in parts]
        table = wide.to(dev)
        got = bf.bfp8_kv_cache_evict(bf.KVCache(*(x.view(torch.float8_e4m3fn) for x in d[:2]), *d[2:4]), d[4], table, ints(c["kv"], dev), n,
                                     budget, recent=7, first=1, out_table=table[:, :columns])
        assert got.tolist() == lens
        assert all(torch.equal(x.cpu(), y) for x, y in zip(d, want)), columns
    assert bf.bfp8_device_status() == 0


def test_lengths_for_the_caller(dev):
    c = make([300, 80], 64)
    lens = torch.empty(2, dtype=torch.int32, device=dev)
    check(dev, c, new_lens=lens)
    assert lens.tolist() == [64, 64]
    kv = ints(c["kv"], dev)
    cache = bf.KVCache(*(c[n].to(dev) for n in ("k", "v", "ks", "vs")))
    with pytest.raises(bf.BFP8Error):
        bf.bfp8_kv_cache_evict(cache, c["w"].to(dev), c["table"].to(dev), kv, 300, 64, new_lens=kv)
    none = torch.zeros(0, 4, dtype=torch.int32, device=dev)
    assert bf.bfp8_kv_cache_evict(cache, c["w"].to(dev), none, kv[:0], 0, 64).shape == (0,)
    got = bf.bfp8_kv_cache_evict(cache, c["w"].to(dev), c["table"].to(dev), torch.zeros_like(kv), 0, 64)
    assert got.tolist() == [0, 0]


@pytest.mark.parametrize("in_place", [False, True])
def test_pages_outside_the_cache(dev, in_place):
    c = make([300, 200], 64)
    d = {n: c[n].to(dev) for n in ("k", "v", "ks", "vs", "w")}
    table, out = c["table"].clone(), c["out"].clone()
    table[0, 2] = 1 << 20
    cache = bf.KVCache(d["k"], d["v"], d["ks"], d["vs"])
    bf.bfp8_kv_cache_evict(cache, d["w"], table.to(dev), ints(c["kv"], dev), 300, 64, recent=64 if in_place else 0,
                           out_table=None if in_place else out.to(dev))
    assert bf.bfp8_device_status(clear=True) == 6
    # the other sequence is as it should be
    want, _ = evict_ref([c["w"]], c["w"], c["table"], [0, 200], 64, 64 if in_place else 0, 0, None if in_place else out)
    at = (c["table"] if in_place else out)[1].long()
    at = at[:1]
    assert torch.equal(d["w"][at].cpu(), want[0][at])


def test_captured(dev):
    c = make([500, 300, 90], 100)
    src = {n: c[n].to(dev) for n in ("k", "v", "ks", "vs", "w")}
    d = {n: x.clone() for n, x in src.items()}
    cache = bf.KVCache(d["k"], d["v"], d["ks"], d["vs"])
    kv, lens, table = ints(c["kv"], dev), torch.empty(3, dtype=torch.int32, device=dev), c["table"].to(dev)

    def call():
        bf.bfp8_kv_cache_evict(cache, d["w"], table, kv, 500, 100, recent=10, first=1, new_lens=lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        call()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            call()
    for n in ([500, 300, 90], [99, 101, 450]):
        for name, x in src.items():
            d[name].view(torch.uint8).copy_(x.view(torch.uint8))
        kv.copy_(ints(n[:2] + [min(n[2], 90)], dev))
        graph.replay()
        torch.cuda.synchronize()
        now = kv.tolist()
        want, new = evict_ref([c["k"].view(torch.uint8), c["w"]], c["w"], c["table"], now, 100, 10, 1)
        assert lens.tolist() == new
        assert torch.equal(d["k"].view(torch.uint8).cpu(), want[0]) and torch.equal(d["w"].cpu(), want[1])
