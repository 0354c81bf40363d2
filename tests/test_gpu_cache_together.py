"""Shared prefixes, accumulated weights and eviction as a serving loop runs them: a batch continues one prompt token by
token, its tokens are weighed under the softmax over both parts, its sequences are cut and go on."""
import pytest
import torch

import block_scaled_fp8_02_gb300 as bf
from attn_ref import check_attention
from block_scaled_fp8_02_gb300 import build as bfbuild
from cache_ref import evict_ref, shared_ref, weigh_ref

pytestmark = pytest.mark.gpu

H, HQ, D, PAGE, B = 2, 8, 128, 16, 5


@pytest.fixture(scope="module")
def dev():
    bfbuild.build()
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


class Batch:
    """B sequences behind one prompt of P tokens, with pages for `most` tokens each."""

    def __init__(self, dev, P, most, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        self.dev, self.P, self.per = dev, P, (most + PAGE - 1) // PAGE
        ahead = (P + PAGE - 1) // PAGE
        pages = ahead + B * self.per
        order = torch.randperm(pages, generator=self.g).int()
        self.ptable, self.table = order[None, :ahead].contiguous(), order[ahead:].view(B, self.per).contiguous()
        self.cache = bf.KVCache.empty(pages, H, PAGE, D, dev)
        self.weights = torch.full((pages, H, PAGE), 99.0, device=dev)                # whatever was there
        j = torch.arange(P)
        self.write(P, self.ptable[0].long()[j // PAGE] * PAGE + j % PAGE)
        # the prompt's sums begin at zero
        at = self.ptable[0].long().to(dev)
        self.weights[at] = 0
        self.lens = [0] * B

    def write(self, n, slots):
        k, v = (torch.randn(n, H, D, generator=self.g).bfloat16().to(self.dev) for _ in range(2))
        bf.bfp8_kv_cache_write(k, v, self.cache, slots.to(self.dev))

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32).to(self.dev, non_blocking=True)

    def step(self, counts):
        """counts[b] new tokens a sequence: written, attended, weighed.  Returns what went in and came out."""
        cu, slots = [0], []
        for b, n in enumerate(counts):
            j = torch.arange(self.lens[b], self.lens[b] + n)
            slots.append(self.table[b].long()[j // PAGE] * PAGE + j % PAGE)
            self.lens[b] += n
            cu.append(cu[-1] + n)
        T = cu[-1]
        self.write(T, torch.cat(slots))
        q = (2 * torch.randn(T, HQ, D, generator=self.g)).bfloat16()
        dq, dcu, dl = q.to(self.dev), self.ints(cu), self.ints(self.lens)
        pcu, plen, pt, table = self.ints([0, T]), self.ints([self.P]), self.ptable.to(self.dev), self.table.to(self.dev)
        mq, mk = max(counts), max(self.lens)
        out, lse = bf.bfp8_shared_prefix_attention(dq, self.cache, pt, pcu, plen, T, self.P, table, dcu, dl, mq, mk, return_lse=True)
        bf.bfp8_kv_cache_weigh(dq, lse, self.cache, self.weights, table, dcu, dl, mq, mk)
        bf.bfp8_kv_cache_weigh(dq, lse, self.cache, self.weights, pt, pcu, plen, T, self.P, causal=False)
        return q, cu, out, lse

    def host(self):
        c = self.cache
        codes = [t.view(torch.uint8).cpu().view(torch.float8_e4m3fn) for t in (c.k, c.v)]
        return (*codes, c.k_scale.cpu(), c.v_scale.cpu())

    def sums(self):
        """Of the own tokens and the prompt's, a kv head each."""
        w = self.weights.cpu().double()
        total = w[self.ptable[0].long()].transpose(1, 2).reshape(-1, H)[: self.P].sum(0)
        for b, n in enumerate(self.lens):
            total += w[self.table[b].long()].transpose(1, 2).reshape(-1, H)[:n].sum(0)
        return total


@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("first,P", [(1, 300), (30, 150)])
def test_a_batch_goes_on(dev, first, P, stream):
    s = torch.cuda.Stream() if stream else torch.cuda.current_stream()
    with torch.cuda.stream(s):
        x = Batch(dev, P, 200)
        rows = 0
        for counts in ([first + b for b in range(B)], [1] * B, [1] * B, [2, 1, 3, 1, 1]):
            before = x.weights.clone()
            q, cu, out, lse = x.step(counts)
            torch.cuda.synchronize()
            k, v, ks, vs = x.host()
            rows += cu[-1]
            check_attention(out, lse, shared_ref(q, k, v, ks, vs, x.ptable, [0, cu[-1]], [P], x.table, cu, x.lens, D ** -0.5))
            want, tol = weigh_ref(q, lse.cpu(), k, ks, before.cpu(), x.table, cu, x.lens, D ** -0.5)
            want, t2 = weigh_ref(q, lse.cpu(), k, ks, want, x.ptable, [0, cu[-1]], [P], D ** -0.5, causal=False)
            assert ((x.weights.cpu().double() - want).abs() <= tol + t2).all()
        # every row's weights, over both parts, sum to one; lse and scores are within 1e-5 or so
        assert torch.allclose(x.sums(), torch.full((H,), rows * HQ / H, dtype=torch.float64), rtol=1e-4)
        # cut, and on
        k, v, ks, vs = x.host()
        parts = [k.view(torch.uint8), v.view(torch.uint8), ks, vs, x.weights.cpu()]
        budget = 4 + first // 2
        want, lens = evict_ref(parts, parts[-1], x.table, x.lens, budget, 2, 1)
        new = bf.bfp8_kv_cache_evict(x.cache, x.weights, x.table.to(dev), x.ints(x.lens), max(x.lens), budget, recent=2, first=1)
        assert new.tolist() == lens
        got = [t.view(torch.uint8).cpu() for t in (x.cache.k, x.cache.v)] + [x.cache.k_scale.cpu(), x.cache.v_scale.cpu(), x.weights.cpu()]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        x.lens = lens
        q, cu, out, lse = x.step([1] * B)
        k, v, ks, vs = x.host()
        check_attention(out, lse, shared_ref(q, k, v, ks, vs, x.ptable, [0, cu[-1]], [P], x.table, cu, x.lens, D ** -0.5))
        torch.cuda.synchronize()
        assert bf.bfp8_device_status() == 0


def test_a_decoding_step_in_one_graph(dev):
    """Write, attention, both sums and the eviction captured together, replayed with growing lengths."""
    x = Batch(dev, 200, 64, seed=3)
    x.step([20] * B)
    table, pt = x.table.to(dev), x.ptable.to(dev)
    k, v = (torch.randn(B, H, D, device=dev).bfloat16() for _ in range(2))
    q = torch.randn(B, HQ, D, device=dev).bfloat16()
    cu, pcu, plen = x.ints(list(range(B + 1))), x.ints([0, B]), x.ints([200])
    lens, new = x.ints([20] * B), torch.empty(B, dtype=torch.int32, device=dev)
    slots = torch.empty(B, dtype=torch.int64, device=dev)
    lse_out = []

    def step():
        lens.add_(1)
        at = (lens - 1).long()
        slots.copy_(table.long().gather(1, (at // PAGE)[:, None])[:, 0] * PAGE + at % PAGE)
        bf.bfp8_kv_cache_write(k, v, x.cache, slots)
        out, lse = bf.bfp8_shared_prefix_attention(q, x.cache, pt, pcu, plen, B, 200, table, cu, lens, 1, 64, return_lse=True)
        bf.bfp8_kv_cache_weigh(q, lse, x.cache, x.weights, table, cu, lens, 1, 64)
        bf.bfp8_kv_cache_evict(x.cache, x.weights, table, lens, 64, 24, recent=4, new_lens=new)
        lens.copy_(new)
        lse_out[:] = [out, lse]

    state = [t.clone() for t in (x.cache.k.view(torch.uint8), x.cache.v.view(torch.uint8), x.cache.k_scale, x.cache.v_scale, x.weights, lens)]

    def reset():
        for t, s in zip((x.cache.k.view(torch.uint8), x.cache.v.view(torch.uint8), x.cache.k_scale, x.cache.v_scale, x.weights, lens), state):
            t.copy_(s)
    eager = []
    for i in range(8):
        q.normal_(generator=torch.Generator(device=dev).manual_seed(i))
        k.normal_(generator=torch.Generator(device=dev).manual_seed(100 + i))
        step()
        eager.append([t.clone() for t in (*lse_out, lens, x.weights)])
    assert lens.tolist() == [24] * B
    reset()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
        reset()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            step()
    for i in range(8):
        q.normal_(generator=torch.Generator(device=dev).manual_seed(i))
        k.normal_(generator=torch.Generator(device=dev).manual_seed(100 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager[i], (*lse_out, lens, x.weights))), i
    assert bf.bfp8_device_status() == 0


def test_calls_of_every_kind_in_turn_on_one_workspace(dev):
    """Nothing waits between them: each finds the counters at zero and leaves the others' partial rows alone."""
    g = torch.Generator().manual_seed(7)
    pages = 400
    codes = [torch.randint(0, 120, (pages, H, PAGE, D), generator=g, dtype=torch.uint8).to(dev) for _ in range(2)]
    scales = [(torch.rand(pages, H, PAGE, generator=g) * 0.01 + 1e-3).to(dev) for _ in range(2)]
    w0 = torch.rand(pages, H, PAGE, generator=g).to(dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def case(plens, pcu, q_lens, kv_lens):
        order = torch.randperm(pages, generator=g).int().to(dev)
        width = (max(kv_lens) + PAGE - 1) // PAGE
        ahead = (max(plens) + PAGE - 1) // PAGE
        cu = [0]
        for m in q_lens:
            cu.append(cu[-1] + m)
        q = torch.randn(cu[-1], HQ, D, generator=g).bfloat16().to(dev)
        table, ptable = order[:len(q_lens) * width].view(len(q_lens), width), order[-len(plens) * ahead:].view(len(plens), ahead)
        pq = max(b - a for a, b in zip(pcu, pcu[1:]))
        i = [ints(v) for v in (pcu, plens, cu, kv_lens)]

        def run():
            cache = bf.KVCache(*(c.clone().view(torch.float8_e4m3fn) for c in codes), *(s.clone() for s in scales))
            w = w0.clone()
            o, lse = bf.bfp8_shared_prefix_attention(q, cache, ptable, i[0], i[1], pq, max(plens), table, i[2], i[3], max(q_lens),
                                                     max(kv_lens), return_lse=True)
            o2, l2 = bf.bfp8_paged_attention(q, cache, table, i[2], i[3], max(q_lens), max(kv_lens), return_lse=True)
            bf.bfp8_kv_cache_weigh(q, lse, cache, w, table, i[2], i[3], max(q_lens), max(kv_lens))
            lens = bf.bfp8_kv_cache_evict(cache, w, table, i[3], max(kv_lens), 20, recent=3)
            return [o, lse, o2, l2, w, lens, cache.k.view(torch.uint8), cache.v_scale]
        return run

    calls = [case([300], [0, 3], [1] * 3, [5, 64, 129]), case([1500], [0, 20], [1] * 20, [3 * i + 1 for i in range(20)]),
             case([700, 33], [0, 30, 33], [1] * 33, [i + 1 for i in range(33)]), case([260], [0, 150], [100, 50], [100, 400]),
             case([515], [0, 88], [1, 40, 1, 45, 1], [300, 40, 1, 200, 77]), case([90, 2000], [0, 2, 60], [2] * 30, [17 + i for i in range(30)])]
    alone = []
    for call in calls:
        alone.append(call())
        torch.cuda.synchronize()
    order = [i for _ in range(6) for i in torch.randperm(len(calls), generator=g).tolist()]
    got = [calls[i]() for i in order]
    torch.cuda.synchronize()
    assert bf.bfp8_device_status() == 0
    for i, r in zip(order, got):
        assert all(torch.equal(a, b) for a, b in zip(r, alone[i])), i
