"""The paged-cache calls together, as a program that serves a model makes them:
prompts in one launch, their keys and values into pages, decode steps that add
up the weights, an eviction, and on (GPU)."""

import math
import threading

import numpy as np
import pytest
import torch

import pass_attention_gb300 as oss
from paged_reference import attend, check, evict, f64

pytestmark = pytest.mark.gpu

D, HQ, HKV, PAGE = 128, 8, 2, 16
G = HQ // HKV
SCALE = 1 / math.sqrt(D)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Serving:
    """Three sequences with room to grow, and their history on the host."""

    def __init__(self, lens, grow, seed):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        self.lens = list(lens)
        columns = max(-(-(n + grow) // PAGE) for n in lens)
        pages = 2 * len(lens) * columns
        self.order = torch.randperm(pages, generator=self.gen, device="cuda").to(torch.int32)
        self.table = self.order[:len(lens) * columns].reshape(len(lens), columns).contiguous()
        self.spare = self.order[len(lens) * columns:].reshape(len(lens), columns).contiguous()
        self.kp = torch.full((pages, HKV, PAGE, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.vp = self.kp.clone()
        self.kv_len = ints(self.lens)
        self.weights = torch.zeros((len(lens), HKV, columns * PAGE), device="cuda")
        # per sequence and key head: keys, values and summed weights, in cache order
        self.k = [[np.zeros((0, D))] * HKV for _ in lens]
        self.v = [[np.zeros((0, D))] * HKV for _ in lens]
        self.w = [[np.zeros(0)] * HKV for _ in lens]

    def rand(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda").to(torch.bfloat16)

    def remember(self, b, k, v):
        for g in range(HKV):
            self.k[b][g] = np.concatenate([self.k[b][g], f64(k[:, g])])
            self.v[b][g] = np.concatenate([self.v[b][g], f64(v[:, g])])
            self.w[b][g] = np.concatenate([self.w[b][g], np.zeros(k.shape[0])])

    def prompt(self):
        total = sum(self.lens)
        qkv = self.rand(total, HQ + 2 * HKV, D)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        cu = ints(np.concatenate([[0], np.cumsum(self.lens)]).tolist())
        o, lse = oss.attention_fwd_packed(q, k, v, cu)
        oss.kv_cache_append(k, v, self.kp, self.vp, self.table, self.kv_len, cu)
        at = 0
        for b, n in enumerate(self.lens):
            self.remember(b, k[at:at + n], v[at:at + n])
            seen = np.tril(np.ones((n, n), bool))
            for h in range(HQ):
                ro, rl, _, bo, bl, _ = attend(f64(q[at:at + n, h]), self.k[b][h // G], self.v[b][h // G], seen, SCALE, 2.0 ** -8, False)
                check(f64(o[at:at + n, h]), ro, bo, f"prompt {b} head {h}")
                check(f64(lse[at:at + n, h]), rl, bl, f"prompt {b} head {h} lse")
            at += n

    def step(self):
        n = len(self.lens)
        q, k, v = self.rand(n, HQ, D), self.rand(n, HKV, D), self.rand(n, HKV, D)
        self.kv_len += 1
        oss.kv_cache_append(k, v, self.kp, self.vp, self.table, self.kv_len)
        o, lse = oss.attention_decode_paged(q, self.kp, self.vp, self.table, self.kv_len, weights=self.weights)
        for b in range(n):
            self.remember(b, k[b:b + 1], v[b:b + 1])
            for h in range(HQ):
                g = h // G
                keys = self.k[b][g]
                ro, rl, p, bo, bl, _ = attend(f64(q[b, h:h + 1]), keys, self.v[b][g], np.ones((1, len(keys)), bool), SCALE, 2.0 ** -8, False)
                check(f64(o[b, h:h + 1]), ro, bo, f"step, sequence {b} head {h}")
                check(f64(lse[b, h:h + 1]), rl, bl, f"step, sequence {b} head {h} lse")
                self.w[b][g] = self.w[b][g] + p[0]

    def evict(self, budget, recent):
        kept, new_len, self.weights = oss.kv_cache_evict(self.kp, self.vp, self.weights, self.table, self.kv_len, self.spare,
                                                         budget, recent)
        self.table, self.spare, self.kv_len = self.spare, self.table, new_len
        for b in range(len(self.lens)):
            n = int(new_len[b])
            assert n == min(len(self.w[b][0]), budget)
            for g in range(HKV):
                pos = kept[b, g, :n].cpu().numpy()
                # weights that differ by less than their error (a relative 4e-4: twice
                # the score's 2 D 2^-24 sum |q k| scale, sum |q k| scale up to 12) may
                # change places: the kept ones weigh as much as the reference's
                ref = evict(self.w[b][g].astype(np.float32), len(self.w[b][g]), budget, recent)
                np.testing.assert_allclose(np.sort(self.w[b][g][pos]), np.sort(self.w[b][g][ref]), rtol=1e-3)
                self.k[b][g], self.v[b][g], self.w[b][g] = self.k[b][g][pos], self.v[b][g][pos], self.w[b][g][pos]


def test_prompts_steps_and_evictions():
    s = Serving([40, 129, 7], grow=12, seed=1)
    s.prompt()
    for _ in range(3):
        s.step()
    s.evict(48, 8)
    for _ in range(3):
        s.step()
    s.evict(40, 0)
    s.step()
    assert oss.check_device_error() == 0


@pytest.mark.parametrize("stale", [0, 1 << 20])
def test_decode_directly_behind_an_eviction(stale):
    # the lengths that eviction writes are the next call's kv_len, with no other
    # kernel between the two: every kernel of the decode has to wait for them,
    # whatever the buffer held before
    batch, hkv, hq, page, n, budget = 4, 2, 8, 16, 8000, 1000
    gen = torch.Generator(device="cuda")
    gen.manual_seed(11)
    columns, new_columns = n // page, -(-budget // page) + 1
    pages = batch * (columns + new_columns)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    kp, vp = (r(pages, hkv, page, 128).to(torch.bfloat16) for _ in range(2))
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = order[:batch * columns].view(batch, columns)
    new_table = order[batch * columns:].view(batch, new_columns)
    kv_len = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    w = r(batch, hkv, n).square_()
    q = r(batch, hq, 128).to(torch.bfloat16)
    new_len = torch.empty(batch, dtype=torch.int32, device="cuda")
    new_w = torch.empty((batch, hkv, new_columns * page), device="cuda")
    want = None
    for i in range(10):
        new_len.fill_(budget if i == 0 else stale)
        oss.kv_cache_evict(kp, vp, w, table, kv_len, new_table, budget, 10, new_len=new_len, new_weights=new_w)
        if i == 0:
            torch.cuda.synchronize()
        o, lse = oss.attention_decode_paged(q, kp, vp, new_table, new_len, weights=new_w)
        got = o.view(torch.int16).clone(), lse.clone(), new_w.clone()
        if i == 0:
            want = got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.all(new_w[:, :, budget:] == 0)
    assert oss.check_device_error() == 0


def test_a_step_in_a_graph_follows_the_cache():
    # length, append, decode and weights in one captured step, replayed token by
    # token beside the same steps made one by one
    one, two = Serving([33, 400], grow=40, seed=2), Serving([33, 400], grow=40, seed=2)
    for s in (one, two):
        s.prompt()
    q, k, v = one.rand(2, HQ, D), one.rand(2, HKV, D), one.rand(2, HKV, D)

    def step(s):
        s.kv_len += 1
        oss.kv_cache_append(k, v, s.kp, s.vp, s.table, s.kv_len)
        return oss.attention_decode_paged(q, s.kp, s.vp, s.table, s.kv_len, weights=s.weights)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step(one)
    for _ in range(30):
        for x in (q, k, v):
            x.copy_(one.rand(*x.shape))
        graph.replay()
        eo, el = step(two)
        assert torch.equal(o, eo) and torch.equal(lse, el)
    assert torch.equal(one.weights, two.weights) and torch.equal(one.kv_len, two.kv_len)
    assert torch.equal(one.kp.view(torch.int16), two.kp.view(torch.int16))
    kept = torch.empty((2, HKV, 64), dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, n1, w1 = oss.kv_cache_evict(one.kp, one.vp, one.weights, one.table, one.kv_len, one.spare, 64, 4, kept=kept)
    graph.replay()
    k2, n2, w2 = oss.kv_cache_evict(two.kp, two.vp, two.weights, two.table, two.kv_len, two.spare, 64, 4)
    assert torch.equal(kept, k2) and torch.equal(n1, n2) and torch.equal(w1, w2)
    assert torch.equal(one.kp.view(torch.int16), two.kp.view(torch.int16))
    assert oss.check_device_error() == 0


def test_calls_from_several_threads():
    # threads that share a stream share its workspace, threads with streams of
    # their own do not: the same bits from all
    s = Serving([1500, 20, 700], grow=4, seed=3)
    s.prompt()
    q = s.rand(3, HQ, D)
    qkv = s.rand(900, HQ + 2 * HKV, D)
    cu = ints([0, 100, 850, 900])
    decode = lambda **kw: oss.attention_decode_paged(q, s.kp, s.vp, s.table, s.kv_len, **kw)  # noqa: E731
    packed = lambda **kw: oss.attention_fwd_packed(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], cu, **kw)  # noqa: E731
    want = {decode: decode(), packed: packed()}
    torch.cuda.synchronize()
    wrong = []

    def work(call, stream):
        outs = [call(stream=stream) if stream else call() for _ in range(40)]
        torch.cuda.synchronize()
        if not all(torch.equal(a, b) for out in outs for a, b in zip(out, want[call])):
            wrong.append(call)

    shared = torch.cuda.Stream()
    threads = [threading.Thread(target=work, args=(c, st)) for c in (decode, packed)
               for st in (None, shared, shared, torch.cuda.Stream())]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert oss.check_device_error() == 0
