"""attention_decode_shared against its definition in 64 bits, and beside
attention_decode_paged (GPU)."""

import math
import random
import threading

import numpy as np
import pytest
import torch

import pass_attention_gb300 as oss
from fp8_reference import check_shared
from paged_reference import DTYPES, f64, gather

pytestmark = pytest.mark.gpu


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# Prefixes that cost little to read again are read by every sequence, by what the table has
# room for: every test runs over tables of the prefixes' own width, and over wide ones, which send
# the prefixes to the tensor cores.
WIDE = False
READ_AGAIN = 80 << 20


@pytest.fixture(params=[False, True], ids=["narrow", "wide"], autouse=True)
def wide(request):
    global WIDE
    WIDE = request.param
    yield
    WIDE = False


class Case:
    """Pools whose pages are in random order, with NaN in every slot that no token has, and -1 behind
    each sequence's and prefix's last page."""

    def __init__(self, sizes, prefixes, own, hq, hkv, d=128, page=16, dtype="bf16", layout="head", seed=0, columns=None,
                 prefix_columns=None, outside=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.gen, self.page, self.heads = gen, page, hkv
        self.own, self.prefixes = list(own), list(prefixes)
        batch = sum(sizes) + outside
        assert len(own) == batch and len(prefixes) == len(sizes)
        need, need0 = [-(-n // page) for n in own], [-(-n // page) for n in prefixes]
        pages = sum(need) + sum(need0) + 3
        r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(DTYPES[dtype])  # noqa: E731
        if layout == "slot":
            self.kp, self.vp = (r(pages, page, hkv, d).transpose(1, 2) for _ in range(2))
        elif layout == "joint":
            both = r(pages, 2, hkv, page, d)
            self.kp, self.vp = both[:, 0], both[:, 1]
        else:
            self.kp, self.vp = r(pages, hkv, page, d), r(pages, hkv, page, d)
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        again = (batch - len(sizes)) * hkv * page * 4 * d  # bytes of a page, for each sequence that reads it again
        if WIDE and prefix_columns is None and again > 0:
            prefix_columns = max(READ_AGAIN // again + 1, max(need0))
        at = 0
        free = torch.ones((pages, page), dtype=torch.bool, device="cuda")
        tables = []
        for lens, count, width in ((own, need, columns), (prefixes, need0, prefix_columns)):
            table = torch.full((len(lens), width or max(max(count), 1)), -1, dtype=torch.int32, device="cuda")
            for b, n in enumerate(lens):
                table[b, :count[b]] = order[at:at + count[b]]
                at += count[b]
                t = torch.arange(n, device="cuda")
                free[table[b, t // page].long(), t % page] = False
            tables.append(table)
        self.table, self.prefix_table = tables
        for x in (self.kp, self.vp):
            x.transpose(1, 2)[free] = float("nan")
        self.kv_len, self.prefix_len = ints(own), ints(prefixes)
        self.cu = ints(np.concatenate([[0], np.cumsum(sizes)]).tolist())
        self.group = [g for g, n in enumerate(sizes) for _ in range(n)] + [-1] * outside
        self.q = r(batch, hq, d)
        self.scale = 1.0 / math.sqrt(d)

    def args(self):
        return self.q, self.kp, self.vp, self.prefix_table, self.prefix_len, self.table, self.kv_len

    def run(self, **kw):
        return oss.attention_decode_shared(*self.args(), self.cu, **kw)

    def seen(self, pool):
        cache = {}

        def rows(b, g):
            own = gather(pool, self.table[b], self.own[b], g)
            if self.group[b] < 0:
                return own
            key = (self.group[b], g)
            if key not in cache:
                cache[key] = gather(pool, self.prefix_table[key[0]], self.prefixes[key[0]], g)
            return np.concatenate([cache[key], own])
        rows.heads = self.heads
        return rows

    def check(self, o, lse, scale=None, rows=None):
        check_shared(o, lse, self.q, self.seen(self.kp), self.seen(self.vp), scale or self.scale, rows)

    def go(self, rows=None, **kw):
        o, lse = self.run(**kw)
        assert oss.check_device_error() == 0
        self.check(o, lse, rows=rows)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 300, 1000])
def test_types_and_prefix_lengths(d, dtype, prefix):
    Case([6], [prefix], [0, 1, 16, 33, 200, 7], 8, 2, d=d, dtype=dtype, seed=prefix).go()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 4), (10, 2), (7, 1), (8, 1), (12, 1), (24, 2), (16, 1),
                                    (17, 1), (33, 1), (64, 1), (128, 1), (256, 1), (35, 5)])
@pytest.mark.parametrize("columns", [None, 40])  # own tokens in one piece, and cut
def test_groups_of_heads(hq, hkv, columns):
    Case([5], [333], [70, 5, 0, 257, 1], hq, hkv, page=32, seed=hq, columns=columns).go()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("layout", ["head", "slot", "joint"])
def test_pages_and_layouts(page, layout):
    Case([2, 3], [2 * page + 5, page - 1], [1, page - 1, page, page + 1, 2 * page + 7], 8, 2, page=page, layout=layout,
         seed=page).go()


@pytest.mark.parametrize("sizes,prefixes", [
    ([1, 1, 1], [100, 0, 500]),              # prefixes of one sequence each
    ([0, 4, 0, 3, 0], [50, 700, 0, 129, 9]),  # groups of none
    ([33, 1, 40, 2], [128, 1000, 17, 2000]),  # tiles that begin inside a group's rows of q
    ([2] * 60, [64 + 3 * i for i in range(60)]),
    ([1] * 70, [5 * i for i in range(70)]),  # more groups than are looked up by every sequence
])
def test_groups_of_sequences(sizes, prefixes):
    own = [(37 * i) % 90 for i in range(sum(sizes))]
    Case(sizes, prefixes, own, 4, 1, seed=len(sizes)).go()
    Case(sizes, prefixes, own, 6, 2, d=64, dtype="f16", seed=len(sizes)).go()


@pytest.mark.parametrize("sizes,prefixes", [([20], [700]), ([17, 3], [300, 900]), ([9, 9], [129, 1])])
def test_many_tiles_of_rows(sizes, prefixes):
    # 128 heads of a key head fill a tile each: a tile or two for every sequence, more than eight a group
    n = sum(sizes)
    Case(sizes, prefixes, [(13 * i) % 40 for i in range(n)], 256, 1, d=64, seed=n).go(rows=[0, n // 2, n - 1])
    Case(sizes, prefixes, [(13 * i) % 40 for i in range(n)], 128, 1, seed=n).go(rows=[0, n // 2, n - 1])


def test_sequences_outside_every_group():
    c = Case([2, 2], [300, 90], [10, 0, 500, 20, 40, 0, 333], 8, 2, outside=3, seed=3)
    c.go()
    # before the first group too
    c.cu = ints([1, 2, 4])
    c.group = [-1, 0, 1, 1, -1, -1, -1]
    c.go()


def test_one_group_without_offsets():
    c = Case([5], [400], [10, 0, 70, 3, 1], 8, 2, seed=4)
    a = oss.attention_decode_shared(*c.args())
    b = c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(*a)


@pytest.mark.parametrize("sizes,prefixes,own,hq,hkv,d,dtype,page", [
    ([1], [40001], [5], 8, 1, 128, "bf16", 64),          # a prefix over the whole GPU for one tile of rows
    ([70], [9000], [64] * 70, 8, 2, 128, "bf16", 128),   # several tiles of rows
    ([300], [700], [3] * 300, 4, 2, 64, "f16", 16),
    ([3, 40, 1], [20000, 5, 3000], [17, 8000] * 22, 4, 1, 128, "bf16", 32),
])
def test_long_and_many(sizes, prefixes, own, hq, hkv, d, dtype, page):
    n = len(own)
    rows = None if n < 50 else sorted({0, 1, n // 2, n - 1})
    Case(sizes, prefixes, own, hq, hkv, d=d, dtype=dtype, page=page, seed=n).go(rows=rows)


def test_a_prefix_that_outweighs_and_one_that_does_not():
    # one key takes nearly all the weight: in the prefix's first, a middle or its last tile, or
    # among the own tokens
    c = Case([4], [900], [100] * 4, 4, 1, page=32, seed=5)
    for b, t in enumerate((3, 450, 899)):
        c.kp[c.prefix_table[0, t // 32].long(), 0, t % 32] = c.q[b, 1] * 8
    c.kp[c.table[3, 2].long(), 0, 30] = c.q[3, 1] * 8
    c.go()


def test_strided_query_given_outputs_and_scale():
    c = Case([3], [200], [50, 300, 0], 4, 2, seed=6)
    wide = torch.zeros((3, 12, 128), dtype=c.q.dtype, device="cuda")
    wide[:, 4:8] = c.q
    o, lse = torch.full_like(c.q, 7.0), torch.full((3, 4), 7.0, device="cuda")
    out = oss.attention_decode_shared(wide[:, 4:8], *c.args()[1:], c.cu, scale=0.3, o=o, lse=lse)
    assert out[0] is o and out[1] is lse
    c.check(o, lse, scale=0.3)


def test_a_query_that_holds_nan():
    c = Case([3, 2], [300, 0], [40, 0, 90, 0, 7], 8, 2, seed=7)
    good = c.run()
    bad = c.q.clone()
    bad[0, 1, 3] = float("nan")
    bad[3] = float("nan")       # without any key
    o, lse = oss.attention_decode_shared(bad, *c.args()[1:], c.cu)
    assert torch.isnan(o[0, 1]).all() and torch.isnan(lse[0, 1])
    assert torch.all(o[3] == 0) and torch.isneginf(lse[3]).all()
    o[0, 1], lse[0, 1] = good[0][0, 1], good[1][0, 1]
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])
    assert oss.check_device_error() == 0


@pytest.mark.parametrize("page", [16, 64, 256])
def test_bad_pages_are_left_out(page):
    prefix = 3 * page
    c = Case([4], [prefix], [20, 0, 5, 40], 8, 2, page=page, seed=8)
    full = c.prefix_table.clone()
    for bad in (-1, c.kp.shape[0], 2 ** 31 - 1):
        c.prefix_table = full.clone()
        c.prefix_table[0, 1] = bad
        o, lse = c.run()
        with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
            oss.check_device_error()
        assert oss.check_device_error() == 0
        c.prefix_table, c.prefixes = torch.cat([full[:, :1], full[:, 2:]], 1), [2 * page]
        c.check(o, lse)
        c.prefix_table = full
        c.prefixes = [prefix]
    c.prefix_table = torch.full_like(full, -5)
    o, lse = c.run()
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()
    c.prefixes = [0]
    c.check(o, lse)


def test_lengths_outside_the_tables_are_clamped():
    c = Case([2, 2], [64, 40], [32, 30, 0, 5], 4, 1, seed=9, prefix_columns=4)
    c.prefix_len, c.kv_len = ints([65, -3]), ints([33, 30, -1, 5])
    c.prefixes = [64, 0]
    c.go()
    # 24 sequences over a table of 1024 tokens, on the tensor cores
    c = Case([24], [1024], [32] + [7] * 23, 16, 8, seed=9, prefix_columns=64)
    c.prefix_len, c.kv_len = ints([2 ** 31 - 1]), ints([33] + [7] * 23)
    c.go(rows=[0, 23])


@pytest.mark.parametrize("cu", [[0, 3, 2], [0, 2, 9], [-1, 2, 4]])
def test_offsets_that_do_not_fit_are_reported(cu):
    c = Case([2, 2], [64, 40], [16, 30, 0, 5], 4, 1, seed=9)
    c.cu = ints(cu)
    c.run()
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()
    assert oss.check_device_error() == 0


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    r = random.Random(seed)
    sizes = [r.choice((0, 1, 1, 2, 7, r.randint(1, 40))) for _ in range(r.choice((1, 1, 2, 5, 34)))]
    sizes[-1] = max(sizes[-1], 1)
    outside = r.choice((0, 0, 2))
    n = sum(sizes) + outside
    prefixes = [r.choice((0, 1, 100, 128, r.randint(1, 3000))) for _ in sizes]
    own = [r.choice((0, 1, r.randint(1, 100), r.randint(1, 900))) for _ in range(n)]
    hkv = r.choice((1, 1, 2, 3, 4))
    hq = hkv * r.choice((1, 2, 3, 4, 6, 8, 9, 16, 17, 40))
    c = Case(sizes, prefixes, own, hq, hkv, d=r.choice((64, 128)), dtype=r.choice(("bf16", "f16")),
             page=r.choice((16, 32, 128, 256)), layout=r.choice(("head", "slot", "joint")), outside=outside, seed=seed)
    c.go(rows=sorted(set(r.sample(range(n), min(n, 3)) + [n - 1])))


def test_as_the_paged_decode_over_the_same_tokens():
    # a prefix of whole pages: the same tokens by one table for each sequence
    c = Case([6], [640], [0, 1, 33, 100, 64, 7], 8, 2, page=32, seed=11)
    o, lse = c.run()
    table = torch.cat([c.prefix_table[:, :20].expand(6, -1), c.table], 1).contiguous()
    ro, rl = oss.attention_decode_paged(c.q, c.kp, c.vp, table, c.kv_len + 640)
    u = torch.finfo(c.q.dtype).eps / 2
    # both round o once and the weights once: 2 (u |o| + u sum p |v|), |v| <= 6
    assert (o.float() - ro.float()).abs().max() <= 2 * u * (ro.float().abs().max() + 6)
    assert (lse - rl).abs().max() <= 1e-4


def test_same_bits_every_time_and_beside_other_calls():
    c = Case([5, 4], [5000, 700], [100, 0, 31, 900, 2000, 1, 1, 1, 1], 8, 2, page=64, seed=10)
    ref = c.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [c.run(stream=s) for s in streams for _ in range(5)]
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_from_several_threads():
    c = Case([5, 4], [3000, 700], [100, 0, 31, 900, 2000, 1, 1, 1, 1], 8, 2, page=64, seed=12)
    want = c.run()
    torch.cuda.synchronize()
    wrong = []

    def work(stream):
        outs = [c.run(stream=stream) for _ in range(30)]
        torch.cuda.synchronize()
        if not all(torch.equal(a, b) for out in outs for a, b in zip(out, want)):
            wrong.append(stream)

    shared = torch.cuda.Stream()
    threads = [threading.Thread(target=work, args=(s,)) for s in (None, shared, shared, torch.cuda.Stream())]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert oss.check_device_error() == 0


def test_outputs_have_guards():
    c = Case([2, 3], [300, 20], [0, 1, 40, 0, 333], 12, 4, d=64, seed=18)
    flat, lse = torch.full((5 * 12 * 64 + 256,), 7.0, dtype=c.q.dtype, device="cuda"), torch.full((5 * 12 + 64,), 7.0, device="cuda")
    o, l = flat[128:-128].view(5, 12, 64), lse[32:-32].view(5, 12)
    c.run(o=o, lse=l)
    c.check(o, l)
    assert torch.all(flat[:128] == 7.0) and torch.all(flat[-128:] == 7.0)
    assert torch.all(lse[:32] == 7.0) and torch.all(lse[-32:] == 7.0)


def test_behind_kernels_that_write_what_it_reads():
    # lengths, tables, queries and cached rows come from kernels right before the call, and
    # what the buffers held before is the last step's
    c = Case([5, 4], [900, 300], [100, 0, 31, 64, 17, 1, 1, 80, 5], 8, 2, page=32, seed=19)
    names = ("q", "kp", "vp", "prefix_table", "prefix_len", "table", "kv_len", "cu")
    want, good = c.run(), {n: getattr(c, n).clone() for n in names}
    torch.cuda.synchronize()
    for i in range(10):
        for n in names:  # empty groups and sequences, other values
            x = getattr(c, n)
            x.zero_() if n in ("kv_len", "prefix_len", "cu") else x.fill_(0 if "table" in n else i)
        c.run()
        for n in names:
            getattr(c, n).copy_(good[n])
        o, lse = c.run()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert oss.check_device_error() == 0


def test_the_binding_refuses():
    c = Case([2, 2], [64, 40], [16, 30, 0, 5], 4, 2, seed=9)
    q, kp, vp, pt, pn, table, kv_len = c.args()
    call = oss.attention_decode_shared
    with pytest.raises(ValueError, match="several groups"):
        call(*c.args())
    with pytest.raises(ValueError, match="one entry more"):
        call(*c.args(), c.cu[:2])
    with pytest.raises(ValueError, match="prefix_len must have one entry"):
        call(q, kp, vp, pt, pn[:1], table, kv_len, c.cu)
    with pytest.raises(TypeError):
        call(q, kp, vp, pt.long(), pn, table, kv_len, c.cu)
    with pytest.raises(ValueError, match="like the cache"):
        call(q[:3], kp, vp, pt, pn, table, kv_len, c.cu)
    with pytest.raises(ValueError, match="cannot share"):
        call(q[:, :3], kp, vp, pt, pn, table, kv_len, c.cu)
    with pytest.raises(ValueError):
        call(q, kp, vp, pt.cpu(), pn, table, kv_len, c.cu)
    assert oss.check_device_error() == 0


# -- together --------------------------------------------------------------------------------

def test_a_prompt_then_steps_of_its_samples():
    # one prompt, attended to and cached once; its samples grow behind it token by token,
    # the last steps from a graph
    gen = torch.Generator(device="cuda")
    gen.manual_seed(33)
    hq, hkv, d, page, dtype, batch, prompt, steps = 8, 2, 128, 16, torch.bfloat16, 5, 173, 6
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    pages, room = 11 + batch, 1300 if WIDE else 11  # (11: 4 sequences read it again, 1.4 MB; 1300: 85 MB)
    kp, vp = (torch.full((pages, hkv, page, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    prefix_table, table = torch.full((1, room), -1, dtype=torch.int32, device="cuda"), order[11:, None].contiguous()
    prefix_table[0, :11] = order[:11]
    prefix_len, cu = ints([prompt]), ints([0, prompt])
    q, k, v = r(prompt, hq, d), r(prompt, hkv, d), r(prompt, hkv, d)
    oss.attention_fwd_packed(q, k, v, cu)
    oss.kv_cache_append(k, v, kp, vp, prefix_table, prefix_len, cu)
    kv_len = ints([0] * batch)
    q1, k1, v1 = r(batch, hq, d), r(batch, hkv, d), r(batch, hkv, d)
    grown_k, grown_v = [], []

    def step():
        kv_len.add_(1)
        oss.kv_cache_append(k1, v1, kp, vp, table, kv_len)
        return oss.attention_decode_shared(q1, kp, vp, prefix_table, prefix_len, table, kv_len)

    graph = None
    for i in range(steps):
        for x in (q1, k1, v1):
            x.copy_(r(*x.shape))
        grown_k.append(f64(k1))
        grown_v.append(f64(v1))
        if i < 2:
            o, lse = step()
        elif graph is None:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                o, lse = step()
            graph.replay()
        else:
            graph.replay()
        assert oss.check_device_error() == 0

        def rows(first, grown):
            def get(b, g):
                return np.concatenate([f64(first[:, g]), np.stack([x[b, g] for x in grown])])
            get.heads = hkv
            return get
        check_shared(o, lse, q1, rows(k, grown_k), rows(v, grown_v), 1 / math.sqrt(d))


def test_two_graphs_with_other_lengths_side_by_side():
    cases = [Case([4, 3], [3000, 500], [700, 0, 3, 90, 40, 1, 2], 8, 2, page=32, seed=s) for s in (14, 15)]
    for c in cases:
        c.run()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(c.run())
        graphs.append(graph)
    other = torch.cuda.Stream()
    for prefixes, own in (([3000, 500], [700, 0, 3, 90, 40, 1, 2]), ([1, 499], [0, 0, 1, 64, 2, 1, 1]), ([0, 0], [0] * 7)):
        for c in cases:
            c.prefixes, c.own = prefixes, own
            c.prefix_len.copy_(ints(prefixes))
            c.kv_len.copy_(ints(own))
        torch.cuda.synchronize()
        for _ in range(3):
            graphs[0].replay()
            with torch.cuda.stream(other):
                graphs[1].replay()
        torch.cuda.synchronize()
        for c, out in zip(cases, outs):
            c.check(*out)
    assert oss.check_device_error() == 0


def test_a_wait_that_gives_up_is_reported(wide):
    # a V tile that never arrives: the launch ends, and the next one works
    c = Case([24], [1000], [20] * 24, 16, 8, seed=17, prefix_columns=64)
    oss.debug_inject_fault(1, 0, 20_000_000)
    c.run()
    with pytest.raises(oss.OssError, match="OS_ERR_TIMEOUT"):
        oss.check_device_error()
    assert oss.check_device_error() == 0
    c.go(rows=[0, 23])


@pytest.mark.slow
def test_offsets_beyond_32_bits():
    # pools of more than 2^32 bytes and 2^31 elements each: the last pages are used
    page, heads, d = 64, 8, 128
    pages = (2 ** 31 + 2 ** 26) // (page * heads * d)
    kp = torch.empty((pages, heads, page, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    prefix_table = torch.full((1, 400 if WIDE else 3), -1, dtype=torch.int32, device="cuda")
    prefix_table[0, :3] = ints([pages - 1, 0, pages - 2])
    table = ints([[pages - 3], [pages - 4], [1]])
    k, v = (torch.randn((150 + 3 * 20, heads, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    own = ints([20, 20, 20])
    oss.kv_cache_append(k[:150], v[:150], kp, vp, prefix_table, ints([150]), ints([0, 150]))
    oss.kv_cache_append(k[150:], v[150:], kp, vp, table, own, ints([0, 20, 40, 60]))
    q = torch.randn((3, 16, d), device="cuda").to(torch.bfloat16)
    o, lse = oss.attention_decode_shared(q, kp, vp, prefix_table, ints([150]), table, own)
    assert oss.check_device_error() == 0

    def rows(x):
        def get(b, g):
            return f64(torch.cat([x[:150, g], x[150 + 20 * b:170 + 20 * b, g]]))
        get.heads = heads
        return get
    check_shared(o, lse, q, rows(k), rows(v), 1 / math.sqrt(d))
