"""kv_cache_append, attention_decode_paged and kv_cache_evict against their
definitions in 64 bits (GPU)."""

import math

import numpy as np
import pytest
import torch

import pass_attention_gb300 as oss
from paged_reference import DTYPES, check_decode, evict, f64, gather

pytestmark = pytest.mark.gpu


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def pools(gen, pages, heads, page, d, dtype, layout="head"):
    """K and V pools [pages, heads, page, d]: dense, as views of [page, slot,
    head, d], or K and V pages side by side in one pool."""
    r = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float32).to(dtype)  # noqa: E731
    if layout == "slot":
        return r(pages, page, heads, d).transpose(1, 2), r(pages, page, heads, d).transpose(1, 2)
    if layout == "joint":
        both = r(pages, 2, heads, page, d)
        return both[:, 0], both[:, 1]
    return r(pages, heads, page, d), r(pages, heads, page, d)


def make(lens, hq, hkv, d=128, page=16, dtype="bf16", layout="head", seed=0, spare=3, columns=None):
    """A cache with the sequences' pages in random order, NaN in every slot
    that no token has, and -1 behind each sequence's last page."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    kp, vp = pools(gen, pages, hkv, page, d, DTYPES[dtype], layout)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), columns or max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    free = torch.ones((pages, page), dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        t = torch.arange(n, device="cuda")
        free[table[b, t // page].long(), t % page] = False
    for x in (kp, vp):
        x.transpose(1, 2)[free] = float("nan")
    q = torch.randn((len(lens), hq, d), generator=gen, device="cuda").to(DTYPES[dtype])
    return q, kp, vp, table, ints(lens), order[at:]


def decode(lens, hq, hkv, weights=False, **kw):
    q, kp, vp, table, kv_len, _ = make(lens, hq, hkv, **kw)
    w = before = None
    if weights:
        w = torch.rand((len(lens), hkv, table.shape[1] * kp.shape[2] + 5), device="cuda")
        before = w.clone()
    scale = 1.0 / math.sqrt(q.shape[-1])
    o, lse = oss.attention_decode_paged(q, kp, vp, table, kv_len, weights=w)
    assert oss.check_device_error() == 0
    check_decode(o, lse, q, kp, vp, table, kv_len, scale, w, before)


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 200, 333]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("weights", [False, True])
def test_decode_types_and_lengths(d, dtype, weights):
    decode(LENS, 8, 2, weights=weights, d=d, dtype=dtype, seed=d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 4), (10, 2), (7, 1), (8, 1), (9, 1), (24, 2),
                                    (16, 1), (17, 1), (33, 1), (64, 1), (35, 5)])
def test_decode_groups(hq, hkv):
    decode([70, 5, 0, 257], hq, hkv, weights=True, page=32, seed=hq)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("layout", ["head", "slot", "joint"])
def test_decode_pages_and_layouts(page, layout):
    decode([1, page - 1, page, page + 1, 2 * page + 7], 8, 2, page=page, layout=layout, seed=page)


@pytest.mark.parametrize("lens,hq,hkv", [
    ([40001], 8, 1),                        # one sequence, one key head, over the whole GPU
    ([1, 20000, 3, 0, 777, 20001], 8, 2),   # long and short ones side by side
    ([130] * 300, 4, 2),                    # many sequences
    ([1, 17, 0, 40] * 600, 2, 1),
])
def test_decode_long_and_many(lens, hq, hkv):
    decode(lens, hq, hkv, weights=True, page=64, seed=len(lens))


def test_decode_one_heavy_key():
    # one key takes nearly all the weight, in the first, a middle or the last tile
    q, kp, vp, table, kv_len, _ = make([900, 900, 900], 4, 1, page=32, seed=5)
    for b, t in enumerate((3, 450, 899)):
        kp[table[b, t // 32].long(), 0, t % 32] = q[b, 1] * 8
    o, lse = oss.attention_decode_paged(q, kp, vp, table, kv_len)
    check_decode(o, lse, q, kp, vp, table, kv_len, 1 / math.sqrt(128))


def test_decode_strided_query_and_given_outputs():
    q, kp, vp, table, kv_len, _ = make([50, 300], 4, 2, seed=6)
    wide = torch.zeros((2, 12, 128), dtype=q.dtype, device="cuda")
    wide[:, 4:8] = q
    o = torch.full_like(q, 7.0)
    lse = torch.full((2, 4), 7.0, device="cuda")
    out = oss.attention_decode_paged(wide[:, 4:8], kp, vp, table, kv_len, scale=0.3, o=o, lse=lse)
    assert out[0] is o and out[1] is lse
    check_decode(o, lse, q, kp, vp, table, kv_len, 0.3)


def test_decode_shared_prefix_pages():
    # two sequences read the same first pages
    q, kp, vp, table, kv_len, _ = make([100, 90, 64], 8, 2, seed=7)
    table[1, :4] = table[0, :4]
    w = torch.zeros((3, 2, table.shape[1] * 16), device="cuda")
    o, lse = oss.attention_decode_paged(q, kp, vp, table, kv_len, weights=w)
    check_decode(o, lse, q, kp, vp, table, kv_len, 1 / math.sqrt(128), w, torch.zeros_like(w))


def test_decode_leaves_out_bad_pages():
    # a page number outside the pool: those keys are masked, and it is reported
    q, kp, vp, table, kv_len, _ = make([64, 64], 4, 1, seed=8)
    for bad in (-1, kp.shape[0], 2 ** 31 - 1):
        broken = table.clone()
        broken[0, 1] = bad
        o, lse = oss.attention_decode_paged(q, kp, vp, broken, kv_len)
        with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
            oss.check_device_error()
        assert oss.check_device_error() == 0
        good = torch.cat([table[0, :1], table[0, 2:]])[None]
        check_decode(o[:1], lse[:1], q[:1], kp, vp, good, kv_len[:1] - 16, 1 / math.sqrt(128))
        check_decode(o[1:], lse[1:], q[1:], kp, vp, table[1:], kv_len[1:], 1 / math.sqrt(128))


def test_decode_every_page_bad():
    q, kp, vp, table, kv_len, _ = make([40], 4, 1, seed=8)
    w = torch.ones((1, 1, table.shape[1] * 16), device="cuda")
    o, lse = oss.attention_decode_paged(q, kp, vp, torch.full_like(table, -5), kv_len, weights=w)
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse)) and torch.all(w == 1)


def test_decode_clamps_lengths():
    # lengths beyond the page table's rows and below zero
    q, kp, vp, table, kv_len, _ = make([64, 30], 4, 1, seed=9)
    o, lse = oss.attention_decode_paged(q, kp, vp, table, ints([65, -3]))
    check_decode(o, lse, q, kp, vp, table, ints([64, 0]), 1 / math.sqrt(128))


def test_decode_same_bits_every_time_and_beside_other_calls():
    q, kp, vp, table, kv_len, _ = make([5000, 31, 900], 8, 2, page=64, seed=10)
    ref = oss.attention_decode_paged(q, kp, vp, table, kv_len)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [oss.attention_decode_paged(q, kp, vp, table, kv_len, stream=s) for s in streams for _ in range(5)]
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_outputs_on_another_stream_take_no_memory_in_use():
    # a block freed while the current stream still has to read it: an output
    # allocated for another stream must not be put there
    q, kp, vp, table, kv_len, _ = make([2000] * 4, 8, 2, page=64, seed=13)
    ref, _ = oss.attention_decode_paged(q, kp, vp, table, kv_len)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        x = [torch.full_like(q, 3.0) for _ in range(8)]
        torch.cuda._sleep(20_000_000)
        y = [t + 0 for t in x]
        del x
        o, _ = oss.attention_decode_paged(q, kp, vp, table, kv_len, stream=side)
        side.synchronize()
        assert torch.equal(o.clone(), ref)
        torch.cuda.synchronize()
        assert all(torch.all(t == 3.0) for t in y)


def test_decode_in_two_graphs_with_new_lengths():
    # captured once, replayed side by side with other lengths in the same tensors
    q, kp, vp, table, kv_len, _ = make([3000, 700], 8, 2, page=32, seed=11)
    other = make([1500, 2999], 8, 2, page=32, seed=12, columns=table.shape[1])
    oss.attention_decode_paged(q, kp, vp, table, kv_len)
    torch.cuda.synchronize()
    graphs, outs, lens = [], [], []
    for args in ((q, kp, vp, table), other[:4]):
        n = torch.ones(2, dtype=torch.int32, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(oss.attention_decode_paged(*args, n))
        graphs.append(graph)
        lens.append(n)
    for real in ([3000, 700], [17, 0], [2999, 64]):
        lens[0].copy_(ints(real))
        lens[1].copy_(ints([min(real[1], 1500), min(real[0], 2999)]))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for _ in range(3):
            graphs[0].replay()
            with torch.cuda.stream(side):
                graphs[1].replay()
        torch.cuda.synchronize()
        check_decode(*outs[0], q, kp, vp, table, lens[0], 1 / math.sqrt(128))
        check_decode(*outs[1], *other[:4], lens[1], 1 / math.sqrt(128))


@pytest.mark.slow
def test_offsets_beyond_32_bits():
    # pools of more than 2^32 bytes and 2^31 elements each: the last pages are used
    page, heads, d = 64, 8, 128
    pages = (2 ** 31 + 2 ** 26) // (page * heads * d)
    kp = torch.empty((pages, heads, page, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    table = ints([[pages - 1, pages - 2, 0], [pages - 3, 1, 2]])
    new = torch.randn((2, 300, heads, d), device="cuda").to(torch.bfloat16)
    k, v = new[0], new[1]
    kv_len, cu = ints([130, 170]), ints([0, 130, 300])
    oss.kv_cache_append(k, v, kp, vp, table, kv_len, cu)
    q = torch.randn((2, 16, d), device="cuda").to(torch.bfloat16)
    o, lse = oss.attention_decode_paged(q, kp, vp, table, kv_len)
    assert oss.check_device_error() == 0
    for g in range(heads):
        assert np.array_equal(gather(kp, table[0], 130, g), f64(k[:130, g]))
        assert np.array_equal(gather(vp, table[1], 170, g), f64(v[130:, g]))
    check_decode(o, lse, q, kp, vp, table, kv_len, 1 / math.sqrt(d))
    w = torch.rand((2, heads, 3 * page), device="cuda")
    kept, _, _ = oss.kv_cache_evict(kp, vp, w, table, kv_len, ints([[pages - 9], [pages - 10]]), 64, 8)
    for g in range(heads):
        want = gather(kp, table[1], 170, g)[kept[1, g].cpu().numpy()]
        assert np.array_equal(gather(kp, ints([pages - 10]), 64, g), want)


# -- append ----------------------------------------------------------------------------------

@pytest.mark.parametrize("d,dtype,page,layout", [(128, "bf16", 16, "head"), (64, "f16", 64, "slot"),
                                                 (128, "f16", 32, "joint"), (64, "bf16", 1024, "head")])
@pytest.mark.parametrize("before,new", [([0, 5, 16, 100, 31], [33, 0, 1, 64, 1]), ([0], [1]), ([15], [2]),
                                        ([7, 0], [0, 0])])
def test_append_writes_the_new_rows_only(d, dtype, page, layout, before, new):
    heads = 3
    lens = [a + b for a, b in zip(before, new)]
    _, kp, vp, table, kv_len, _ = make(lens, heads, heads, d=d, page=page, dtype=dtype, layout=layout, seed=d + page)
    total = sum(new)
    # k and v are slices of one projection, with rows behind the last sequence
    qkv = torch.randn((total + 2, 5 * heads, d), device="cuda").to(kp.dtype)
    k, v = qkv[:, heads:2 * heads], qkv[:, 3 * heads:4 * heads]
    cu = ints(np.concatenate([[0], np.cumsum(new)]).tolist())
    want = []
    for pool, x in ((kp, k), (vp, v)):
        ref = pool.clone()
        for b in range(len(lens)):
            for i in range(new[b]):
                t = before[b] + i
                ref[table[b, t // page].long(), :, t % page] = x[int(cu[b]) + i]
        want.append(ref)
    oss.kv_cache_append(k, v, kp, vp, table, kv_len, cu)
    assert oss.check_device_error() == 0
    for pool, ref in ((kp, want[0]), (vp, want[1])):
        assert torch.equal(pool.contiguous().view(torch.int16), ref.contiguous().view(torch.int16))


def test_append_one_token_each():
    lens = [1, 17, 16, 40]
    _, kp, vp, table, kv_len, _ = make(lens, 2, 2, seed=21)
    k, v = (torch.randn((4, 2, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    wk, wv = kp.clone(), vp.clone()
    for b, n in enumerate(lens):
        at = table[b, (n - 1) // 16].long()
        wk[at, :, (n - 1) % 16], wv[at, :, (n - 1) % 16] = k[b], v[b]
    oss.kv_cache_append(k, v, kp, vp, table, kv_len)
    assert torch.equal(kp.view(torch.int16), wk.view(torch.int16))
    assert torch.equal(vp.view(torch.int16), wv.view(torch.int16))


@pytest.mark.parametrize("cu", [False, True])
def test_append_and_decode_of_a_padded_batch(cu):
    # places of the batch without a sequence: kv_len 0, no page, a row that is
    # not read; with offsets, a new token that has no position is reported
    lens = [0, 17, 0, 40]
    q, kp, vp, table, kv_len, _ = make(lens, 4, 2, seed=24)
    k, v = (torch.randn((4, 2, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    wk, wv = kp.clone(), vp.clone()
    for b, n in ((1, 17), (3, 40)):
        at = table[b, (n - 1) // 16].long()
        wk[at, :, (n - 1) % 16], wv[at, :, (n - 1) % 16] = k[b], v[b]
    oss.kv_cache_append(k, v, kp, vp, table, kv_len, ints([0, 1, 2, 3, 4]) if cu else None)
    if cu:
        with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
            oss.check_device_error()
    assert oss.check_device_error() == 0
    assert torch.equal(kp.view(torch.int16), wk.view(torch.int16))
    assert torch.equal(vp.view(torch.int16), wv.view(torch.int16))
    o, lse = oss.attention_decode_paged(q, kp, vp, table, kv_len)
    assert oss.check_device_error() == 0
    check_decode(o, lse, q, kp, vp, table, kv_len, 1.0 / math.sqrt(128))


def test_append_many_tokens():
    lens = [4000, 1, 2500]
    _, kp, vp, table, kv_len, _ = make(lens, 8, 8, page=64, seed=22)
    k, v = (torch.randn((sum(lens), 8, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    oss.kv_cache_append(k, v, kp, vp, table, kv_len, ints([0, 4000, 4001, 6501]))
    at = 0
    for b, n in enumerate(lens):
        for g in (0, 7):
            assert np.array_equal(gather(kp, table[b], n, g), f64(k[at:at + n, g]))
            assert np.array_equal(gather(vp, table[b], n, g), f64(v[at:at + n, g]))
        at += n


@pytest.mark.parametrize("kv_len,entry", [([16, 40], -1), ([16, 40], 99999), ([-1, 40], None), ([16, 65], None)])
def test_append_leaves_out_what_has_no_place(kv_len, entry):
    # a bad page, a position before the first, one behind the last page: the
    # other sequence's row is written, nothing else is, and it is reported
    _, kp, vp, table, _, _ = make([16, 64], 2, 2, seed=23)
    k, v = (torch.randn((2, 2, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    good = 0 if kv_len[1] == 65 else 1
    if entry is not None:
        table[0, 0] = entry
    wk, wv = kp.clone(), vp.clone()
    n = kv_len[good] - 1
    at = table[good, n // 16].long()
    wk[at, :, n % 16], wv[at, :, n % 16] = k[good], v[good]
    oss.kv_cache_append(k, v, kp, vp, table, ints(kv_len))
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()
    assert torch.equal(kp.view(torch.int16), wk.view(torch.int16))
    assert torch.equal(vp.view(torch.int16), wv.view(torch.int16))


# -- evict -----------------------------------------------------------------------------------

def run_evict(lens, heads, budget, recent, make_weights, d=128, page=16, dtype="bf16", layout="head", seed=0,
              extra=0, wide=0):
    _, kp, vp, table, kv_len, _ = make(lens, heads, heads, d=d, page=page, dtype=dtype, layout=layout, seed=seed,
                                       spare=len(lens) * (-(-budget // page) + extra) + 1)
    used = set(table.flatten().tolist())
    free = [x for x in range(kp.shape[0]) if x not in used]
    columns = -(-budget // page) + extra
    new_table = ints(np.array(free[:len(lens) * columns]).reshape(len(lens), columns).tolist())
    cap = table.shape[1] * page
    w = make_weights((len(lens), heads, cap + wide))
    before = kp.clone(), vp.clone()
    kept, new_len, new_w = oss.kv_cache_evict(kp, vp, w, table, kv_len, new_table, budget, recent)
    assert oss.check_device_error() == 0
    wk, wv = before
    wh = w.cpu().numpy()
    for b, n in enumerate(lens):
        keep = min(n, budget)
        assert int(new_len[b]) == keep
        for g in range(heads):
            ref = evict(wh[b, g], n, budget, recent)
            got = kept[b, g].cpu().numpy()
            assert np.array_equal(got[:keep], ref), f"sequence {b} head {g}"
            assert np.all(got[keep:] == -1)
            nw = new_w[b, g].cpu().numpy()
            assert np.array_equal(nw[:keep], wh[b, g][ref], equal_nan=True) and np.all(nw[keep:] == 0)
            t, r = torch.arange(keep), torch.tensor(ref)
            src, dst = table[b].cpu().long()[r // page], new_table[b].cpu().long()[t // page]
            wk[dst.cuda(), g, (t % page).cuda()] = wk[src.cuda(), g, (r % page).cuda()]
            wv[dst.cuda(), g, (t % page).cuda()] = wv[src.cuda(), g, (r % page).cuda()]
    assert torch.equal(kp.contiguous().view(torch.int16), wk.contiguous().view(torch.int16))
    assert torch.equal(vp.contiguous().view(torch.int16), wv.contiguous().view(torch.int16))


def spread(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return lambda shape: torch.randn(shape, generator=gen, device="cuda").mul_(2).exp_()


@pytest.mark.parametrize("d,dtype,page,layout", [(128, "bf16", 16, "head"), (64, "f16", 64, "slot"), (128, "f16", 32, "joint")])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (40, 0), (40, 40), (100, 7), (300, 16)])
def test_evict_budgets(d, dtype, page, layout, budget, recent):
    run_evict([0, 1, 39, 40, 41, 100, 257], 2, budget, recent, spread(budget), d=d, dtype=dtype, page=page,
              layout=layout, seed=budget, extra=2, wide=3)


@pytest.mark.parametrize("n,budget,recent", [(1025, 1000, 3), (4096, 1024, 0), (9001, 2000, 200), (50000, 300, 100),
                                             (70001, 69000, 5), (131072, 16384, 1000), (200003, 1, 0)])
def test_evict_long(n, budget, recent):
    run_evict([n, n // 3], 2, budget, recent, spread(n), page=64, d=64, seed=n)


@pytest.mark.parametrize("n,budget", [(70, 20), (5000, 1200), (40000, 30000)])
def test_evict_ties_go_to_the_lowest_position(n, budget):
    # few distinct weights, all equal, and all zero
    run_evict([n], 1, budget, 5, lambda s: torch.randint(0, 3, s, device="cuda").float(), page=64, seed=1)
    run_evict([n], 1, budget, 0, lambda s: torch.full(s, 0.25, device="cuda"), page=64, seed=2)
    run_evict([n], 1, budget, 0, lambda s: torch.zeros(s, device="cuda"), page=64, seed=3)


def test_evict_order_of_special_weights():
    def special(shape):
        w = torch.randn(shape, device="cuda")
        pick = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 1e-45, -1e-45, 3.4e38], device="cuda")
        return torch.where(torch.rand(shape, device="cuda") < 0.6, pick[torch.randint(0, 8, shape, device="cuda")], w)
    for budget in (1, 10, 60, 200, 299):
        run_evict([300], 3, budget, 0, special, seed=budget)


def test_evict_from_shared_pages():
    # both sequences name the same pages; each keeps its own choice of them
    _, kp, vp, table, kv_len, free = make([96, 96], 2, 2, seed=31, spare=8)
    table[1] = table[0]
    w = torch.rand((2, 2, 96), device="cuda")
    new_table = free[:4].reshape(2, 2)
    kept, _, _ = oss.kv_cache_evict(kp, vp, w, table, kv_len, new_table, 32, 4)
    for b in range(2):
        for g in range(2):
            ref = evict(w[b, g].cpu().numpy(), 96, 32, 4)
            assert np.array_equal(kept[b, g].cpu().numpy(), ref)
            assert np.array_equal(gather(kp, new_table[b], 32, g), gather(kp, table[b], 96, g)[ref])


def test_evict_leaves_out_bad_pages():
    _, kp, vp, table, kv_len, free = make([40, 40], 1, 1, seed=32, spare=4)
    before = kp.clone()
    new_table = torch.stack([torch.full_like(free[:1], kp.shape[0]), free[:1]])
    w = torch.rand((2, 1, 48), device="cuda")
    kept, _, _ = oss.kv_cache_evict(kp, vp, w, table, kv_len, new_table, 16, 0)
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()
    at = free[0].long()
    rest = torch.arange(kp.shape[0], device="cuda") != at
    assert torch.equal(kp[rest].view(torch.int16), before[rest].view(torch.int16))
    assert np.array_equal(gather(kp, new_table[1], 16, 0), gather(before, table[1], 40, 0)[kept[1, 0].cpu().numpy()])


# -- refusals --------------------------------------------------------------------------------

def test_refusals():
    q, kp, vp, table, kv_len, free = make([20, 20], 4, 2, seed=41, spare=6)
    k = torch.zeros((2, 2, 128), dtype=kp.dtype, device="cuda")
    w = torch.zeros((2, 2, 32), device="cuda")
    dec = lambda **c: oss.attention_decode_paged(**{**dict(q=q, k_pages=kp, v_pages=vp, page_table=table, kv_len=kv_len), **c})  # noqa: E731
    app = lambda **c: oss.kv_cache_append(**{**dict(k=k, v=k, k_pages=kp, v_pages=vp, page_table=table, kv_len=kv_len), **c})  # noqa: E731
    evi = lambda **c: oss.kv_cache_evict(**{**dict(k_pages=kp, v_pages=vp, weights=w, page_table=table, kv_len=kv_len, new_page_table=free[:2].reshape(2, 1), budget=8), **c})  # noqa: E731
    for call in (dec, app, evi):
        with pytest.raises(TypeError):
            call(k_pages=kp.float(), v_pages=vp.float())
        with pytest.raises(TypeError):
            call(v_pages=vp.half())
        with pytest.raises(TypeError):
            call(page_table=table.long())
        with pytest.raises(ValueError):
            call(v_pages=vp[:, :, :, :64])
        with pytest.raises(ValueError):
            call(kv_len=kv_len[:1])
        with pytest.raises(ValueError):
            call(kv_len=kv_len.cpu())
        with pytest.raises(ValueError):
            call(k_pages=kp[..., ::2], v_pages=vp[..., ::2])
        with pytest.raises((oss.OssError, ValueError), match="UNSUPPORTED|weights|like the cache"):
            call(k_pages=kp[:, :, :8], v_pages=vp[:, :, :8])
        with pytest.raises((oss.OssError, ValueError), match="UNSUPPORTED|like the cache"):
            call(k_pages=kp[..., :32], v_pages=vp[..., :32])
    for bad in (dict(q=q[:1]), dict(q=q[..., :64]), dict(q=q[:, :3]), dict(weights=w[..., :31]), dict(weights=w[:, :1]),
                dict(o=q[:, :2]), dict(lse=w)):
        with pytest.raises(ValueError):
            dec(**bad)
    for bad in (dict(weights=w.half()), dict(q=q.half())):
        with pytest.raises(TypeError):
            dec(**bad)
    with pytest.raises(oss.OssError, match="INVALID"):
        dec(scale=0.0)
    with pytest.raises(oss.OssError, match="INVALID"):
        dec(weights=w[:, :1].expand(2, 2, 32))  # the heads' sums in one place
    with pytest.raises(oss.OssError, match="MISALIGNED"):
        dec(q=torch.zeros(2, 4, 132, dtype=q.dtype, device="cuda")[..., :128])
    for bad in (dict(k=k[:, :1], v=k[:, :1]), dict(v=k[:1]), dict(cu_seqlens=kv_len), dict(k=k[..., :64], v=k[..., :64])):
        with pytest.raises(ValueError):
            app(**bad)
    with pytest.raises(oss.OssError, match="INVALID"):
        app(k=k[:1], v=k[:1])  # one token for two sequences without offsets
    for bad in (dict(budget=0), dict(budget=17), dict(recent=9), dict(recent=-1), dict(new_page_table=free[:1].reshape(1, 1)),
                dict(weights=w[..., :31]), dict(kept=w), dict(new_weights=w)):
        with pytest.raises((ValueError, TypeError)):
            evi(**bad)
    for bad in (dict(new_page_table=table), dict(new_len=kv_len),
                dict(new_page_table=free[:4].reshape(2, 2), new_weights=w)):
        with pytest.raises(oss.OssError, match="INVALID"):
            evi(**bad)
    assert oss.check_device_error() == 0
