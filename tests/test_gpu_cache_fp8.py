"""kv_cache_append_fp8, kv_cache_read_fp8 and attention_decode_paged_fp8 against their
definitions in 64 bits (GPU)."""

import math
import random
import threading

import numpy as np
import pytest
import torch

import pass_attention_gb300 as oss
from fp8_reference import check_decode_fp8, codes, gather8, quantise, scales
from paged_reference import DTYPES, check_packed, f64

pytestmark = pytest.mark.gpu
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def pools(pages, heads, page, d, layout, byte=0x7f, scale=255):
    """Pools and scales with every byte set (NaN by default): dense, as views of [page,
    slot, head, d], or K and V side by side in one pool."""
    full = lambda *s: torch.full(s, byte, dtype=torch.uint8, device="cuda")  # noqa: E731
    sc = torch.full((2, pages, heads, page), scale, dtype=torch.uint8, device="cuda")
    if layout == "slot":
        kp, vp = full(pages, page, heads, d).transpose(1, 2), full(pages, page, heads, d).transpose(1, 2)
    elif layout == "joint":
        both, sc = full(pages, 2, heads, page, d), sc.transpose(0, 1).contiguous().transpose(0, 1)
        kp, vp = both[:, 0], both[:, 1]
    else:
        kp, vp = full(pages, heads, page, d), full(pages, heads, page, d)
    return kp.view(F8), vp.view(F8), sc[0].view(E8), sc[1].view(E8)


def tables(lens, page, gen, spare=3, columns=None):
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), columns or max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def rows(gen, shape, dtype):
    """Rows of very different sizes, some of zeros."""
    x = torch.randn(shape, generator=gen, device="cuda")
    size = torch.randn(shape[:-1] + (1,), generator=gen, device="cuda").mul_(1.5).exp2_()
    zero = torch.rand(shape[:-1] + (1,), generator=gen, device="cuda") < 0.02
    return (x * size).masked_fill_(zero, 0.0).to(dtype)


def fill(pages_, scales_, table, lens, x):
    """Rows x [tokens, heads, D] into the pages, quantised by the definition."""
    c, s = quantise(x)
    c = torch.from_numpy(c).to("cuda").float().to(F8).view(torch.uint8)
    s = torch.from_numpy(np.log2(s) + 127).to("cuda").to(torch.uint8)
    at, page = 0, pages_.shape[2]
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        where = table[b, t // page].long()
        pages_.view(torch.uint8)[where, :, t % page] = c[at:at + n]
        scales_.view(torch.uint8)[where, :, t % page] = s[at:at + n]
        at += n


def make(lens, hq, hkv, d=128, page=16, dtype="bf16", layout="head", seed=0, columns=None):
    """A cache with NaN in every slot and scale that no token has."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    table, pages = tables(lens, page, gen, columns=columns)
    kp, vp, ks, vs = pools(pages, hkv, page, d, layout)
    k, v = (rows(gen, (sum(lens), hkv, d), DTYPES[dtype]) for _ in range(2))
    k = k / k.float().abs().amax(-1, keepdim=True).clamp(min=1).to(k.dtype)
    fill(kp, ks, table, lens, k)
    fill(vp, vs, table, lens, v)
    q = torch.randn((len(lens), hq, d), generator=gen, device="cuda").mul_(3).to(DTYPES[dtype])
    return q, (kp, vp, ks, vs, table, ints(lens))


def decode(lens, hq, hkv, **kw):
    q, cache = make(lens, hq, hkv, **kw)
    o, lse = oss.attention_decode_paged_fp8(q, *cache)
    assert oss.check_device_error() == 0
    check_decode_fp8(o, lse, q, *cache, 1.0 / math.sqrt(q.shape[-1]))


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 200, 333]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_decode_types_and_lengths(d, dtype):
    decode(LENS, 8, 2, d=d, dtype=dtype, seed=d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 4), (10, 2), (7, 1), (8, 1), (9, 1), (24, 2),
                                    (16, 1), (17, 1), (33, 1), (64, 1), (35, 5)])
@pytest.mark.parametrize("columns", [None, 40])  # whole items, and items that may be cut
def test_decode_groups(hq, hkv, columns):
    decode([70, 5, 0, 257], hq, hkv, page=32, seed=hq, columns=columns)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("layout", ["head", "slot", "joint"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_pages_and_layouts(page, layout, d):
    decode([1, page - 1, page, page + 1, 2 * page + 7], 8, 2, page=page, layout=layout, d=d, seed=page)


@pytest.mark.parametrize("lens,hq,hkv,d,dtype", [
    ([40001], 8, 1, 128, "bf16"),                       # one sequence, one key head, over the whole GPU
    ([20000], 16, 1, 64, "f16"),
    ([1, 20000, 3, 0, 777, 20001], 8, 2, 128, "bf16"),  # long and short ones side by side
    ([130] * 300, 4, 2, 64, "bf16"),                    # many sequences
    ([1, 17, 0, 40] * 400, 2, 1, 128, "f16"),
])
def test_decode_long_and_many(lens, hq, hkv, d, dtype):
    decode(lens, hq, hkv, page=64, d=d, dtype=dtype, seed=len(lens))


@pytest.mark.parametrize("seed", range(24))
def test_decode_random_batches(seed):
    r = random.Random(seed)
    lens = [r.choice((0, 1, 16, r.randint(1, 300), r.randint(1, 3000))) for _ in range(r.choice((1, 2, 5, 12)))]
    hkv = r.choice((1, 1, 2, 3, 5))
    hq = hkv * r.choice((1, 2, 3, 4, 6, 8, 9, 16, 17, 40))
    decode(lens, hq, hkv, d=r.choice((64, 128)), dtype=r.choice(("bf16", "f16")), page=r.choice((16, 32, 128, 256)),
           layout=r.choice(("head", "slot", "joint")), columns=r.choice((None, 250)), seed=seed)


def test_decode_one_heavy_key():
    # one key takes nearly all the weight, in the first, a middle or the last tile, and
    # its value row is far smaller than the others
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    lens, page = [900, 900, 900], 32
    table, pages = tables(lens, page, gen)
    kp, vp, ks, vs = pools(pages, 1, page, 128, "head")
    q = torch.randn((3, 4, 128), generator=gen, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn((2700, 1, 128), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    for b, t in enumerate((3, 450, 899)):
        k[900 * b + t, 0] = q[b, 1] * 8
        v[900 * b + t] *= 2.0 ** -12
    fill(kp, ks, table, lens, k)
    fill(vp, vs, table, lens, v)
    cache = (kp, vp, ks, vs, table, ints(lens))
    o, lse = oss.attention_decode_paged_fp8(q, *cache)
    check_decode_fp8(o, lse, q, *cache, 1 / math.sqrt(128))


@pytest.mark.parametrize("power", [-118, -60, 60, 100])
def test_decode_values_of_extreme_sizes(power):
    # bf16 reaches from 2^-126 to 2^127: value rows of such sizes, and a key and a
    # query whose product is ordinary
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    lens, page = [700, 33], 16
    table, pages = tables(lens, page, gen)
    kp, vp, ks, vs = pools(pages, 2, page, 64, "head")
    k = (torch.randn((733, 2, 64), generator=gen, device="cuda") * 2.0 ** (power // 2)).to(torch.bfloat16)
    v = (torch.randn((733, 2, 64), generator=gen, device="cuda") * 2.0 ** power).to(torch.bfloat16)
    q = (torch.randn((2, 8, 64), generator=gen, device="cuda") * 2.0 ** -(power // 2)).to(torch.bfloat16)
    fill(kp, ks, table, lens, k)
    fill(vp, vs, table, lens, v)
    cache = (kp, vp, ks, vs, table, ints(lens))
    o, lse = oss.attention_decode_paged_fp8(q, *cache)
    check_decode_fp8(o, lse, q, *cache, 1 / math.sqrt(64))


def test_decode_a_query_with_one_large_element():
    # a bf16 q is held in fp16 relative to its largest element
    q, cache = make([300, 40], 4, 2, seed=7)
    q[:, :, 5] *= 2.0 ** 30
    cache[0].view(torch.uint8)[:, :, :, 5] = 0  # which meets zeros: the small ones decide
    o, lse = oss.attention_decode_paged_fp8(q, *cache)
    check_decode_fp8(o, lse, q, *cache, 1 / math.sqrt(128))


def test_decode_strided_query_and_given_outputs():
    q, cache = make([50, 300], 4, 2, seed=6)
    wide = torch.zeros((2, 12, 128), dtype=q.dtype, device="cuda")
    wide[:, 4:8] = q
    o = torch.full_like(q, 7.0)
    lse = torch.full((2, 4), 7.0, device="cuda")
    out = oss.attention_decode_paged_fp8(wide[:, 4:8], *cache, scale=0.3, o=o, lse=lse)
    assert out[0] is o and out[1] is lse
    check_decode_fp8(o, lse, q, *cache, 0.3)


@pytest.mark.parametrize("lens,columns", [([70, 200, 0, 16], None), ([3000, 100, 0, 1500], 128)])
@pytest.mark.parametrize("hq", [4, 12, 20])
def test_decode_nan(lens, columns, hq):
    # a NaN query, key row or value row: NaN where it reaches, answers elsewhere
    q, cache = make(lens, hq, 1, page=32, columns=columns, seed=hq)
    kp, vp, ks, vs, table, kv_len = cache
    bad = q.clone()
    bad[0, 1, 3] = float("nan")
    bad[2] = float("nan")               # a sequence without keys
    o, lse = oss.attention_decode_paged_fp8(bad, *cache)
    assert torch.isnan(o[0, 1]).all() and torch.isnan(lse[0, 1])
    assert torch.all(o[2] == 0) and torch.isneginf(lse[2]).all()
    good, good_lse = oss.attention_decode_paged_fp8(q, *cache)
    o[0, 1], lse[0, 1] = good[0, 1], good_lse[0, 1]
    check_decode_fp8(o, lse, q, *cache, 1 / math.sqrt(128))
    t = lens[1] - 3
    ks.view(torch.uint8)[table[1, t // 32].long(), 0, t % 32] = 255
    o, lse = oss.attention_decode_paged_fp8(q, *cache)
    assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
    assert torch.equal(o[[0, 2, 3]], good[[0, 2, 3]]) and torch.equal(lse[[0, 2, 3]], good_lse[[0, 2, 3]])
    vs.view(torch.uint8)[table[3, 0].long(), 0, 2] = 255
    o, lse = oss.attention_decode_paged_fp8(q, *cache)
    assert torch.isnan(o[3]).all() and torch.equal(lse[3], good_lse[3])
    assert torch.equal(o[0], good[0])
    assert oss.check_device_error() == 0


def test_decode_infinite_query():
    q, cache = make([70, 30], 4, 2, seed=9)
    bad = q.clone()
    bad[0, 0, 0] = float("inf")
    o, lse = oss.attention_decode_paged_fp8(bad, *cache)
    good, good_lse = oss.attention_decode_paged_fp8(q, *cache)
    assert torch.equal(o[1], good[1]) and torch.equal(o[0, 1:], good[0, 1:])
    # +inf and -inf scores: the sum of weights is NaN
    assert torch.isnan(o[0, 0]).any()


def test_decode_leaves_out_bad_pages():
    q, cache = make([64, 64], 4, 1, seed=8)
    table, kv_len = cache[4:]
    for bad in (-1, cache[0].shape[0], 2 ** 31 - 1):
        broken = table.clone()
        broken[0, 1] = bad
        o, lse = oss.attention_decode_paged_fp8(q, *cache[:4], broken, kv_len)
        with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
            oss.check_device_error()
        assert oss.check_device_error() == 0
        good = torch.cat([table[0, :1], table[0, 2:]])[None]
        check_decode_fp8(o[:1], lse[:1], q[:1], *cache[:4], good, kv_len[:1] - 16, 1 / math.sqrt(128))
        check_decode_fp8(o[1:], lse[1:], q[1:], *cache[:4], table[1:], kv_len[1:], 1 / math.sqrt(128))
    o, lse = oss.attention_decode_paged_fp8(q, *cache[:4], torch.full_like(table, -5), kv_len)
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))


def test_decode_clamps_lengths():
    q, cache = make([64, 30], 4, 1, seed=9)
    o, lse = oss.attention_decode_paged_fp8(q, *cache[:5], ints([65, -3]))
    check_decode_fp8(o, lse, q, *cache[:5], ints([64, 0]), 1 / math.sqrt(128))


def test_decode_same_bits_every_time_and_beside_other_calls():
    q, cache = make([5000, 31, 900], 8, 2, page=64, seed=10)
    ref = oss.attention_decode_paged_fp8(q, *cache)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [oss.attention_decode_paged_fp8(q, *cache, stream=s) for s in streams for _ in range(5)]
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


# -- append and read ---------------------------------------------------------------------------

def expect(pool, sc, table, page, pos, x):
    """Bytes of a pool and its scales after the rows x [n, heads, D] went to `pos` of a sequence."""
    c, s = quantise(x)
    bad = np.isnan(s)
    cb = torch.from_numpy(np.where(bad[..., None], 0.0, c)).float().to(F8).view(torch.uint8)
    cb[torch.from_numpy(bad)] = 0x7f
    sb = torch.from_numpy(np.where(bad, 255, np.log2(np.where(bad, 1.0, s)) + 127)).to(torch.uint8)
    t = torch.as_tensor(pos)
    where = table[t // page].long()
    pool[where, :, t % page], sc[where, :, t % page] = cb, sb


def bytes_of(*tensors):
    return [t.contiguous().view(torch.uint8).cpu() for t in tensors]


@pytest.mark.parametrize("d,dtype,page,layout", [(128, "bf16", 16, "head"), (64, "f16", 64, "slot"),
                                                 (128, "f16", 32, "joint"), (64, "bf16", 1024, "head")])
@pytest.mark.parametrize("before,new", [([0, 5, 16, 100, 31], [33, 0, 1, 64, 1]), ([0], [1]), ([15], [2]),
                                        ([7, 0], [0, 0])])
def test_append_writes_the_new_rows_only_and_read_gives_them_back(d, dtype, page, layout, before, new):
    heads = 3
    gen = torch.Generator(device="cuda")
    gen.manual_seed(d + page)
    lens = [a + b for a, b in zip(before, new)]
    table, pages = tables(lens, page, gen)
    cache = pools(pages, heads, page, d, layout, byte=0x33, scale=99)
    total = sum(new)
    # k and v are slices of one projection, with rows behind the last sequence
    qkv = rows(gen, (total + 2, 5 * heads, d), DTYPES[dtype])
    k, v = qkv[:, heads:2 * heads], qkv[:, 3 * heads:4 * heads]
    want = bytes_of(*cache)
    at = 0
    for b, n in enumerate(new):
        pos = torch.arange(before[b], lens[b])
        for pool, sc, x in ((want[0], want[2], k), (want[1], want[3], v)):
            expect(pool, sc, table[b].cpu(), page, pos, x[at:at + n])
        at += n
    cu = ints(np.concatenate([[0], np.cumsum(new)]).tolist())
    oss.kv_cache_append_fp8(k, v, *cache, table, ints(lens), cu)
    assert oss.check_device_error() == 0
    for got, ref in zip(bytes_of(*cache), want):
        assert torch.equal(got, ref)
    # back: into slices of a wide buffer, rows behind the last sequence left as they were
    wide = torch.full((total + 2, 4, heads, d), 5.0, dtype=DTYPES[dtype], device="cuda")
    out = oss.kv_cache_read_fp8(*cache, table, ints(lens), cu, total + 2, DTYPES[dtype], wide[:, 1], wide[:, 3])
    assert oss.check_device_error() == 0
    assert out[0].data_ptr() == wide[:, 1].data_ptr()
    for x, y in ((k, wide[:, 1]), (v, wide[:, 3])):
        c, s = quantise(x[:total])
        ref = torch.from_numpy(c * s[..., None]).to(DTYPES[dtype]).cuda()
        assert torch.equal(y[:total], ref) and torch.all(y[total:] == 5.0)
    assert torch.all(wide[:, 0] == 5.0) and torch.all(wide[:, 2] == 5.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_at_the_borders_of_the_format(d, dtype):
    # largest magnitudes around 448 * 2^e, subnormal and largest numbers, halfway cases of
    # the rounding, zeros, NaN and infinities, one row each
    t = DTYPES[dtype]
    top = torch.finfo(t).max
    x = torch.zeros((24, 1, d), dtype=torch.float64)
    for i, a in enumerate((448.0, 449.0, 450.0, 464.0, 447.0, 0.4375, 1.75, 1.7578125, top, torch.finfo(t).tiny,
                           torch.finfo(t).smallest_normal * torch.finfo(t).eps)):
        x[i, 0, i % d] = -a if i % 2 else a
    ramp = torch.arange(d, dtype=torch.float64)
    x[11, 0] = 256 + 16 * ramp.clamp(max=12)        # halfway between codes: 256 + 16 (2 n + 1)
    x[12, 0] = 2.0 ** -6 * (ramp.clamp(max=60) / 16)  # subnormal codes, halfway ones among them
    x[12, 0, -1] = 448
    x[13, 0] = 1 + ramp.clamp(max=15) / 16
    x[14, 0] = -x[13, 0]
    x[15, 0, 0] = 448
    x[15, 0, 1] = 2.0 ** -10                        # half the least code: to zero
    x[15, 0, 2] = 1.5 * 2.0 ** -10
    x[16, 0, 3] = float("nan")
    x[17, 0, 4] = float("inf")
    x[18, 0, 5] = -float("inf")
    x[19, 0] = float("nan")
    x[20, 0] = -0.0
    x = x.to(t).cuda()
    cache = pools(3, 1, 16, d, "head", byte=0x33, scale=99)
    table, kv_len, cu = ints([[2, 0]]), ints([24]), ints([0, 24])
    want = bytes_of(*cache)
    v = x.flip(0).contiguous()
    expect(want[0], want[2], table[0].cpu(), 16, torch.arange(24), x)
    expect(want[1], want[3], table[0].cpu(), 16, torch.arange(24), v)
    oss.kv_cache_append_fp8(x, v, *cache, table, kv_len, cu)
    for got, ref in zip(bytes_of(*cache), want):
        same = (got == ref) | ((got & 0x7f == 0) & (ref & 0x7f == 0) if got.dim() == 4 else got == ref)  # -0 and 0
        assert same.all(), torch.nonzero(~same)[:5]
    k2, v2 = oss.kv_cache_read_fp8(*cache, table, kv_len, cu, 24, t)
    c, s = quantise(x)
    ref = torch.from_numpy(c * s[..., None]).to(t)
    assert torch.equal(torch.nan_to_num(k2.cpu(), nan=7.0), torch.nan_to_num(ref, nan=7.0))
    assert torch.equal(torch.nan_to_num(v2.cpu().flip(0), nan=7.0), torch.nan_to_num(ref, nan=7.0))


def test_a_bf16_cache_read_as_fp16():
    # values beyond fp16's range become infinity, small ones are rounded to its grid
    x = torch.tensor([2.0 ** 20, 448.0, 2.0 ** -18, -(2.0 ** 17)], dtype=torch.bfloat16, device="cuda")
    x = x[:, None, None].expand(4, 1, 64).contiguous()
    cache = pools(1, 1, 16, 64, "head")
    table, kv_len, cu = ints([[0]]), ints([4]), ints([0, 4])
    oss.kv_cache_append_fp8(x, x, *cache, table, kv_len, cu)
    k, _ = oss.kv_cache_read_fp8(*cache, table, kv_len, cu, 4, torch.float16)
    assert torch.equal(k, x.double().to(torch.float16))


def test_append_one_token_each_and_a_padded_batch():
    lens = [1, 0, 17, 16, 40, 0]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(21)
    table, pages = tables(lens, 16, gen)
    cache = pools(pages, 2, 16, 128, "head", byte=0x33, scale=99)
    k, v = (rows(gen, (6, 2, 128), torch.bfloat16) for _ in range(2))
    want = bytes_of(*cache)
    for b, n in enumerate(lens):
        if n:
            expect(want[0], want[2], table[b].cpu(), 16, [n - 1], k[b:b + 1])
            expect(want[1], want[3], table[b].cpu(), 16, [n - 1], v[b:b + 1])
    oss.kv_cache_append_fp8(k, v, *cache, table, ints(lens))
    assert oss.check_device_error() == 0
    for got, ref in zip(bytes_of(*cache), want):
        assert torch.equal(got, ref)


@pytest.mark.parametrize("lens,heads,d,dtype", [([4000, 1, 2500], 8, 128, "bf16"), ([1, 0, 999], 5, 64, "f16")])
def test_append_many_tokens_and_read_the_last_ones(lens, heads, d, dtype):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(22)
    table, pages = tables(lens, 64, gen)
    cache = pools(pages, heads, 64, d, "head")
    k, v = (rows(gen, (sum(lens), heads, d), DTYPES[dtype]) for _ in range(2))
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    oss.kv_cache_append_fp8(k, v, *cache, table, ints(lens), ints(cu))
    for x, pool, sc in ((k, cache[0], cache[2]), (v, cache[1], cache[3])):
        c, s = quantise(x)
        for b, n in enumerate(lens):
            for g in (0, heads - 1):
                ref = c[cu[b]:cu[b] + n, g] * s[cu[b]:cu[b] + n, g, None]
                assert np.array_equal(gather8(pool, sc, table[b], n, g), ref)
    # the last 1000 tokens at most of each
    few = [min(n, 1000) for n in lens]
    cf = np.concatenate([[0], np.cumsum(few)]).tolist()
    k2, v2 = oss.kv_cache_read_fp8(*cache, table, ints(lens), ints(cf), sum(few), DTYPES[dtype])
    assert oss.check_device_error() == 0
    c, s = quantise(k)
    for b, n in enumerate(few):
        ref = (c * s[..., None])[cu[b + 1] - n:cu[b + 1]]
        assert np.array_equal(f64(k2[cf[b]:cf[b + 1]]), ref)


@pytest.mark.parametrize("kv_len,entry", [([16, 40], -1), ([16, 40], 99999), ([-1, 40], None), ([16, 65], None)])
def test_append_and_read_leave_out_what_has_no_place(kv_len, entry):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(23)
    table, pages = tables([16, 64], 16, gen)
    cache = pools(pages, 2, 16, 128, "head", byte=0x33, scale=99)
    k, v = (rows(gen, (2, 2, 128), torch.bfloat16) for _ in range(2))
    good = 0 if kv_len[1] == 65 else 1
    if entry is not None:
        table[0, 0] = entry
    want = bytes_of(*cache)
    expect(want[0], want[2], table[good].cpu(), 16, [kv_len[good] - 1], k[good:good + 1])
    expect(want[1], want[3], table[good].cpu(), 16, [kv_len[good] - 1], v[good:good + 1])
    cu = ints([0, 1, 2])
    oss.kv_cache_append_fp8(k, v, *cache, table, ints(kv_len), cu)
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()
    for got, ref in zip(bytes_of(*cache), want):
        assert torch.equal(got, ref)
    out = torch.full((2, 2, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    oss.kv_cache_read_fp8(*cache, table, ints(kv_len), cu, 2, k=out[0], v=out[1])
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()
    assert torch.all(out[:, 1 - good] == 5.0)
    c, s = quantise(k[good])
    assert np.array_equal(f64(out[0, good]), c * s[..., None])


@pytest.mark.parametrize("cu", [[0, 2, 1], [0, 1, 4], [-1, 1, 2]])
def test_offsets_that_do_not_fit_are_reported(cu):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(24)
    table, pages = tables([16, 64], 16, gen)
    cache = pools(pages, 1, 16, 64, "head")
    k = rows(gen, (3, 1, 64), torch.bfloat16)
    oss.kv_cache_append_fp8(k, k, *cache, table, ints([16, 40]), ints(cu))
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()
    oss.kv_cache_read_fp8(*cache, table, ints([16, 40]), ints(cu), 3)
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()


def test_nothing_to_do():
    cache = pools(1, 2, 16, 64, "head")
    empty = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    table, kv_len = ints([[0]]), ints([0])
    oss.kv_cache_append_fp8(empty, empty, *cache, table, kv_len, ints([0, 0]))
    k, v = oss.kv_cache_read_fp8(*cache, table, kv_len, ints([0, 0]), 0, torch.float16)
    assert k.shape == v.shape == (0, 2, 64) and k.dtype == torch.float16
    assert oss.check_device_error() == 0


def test_the_binding_refuses():
    q, (kp, vp, ks, vs, table, kv_len) = make([50, 20], 4, 2, seed=3)
    cu = ints([0, 50, 70])
    call = oss.attention_decode_paged_fp8
    with pytest.raises(TypeError, match="float8_e8m0fnu"):
        call(q, kp, vp, ks.view(torch.uint8), vs, table, kv_len)
    with pytest.raises(ValueError, match="scale for each row"):
        call(q, kp, vp, ks[:, :1], vs, table, kv_len)
    with pytest.raises(ValueError, match="same strides"):
        call(q, kp, vp, ks, torch.stack([vs.view(torch.uint8)] * 2, 1)[:, 0].view(E8), table, kv_len)
    with pytest.raises(ValueError, match="unit stride"):
        call(q, kp, vp, ks, vs.view(torch.uint8).repeat(1, 1, 2)[:, :, ::2].view(E8), table, kv_len)
    with pytest.raises(ValueError, match="cannot share"):
        call(q[:, :3], kp, vp, ks, vs, table, kv_len)
    with pytest.raises(ValueError, match="like the cache"):
        call(q[:1], kp, vp, ks, vs, table, kv_len)
    with pytest.raises(ValueError, match="kv_len must have one entry"):
        call(q, kp, vp, ks, vs, table, kv_len[:1])
    with pytest.raises(ValueError, match="given together"):
        oss.kv_cache_read_fp8(kp, vp, ks, vs, table, kv_len, cu, 70, k=torch.empty((70, 2, 128), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="must be"):
        x = torch.empty((2, 69, 2, 128), dtype=torch.bfloat16, device="cuda")
        oss.kv_cache_read_fp8(kp, vp, ks, vs, table, kv_len, cu, 70, k=x[0], v=x[1])
    with pytest.raises(TypeError, match="neither"):
        oss.kv_cache_read_fp8(kp, vp, ks, vs, table, kv_len, cu, 70, torch.float32)
    with pytest.raises(ValueError, match="batch . 1 entries"):
        oss.kv_cache_read_fp8(kp, vp, ks, vs, table, kv_len, cu[:2], 70)
    with pytest.raises(TypeError):
        oss.kv_cache_append_fp8(q[:, :2], q[:, :2].half(), kp, vp, ks, vs, table, kv_len)
    assert oss.check_device_error() == 0


@pytest.mark.slow
def test_offsets_beyond_32_bits():
    # pools of more than 2^32 bytes: the last pages are used
    page, heads, d = 64, 8, 128
    pages = (2 ** 32 + 2 ** 26) // (page * heads * d)
    kp = torch.empty((pages, heads, page, d), dtype=torch.uint8, device="cuda").view(F8)
    vp = torch.empty((pages, heads, page, d), dtype=torch.uint8, device="cuda").view(F8)
    ks, vs = (torch.empty((pages, heads, page), dtype=torch.uint8, device="cuda").view(E8) for _ in range(2))
    table = ints([[pages - 1, pages - 2, 0], [pages - 3, 1, 2]])
    new = torch.randn((2, 300, heads, d), device="cuda").to(torch.bfloat16)
    kv_len, cu = ints([130, 170]), ints([0, 130, 300])
    oss.kv_cache_append_fp8(new[0], new[1], kp, vp, ks, vs, table, kv_len, cu)
    k, v = oss.kv_cache_read_fp8(kp, vp, ks, vs, table, kv_len, cu, 300)
    for x, y in ((new[0], k), (new[1], v)):
        c, s = quantise(x)
        assert np.array_equal(f64(y), c * s[..., None])
    q = torch.randn((2, 16, d), device="cuda").to(torch.bfloat16)
    o, lse = oss.attention_decode_paged_fp8(q, kp, vp, ks, vs, table, kv_len)
    assert oss.check_device_error() == 0
    check_decode_fp8(o, lse, q, kp, vp, ks, vs, table, kv_len, 1 / math.sqrt(d))


# -- together --------------------------------------------------------------------------------

def test_prompts_steps_and_a_continued_prompt():
    # prompts in one launch, their rows quantised into pages, decode steps, then the
    # next piece of the prompts behind what is cached
    gen = torch.Generator(device="cuda")
    gen.manual_seed(31)
    hq, hkv, d, page, dtype = 8, 2, 128, 16, torch.bfloat16
    lens, piece = [40, 129, 7], [20, 3, 50]
    table, pages = tables([n + 2 + p for n, p in zip(lens, piece)], page, gen)
    cache = pools(pages, hkv, page, d, "head")
    total = sum(lens)
    q, k, v = (torch.randn((total, h, d), generator=gen, device="cuda").to(dtype) for h in (hq, hkv, hkv))
    cu = ints(np.concatenate([[0], np.cumsum(lens)]).tolist())
    kv_len = ints(lens)
    oss.kv_cache_append_fp8(k, v, *cache, table, kv_len, cu)
    o, lse = oss.attention_fwd_packed(q, k, v, cu)
    for _ in range(2):
        q1, k1, v1 = (torch.randn((3, h, d), generator=gen, device="cuda").to(dtype) for h in (hq, hkv, hkv))
        kv_len += 1
        oss.kv_cache_append_fp8(k1, v1, *cache, table, kv_len)
        o1, lse1 = oss.attention_decode_paged_fp8(q1, *cache, table, kv_len)
        check_decode_fp8(o1, lse1, q1, *cache, table, kv_len, 1 / math.sqrt(d))
    n2 = sum(piece)
    q2, k2, v2 = (torch.randn((n2, h, d), generator=gen, device="cuda").to(dtype) for h in (hq, hkv, hkv))
    cu2 = ints(np.concatenate([[0], np.cumsum(piece)]).tolist())
    kv_len += ints(piece)
    oss.kv_cache_append_fp8(k2, v2, *cache, table, kv_len, cu2)
    full = [n + 2 + p for n, p in zip(lens, piece)]
    cu_k = ints(np.concatenate([[0], np.cumsum(full)]).tolist())
    kk, vv = oss.kv_cache_read_fp8(*cache, table, kv_len, cu_k, sum(full), dtype)
    o2, lse2 = oss.attention_fwd_packed(q2, kk, vv, cu2, cu_k)
    assert oss.check_device_error() == 0
    for b, (n, at) in enumerate(zip(full, cu_k.tolist())):
        for g in range(hkv):
            assert np.array_equal(f64(kk[at:at + n, g]), gather8(cache[0], cache[2], table[b], n, g))
            assert np.array_equal(f64(vv[at:at + n, g]), gather8(cache[1], cache[3], table[b], n, g))
    check_packed(o2, lse2, q2, kk, vv, piece, full, 1 / math.sqrt(d), True)


def test_a_step_in_a_graph_follows_the_cache():
    # length, append and decode in one captured step, replayed token by token; two graphs
    # captured on one stream and replayed side by side
    gen = torch.Generator(device="cuda")
    gen.manual_seed(32)
    lens, d = [33, 4000], 128
    sides = []
    for _ in range(2):
        table, pages = tables([n + 40 for n in lens], 32, gen)
        cache = pools(pages, 2, 32, d, "head")
        k, v = (rows(gen, (sum(lens), 2, d), torch.bfloat16) for _ in range(2))
        kv_len = ints(lens)
        oss.kv_cache_append_fp8(k, v, *cache, table, kv_len, ints([0, 33, 4033]))
        new = [torch.zeros((2, h, d), dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2)]
        oss.attention_decode_paged_fp8(new[0], *cache, table, kv_len)
        sides.append((cache, table, kv_len, new))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for cache, table, kv_len, (q1, k1, v1) in sides:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kv_len += 1
            oss.kv_cache_append_fp8(k1, v1, *cache, table, kv_len)
            outs.append(oss.attention_decode_paged_fp8(q1, *cache, table, kv_len))
        graphs.append(graph)
    other = torch.cuda.Stream()
    for _ in range(20):
        for _, _, _, new in sides:
            for x in new:
                x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
        torch.cuda.synchronize()
    for (cache, table, kv_len, new), (o, lse) in zip(sides, outs):
        assert kv_len.tolist() == [53, 4020]
        check_decode_fp8(o, lse, new[0], *cache, table, kv_len, 1 / math.sqrt(d))
        assert torch.equal(o, oss.attention_decode_paged_fp8(new[0], *cache, table, kv_len)[0])
    assert oss.check_device_error() == 0


def test_on_other_streams_and_from_several_threads():
    # calls on streams of their own, and threads that share one: the same bytes from all
    lens = [1500, 20, 700]
    q, cache = make(lens, 8, 2, page=32, seed=33)
    cu, total = ints([0, 1500, 1520, 2220]), 2220
    want = (*oss.attention_decode_paged_fp8(q, *cache), *oss.kv_cache_read_fp8(*cache, cu, total))
    torch.cuda.synchronize()
    wrong = []

    def work(stream):
        out = pools(cache[0].shape[0], 2, 32, 128, "head")
        for _ in range(20):
            got = (*oss.attention_decode_paged_fp8(q, *cache, stream=stream),
                   *oss.kv_cache_read_fp8(*cache, cu, total, stream=stream))
            oss.kv_cache_append_fp8(want[2], want[3], *out, *cache[4:], cu, stream=stream)
            torch.cuda.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                wrong.append(stream)
        k, _ = oss.kv_cache_read_fp8(*out, *cache[4:], cu, total)
        if not torch.equal(k, want[2]):
            wrong.append("append")

    shared = torch.cuda.Stream()
    threads = [threading.Thread(target=work, args=(s,)) for s in (None, shared, shared, torch.cuda.Stream())]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert oss.check_device_error() == 0


def test_a_captured_read_follows_the_lengths():
    q, cache = make([300, 40], 4, 2, seed=34)
    kv_len, cu = cache[5], ints([0, 300, 340])
    full = oss.kv_cache_read_fp8(*cache, cu, 340)
    torch.cuda.synchronize()
    k, v = (torch.zeros((340, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        oss.kv_cache_read_fp8(*cache, cu, 340, k=k, v=v)
    for n in ([300, 40], [17, 3], [0, 40]):
        kv_len.copy_(ints(n))
        cu.copy_(ints([0, n[0], sum(n)]))
        k.fill_(5.0)
        v.fill_(5.0)
        graph.replay()
        for got, ref in ((k, full[0]), (v, full[1])):
            assert torch.equal(got[:n[0]], ref[:n[0]]) and torch.equal(got[n[0]:sum(n)], ref[300:300 + n[1]])
            assert torch.all(got[sum(n):] == 5.0)
    assert oss.check_device_error() == 0


def test_outputs_have_guards():
    # nothing around o and lse, and around the rows read back, is written
    q, cache = make([70, 0, 333], 12, 4, d=64, seed=35)
    cu = ints([0, 70, 70, 403])
    for n, call in (((3, 12, 64), "o"), ((403, 4, 64), "k")):
        size = math.prod(n)
        flat = [torch.full((size + 256,), 7.0, dtype=q.dtype, device="cuda") for _ in range(2)]
        x, y = (f[128:128 + size].view(n) for f in flat)
        lse = torch.full((3 * 12 + 64,), 7.0, device="cuda")
        if call == "o":
            oss.attention_decode_paged_fp8(q, *cache, o=x, lse=lse[32:32 + 36].view(3, 12))
            assert torch.all(lse[:32] == 7.0) and torch.all(lse[68:] == 7.0) and not torch.any(lse[32:68] == 7.0)
        else:
            oss.kv_cache_read_fp8(*cache, cu, 403, k=x, v=y)
        for f in flat:
            assert torch.all(f[:128] == 7.0) and torch.all(f[128 + size:] == 7.0)
    assert oss.check_device_error() == 0
