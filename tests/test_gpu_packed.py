"""attention_fwd_packed against its definition in 64 bits (GPU)."""

import math

import pytest
import torch

import pass_attention_gb300 as oss
from paged_reference import DTYPES, check_packed

pytestmark = pytest.mark.gpu


def offsets(lens, at=0):
    out = [at]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def rand(seed, *shape, dtype="bf16"):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(DTYPES[dtype])


def run(lens_q, lens_k, hq, hkv, d=128, dtype="bf16", causal=True, seed=0, scale=None):
    q = rand(seed, sum(lens_q), hq, d, dtype=dtype)
    k = rand(seed + 1, sum(lens_k), hkv, d, dtype=dtype)
    v = rand(seed + 2, sum(lens_k), hkv, d, dtype=dtype)
    o, lse = oss.attention_fwd_packed(q, k, v, offsets(lens_q), offsets(lens_k), scale=scale, causal=causal)
    assert oss.check_device_error() == 0
    check_packed(o, lse, q, k, v, lens_q, lens_k, scale or 1 / math.sqrt(d), causal)


LENS = [1, 0, 31, 32, 33, 127, 128, 129, 300, 2]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
def test_types_and_lengths(d, dtype, causal):
    run(LENS, LENS, 4, 1, d=d, dtype=dtype, causal=causal, seed=d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 4), (6, 1), (7, 1), (10, 2), (12, 1), (16, 1), (24, 2),
                                    (32, 1), (64, 1), (128, 1), (256, 1)])
def test_groups(hq, hkv):
    run([3, 130, 65], [3, 130, 65], hq, hkv, seed=hq)


@pytest.mark.parametrize("lens_q,lens_k", [
    ([1, 1, 5], [1, 500, 133]),          # a few queries behind long prefixes
    ([64, 200, 100], [1000, 200, 700]),  # pieces of prompts
    ([130, 40, 3], [5, 0, 2]),           # more queries than keys: the first rows see none
    ([0, 0], [10, 0]),
    ([257], [256]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_queries_and_keys_of_different_lengths(lens_q, lens_k, causal):
    if sum(lens_q):
        run(lens_q, lens_k, 8, 2, causal=causal, seed=len(lens_q))
    else:
        q, k = rand(1, 4, 8, 128), rand(2, 10, 2, 128)
        o = torch.full_like(q, 3.0)
        oss.attention_fwd_packed(q, k, k, offsets(lens_q), offsets(lens_k), causal=causal, o=o)
        assert torch.all(o == 3.0)


@pytest.mark.parametrize("lens,hq,hkv", [([1500, 2, 999], 8, 2), ([2049], 2, 2), ([5] * 500, 4, 2), ([700] * 12, 4, 4),
                                         ([1, 0, 2, 3] * 700, 2, 1)])
def test_long_and_many(lens, hq, hkv):
    run(lens, lens, hq, hkv, seed=len(lens))


def test_one_heavy_key_per_row():
    # scores up to several hundred in base 2, rising along the keys
    q, k, v = (rand(s, 600, 2, 128) for s in (1, 2, 3))
    k = k * torch.linspace(0.1, 6.0, 600, device="cuda").to(k.dtype)[:, None, None]
    for causal in (True, False):
        o, lse = oss.attention_fwd_packed(q, k, v, offsets([600]), causal=causal)
        check_packed(o, lse, q, k, v, [600], [600], 1 / math.sqrt(128), causal)


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_padded_batch_and_poison_around_it(poison):
    # rows before the first, behind the last sequence and between: not
    # read into any result, and not written
    lens = [40, 129, 7]
    total = sum(lens)
    q, k, v = (torch.full((total + 150, 4, 128), poison, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    good = [rand(s, total, 4, 128) for s in (1, 2, 3)]
    for x, y in zip((q, k, v), good):
        x[20:20 + total] = y
    o, lse = torch.full_like(q, 5.0), torch.full((total + 150, 4), 5.0, device="cuda")
    oss.attention_fwd_packed(q, k, v, offsets(lens, 20), causal=True, o=o, lse=lse)
    assert oss.check_device_error() == 0
    check_packed(o[20:], lse[20:], *good, lens, lens, 1 / math.sqrt(128), True)
    for x in (o, lse):
        assert torch.all(x[:20] == 5.0) and torch.all(x[20 + total:] == 5.0)


def test_a_neighbour_of_nan_stays_out():
    lens = [50, 60, 70]
    q, k, v = (rand(s, 180, 4, 128) for s in (1, 2, 3))
    bad = [x.clone() for x in (q, k, v)]
    for x in bad:
        x[50:110] = float("nan")
    for causal in (True, False):
        good, _ = oss.attention_fwd_packed(q, k, v, offsets(lens), causal=causal)
        o, _ = oss.attention_fwd_packed(*bad, offsets(lens), causal=causal)
        assert torch.equal(o[:50], good[:50]) and torch.equal(o[110:], good[110:])


def test_views_of_a_fused_projection():
    lens = [33, 200]
    qkv = rand(1, 233, 4 + 2 + 2, 128)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    o, lse = oss.attention_fwd_packed(q, k, v, offsets(lens), scale=0.05)
    check_packed(o, lse, q, k, v, lens, lens, 0.05, True)
    # head-major storage
    t, kv = rand(2, 4, 233, 128).transpose(0, 1), rand(3, 2, 233, 128).transpose(0, 1)
    o, lse = oss.attention_fwd_packed(t, kv, kv, offsets(lens))
    check_packed(o, lse, t, kv, kv, lens, lens, 1 / math.sqrt(128), True)


def test_same_bits_every_time_and_beside_other_calls():
    lens = [700, 3, 250]
    q, k, v = rand(1, 953, 8, 128), rand(2, 953, 2, 128), rand(3, 953, 2, 128)
    cu = offsets(lens)
    ref = oss.attention_fwd_packed(q, k, v, cu)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [oss.attention_fwd_packed(q, k, v, cu, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    assert oss.check_device_error() == 0
    for o, lse in outs:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_in_a_graph_with_new_lengths():
    q, k, v = rand(1, 600, 8, 128), rand(2, 600, 2, 128), rand(3, 600, 2, 128)
    cu = offsets([600, 0, 0])
    oss.attention_fwd_packed(q, k, v, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = oss.attention_fwd_packed(q, k, v, cu)
    for lens in ([600, 0, 0], [100, 200, 300], [1, 1, 598], [0, 599, 0]):
        cu.copy_(offsets(lens))
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert oss.check_device_error() == 0
        check_packed(o, lse, q, k, v, lens, lens, 1 / math.sqrt(128), True)


def test_offsets_outside_the_tokens_are_clamped():
    q, k, v = (rand(s, 100, 2, 128) for s in (1, 2, 3))
    cu = torch.tensor([0, 40, 160], dtype=torch.int32, device="cuda")
    o, lse = oss.attention_fwd_packed(q, k, v, cu)
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()
    check_packed(o, lse, q, k, v, [40], [40], 1 / math.sqrt(128), True)
    for bad in ([0, 60, 30], [-5, 10, 20], [0, 2 ** 31 - 1, 50], [50, 0, 100]):
        oss.attention_fwd_packed(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"))
        with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
            oss.check_device_error()


def test_no_keys_at_all():
    q = rand(1, 10, 4, 128)
    k = torch.empty((0, 2, 128), dtype=q.dtype, device="cuda")
    o, lse = oss.attention_fwd_packed(q, k, k, offsets([10]), offsets([0]))
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))
    o, lse = oss.attention_fwd_packed(q[:0], k, k, offsets([0]), offsets([0]))
    assert o.shape == (0, 4, 128) and lse.shape == (0, 4)


def test_refusals():
    q, k = rand(1, 20, 4, 128), rand(2, 20, 2, 128)
    cu = offsets([20])
    call = lambda **c: oss.attention_fwd_packed(**{**dict(q=q, k=k, v=k, cu_seqlens_q=cu), **c})  # noqa: E731
    for bad in (dict(k=k.half()), dict(q=q.float()), dict(cu_seqlens_q=cu.long()), dict(q=None)):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(v=k[:10]), dict(k=k[..., :64], v=k[..., :64]), dict(q=q[:, :3]), dict(cu_seqlens_q=cu[:1]),
                dict(cu_seqlens_k=offsets([5, 15])), dict(cu_seqlens_k=cu.cpu()), dict(q=q[..., ::2], k=k[..., ::2], v=k[..., ::2]),
                dict(o=q[:10]), dict(v=rand(2, 20, 4, 128)[:, ::2]), dict(q=q[0])):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(oss.OssError, match="UNSUPPORTED"):
        call(q=q[..., :32], k=k[..., :32], v=k[..., :32])
    with pytest.raises(oss.OssError, match="INVALID"):
        call(scale=-1.0)
    with pytest.raises(oss.OssError, match="INVALID"):
        call(k=k[:, :1].expand(20, 2, 128), v=k[:, :1].expand(20, 2, 128))
    with pytest.raises(oss.OssError, match="MISALIGNED"):
        call(q=torch.zeros(20, 4, 132, dtype=q.dtype, device="cuda")[..., :128])
    assert oss.check_device_error() == 0


def test_a_wait_that_runs_out_is_reported():
    q, k, v = rand(1, 300, 4, 128), rand(2, 300, 1, 128), rand(3, 300, 1, 128)
    cu = offsets([300])
    oss.debug_inject_fault(1, step=1, timeout_ns=2_000_000)
    oss.attention_fwd_packed(q, k, v, cu)
    with pytest.raises(oss.OssError, match="OS_ERR_TIMEOUT"):
        oss.check_device_error()
    o, lse = oss.attention_fwd_packed(q, k, v, cu)
    assert oss.check_device_error() == 0
    check_packed(o, lse, q, k, v, [300], [300], 1 / math.sqrt(128), True)


def test_many_rounds():
    # more than 64 MB of K and V: shares in several rounds, a window of heads at a time
    lens = [9000, 300]
    q, k, v = (rand(s, sum(lens), 16, 128) for s in (1, 2, 3))
    o, lse = oss.attention_fwd_packed(q, k, v, offsets(lens))
    assert oss.check_device_error() == 0
    heads = (0, 7, 15)
    check_packed(o[9000:], lse[9000:], q[9000:], k[9000:], v[9000:], [300], [300], 1 / math.sqrt(128), True)
    pick = torch.cat([torch.arange(40), torch.randint(40, 8900, (60,), generator=torch.Generator().manual_seed(1)),
                      torch.arange(8940, 9000)]).cuda()
    for i in pick.tolist():
        check_packed(o[i:i + 1, heads], lse[i:i + 1, heads], q[i:i + 1, heads], k[:i + 1, heads], v[:i + 1, heads],
                     [1], [i + 1], 1 / math.sqrt(128), True)
