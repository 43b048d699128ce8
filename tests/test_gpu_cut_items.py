"""Work that is cut between the GPU's SMs along the keys, and joined, in every
type, head size and head group (GPU). (The page table's width decides whether the
decode cuts, and the packed forward cuts tiles of more than five KV steps.)"""

import pytest
import torch

import pass_attention_gb300 as oss
from paged_reference import DTYPES, check_packed
from test_gpu_packed import offsets, rand, run
from test_gpu_paged_cache import decode

pytestmark = pytest.mark.gpu

TYPES = [(64, "bf16"), (64, "f16"), (128, "bf16"), (128, "f16")]


@pytest.mark.parametrize("d,dtype", TYPES)
@pytest.mark.parametrize("group", [1, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("hkv", [1, 3])
@pytest.mark.parametrize("weights", [False, True])
def test_decode(d, dtype, group, hkv, weights):
    decode([1000, 3217, 17, 0, 2049, 64], group * hkv, hkv, weights=weights, d=d, dtype=dtype, page=64, columns=100,
           seed=group + d)


@pytest.mark.parametrize("d,dtype", TYPES)
@pytest.mark.parametrize("lens,hq,hkv", [([0, 1, 15, 16, 17, 63, 64, 65, 127, 200, 333], 8, 2),  # short ones in a wide table
                                         ([20001], 16, 1), ([700] * 40, 4, 4)])
def test_decode_lengths(lens, hq, hkv, d, dtype):
    decode(lens, hq, hkv, weights=True, d=d, dtype=dtype, page=32, columns=640, seed=d)


@pytest.mark.parametrize("d,dtype", TYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens_q,lens_k,hq,hkv", [
    ([1500, 2, 999], [1500, 2, 999], 8, 2),
    ([1, 1, 5], [1, 3000, 133], 8, 2),         # a few queries behind long prefixes
    ([9], [20000], 2, 1),                      # one item over a hundred shares
    ([64, 200, 100], [2500, 200, 1700], 6, 3),
    ([2049], [2049], 2, 2),
])
def test_packed(lens_q, lens_k, hq, hkv, d, dtype, causal):
    run(lens_q, lens_k, hq, hkv, d=d, dtype=dtype, causal=causal, seed=d + len(lens_q))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,dtype,lens", [(64, "f16", [17000, 1300]), (64, "bf16", [700, 17500]), (128, "f16", [400, 8700])])
def test_packed_in_several_rounds(d, dtype, lens, causal):
    # more than 64 MB of K and V: a CTA's shares in several rounds
    heads = (0, 9, 15)
    q, k, v = (rand(s, sum(lens), 16, d, dtype=dtype) for s in (1, 2, 3))
    assert k.numel() * 4 > 64 << 20 and k.dtype == DTYPES[dtype]
    o, lse = oss.attention_fwd_packed(q, k, v, offsets(lens), causal=causal)
    assert oss.check_device_error() == 0
    gen = torch.Generator().manual_seed(d)
    at = 0
    for n in lens:
        pick = sorted({0, 1, 127, 128, n - 1, *torch.randint(0, n, (40,), generator=gen).tolist()})
        for i in pick:
            m = i + 1 if causal else n
            check_packed(o[at + i:at + i + 1, heads], lse[at + i:at + i + 1, heads], q[at + i:at + i + 1, heads],
                         k[at:at + m, heads], v[at:at + m, heads], [1], [m], d ** -0.5, causal)
        at += n
