"""The 8-bit decode of a bf16 query whose elements differ by up to 2^40 within a head: every
element is off by at most 2^-40 of its head's largest, the term of fp8_reference (GPU)."""

import math

import pytest
import torch

import pass_attention_gb300 as oss
from fp8_reference import check_decode_fp8

pytestmark = pytest.mark.gpu
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def one_key(q, exponent, page=16):
    """A cache of one token whose key is 0 in dim 0 (the queries' largest) and 448 * 2^exponent
    elsewhere: the score, which is lse, is the small elements' alone."""
    d = q.shape[2]
    kp, vp = (torch.zeros((1, 1, page, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    kp[0, 0, 0, 1:] = 0x7e  # 448
    vp[0, 0, 0] = 0x38      # 1
    ks, vs = (torch.full((1, 1, page), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks[0, 0, 0] = 127 + exponent
    table, n = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    cache = (kp.view(F8), vp.view(F8), ks.view(E8), vs.view(E8), table, n)
    o, lse = oss.attention_decode_paged_fp8(q, *cache)
    assert oss.check_device_error() == 0
    check_decode_fp8(o, lse, q, *cache, 1.0 / math.sqrt(d))
    return lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("base", [-90, -3, 0, 60])
def test_elements_far_below_the_largest(d, base):
    # head h: all small elements 2^(-28 - h) of the largest, 2^base; the last at 2^-39
    q = torch.zeros((1, 12, d), dtype=torch.bfloat16, device="cuda")
    for h in range(12):
        q[0, h] = 2.0 ** (base - 28 - h)
    q[0, :, 0] = 2.0 ** base
    lse = one_key(q, 31 - base)
    # powers of two from 2^-39 of the largest on are exact in fp16: d - 1 products of one size
    for h in range(12):
        want = (d - 1) * 448 * 2.0 ** (31 - 28 - h) / math.sqrt(d)
        assert abs(lse[0, h].item() - want) <= 2.0 ** -20 * (want + 2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("largest", [1.0, 1.5, 1.9921875, -1.9921875])
def test_random_elements_below_any_largest(d, largest):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(d)
    q = torch.randn((1, 16, d), generator=gen, device="cuda") * torch.exp2(-40 + 14 * torch.rand((1, 16, d), generator=gen, device="cuda"))
    q[0, :, 0] = largest
    one_key(q.to(torch.bfloat16), 31)
