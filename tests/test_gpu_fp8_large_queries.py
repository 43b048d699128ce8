"""The 8-bit decode of queries up to bf16's largest, over keys so small, or so far from them in
direction, that the scores are ordinary numbers (GPU)."""

import math

import pytest
import torch

import pass_attention_gb300 as oss
from fp8_reference import check_decode_fp8

pytestmark = pytest.mark.gpu
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
TOP = torch.finfo(torch.bfloat16).max


def cache(codes, k_bytes, page=16):
    """One sequence of one key head, whose keys are `codes` [n, D] uint8 with scale bytes k_bytes
    [n], and whose values are 1, 2, 4, ... (times 2^(t % 4)) in all dims."""
    n, d = codes.shape
    pages = -(-n // page)
    kp, vp = (torch.zeros((pages, 1, page, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, 1, page), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    t = torch.arange(n, device="cuda")
    kp[t // page, 0, t % page] = codes.cuda()
    ks[t // page, 0, t % page] = k_bytes.cuda()
    vp[t // page, 0, t % page] = 0x38
    vs[t // page, 0, t % page] = (127 + t % 4).to(torch.uint8)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return kp.view(F8), vp.view(F8), ks.view(E8), vs.view(E8), ints([list(range(pages))]), ints([n])


def run(q, c, scale=None):
    o, lse = oss.attention_decode_paged_fp8(q, *c, scale=scale)
    assert oss.check_device_error() == 0
    check_decode_fp8(o, lse, q, *c, scale or 1.0 / math.sqrt(q.shape[2]))
    return o, lse


@pytest.mark.parametrize("heads", [4, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("exponent", [100, 111, 120, 127])
def test_large_queries_over_small_keys(d, heads, exponent):
    # scores of up to 80: q of 2^exponent, keys of 2^-exponent
    codes = torch.zeros((40, d), dtype=torch.uint8)
    codes[:, 1] = torch.arange(40) % 8 + 0x70  # 128 .. 240
    codes[1::2, 1] |= 0x80
    q = torch.zeros((1, heads, d), dtype=torch.bfloat16, device="cuda")
    q[0, :, 1] = 2.0 ** exponent
    q[0, 0, 1] = TOP if exponent == 127 else 1.9921875 * 2.0 ** exponent
    run(q, cache(codes, torch.full((40,), 127 - exponent, dtype=torch.uint8)))


@pytest.mark.parametrize("d", [64, 128])
def test_large_queries_beside_large_keys(d):
    # products of zeros alone: scores of 0, however large the factors beside them
    codes = torch.zeros((20, d), dtype=torch.uint8)
    codes[:, 2] = 0x7e
    q = torch.zeros((1, 8, d), dtype=torch.bfloat16, device="cuda")
    q[0, :, 1] = TOP
    o, lse = oss.attention_decode_paged_fp8(q, *cache(codes, torch.full((20,), 246, dtype=torch.uint8)))
    assert oss.check_device_error() == 0
    # equal weights of 20 keys; the values are 1, 2, 4 and 8, of which every sum is exact, and o
    # rounds once more to bf16 (3.75 is one)
    assert (lse - math.log(20)).abs().max() <= 2.0 ** -20
    assert (o.float() - 3.75).abs().max() <= 3.75 * torch.finfo(torch.bfloat16).eps / 2


def test_scales_of_nan_beside_large_factors():
    # a key row whose scale alone is NaN (its codes are not) makes lse and o NaN
    codes = torch.zeros((20, 128), dtype=torch.uint8)
    k_bytes = torch.full((20,), 246, dtype=torch.uint8)
    k_bytes[7] = 255
    q = torch.full((1, 4, 128), TOP, dtype=torch.bfloat16, device="cuda")
    o, lse = oss.attention_decode_paged_fp8(q, *cache(codes, k_bytes))
    assert torch.isnan(o).all() and torch.isnan(lse).all()
    assert oss.check_device_error() == 0
