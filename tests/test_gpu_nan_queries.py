"""A query that holds NaN gets NaN, not the answer of a query without keys (GPU)."""

import math

import numpy as np
import pytest
import torch

import pass_attention_gb300 as oss
from paged_reference import attend, check, check_decode, check_packed, f64, gather
from test_gpu_packed import offsets, rand
from test_gpu_paged_cache import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (12, 1), (20, 1)])
@pytest.mark.parametrize("lens,columns", [([70, 200, 0, 16], None),             # answered in one piece
                                          ([3000, 100, 0, 1500], 128)])         # cut and joined
def test_decode(lens, columns, hq, hkv, d, dtype):
    q, kp, vp, table, kv_len, _ = make(lens, hq, hkv, d=d, dtype=dtype, page=32, columns=columns, seed=hq + d)
    bad = q.clone()
    bad[0, 1, 3] = float("nan")         # one head of one sequence
    bad[2] = float("nan")               # a sequence without keys
    bad[3] = float("nan")               # every head of a sequence
    w = torch.rand((4, hkv, table.shape[1] * 32), device="cuda")
    before = w.clone()
    o, lse = oss.attention_decode_paged(bad, kp, vp, table, kv_len, weights=w)
    assert oss.check_device_error() == 0
    for rows in ((0, 1), (3, slice(None))):
        assert torch.isnan(o[rows]).all() and torch.isnan(lse[rows]).all()
    assert torch.all(o[2] == 0) and torch.isneginf(lse[2]).all()
    # the other sequences, and the other heads of the first one
    scale = 1 / math.sqrt(d)
    check_decode(o[1:2], lse[1:2], q[1:2], kp, vp, table[1:2], kv_len[1:2], scale, w[1:2], before[1:2])
    u = torch.finfo(q.dtype).eps / 2
    group = hq // hkv
    for h in [x for x in range(hq) if x != 1]:
        g = h // group
        k, v = gather(kp, table[0], lens[0], g), gather(vp, table[0], lens[0], g)
        ro, rl, _, bo, bl, _ = attend(f64(q[0, h:h + 1]), k, v, np.ones((1, lens[0]), bool), scale, u, dtype == "f16")
        check(f64(o[0, h:h + 1]), ro, bo, f"head {h} o")
        check(f64(lse[0, h:h + 1]), rl, bl, f"head {h} lse")
    # sums over a group with such a head are NaN up to the length
    assert torch.isnan(w[0, 0, :lens[0]]).all() and torch.isnan(w[3, :, :lens[3]]).all()
    assert torch.equal(w[0, :, lens[0]:], before[0, :, lens[0]:]) and torch.equal(w[2], before[2])
    if hkv > 1:
        assert torch.isfinite(w[0, 1:]).all()


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2)])
@pytest.mark.parametrize("lens", [[40, 0, 130], [5, 2500]])  # whole tiles; tiles cut along the keys and joined
def test_packed(lens, hq, hkv, d, dtype):
    total = sum(lens)
    q, k, v = rand(1, total, hq, d, dtype=dtype), rand(2, total, hkv, d, dtype=dtype), rand(3, total, hkv, d, dtype=dtype)
    rows = [2, total - 1, total - 57]
    bad = q.clone()
    bad[rows, 0, 5] = float("nan")
    for causal in (True, False):
        o, lse = oss.attention_fwd_packed(bad, k, v, offsets(lens), causal=causal)
        assert oss.check_device_error() == 0
        assert torch.isnan(o[rows, 0]).all() and torch.isnan(lse[rows, 0]).all()
        # every other row has its answer
        clean, clean_lse = oss.attention_fwd_packed(q, k, v, offsets(lens), causal=causal)
        o[rows, 0], lse[rows, 0] = clean[rows, 0], clean_lse[rows, 0]
        check_packed(o, lse, q, k, v, lens, lens, 1 / math.sqrt(d), causal)
