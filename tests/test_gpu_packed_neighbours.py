"""A packed sequence's results do not depend on the rows around it: the same
bits whatever the queries that share its last tile hold (GPU)."""

import pytest
import torch

import pass_attention_gb300 as oss
from paged_reference import check_packed
from test_gpu_packed import offsets, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d,dtype", [(1, 1, 128, "bf16"), (4, 1, 128, "bf16"), (6, 3, 64, "bf16"), (8, 1, 64, "f16")])
def test_the_queries_behind_a_sequence_stay_out(hq, hkv, d, dtype, causal):
    # sequences of several KV tiles whose last query tile is partial: its other rows
    # are the next sequence's queries, or rows that no sequence has
    lens = [905, 1301, 677]
    total, tail = sum(lens), 130
    q = rand(1, total + tail, hq, d, dtype=dtype)
    k, v = (rand(s, total, hkv, d, dtype=dtype) for s in (2, 3))
    cu = offsets(lens)
    clean = oss.attention_fwd_packed(q, k, v, cu, causal=causal)
    check_packed(*clean, q, k, v, lens, lens, d ** -0.5, causal)
    first, last = slice(0, lens[0]), slice(lens[0] + lens[1], total)
    for value in (200.0, -77.0, float("nan"), float("inf")):
        other = q.clone()
        for rows in (slice(lens[0], lens[0] + lens[1]), slice(total, total + tail)):
            other[rows] = other[rows] * value if value == value and abs(value) < 1e4 else value
        o, lse = oss.attention_fwd_packed(other, k, v, cu, causal=causal)
        for rows in (first, last):
            assert torch.equal(o[rows], clean[0][rows]) and torch.equal(lse[rows], clean[1][rows]), value
    assert oss.check_device_error() == 0
