"""kv_cache_append with offsets that do not fit its rows: reported, and no row
is written that has no place (GPU)."""

import pytest
import torch

import pass_attention_gb300 as oss
from test_gpu_paged_cache import ints, make

pytestmark = pytest.mark.gpu


def append(lens, rows, cu):
    """Appends `rows` rows; returns the pools, what they held before, k, v and the table."""
    _, kp, vp, table, kv_len, _ = make(lens, 2, 2, seed=len(lens) + rows)
    k, v = (torch.randn((rows, 2, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    before = kp.clone(), vp.clone()
    oss.kv_cache_append(k, v, kp, vp, table, kv_len, ints(cu))
    return (kp, vp), before, (k, v), table


def bits(x):
    return x.view(torch.int16)


@pytest.mark.parametrize("cu", [
    [0, 4, 10],               # past the rows
    [0, 4, 2 ** 31 - 1],
    [0, 9, 8],                # one sequence past the rows, the next one backwards
    [-2, 4, 8],               # from below the first row
    [0, 6, 4],                # backwards
    [8, 4, 8],
    [4, 8, -1],
    [0] * 300 + [9] * 2,      # far from the first sequence
])
def test_offsets_that_do_not_fit_are_reported(cu):
    append([40] * (len(cu) - 1), 8, cu)
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()
    assert oss.check_device_error() == 0


@pytest.mark.parametrize("cu", [[0, 4, 8], [3, 4, 8], [0, 0, 0], [2, 2, 2], [8, 8, 8], [0, 8, 8], [0] * 300 + [8]])
def test_offsets_that_fit_are_not(cu):
    append([40] * (len(cu) - 1), 8, cu)
    assert oss.check_device_error() == 0


def test_rows_that_are_there_are_written():
    # six new tokens by the offsets, four rows: those four go to their places
    pools, before, new, table = append([20, 37], 8, [0, 4, 10])
    with pytest.raises(oss.OssError, match="OS_ERR_BAD_INDEX"):
        oss.check_device_error()
    for pool, old, x in zip(pools, before, new):
        for b, first, at, n in ((0, 16, 0, 4), (1, 31, 4, 4)):
            for i in range(n):
                old[table[b, (first + i) // 16].long(), :, (first + i) % 16] = x[at + i]
        assert torch.equal(bits(pool), bits(old))
