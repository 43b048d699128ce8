"""attention_decode_shared where the way to its prefixes is decided: which way a call takes, by the
workspace that it asks for, and that the answers are right there (GPU)."""

import pytest

import pass_attention_gb300 as oss
from test_gpu_shared_prefix import Case

pytestmark = pytest.mark.gpu


def on_tensor_cores(c):
    """Whether the case's prefixes go to the tensor cores: their workspace does not depend on the
    prefix table's size."""
    lib = oss.load()
    cache = oss._cache(c.kp, c.vp, c.table, c.kv_len)[0]
    groups, pages = c.prefix_table.shape
    need = [lib.os_attention_decode_shared_workspace_bytes(c.q.shape[1], cache, *x) for x in ((pages, groups), (2 ** 30 // c.page, 65))]
    assert need[0] > 0 and need[1] > 0
    return need[0] == need[1]


def shared(c, rows=None):
    o, lse = c.run()
    assert oss.check_device_error() == 0
    c.check(o, lse, rows=rows)


@pytest.mark.parametrize("prefix,tensor", [(300, False), (4000, True)])
def test_blocks_of_query_heads_read_their_prefix_each(prefix, tensor):
    # 8 blocks of 16 query heads: 16 sequences read a prefix 128 times
    c = Case([16], [prefix], [(7 * i) % 60 for i in range(16)], 128, 1, seed=1)
    assert on_tensor_cores(c) == tensor
    shared(c, rows=[0, 15])


@pytest.mark.parametrize("hq,hkv,prefix,tensor", [(128, 1, 4001, False), (128, 1, 40001, True), (8, 1, 40001, False)])
def test_one_sequence(hq, hkv, prefix, tensor):
    c = Case([1], [prefix], [5], hq, hkv, page=64, seed=2)
    assert on_tensor_cores(c) == tensor
    shared(c)
