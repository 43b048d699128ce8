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


@pytest.mark.parametrize("n,prefix,tensor", [(20, 900, False), (20, 9000, True), (64, 2000, True)])
@pytest.mark.parametrize("at", [0, 1, -1])
def test_as_many_groups_as_sequences_and_all_in_one(n, prefix, tensor, at):
    # a slot for every sequence, and only one in use
    sizes, prefixes = [0] * n, [0] * n
    sizes[at], prefixes[at] = n, prefix
    c = Case(sizes, prefixes, [(5 * i) % 70 for i in range(n)], 16, 8, page=64, seed=n)
    assert on_tensor_cores(c) == tensor
    shared(c, rows=[0, 1, n - 1])


@pytest.mark.parametrize("n,prefix,tensor", [(5, 2000, False), (20, 9000, True), (64, 2000, True)])
def test_as_many_groups_as_sequences_and_one_in_each(n, prefix, tensor):
    c = Case([1] * n, [prefix - 31 * i for i in range(n)], [(5 * i) % 70 for i in range(n)], 16, 8, page=64, seed=n)
    assert on_tensor_cores(c) == tensor
    shared(c, rows=[0, n // 2, n - 1])


def test_one_tile_of_rows_over_the_whole_gpu():
    # 16 rows of a tile (two sequences of 8 heads), whose 1251 KV steps are cut over all SMs and joined
    # from their parts. (In a table of its own width the prefix would be read twice, 82 MB.)
    c = Case([2], [160001], [5, 40], 8, 1, page=64, seed=3, prefix_columns=3000)
    assert on_tensor_cores(c)
    shared(c)
