"""Eviction of rows too long for a cluster's shared memory (more than 393216
positions in a row of the page table), whose selection reads the weights again
for every digit (GPU)."""

import pytest
import torch

from test_gpu_paged_cache import run_evict, spread

pytestmark = pytest.mark.gpu


def evict_wide(lens, heads, budget, recent, make_weights, seed, **kw):
    assert -(-max(lens) // 1024) * 1024 > 8 * 48 * 1024
    run_evict(lens, heads, budget, recent, make_weights, page=1024, d=64, seed=seed, **kw)


@pytest.mark.parametrize("budget,recent", [(1, 0), (700, 700), (5000, 77), (393000, 10), (400001, 3)])
def test_budgets(budget, recent):
    evict_wide([400001, 0, 700, 5001], 1, budget, recent, spread(budget), seed=budget)


def test_heads_and_strided_weights():
    evict_wide([393217, 399999], 3, 2000, 100, spread(4), seed=4, extra=1, wide=5, dtype="f16", layout="slot")


@pytest.mark.parametrize("budget,recent", [(20, 5), (150000, 0), (399000, 1000)])
def test_ties_go_to_the_lowest_position(budget, recent):
    evict_wide([400003], 1, budget, recent, lambda s: torch.randint(0, 3, s, device="cuda").float(), seed=1)
    evict_wide([400003], 1, budget, recent, lambda s: torch.full(s, 0.25, device="cuda"), seed=2)


def test_order_of_special_weights():
    def special(shape):
        w = torch.randn(shape, device="cuda")
        pick = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 1e-45, -1e-45, 3.4e38], device="cuda")
        return torch.where(torch.rand(shape, device="cuda") < 0.6, pick[torch.randint(0, 8, shape, device="cuda")], w)
    for budget in (60, 100000, 300000):
        evict_wide([395000], 1, budget, 0, special, seed=budget)
