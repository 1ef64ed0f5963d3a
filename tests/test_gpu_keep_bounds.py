"""Moves whose first new token has no place: where a sequence's starts or length had to be cut, nothing of it moves."""

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from oracle import eviction as ev
from test_gpu_eviction import filled
from test_gpu_serving import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("starts,lens", [
    ([0, 101], [100]),              # one new token more than cached ones
    ([0, (1 << 31) - 1], [100]),
    ([0, -3], [100]),               # fewer than none
    ([3, 0], [100]),
    ([-(1 << 31), (1 << 31) - 1], [100]),
    ([0, 6], [113]),                # longer than the table's 112 places
    ([0, 6], [1 << 30]),
    ([0, 6], [-1]),
    ([0, 1], [0]),
])
@pytest.mark.parametrize("counted", [False, True])
def test_nothing_moves_from_a_place_that_is_not_known(kind, starts, lens, counted):
    su, w = filled(kind, 2, 64, 16, [0], [100], seed=81)
    clean, weights, err = su.pool.clone(), dev(w), torch.zeros(1, dtype=torch.int32, device="cuda")
    lists = np.array([[[0, 2, 5]]], np.int32)
    wd.kv_keep(su.desc, su.pool, dev(lists), dev(np.asarray(lens, np.int32)), dev(su.table), starts=dev(np.asarray(starts, np.int32)),
               counts=dev(np.array([3], np.int32)) if counted else None, weights=weights, err_count=err)
    assert torch.equal(su.pool, clean)
    assert np.array_equal(weights.cpu().numpy().view(np.uint32), w.view(np.uint32))
    assert err.item() >= 1


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_other_sequences_move_all_the_same(kind):
    """A sequence whose places are not known beside two that move."""
    su, w = filled(kind, 3, 96, 16, [8, 8, 8], [60, 40, 33], seed=82)
    lists = np.array([[[0, 3, 7]], [[0, 3, 7]], [[0, 1, 6]]], np.int32)
    starts, lens = np.array([0, 8, 50, 58], np.int32), [60, 40, 33]      # 42 new tokens of 40 in the middle
    pool, weights = su.pool.cpu().numpy(), w.copy()
    ev.keep(su.lay, pool, weights, su.table, lens, lists, [3, 0, 3], [52, 0, 25])
    got_w, err = dev(w), torch.zeros(1, dtype=torch.int32, device="cuda")
    wd.kv_keep(su.desc, su.pool, dev(lists), dev(np.asarray(lens, np.int32)), dev(su.table), starts=dev(starts), weights=got_w, err_count=err)
    assert np.array_equal(su.pool.cpu().numpy(), pool)
    assert np.array_equal(got_w.cpu().numpy().view(np.uint32), weights.view(np.uint32))
    assert err.item() == 3          # one for each key head of the middle one
