"""The choice counts page numbers outside the pool for every sequence, those within their budget among them."""

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from test_gpu_serving import dev

pytestmark = pytest.mark.gpu


def choose(table, lens, budget, pages, err):
    desc = wd.make_kv_desc(wd.KV_FP8, 2, 64, 16, pages)
    weights = torch.zeros(pages, 2, 16, device="cuda")
    keep = torch.full((len(lens), 2, budget), 7, dtype=torch.int32, device="cuda")
    counts = torch.full((len(lens),), 7, dtype=torch.int32, device="cuda")
    wd.kv_choose(desc, weights, dev(np.asarray(lens, np.int32)), dev(np.asarray(table, np.int32)), keep, counts, err_count=err)
    return keep.cpu().numpy(), counts.cpu().numpy()


@pytest.mark.parametrize("width", [40, 300, 2100])       # tables of each form of the choice
@pytest.mark.parametrize("bad", [-1, 2100, (1 << 31) - 1])
@pytest.mark.parametrize("at", [0, 36])
def test_a_lost_page_of_a_short_sequence_is_counted(width, bad, at):
    table = np.tile(np.arange(width, dtype=np.int64), (2, 1))
    table[0, at] = bad
    m = at * 16 + 1                                      # one place of the page
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep, counts = choose(table, [m, 5], 600, 2100, err)
    assert err.item() >= 1
    assert counts.tolist() == [m, 5]
    for b, n in enumerate((m, 5)):
        for h in range(2):
            assert keep[b, h].tolist() == list(range(n)) + [-1] * (600 - n)


@pytest.mark.parametrize("width", [40, 300, 2100])
def test_pages_past_a_short_sequence_are_not_looked_at(width):
    table = np.full((3, width), -1, np.int64)
    table[0, :3] = [5, 0, 9]
    table[1, 0] = 2
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep, counts = choose(table, [48, 16, 0], 100, 2100, err)
    assert err.item() == 0 and counts.tolist() == [48, 16, 0]
    assert (keep[2] == -1).all() and keep[0, 1, :48].tolist() == list(range(48))


def test_a_long_run_of_pages_is_looked_at_whole():
    """More pages than a workgroup has threads, each of one token; the last is lost."""
    desc = wd.make_kv_desc(wd.KV_BF16, 1, 32, 1, 3000)
    table = np.arange(3000, dtype=np.int32)[None].copy()
    weights = torch.zeros(3000, 1, 1, device="cuda")
    keep, counts = torch.empty(1, 1, 3000, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    for bad, want in ((2999, 0), (3000, 1)):
        table[0, 2999] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        wd.kv_choose(desc, weights, dev(np.array([3000], np.int32)), dev(table), keep, counts, err_count=err)
        assert (err.item() >= 1) == bool(want)
        assert keep[0, 0].tolist() == list(range(3000))
