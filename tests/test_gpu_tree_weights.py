"""The weights that cached tokens receive from a step of drafted trees: the accepted nodes move together, then attend and are
weighed as the chain that they are.  Bounds as in the tests of the weights, with the log-sum that the call itself gave."""

import math

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from test_gpu_attn_lse import run_lse
from test_gpu_eviction import check_weights, run_weigh
from test_gpu_serving import Setup, dev, f64
from test_gpu_trees import random_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_accepted_nodes_are_weighed_as_a_chain(kind, dtype):
    nodes, lens = 14, [64, 33, 214]
    su = Setup(kind, 2, 64, 16, [nodes] * 3, lens, seed=101)
    caches = su.fill()
    q = dev(su.rng.randn(3 * nodes, 6, 64).astype(np.float32), dtype)
    paths = []
    for b in range(3):
        parents, way = random_tree(su.rng, nodes), [nodes - 1 - b]
        while parents[way[0]] >= 0:
            way.insert(0, parents[way[0]])
        paths.append(way)
    width = max(len(way) for way in paths)
    lists = np.full((3, 1, width), -1, np.int32)
    for b, way in enumerate(paths):
        lists[b, 0, :len(way)] = way
    starts, full, table = su.plan()
    # the text has no weight yet; what the nodes' places held is of tokens that are gone
    weights = torch.zeros(su.pages, 2, 16, device="cuda")
    for b, m in enumerate(lens):
        for j in range(m - nodes, m):
            weights[int(su.table[b, j // 16]), :, j % 16] = math.nan
    wd.kv_keep(su.desc, su.pool, dev(lists), full, table, starts=starts, weights=weights)
    rows = np.concatenate([b * nodes + np.asarray(way) for b, way in enumerate(paths)])
    caches = [tuple(np.concatenate((x[:m - nodes], x[m - nodes:][way])) for x in both) for both, m, way in zip(caches, lens, paths)]
    su.new, su.lens = [len(way) for way in paths], [len(k) for k, _ in caches]
    su.starts = np.concatenate(([0], np.cumsum(su.new))).astype(np.int32)
    mine = q[dev(rows)].contiguous()
    _, lse = run_lse(su, mine)
    before = weights.cpu().numpy()
    run_weigh(su, weights, mine, lse)
    check_weights(su, caches, f64(mine), lse.cpu().numpy(), before, weights.cpu().numpy(), 0, True, False)
    for b, m in enumerate(su.lens):
        at = np.arange(m)
        page, slot = dev(su.table[b][at // 16]).long(), dev(at % 16)
        assert torch.isfinite(weights[page, :, slot]).all()
