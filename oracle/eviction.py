"""CPU oracle of eviction from the paged cache (numpy, 64 bits): the weight that cached tokens receive, the choice of those that
stay and their move, written from their definitions in include/llvq.h.  Shares no code with the GPU path."""

import numpy as np


def weigh(q, k, lse, see, scale):
    """One sequence: q [n][heads][D], k [m][kv_heads][D], lse [n][heads], see [n][m].  Returns (sums [m][kv_heads], slack):
    slack_j = sum_i p_ij (2 (3 D + 8) 2^-24 scale sum |q_d k_d| + 2^-21 (|s| + |lse| + 1))."""
    n, heads, dim = q.shape
    kv_heads = k.shape[1]
    sums, slack = np.zeros((len(k), kv_heads)), np.zeros((len(k), kv_heads))
    for h in range(heads):
        kk = k[:, h * kv_heads // heads]
        s = scale * (q[:, h] @ kk.T)
        with np.errstate(all="ignore"):
            p = np.where(see, np.exp(s - lse[:, h, None]), 0.0)
        size = 2 * (3 * dim + 8) * 2.0 ** -24 * scale * (np.abs(q[:, h]) @ np.abs(kk).T) + 2.0 ** -21 * (np.abs(s) + np.abs(lse[:, h, None]) + 1)
        sums[:, h * kv_heads // heads] += p.sum(0)
        slack[:, h * kv_heads // heads] += np.where(see, p * np.where(see, size, 0.0), 0.0).sum(0)
    return sums, slack


def choose(weights, budget, sinks, recent):
    """Places that stay of weights [m] (one sequence and head)."""
    m = len(weights)
    if m <= budget:
        return list(range(m))
    sure = list(range(sinks)) + list(range(m - recent, m))
    w = np.where(np.isnan(weights), -np.inf, weights).astype(np.float64)
    between = sorted(range(sinks, m - recent), key=lambda j: (-w[j], j))
    return sorted(sure + between[:budget - sinks - recent])


def keep(lay, pool, weights, tables, lens, lists, counts, firsts):
    """Moves tokens in pool (uint8 bytes) and weights ([pages][heads][page] or None) one entry after the other, in order."""
    for b in range(len(lens)):
        for h in range(lay.heads):
            mine = lists[b][h if len(lists[b]) > 1 else 0]
            for i in range(counts[b]):
                j = int(mine[i])
                if j in (-1, i):
                    continue
                (sp, ss), (dp, ds) = divmod(firsts[b] + j, lay.page), divmod(firsts[b] + i, lay.page)
                sp, dp = int(tables[b][sp]), int(tables[b][dp])
                for is_v in (0, 1):
                    for at, size in ((lay.codes, lay.row), (lay.scales, lay.groups)):
                        src, dst = at(sp, h, ss, is_v), at(dp, h, ds, is_v)
                        pool[dst:dst + size] = pool[src:src + size].copy()
                if weights is not None:
                    weights[dp, h, ds] = weights[sp, h, ss]
