"""CPU oracle of attention over trees of drafted tokens, of the rows' log-sums and of the check of drafted trees (numpy,
64 bits), written from their definitions in include/llvq.h.  Shares no code with the GPU path."""

import numpy as np

from oracle.serving import draw


def sees(parents, text, window=0):
    """[n][text + n]: what each node of one sequence sees."""
    n = len(parents)
    path = []
    for i, p in enumerate(parents):
        path.append((path[p] if 0 <= p < i else []) + [i])
    see = np.zeros((n, text + n), bool)
    for i in range(n):
        here = text + len(path[i]) - 1
        for j in range(text):
            see[i, j] = not window or j > here - window
        for depth, j in enumerate(path[i]):
            see[i, text + j] = not window or text + depth > here - window
    return see


def attend(q, k, v, see, scale):
    """One sequence: q [n][heads][D], k and v [len][kv_heads][D], see [n][len].  Returns (out, mass, spread, lse): mass =
    sum p |v| / sum p, spread = the largest scale * sum |q_d k_d| over the keys that a row sees."""
    n, heads, dim = q.shape
    share = heads // k.shape[1]
    out, mass = np.zeros((n, heads, dim)), np.zeros((n, heads, dim))
    spread, lse = np.zeros((n, heads)), np.full((n, heads), -np.inf)
    for i in range(n):
        if not see[i].any():
            continue
        for h in range(heads):
            kk, vv = k[see[i], h // share], v[see[i], h // share]
            s = scale * (kk @ q[i, h])
            spread[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
            p = np.exp(s - s.max())
            lse[i, h] = s.max() + np.log(p.sum())
            out[i, h] = p @ vv / p.sum()
            mass[i, h] = p @ np.abs(vv) / p.sum()
    return out, mass, spread, lse


def verify(target, starts, tokens, parents, uniforms, noise, width):
    """Trees checked node by node: (accepted [B], path [B][width], out [B][width])."""
    b, vocab = noise.shape
    accepted = np.zeros(b, np.int32)
    path, out = np.full((b, width), -1, np.int32), np.full((b, width), -1, np.int32)
    for s in range(b):
        n = min(starts[s + 1] - starts[s], 64)
        if n <= 0:
            continue
        at = starts[s]
        cur, left, gone, walk = 0, 1.0, set(), [0]
        for i in range(1, n):
            if len(walk) >= width:
                break
            if parents[at + i] != cur:
                continue
            x = int(tokens[at + i])
            w = float(target[at + cur][x]) if 0 <= x < vocab and x not in gone else 0.0
            w = w if w > 0 else 0.0
            if float(uniforms[at + i]) * max(left, 0.0) < w:
                cur, left, gone = i, 1.0, set()
                walk.append(i)
            else:
                left -= w
                gone.add(x)
        row = np.float32(target[at + cur])
        rest = row.copy()
        for x in gone:
            if 0 <= x < vocab:
                rest[x] = 0
        last = draw(rest, noise[s])
        accepted[s] = len(walk) - 1
        path[s, :len(walk)] = walk
        out[s, :len(walk) - 1] = [tokens[at + i] for i in walk[1:]]
        out[s, len(walk) - 1] = last if last >= 0 else draw(row, noise[s])
    return accepted, path, out
