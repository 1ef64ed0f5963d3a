"""CPU oracle of the serving operators (numpy, 64 bits): the paged cache's bytes, the
attention over it and the check of drafted tokens, written from their definitions in
include/llvq.h.  Shares no code with the GPU path."""

import numpy as np

BF16, FP8, FP4 = 0, 1, 2
GROUP = 32
# magnitudes by code
E4M3 = np.array([m * 2.0 ** -9 if x == 0 else (8 + m) * 2.0 ** (x - 10) for x in range(16) for m in range(8)][:-1])
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
GRID = {FP8: E4M3, FP4: E2M1}
E_LOW, E_HIGH = -100, {FP8: 119, FP4: 125}


def bf16_bits(x):
    """Nearest bf16 (ties to even) of f32 values, as uint16; NaN stays NaN."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16_value(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def nearest_code(a, grid):
    """Index of the nearest grid value to each a >= 0, ties to the even index, past the end the last."""
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    low, up = a - grid[hi - 1], grid[hi] - a
    return np.where((low < up) | ((low == up) & (hi % 2 == 1)), hi - 1, hi)


def quantise(x, kind):
    """(codes [..., D] with sign, scale bytes [..., D / 32]) of x [..., D]."""
    g = np.asarray(x, np.float64).reshape(x.shape[:-1] + (-1, GROUP))
    amax = np.abs(g).max(-1)
    bad = ~np.isfinite(amax)
    safe = np.where(bad | (amax == 0), 1.0, amax)
    # the smallest e with amax <= top * 2^e
    mant, ex = np.frexp(safe / GRID[kind][-1])
    e = np.where(mant == 0.5, ex - 1, ex)
    e = np.clip(np.where(amax == 0, E_LOW, e), E_LOW, E_HIGH[kind])
    y = np.where(bad[..., None], 0.0, g) / 2.0 ** e[..., None]
    code = nearest_code(np.abs(y), GRID[kind])
    sign = np.signbit(y) & ~bad[..., None]
    code = code + sign * (128 if kind == FP8 else 8)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scales, kind):
    top = 128 if kind == FP8 else 8
    grid = np.concatenate((GRID[kind], [np.nan])) if kind == FP8 else GRID[kind]
    v = grid[codes % top] * np.where(codes >= top, -1.0, 1.0)
    f = np.where(scales > E_HIGH[kind] + 127, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v.reshape(v.shape[:-1] + (-1, GROUP)) * f[..., None]).reshape(v.shape)


def held(x, kind):
    """What the cache holds for x (f32 values)."""
    if kind == BF16:
        return bf16_value(bf16_bits(x)).astype(np.float64)
    return values(*quantise(x, kind), kind)


class Layout:
    """Byte offsets of a pool."""

    def __init__(self, kind, heads, dim, page):
        self.kind, self.heads, self.dim, self.page = kind, heads, dim, page
        self.row = {BF16: 2 * dim, FP8: dim, FP4: dim // 2}[kind]
        self.groups = 0 if kind == BF16 else dim // GROUP
        self.block = (2 * page * (self.row + self.groups) + 15) // 16 * 16

    def codes(self, page, head, slot, is_v):
        return (page * self.heads + head) * self.block + (is_v * self.page + slot) * self.row

    def scales(self, page, head, slot, is_v):
        return (page * self.heads + head) * self.block + 2 * self.page * self.row + (is_v * self.page + slot) * self.groups


def place(starts, lens, table, page_tokens, pages, t):
    """(page, slot) of new token t, or None."""
    for b in range(len(lens)):
        if starts[b] <= t < starts[b + 1]:
            pos = lens[b] - (starts[b + 1] - starts[b]) + (t - starts[b])
            if pos < 0 or pos // page_tokens >= table.shape[1]:
                return None
            page = table[b][pos // page_tokens]
            return (int(page), int(pos % page_tokens)) if 0 <= page < pages else None
    return None


def write(lay, pool, pages, k, v, starts, lens, table):
    """Writes k, v [tokens][heads][dim] (f32 values) into pool (uint8); returns the error count."""
    err = 0
    for t in range(k.shape[0]):
        at = place(starts, lens, table, lay.page, pages, t)
        if at is None:
            err += 1
            continue
        for is_v, x in enumerate((k, v)):
            for h in range(lay.heads):
                if lay.kind == BF16:
                    raw, sc = bf16_bits(x[t, h]).view(np.uint8), None
                else:
                    raw, sc = quantise(x[t, h], lay.kind)
                    err += int((sc == 255).sum())
                    if lay.kind == FP4:
                        raw = raw[0::2] | (raw[1::2] << 4)
                    o = lay.scales(at[0], h, at[1], is_v)
                    pool[o:o + lay.groups] = sc
                o = lay.codes(at[0], h, at[1], is_v)
                pool[o:o + lay.row] = raw
    return err


def attend(q, k, v, pos, scale, causal=True, window=0):
    """One sequence: q [n][heads][D], k and v [len][kv_heads][D], positions [n].  Returns (out, mass, spread):
    mass = sum p |v| / sum p, spread = the largest scale * sum |q_d k_d| over the keys a row sees."""
    n, heads, dim = q.shape
    kv_heads, share = k.shape[1], heads // k.shape[1]
    out, mass, spread = np.zeros((n, heads, dim)), np.zeros((n, heads, dim)), np.zeros((n, heads))
    j = np.arange(k.shape[0])
    for i in range(n):
        see = np.ones(len(j), bool)
        if causal:
            see &= j <= pos[i]
        if window:
            see &= j > pos[i] - window
        if not see.any():
            continue
        for h in range(heads):
            kk, vv = k[see, h // share], v[see, h // share]
            s = scale * (kk @ q[i, h])
            spread[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
            p = np.exp(s - s.max())
            out[i, h] = p @ vv / p.sum()
            mass[i, h] = p @ np.abs(vv) / p.sum()
    assert kv_heads * share == heads
    return out, mass, spread


def draw(w, noise):
    """argmax w / noise over w > 0 in f32, lowest index of equals; -1 if there is none."""
    with np.errstate(all="ignore"):
        ok = (w > 0) & (noise >= 0)
        s = np.where(ok, np.float32(w) / np.float32(noise), np.float32(-1))
    s = np.where(np.isnan(s), np.float32(-1), s)
    return int(np.argmax(s)) if s.max() >= 0 else -1


def verify(target, draft, tokens, counts, uniforms, noise):
    """Drafts checked one by one; everything in f32.  Returns (accepted, out)."""
    b, s1, vocab = target.shape
    accepted, out = np.zeros(b, np.int32), np.full((b, s1), -1, np.int32)
    for i in range(b):
        n = s1 - 1 if counts is None else min(max(int(counts[i]), 0), s1 - 1)
        a = 0
        while a < n:
            x = int(tokens[i, a])
            if not 0 <= x < vocab:
                break
            q = np.float32(1) if draft is None else np.float32(draft[i, a, x])
            if not np.float32(uniforms[i, a]) * q < np.float32(target[i, a, x]):
                break
            a += 1
        row = np.float32(target[i, a])
        rest = row
        if a < n:
            if draft is None:
                rest = row.copy()
                if 0 <= int(tokens[i, a]) < vocab:
                    rest[int(tokens[i, a])] = 0
            else:
                rest = row - np.float32(draft[i, a])
        last = draw(rest, noise[i])
        accepted[i] = a
        out[i, :a] = tokens[i, :a]
        out[i, a] = last if last >= 0 else draw(row, noise[i])
    return accepted, out
