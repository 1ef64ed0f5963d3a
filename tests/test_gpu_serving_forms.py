"""Every form in which the attention and the cache's calls are launched, at sizes that select it: attention of few rows
by one, four and eight waves a row block, in one and two column tiles, whole and split; of many rows by four and eight
waves; the cache's kernels with four tokens a wave.  Attention is compared with the 64-bit oracle at some rows and heads
of some sequences, within the bounds that test_gpu_serving.py derives; the cache exactly."""

import math

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from oracle import serving as sv
from test_gpu_serving import Setup, dev, f64, run_attn

pytestmark = pytest.mark.gpu


class Batch(Setup):
    """Sequences of given lengths, their caches filled; the oracle's values of some of them."""

    def __init__(self, kind, kv_heads, dim, page, new, lens, seed, sample):
        super().__init__(kind, kv_heads, dim, page, new, lens, seed=seed, max_pages=-(-max(lens) // page) + 1)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        k, v = (torch.randn(sum(lens), kv_heads, dim, device="cuda", generator=gen) for _ in range(2))
        ends = np.concatenate(([0], np.cumsum(lens)))
        wd.kv_write(self.desc, self.pool, k, v, *self.plan(starts=ends))
        self.held = {b: [sv.held(x[ends[b]:ends[b + 1]].cpu().numpy(), self.kind) for x in (k, v)] for b in sample}

    def check(self, q, out, dtype, window, causal):
        heads = q.shape[1]
        share, scale = heads // self.kv_heads, 1.0 / math.sqrt(self.dim)
        for b, (k, v) in self.held.items():
            n = self.new[b]
            rows = sorted(set([0, n // 3, n - 2, n - 1]) & set(range(n)))
            if not rows:
                continue
            hs = sorted({0, self.kv_heads - 1})
            at = [self.starts[b] + r for r in rows]
            pos = np.array([self.lens[b] - n + r for r in rows])
            pick = [h * share + g for h in hs for g in range(share)]
            q64, got = f64(q[at][:, pick]), f64(out[at][:, pick])
            ref, mass, spread = sv.attend(q64, k[:, hs], v[:, hs], pos, scale, causal, window)
            bound = mass * (2 * (3 * self.dim + 8) * 2.0 ** -24 * spread[..., None] + (len(k) + 64) * 2.0 ** -23)
            if dtype == torch.bfloat16:
                bound = bound + 2 * 2.0 ** -9 * mass + 2.0 ** -9 * (np.abs(ref) + bound)
            off = np.abs(got - ref) - bound
            assert np.isfinite(got).all() and (off <= 0).all(), (b, np.abs(got - ref).max(), off.max())


# name: (sequences, key heads, query heads of each, new tokens, longest length, max_len that is told)
FORMS = {
    "eight waves a row block": (5, 2, 5, 3, 290, 290),
    "four waves a row block": (65, 4, 4, 3, 200, 1),
    "four waves a row block, split": (5, 3, 4, 3, 700, 100000),
    "a wave a row block": (257, 8, 3, 2, 90, 90),
    "two column tiles": (5, 2, 7, 4, 300, 1),
    "two column tiles, split": (3, 2, 11, 5, 600, 100000),
    "two column tiles, a wave a row block": (257, 8, 5, 5, 60, 60),
    "many rows, four waves": (3, 2, 5, 23, 300, 1),
    "many rows, four waves, split": (2, 2, 3, 41, 700, 100000),
    "many rows, eight waves": (33, 8, 7, 19, 200, 200),
    "many rows, eight waves, split": (17, 8, 3, 101, 420, 100000),
}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 256])
def test_attention_in_every_form(form, kind, dim):
    batch, kv_heads, share, chunk, longest, max_len = FORMS[form]
    seed = dim + len(form)
    rng = np.random.RandomState(seed)
    lens = rng.randint(1, longest + 1, batch)
    new = np.minimum(rng.randint(1, chunk + 1, batch), lens)
    lens[0], new[0] = longest, chunk
    lens[1], new[1] = chunk - 1, chunk                 # a row that sees nothing
    sample = [0, 1, batch // 2, batch - 1]
    page = int(rng.choice([7, 16, 48]))
    su = Batch(kind, kv_heads, dim, page, new.tolist(), lens.tolist(), seed, sample)
    for dtype in (torch.bfloat16, torch.float32):
        q = 1.5 * torch.randn(int(new.sum()), kv_heads * share, dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
        q = q.to(dtype)
        for window, causal in ((0, True), (29, True), (0, False)):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = run_attn(su, q, dtype, window, causal, max_len=max_len, err=err)
            assert err.item() == 0
            su.check(q, out, dtype, window, causal)
        assert torch.equal(out, run_attn(su, q, dtype, window, causal, max_len=max_len))


# tokens * heads * channels from 2^22 on, token counts that no wave's or workgroup's share divides
@pytest.mark.parametrize("heads,dim,page,tokens", [(8, 128, 16, 4111), (32, 256, 48, 519), (1, 32, 7, 131075), (3, 96, 64, 14573)])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("wide", [True, False])
def test_cache_with_four_tokens_a_wave(heads, dim, page, tokens, kind, dtype, wide):
    assert tokens * heads * dim >= 1 << 22
    lens = [tokens // 3, 5, 0, tokens - tokens // 3 - 5 - 1, 1]
    new = [n - n // 7 for n in lens]                  # the last of each sequence's tokens
    extra = tokens - sum(new)
    lens[3], new[3] = lens[3] + extra, new[3] + extra
    assert sum(new) == tokens
    su = Setup(kind, heads, dim, page, new, lens, seed=heads + dim)
    gen = torch.Generator(device="cuda").manual_seed(dim)
    pad = 8 if wide else 3                            # not wide: rows that start off 16 bytes
    fused = torch.randn(tokens, 2 * heads, dim + pad, device="cuda", generator=gen).to(dtype)
    fused[7, 0, 3], fused[11, heads, 5] = math.inf, math.nan
    k, v = fused[:, :heads, :dim], fused[:, heads:, :dim]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    wd.kv_write(su.desc, su.pool, k, v, *su.plan(), err_count=err)
    assert err.item() == (0 if kind == "bf16" else 2)
    # the same bytes, and no others, as the kernels write that take a token a wave
    whole = su.pool.clone()
    su.pool.fill_(255)
    most = ((1 << 22) - 1) // (heads * dim)
    plans = []
    for b in range(len(lens)):
        a = int(su.starts[b])
        for i in range(0, new[b], most):
            n = min(most, new[b] - i)
            plans.append((a + i, n, dev(np.array([0, n], np.int32)), dev(np.array([lens[b] - new[b] + i + n], np.int32)),
                          dev(su.table[b:b + 1])))
    for a, n, *plan in plans:
        wd.kv_write(su.desc, su.pool, k[a:a + n], v[a:a + n], *plan)
    assert torch.equal(whole, su.pool)
    some = np.unique(np.concatenate((np.arange(20), tokens - 1 - np.arange(20), np.random.RandomState(1).randint(0, tokens, 60))))
    for out_dtype in (torch.float32, torch.bfloat16):
        out = torch.full((2, tokens, heads, dim + pad), 7.0, device="cuda", dtype=out_dtype)
        err.zero_()
        wd.kv_read(su.desc, su.pool, out[0][..., :dim], out[1][..., :dim], *su.plan(), err_count=err)
        assert err.item() == 0 and (out[..., dim:] == 7.0).all()
        for got, x in zip(out, (k, v)):
            assert np.array_equal(f64(got[some][..., :dim]), sv.held(x[some].float().cpu().numpy(), su.kind), equal_nan=True)
        apart = torch.empty(2, tokens, heads, dim, device="cuda", dtype=out_dtype)
        for a, n, *plan in plans:
            wd.kv_read(su.desc, su.pool, apart[0][a:a + n], apart[1][a:a + n], *plan)
        assert torch.equal(torch.nan_to_num(out[..., :dim], 1e9), torch.nan_to_num(apart, 1e9))


