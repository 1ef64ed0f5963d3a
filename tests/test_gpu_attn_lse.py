"""The rows' log-sums that attention gives beside its output, against the 64-bit oracle.

A score's error is below e = (3 D + 8) 2^-24 times scale * sum |q_d k_d| (f32 sums of exact products of bf16 terms): it moves
the log-sum by no more than its largest.  v_exp_f32 and the sum over n keys add a relative (n + 64) 2^-23 to the sum, as
much to its logarithm; v_log_f32, its sum with the maximum and the product with ln 2 are three roundings of numbers up to
the log-sum's size and the maximum's lead of 8: 2^-21 (|lse| + 8)."""

import math

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from oracle import serving as sv
from oracle import trees
from test_gpu_serving import Setup, check_attn, dev, f64, run_attn
from test_gpu_serving_forms import FORMS

pytestmark = pytest.mark.gpu


def run_lse(su, q, window=0, causal=True, max_len=None, err=None):
    out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
    chunk, max_len = max(max(su.new), 1), max(max(su.lens), 1) if max_len is None else max_len
    ws = torch.empty(wd.attn_workspace_bytes(su.desc, q.shape[1], q.shape[0], len(su.lens), chunk, max_len), dtype=torch.uint8, device="cuda")
    wd.attn(su.desc, su.pool, q, out, *su.plan(), ws, max_chunk=chunk, max_len=max_len, window=window, causal=causal, lse=lse, err_count=err)
    return out, lse


def seen(n, m, window, causal):
    gap = np.arange(m - n, m)[:, None] - np.arange(m)[None]
    see = gap >= 0 if causal else np.ones_like(gap, bool)
    return see & (gap < window) if window else see


def check_lse(got, q64, k, see, dim):
    _, _, spread, lse = trees.attend(q64, k, k, see, 1.0 / math.sqrt(dim))
    empty = np.isinf(lse)
    assert (got[empty] == -np.inf).all()
    bound = (3 * dim + 8) * 2.0 ** -24 * spread + (len(k) + 64) * 2.0 ** -23 + 2.0 ** -21 * (np.abs(lse) + 8)
    off = np.abs(got[~empty] - lse[~empty]) - bound[~empty]
    ok = bool(np.isfinite(got[~empty]).all() and (off <= 0).all())
    assert ok, off.max()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 256])
def test_log_sums_in_every_form(form, kind, dim):
    batch, kv_heads, share, chunk, longest, max_len = FORMS[form]
    seed = dim + len(form)
    rng = np.random.RandomState(seed)
    lens = rng.randint(1, longest + 1, batch)
    new = np.minimum(rng.randint(1, chunk + 1, batch), lens)
    lens[0], new[0] = longest, chunk
    lens[1], new[1] = chunk - 1, chunk                 # a row that sees nothing
    page = int(rng.choice([7, 16, 48]))
    su = Setup(kind, kv_heads, dim, page, new.tolist(), lens.tolist(), seed=seed, max_pages=-(-max(longest, chunk) // page) + 1)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(int(lens.sum()), kv_heads, dim, device="cuda", generator=gen) for _ in range(2))
    ends = np.concatenate(([0], np.cumsum(lens)))
    wd.kv_write(su.desc, su.pool, k, v, *su.plan(starts=ends))
    for dtype in (torch.bfloat16, torch.float32):
        q = (1.5 * torch.randn(int(new.sum()), kv_heads * share, dim, device="cuda", generator=gen)).to(dtype)
        for window, causal in ((0, True), (29, True), (0, False)):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            out, lse = run_lse(su, q, window, causal, max_len, err)
            again = run_lse(su, q, window, causal, max_len)
            assert err.item() == 0 and torch.equal(out, again[0]) and torch.equal(lse, again[1])
            plain = run_attn(su, q, dtype, window, causal, max_len=max_len)
            if dtype == torch.float32 or "split" not in form:
                assert torch.equal(out, plain)
            q64, got = f64(q), f64(lse)
            for b in sorted({0, 1, batch - 1}):
                a, n, m = su.starts[b], int(new[b]), int(lens[b])
                rows = sorted(set([0, n // 3, n - 2, n - 1]) & set(range(n)))
                at = [a + r for r in rows]
                h = b % kv_heads
                kk = sv.held(k[ends[b]:ends[b + 1], h:h + 1].cpu().numpy(), su.kind)
                mine = slice(h * share, (h + 1) * share)
                check_lse(got[at][:, mine], q64[at][:, mine], kk, seen(n, m, window, causal)[rows], dim)


@pytest.mark.parametrize("share", [1, 40])
def test_out_with_log_sums_stays_within_attentions_bound(share):
    su = Setup("fp8", 1, 128, 16, [9, 3], [800, 300], seed=31)
    caches = su.fill()
    q = dev(su.rng.randn(12, share, 128).astype(np.float32), torch.bfloat16)
    for max_len in (1, 100000):
        out, _ = run_lse(su, q, max_len=max_len)
        check_attn(su, caches, q, out, torch.bfloat16)


def test_log_sums_of_spoilt_rows():
    """A key that is not finite: NaN for the rows that see it, the others as they were."""
    su = Setup("fp8", 1, 64, 16, [6], [50], seed=32)
    su.fill()
    q = dev(su.rng.randn(6, 2, 64).astype(np.float32))
    _, clean = run_lse(su, q)
    bad = torch.full((1, 1, 64), math.nan, device="cuda")
    wd.kv_write(su.desc, su.pool, bad, bad, dev(np.array([0, 1], np.int32)), dev(np.array([48], np.int32)), dev(su.table))
    _, lse = run_lse(su, q)
    assert torch.equal(lse[:3], clean[:3]) and torch.isnan(lse[3:]).all()


def test_rows_of_no_sequence_are_left():
    su = Setup("fp8", 1, 64, 16, [2, 1], [50, 70], seed=33)
    su.fill()
    q = dev(su.rng.randn(8, 2, 64).astype(np.float32))
    for max_len in (1, 100000):
        ws = torch.empty(wd.attn_workspace_bytes(su.desc, 2, 8, 2, 4, max_len), dtype=torch.uint8, device="cuda")
        out, lse = torch.full_like(q, 9.0), torch.full((8, 2), 9.0, device="cuda")
        wd.attn(su.desc, su.pool, q, out, *su.plan(), ws, max_chunk=4, max_len=max_len, lse=lse)
        assert (lse[3:] == 9.0).all() and (out[3:] == 9.0).all() and (lse[:3] != 9.0).all()
