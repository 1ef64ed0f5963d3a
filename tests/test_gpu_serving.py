"""The serving operators on the GPU against the 64-bit oracle (oracle/serving.py).

The cache's bytes and the values read back are compared exactly.  Attention is compared within bounds
that follow from its roundings, per output, with A = sum p |v| / sum p:
* a score is a sum of D exact products of bf16 numbers (three terms a query for f32 queries) in f32: its
  error is below (3 D + 8) 2^-24 times scale * sum |q_d k_d|, and exp turns it into a relative error of p,
  in the numerator and in the sum of p: 2 A times that; v_exp_f32 and the sums over n keys add
  (n + 64) 2^-23 A;
* bf16 queries: p is rounded to bf16 in the numerator and in the sum alike, and the output is.  One
  rounding is 2^-8 relative at most and 2^-9 on average; the roundings of p enter as
  sum p d (v - out) / sum p, |d| <= 2^-8.  The bound takes 2 * 2^-9 A for them and the average for the
  output, 2^-9 |out|: less than the worst case of both together, which needs every rounding at its
  worst with the sign of v - out;
* f32 queries: three bf16 terms of p leave 2^-26, below the term above."""

import math

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from oracle import serving as sv

pytestmark = pytest.mark.gpu
KINDS = {"bf16": wd.KV_BF16, "fp8": wd.KV_FP8, "fp4": wd.KV_FP4}


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.double().cpu().numpy()


class Setup:
    """A batch over a pool: lens and new-token numbers given, pages in random order."""

    def __init__(self, kind, kv_heads, dim, page, new, lens, seed=0, spare=2, max_pages=None):
        self.rng = np.random.RandomState(seed)
        self.kind, self.kv_heads, self.dim, self.page = KINDS[kind], kv_heads, dim, page
        self.new, self.lens = list(new), list(lens)
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        width = max(max(need), 1) if max_pages is None else max_pages
        ids = self.rng.permutation(self.pages)
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        self.desc = wd.make_kv_desc(self.kind, kv_heads, dim, page, self.pages)
        self.lay = sv.Layout(self.kind, kv_heads, dim, page)
        # unwritten places hold bytes that read as NaN
        self.pool = torch.full((wd.kv_pool_bytes(self.desc),), 255, dtype=torch.uint8, device="cuda")
        assert self.pool.numel() == self.pages * kv_heads * self.lay.block

    def plan(self, starts=None, lens=None):
        return (dev(self.starts if starts is None else np.asarray(starts, np.int32)),
                dev(np.asarray(self.lens if lens is None else lens, np.int32)), dev(self.table))

    def fill(self, bf16=True):
        """Writes every sequence's whole cache; returns the held values per sequence."""
        total = sum(self.lens)
        k = self.rng.randn(total, self.kv_heads, self.dim).astype(np.float32)
        v = self.rng.randn(total, self.kv_heads, self.dim).astype(np.float32)
        ends = np.concatenate(([0], np.cumsum(self.lens))).astype(np.int32)
        if total:
            wd.kv_write(self.desc, self.pool, dev(k), dev(v), *self.plan(starts=ends))
        hk, hv = sv.held(k, self.kind), sv.held(v, self.kind)
        return [(hk[ends[b]:ends[b + 1]], hv[ends[b]:ends[b + 1]]) for b in range(len(self.lens))]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,dim,page", [(1, 32, 1), (2, 128, 16), (3, 96, 7), (5, 256, 48), (8, 64, 5)])
@pytest.mark.parametrize("wide", [True, False])
def test_write_gives_the_oracles_bytes(kind, dtype, heads, dim, page, wide):
    su = Setup(kind, heads, dim, page, [3, 0, 1, 17, 2], [9, 4, 1, 17, 70], seed=dim + page)
    n = int(su.starts[-1])
    # slices of a fused projection; not wide: rows that start off 16 bytes
    pad = 8 if wide else 3
    fused = torch.zeros(n, 2 * heads + 1, dim + pad, device="cuda", dtype=dtype)
    scale = 2.0 ** su.rng.randint(-20, 20, (n, 2 * heads + 1, 1))
    fused[:, :, :dim] = dev((su.rng.randn(n, 2 * heads + 1, dim) * scale).astype(np.float32)).to(dtype)
    k, v = fused[:, 1:heads + 1, :dim], fused[:, heads + 1:, :dim]
    want = su.pool.cpu().numpy().copy()
    assert sv.write(su.lay, want, su.pages, k.float().cpu().numpy(), v.float().cpu().numpy(), su.starts, su.lens, su.table) == 0
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    wd.kv_write(su.desc, su.pool, k, v, *su.plan(), err_count=err)
    assert np.array_equal(su.pool.cpu().numpy(), want)
    assert err.item() == 0
    for out_dtype in (torch.float32, torch.bfloat16):
        # into a wider tensor: strides of the output
        out = torch.full((2, n, heads, dim + pad), 7.0, device="cuda", dtype=out_dtype)
        wd.kv_read(su.desc, su.pool, out[0][..., :dim], out[1][..., :dim], *su.plan(), err_count=err)
        for got, x in zip(out, (k, v)):
            assert np.array_equal(f64(got[..., :dim]), sv.held(x.float().cpu().numpy(), su.kind))
            assert (got[..., dim:] == 7.0).all()
    assert err.item() == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_write_of_extreme_values(kind):
    su = Setup(kind, 2, 64, 16, [8], [8], seed=5)
    top = np.finfo(np.float32).max
    k = su.rng.randn(8, 2, 64).astype(np.float32)
    v = su.rng.randn(8, 2, 64).astype(np.float32)
    k[0] = 0.0
    k[1] *= 1e-39
    k[2, 0, 5] = np.nan
    k[3, 1, 40] = np.inf
    v[3, 0, 0] = -np.inf
    k[4] = -0.0
    k[5, 0, :4] = [top, -top, top / 2, 1e30]
    v[6, 1, 32:] = np.tile([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5], 4)     # ties of e2m1
    v[7, 0, :32] = np.tile([448, 17, 19, 2.0 ** -10, 3 * 2.0 ** -10, -464, 1, 0], 4)   # past the top, ties and subnormals of e4m3
    want = su.pool.cpu().numpy().copy()
    bad = sv.write(su.lay, want, su.pages, k, v, su.starts, su.lens, su.table)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    wd.kv_write(su.desc, su.pool, dev(k), dev(v), *su.plan(), err_count=err)
    got = su.pool.cpu().numpy()
    if su.kind == wd.KV_BF16:       # a NaN's payload is not fixed
        a, b = got.view(np.uint16), want.view(np.uint16)
        nan = (b & 0x7FFF) > 0x7F80
        assert ((a[nan] & 0x7FFF) > 0x7F80).all() and np.array_equal(a[~nan], b[~nan])
    else:
        assert np.array_equal(got, want)
    assert err.item() == bad == (0 if su.kind == wd.KV_BF16 else 3)
    out = torch.empty(2, 8, 2, 64, device="cuda")
    wd.kv_read(su.desc, su.pool, out[0], out[1], *su.plan())
    assert np.array_equal(f64(out[0]), sv.held(k, su.kind), equal_nan=True)
    assert np.array_equal(f64(out[1]), sv.held(v, su.kind), equal_nan=True)


def test_tokens_without_a_place_are_counted_and_not_written():
    su = Setup("fp8", 2, 64, 4, [5, 2, 3], [3, 2, 12], seed=2)     # 5 new tokens of 3: two positions are negative
    su.table[2, 2] = su.pages                                       # a page outside the pool: positions 8..11
    n = 10
    k, v = su.rng.randn(2, n, 2, 64).astype(np.float32)
    want = su.pool.cpu().numpy().copy()
    bad = sv.write(su.lay, want, su.pages, k, v, su.starts, su.lens, su.table)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    wd.kv_write(su.desc, su.pool, dev(k), dev(v), *su.plan(), err_count=err)
    assert np.array_equal(su.pool.cpu().numpy(), want) and err.item() == bad == 5
    out = torch.full((2, n, 2, 64), 3.0, device="cuda")
    wd.kv_read(su.desc, su.pool, out[0], out[1], *su.plan(), err_count=err)
    there = np.array([0, 0, 1, 1, 1, 1, 1, 0, 0, 0], bool)
    assert np.array_equal(f64(out[0])[there], sv.held(k, su.kind)[there]) and (f64(out)[:, ~there] == 0).all()
    assert err.item() == 10


def run_attn(su, q, dtype, window=0, causal=True, max_len=None, stream=None, out=None, max_chunk=None, plan=None, err=None, scale=None):
    q = q if isinstance(q, torch.Tensor) else dev(q, dtype)
    n, heads, _ = q.shape
    max_chunk = max(su.new + [1]) if max_chunk is None else max_chunk
    max_len = max(su.lens + [1]) if max_len is None else max_len
    out = torch.full((n, heads, su.dim), 99.0, device="cuda", dtype=dtype) if out is None else out
    size = wd.attn_workspace_bytes(su.desc, heads, n, len(su.lens), max_chunk, max_len)
    # what the workspace holds before the call must not matter
    ws = torch.full((max(size, 16),), 255, dtype=torch.uint8, device="cuda")
    wd.attn(su.desc, su.pool, q, out, *(plan or su.plan()), ws, max_chunk=max_chunk, max_len=max_len, window=window,
            causal=causal, err_count=err, stream=stream, scale=scale)
    return out


def check_attn(su, caches, q, out, dtype, window=0, causal=True, scale=None):
    """Compares every sequence's rows with the oracle within the module's bound."""
    q64, got = f64(q if isinstance(q, torch.Tensor) else dev(q, dtype)), f64(out)
    scale = 1.0 / math.sqrt(su.dim) if scale is None else scale
    for b, (k, v) in enumerate(caches):
        a, e = su.starts[b], su.starts[b + 1]
        pos = su.lens[b] - (e - a) + np.arange(e - a)
        ref, mass, spread = sv.attend(q64[a:e], k, v, pos, scale, causal, window)
        rel = 2 * (3 * su.dim + 8) * 2.0 ** -24 * spread[..., None] + (len(k) + 64) * 2.0 ** -23
        bound = mass * rel
        if dtype == torch.bfloat16:
            bound = bound + 2 * 2.0 ** -9 * mass + 2.0 ** -9 * (np.abs(ref) + bound)
        off = np.abs(got[a:e] - ref) - bound
        assert np.isfinite(got[a:e]).all() and (off <= 0).all(), (b, np.abs(got[a:e] - ref).max(), off.max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind,kv_heads,share,dim,page,new,lens,window", [
    ("bf16", 1, 1, 32, 1, [1], [1], 0),                                    # one token that sees itself
    ("fp8", 2, 1, 64, 16, [1, 1, 0, 1], [1, 63, 5, 300], 0),               # decode; a sequence with nothing new
    ("fp4", 1, 8, 128, 16, [1, 1], [64, 513], 0),                          # shared heads
    ("fp8", 3, 4, 96, 7, [1, 3, 8], [5, 130, 257], 0),                     # drafts, odd pages, a dim between the tiles
    ("bf16", 2, 2, 160, 48, [2, 17], [2, 200], 0),                         # whole prompt; dim 160
    ("fp4", 2, 5, 256, 16, [13, 1], [100, 129], 0),                        # 65 rows
    ("fp8", 1, 6, 128, 64, [70, 33], [70, 201], 0),                        # several row blocks
    ("fp4", 4, 1, 64, 128, [150, 129, 1], [150, 400, 128], 0),
    ("bf16", 1, 2, 256, 32, [90], [333], 0),
    ("fp8", 2, 3, 128, 16, [40, 7, 1], [300, 7, 200], 9),                  # windows
    ("fp4", 1, 1, 64, 48, [130], [400], 100),
    ("bf16", 2, 1, 96, 16, [5, 1], [70, 90], 1),                           # each row sees itself alone
    ("fp8", 1, 4, 128, 16, [1, 2], [0, 1], 0),                             # lens shorter than the chunk: empty rows
    ("fp8", 32, 1, 32, 4, [1] * 70, list(range(70)), 0),                   # workgroups enough without a split
    ("fp4", 1, 70, 64, 16, [1, 1], [65, 1000], 0),                         # more than 64 rows of one token
])
def test_attention(kind, kv_heads, share, dim, page, new, lens, window, dtype):
    su = Setup(kind, kv_heads, dim, page, new, lens, seed=dim + len(new), max_pages=max(1, -(-max(lens) // page)) + 2)
    caches = su.fill()
    q = su.rng.randn(sum(new), kv_heads * share, dim).astype(np.float32) * 1.5
    for max_len in (None, 1, 100000):       # the split rule: as it comes, none, many
        out = run_attn(su, q, dtype, window, max_len=max_len)
        check_attn(su, caches, q, out, dtype, window)
        again = run_attn(su, q, dtype, window, max_len=max_len)
        assert torch.equal(out, again)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_attention_without_causal_mask(kind):
    su = Setup(kind, 2, 128, 16, [5, 40], [37, 150], seed=11)
    caches = su.fill()
    q = su.rng.randn(45, 4, 128).astype(np.float32)
    for window in (0, 20):
        check_attn(su, caches, q, run_attn(su, q, torch.bfloat16, window, causal=False), torch.bfloat16, window, causal=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_strides_and_alignment(dtype):
    su = Setup("fp8", 2, 64, 16, [3, 30], [40, 90], seed=12)
    caches = su.fill()
    base = torch.randn(33, 7, 64 + 3, device="cuda", dtype=dtype)
    q = base[:, 2:6, 1:65]                           # rows that start off 16 bytes
    wide = torch.full((33, 6, 72), 5.0, device="cuda", dtype=dtype)
    run_attn(su, q, dtype, out=wide[:, 1:5, 4:68])
    check_attn(su, caches, q, wide[:, 1:5, 4:68], dtype)
    keep = torch.ones_like(wide, dtype=torch.bool)
    keep[:, 1:5, 4:68] = False
    assert (wide[keep] == 5.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_of_large_scores_and_a_late_maximum(dtype):
    # maxima that rise along the keys (every tile rescales), and scores far past the range of exp in f32
    su = Setup("bf16", 1, 64, 16, [2, 70], [700, 300], seed=13)
    total = sum(su.lens)
    ramp = np.concatenate([np.linspace(0, 1, n) for n in su.lens])[:, None, None]
    k = (np.ones((total, 1, 64)) * ramp * 8).astype(np.float32)
    v = su.rng.randn(total, 1, 64).astype(np.float32)
    ends = np.concatenate(([0], np.cumsum(su.lens))).astype(np.int32)
    wd.kv_write(su.desc, su.pool, dev(k), dev(v), *su.plan(starts=ends))
    hk, hv = sv.held(k, 0), sv.held(v, 0)
    caches = [(hk[ends[b]:ends[b + 1]], hv[ends[b]:ends[b + 1]]) for b in range(2)]
    for sign in (1.0, -1.0):
        q = (sign * np.abs(su.rng.randn(72, 2, 64)) * 4).astype(np.float32)
        for max_len in (1, 100000):
            check_attn(su, caches, q, run_attn(su, q, dtype, max_len=max_len), dtype)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("new", [6, 140])
@pytest.mark.parametrize("max_len", [1, 100000])
def test_what_a_row_does_not_see_has_no_effect(kind, new, max_len):
    """A key and a value that are not finite, at a place that only later rows see."""
    su = Setup(kind, 2, 64, 16, [new], [new + 50], seed=14)
    caches = su.fill()
    q = su.rng.randn(new, 4, 64).astype(np.float32)
    clean = run_attn(su, q, torch.bfloat16, max_len=max_len)
    at = 50 + new // 2                                 # position of the token that is spoilt
    k, v = (torch.randn(1, 2, 64, device="cuda") for _ in range(2))
    v[0, 0, 40] = math.inf
    v[0, 1, 3] = math.nan
    wd.kv_write(su.desc, su.pool, k, v, dev(np.array([0, 1], np.int32)), dev(np.array([at + 1], np.int32)), dev(su.table))
    out = run_attn(su, q, torch.bfloat16, max_len=max_len)
    first = at - 50                                    # the first row that sees it
    assert torch.equal(out[:first], clean[:first])
    got = f64(out[first:])
    if su.kind == wd.KV_BF16:
        assert (got[:, :2, 40] == np.inf).all() and np.isnan(got[:, 2:, 3]).all()
        rest = np.ones((4, 64), bool)
        rest[:2, 40] = rest[2:, 3] = False
    else:                                              # the value's group of 32 channels
        assert np.isnan(got[:, :2, 32:]).all() and np.isnan(got[:, 2:, :32]).all()
        rest = np.ones((4, 64), bool)
        rest[:2, 32:] = rest[2:, :32] = False
    assert np.isfinite(got[:, rest]).all()
    # a key that is not finite spoils the rows that see it, and no others
    k[0, 0, 1] = math.nan
    wd.kv_write(su.desc, su.pool, k, v.nan_to_num(0.0, 0.0), dev(np.array([0, 1], np.int32)), dev(np.array([at + 1], np.int32)),
                dev(su.table))
    out = run_attn(su, q, torch.bfloat16, max_len=max_len)
    assert torch.equal(out[:first], clean[:first]) and torch.isnan(out[first:, :2]).all() and torch.isfinite(out[first:, 2:]).all()
    assert len(caches) == 1


def test_a_window_hides_what_lies_before_it():
    su = Setup("fp8", 1, 64, 16, [4], [200], seed=15)
    su.fill()
    q = su.rng.randn(4, 2, 64).astype(np.float32)
    clean = run_attn(su, q, torch.bfloat16, window=30)
    bad = torch.full((160, 1, 64), math.nan, device="cuda")
    wd.kv_write(su.desc, su.pool, bad, bad, dev(np.array([0, 160], np.int32)), dev(np.array([160], np.int32)), dev(su.table))
    assert torch.equal(run_attn(su, q, torch.bfloat16, window=30), clean)


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_a_pool_past_32_bits(kind):
    """Pages whose offsets pass 2^32 bytes."""
    su = Setup(kind, 2, 128, 16, [3], [100], seed=16)
    pages = (5 << 30) // (2 * su.lay.block)
    su.desc = wd.make_kv_desc(su.kind, 2, 128, 16, pages)
    su.pages = pages
    su.pool = torch.empty(wd.kv_pool_bytes(su.desc), dtype=torch.uint8, device="cuda")
    assert su.pool.numel() > 1 << 32
    su.table[0] = pages - 1 - np.arange(su.table.shape[1])
    caches = su.fill()
    q = su.rng.randn(3, 4, 128).astype(np.float32)
    check_attn(su, caches, q, run_attn(su, q, torch.bfloat16), torch.bfloat16)
    out = torch.empty(2, 100, 2, 128, device="cuda")
    wd.kv_read(su.desc, su.pool, out[0], out[1], *su.plan(starts=[0, 100]))
    assert np.array_equal(f64(out[0]), caches[0][0]) and np.array_equal(f64(out[1]), caches[0][1])


def test_arrays_that_do_not_fit_are_bounded_and_counted():
    su = Setup("fp8", 2, 64, 16, [2, 2], [40, 40], seed=17)
    su.fill()
    q = su.rng.randn(4, 2, 64).astype(np.float32)
    fine = run_attn(su, q, torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_attn(su, q, torch.bfloat16, err=err)
    assert err.item() == 0
    for starts, lens in (([0, 2, 900], [40, 40]), ([-5, 2, 4], [40, 40]), ([0, 2, 4], [40, 1 << 29]), ([0, 2, 4], [40, -7]),
                         ([3, 1, 4], [40, 40])):
        err.zero_()
        run_attn(su, q, torch.bfloat16, plan=su.plan(starts, lens), err=err)
        assert err.item() > 0, (starts, lens)
    for page in (-1, su.pages, 1 << 30, -2 ** 31):
        table = su.table.copy()
        table[1, 1] = page
        err.zero_()
        out = run_attn(su, q, torch.bfloat16, plan=(dev(su.starts), dev(np.array(su.lens, np.int32)), dev(table)), err=err)
        assert err.item() > 0 and torch.equal(out[:2], fine[:2]) and torch.isfinite(out).all()
    err.zero_()
    run_attn(su, dev(su.rng.randn(100, 2, 64).astype(np.float32), torch.bfloat16), torch.bfloat16,
             plan=su.plan([0, 90, 100], [40, 90]), max_chunk=50, err=err)     # more rows than max_chunk
    assert err.item() > 0


def test_empty_calls():
    su = Setup("fp8", 2, 64, 16, [0, 0], [5, 0], seed=18)
    empty = torch.empty(0, 2, 64, device="cuda")
    wd.kv_write(su.desc, su.pool, empty, empty, *su.plan())
    wd.kv_read(su.desc, su.pool, empty, empty, *su.plan())
    assert run_attn(su, empty, torch.float32).shape == (0, 2, 64)


def test_another_stream_and_a_captured_graph():
    su = Setup("fp8", 2, 128, 16, [1, 1], [900, 300], seed=19)
    caches = su.fill()
    plan = su.plan()
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    kv = torch.randn(2, 2, 2, 128, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(max(16, wd.attn_workspace_bytes(su.desc, 8, 2, 2, 1, 900)), dtype=torch.uint8, device="cuda")
    target, draft = torch.rand(2, 4, 999, device="cuda"), torch.rand(2, 3, 999, device="cuda")
    tokens = torch.randint(0, 999, (2, 3), device="cuda", dtype=torch.int32)
    uni, noise = torch.rand(2, 3, device="cuda"), torch.rand(2, 999, device="cuda") + 0.1
    acc, tok = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(2, 4, dtype=torch.int32, device="cuda")
    dws = torch.empty(wd.draft_workspace_bytes(2, 999), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        wd.kv_write(su.desc, su.pool, kv[0], kv[1], *plan, stream=stream)
        wd.attn(su.desc, su.pool, q, out, *plan, ws, max_chunk=1, max_len=900, stream=stream)
        wd.draft_verify(target, draft, tokens, uni, noise, acc, tok, dws, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side.cuda_stream)
    side.synchronize()
    for b in range(2):
        caches[b][0][-1], caches[b][1][-1] = (sv.held(x[b].cpu().numpy(), su.kind) for x in kv)
    check_attn(su, caches, q, out, torch.bfloat16)
    first = [out.clone(), acc.clone(), tok.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        q.normal_()
        uni.uniform_()
        kv.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [out.clone(), acc.clone(), tok.clone()]
        out.zero_(), acc.zero_(), tok.zero_()
        step()
        assert all(torch.equal(x, y) for x, y in zip(got, (out, acc, tok))), i
    assert not torch.equal(first[0], out)


def draft_case(b, s, vocab, dtype, seed, certain=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    logits = 2 * torch.randn(b, s + 1, vocab, device="cuda", generator=gen)
    target = torch.softmax(logits, -1).to(dtype)
    draft = torch.softmax(logits[:, :s] + 0.5 * torch.randn(b, s, vocab, device="cuda", generator=gen), -1).to(dtype)
    noise = torch.empty(b, vocab, device="cuda").exponential_(generator=gen).clamp_(min=1e-30)
    tokens = draft.float().argmax(-1).int()
    return target, None if certain else draft, tokens, torch.rand(b, s, device="cuda", generator=gen), noise


def run_draft(target, draft, tokens, uni, noise, counts=None, err=None):
    b, s1, vocab = target.shape
    acc = torch.full((b,), 77, dtype=torch.int32, device="cuda")
    out = torch.full((b, s1), 77, dtype=torch.int32, device="cuda")
    ws = torch.full((wd.draft_workspace_bytes(b, vocab),), 255, dtype=torch.uint8, device="cuda")
    wd.draft_verify(target, draft, tokens, uni, noise, acc, out, ws, counts=counts, err_count=err)
    return acc.cpu().numpy(), out.cpu().numpy()


def check_draft(case, counts=None, errors=0):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc, out = run_draft(*case, counts=counts, err=err)
    host = [None if t is None else t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy() for t in case]
    want = sv.verify(host[0], host[1], host[2], None if counts is None else counts.cpu().numpy(), host[3], host[4])
    assert np.array_equal(acc, want[0]) and np.array_equal(out, want[1])
    assert err.item() == errors
    return acc, out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,s,vocab", [(1, 0, 1), (1, 4, 7), (3, 1, 2049), (5, 7, 32000), (40, 3, 1001), (2, 63, 300),
                                       (1, 2, 100003), (600, 2, 50), (3, 2, 8193)])
@pytest.mark.parametrize("certain", [False, True])
def test_draft_verify(b, s, vocab, dtype, certain):
    case = draft_case(b, s, vocab, dtype, seed=b + s, certain=certain)
    check_draft(case)
    if s:
        counts = torch.randint(0, s + 1, (b,), device="cuda", dtype=torch.int32)
        acc, out = check_draft(case, counts)
        assert (acc <= counts.cpu().numpy()).all()


def test_draft_verify_edges():
    target, draft, tokens, uni, noise = draft_case(6, 2, 5000, torch.float32, seed=9)
    noise[0] = 1.0                        # equal noise and equal weights: ties
    target[0], draft[0] = 0.25, 0.125
    uni[0] = 0.999
    draft[1] = target[1, :2]              # the rest is empty: drawn from the target alone
    uni[1] = 1.0
    target[2, :, ::2] = math.nan          # NaN weights are never drawn
    draft[2, 0, tokens[2, 0].item()] = math.nan
    target[3] = 0.0                       # nothing to draw
    tokens[4, 0] = 5000                   # outside the vocabulary
    noise[5, :4000] = math.nan
    noise[5, 4500] = 0.0
    acc, out = check_draft((target, draft, tokens, uni, noise), errors=2)
    assert out[3, 0] == -1 and acc[4] == 0 and out[5, acc[5]] >= 4000
    check_draft((target, draft, tokens, uni, noise), torch.tensor([2, 9, -1, 0, 1, 2], dtype=torch.int32, device="cuda"), errors=4)
