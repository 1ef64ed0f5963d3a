"""Eviction from the paged cache on the GPU against the oracle (oracle/eviction.py): choices and moves equal, the weights
within bounds that follow from their roundings.  A score is a sum of D exact products of bf16 numbers (three terms a query
for f32 queries) in f32, (3 D + 8) 2^-24 of scale * sum |q_d k_d| off at most; its product with scale log2(e), the log-sum's with
log2(e), their difference and v_exp_f32 each round numbers up to |s| and |lse| in f32: 2^-21 (|s| + |lse| + 1) in all, a relative
error of p like the first.  The sum over R rows adds (R + 8) 2^-24 of it, the last addition 2^-24 of the weight."""

import math

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from oracle import eviction as ev
from oracle import serving as sv
from test_gpu_attn_lse import run_lse, seen
from test_gpu_serving import Setup, dev, f64

pytestmark = pytest.mark.gpu


def places(su, b, m):
    at = np.arange(m)
    return su.table[b][at // su.page], at % su.page


def run_weigh(su, weights, q, lse, window=0, causal=True, fresh=False, max_len=None, err=None, plan=None, stream=None, max_chunk=None):
    wd.kv_weigh(su.desc, su.pool, weights, q, lse, *(plan or su.plan()), max_chunk=max(max(su.new), 1) if max_chunk is None else max_chunk,
                max_len=max(max(su.lens), 1) if max_len is None else max_len, window=window, causal=causal, fresh=fresh, err_count=err,
                stream=stream)


def true_lse(su, caches, q64, window, causal):
    """The rows' log-sums as f32, from the oracle."""
    out = np.zeros(q64.shape[:2], np.float32)
    for b, (k, _) in enumerate(caches):
        a, e = su.starts[b], su.starts[b + 1]
        if e > a:
            out[a:e] = true_lse_of(q64[a:e], k, seen(e - a, su.lens[b], window, causal), su.dim)
    return out


def true_lse_of(q, k, see, dim):
    heads = q.shape[1]
    out = np.full(q.shape[:2], -np.inf)
    for h in range(heads):
        s = q[:, h] @ k[:, h * k.shape[1] // heads].T / math.sqrt(dim)
        s = np.where(see, s, -np.inf)
        top = s.max(-1, initial=-np.inf)
        top = np.where(np.isfinite(top), top, 0.0)
        with np.errstate(divide="ignore"):
            out[:, h] = np.log(np.exp(s - top[:, None]).sum(-1)) + top
    return out.astype(np.float32)


def check_weights(su, caches, q64, lse, before, after, window, causal, fresh, heads=None):
    touched = np.zeros(before.shape, bool)
    share = q64.shape[1] // su.kv_heads
    for b, (k, _) in enumerate(caches):
        a, e = su.starts[b], su.starts[b + 1]
        n, m = e - a, su.lens[b]
        if n == 0 or m == 0:
            continue
        see = seen(n, m, window, causal)
        sums, slack = ev.weigh(q64[a:e], k, lse[a:e].astype(np.float64), see, 1.0 / math.sqrt(su.dim))
        page, slot = places(su, b, m)
        old = before[page, :, slot].astype(np.float64)
        starts_anew = (np.arange(m) >= m - n)[:, None] | fresh
        want = np.where(starts_anew, 0.0, old) + sums
        bound = slack + sums * (n * share + 8) * 2.0 ** -24 + 2.0 ** -24 * np.abs(want)
        got = after[page, :, slot].astype(np.float64)
        ok = bool(np.isfinite(got).all() and (np.abs(got - want) <= bound).all())
        assert ok, (b, np.abs(got - want).max(), (np.abs(got - want) - bound).max())
        touched[page, :, slot] = True
    assert np.array_equal(before[~touched].view(np.uint32), after[~touched].view(np.uint32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind,kv_heads,share,dim,page,new,lens,window,causal", [
    ("bf16", 1, 1, 32, 1, [1], [1], 0, True),                                  # one token that sees itself
    ("fp8", 2, 1, 64, 16, [1, 1, 0, 1], [1, 63, 5, 300], 0, True),             # a step; a sequence with nothing new
    ("fp4", 1, 8, 128, 16, [1, 1], [64, 513], 0, True),                        # shared heads
    ("fp8", 3, 4, 96, 7, [1, 3, 8], [5, 130, 257], 0, True),                   # odd pages, a dim between the tiles
    ("bf16", 2, 2, 160, 48, [2, 17], [2, 200], 0, True),
    ("fp4", 2, 5, 256, 16, [13, 1], [100, 129], 0, True),
    ("fp8", 1, 6, 128, 64, [70, 33], [70, 601], 0, True),                      # several row blocks, a whole prompt
    ("fp4", 4, 1, 64, 128, [150, 129, 1], [150, 400, 128], 0, True),
    ("bf16", 1, 2, 256, 32, [90], [333], 0, True),
    ("fp8", 2, 3, 128, 16, [40, 7, 1], [300, 7, 200], 9, True),                # windows
    ("fp4", 1, 1, 64, 48, [130], [700], 100, True),
    ("bf16", 2, 1, 96, 16, [5, 1], [70, 90], 1, True),                         # each row sees itself alone
    ("fp8", 1, 4, 128, 16, [1, 2], [0, 1], 0, True),                           # lens shorter than the chunk: empty rows
    ("fp4", 32, 1, 32, 4, [1] * 70, list(range(70)), 0, True),
    ("fp4", 1, 70, 64, 16, [1, 1], [65, 1000], 0, True),                       # many rows of one token
    ("bf16", 2, 2, 128, 16, [5, 40], [37, 550], 0, False),                     # no causal mask
    ("fp8", 2, 3, 64, 16, [5, 40], [37, 550], 20, False),
])
def test_weights(kind, kv_heads, share, dim, page, new, lens, window, causal, dtype):
    su = Setup(kind, kv_heads, dim, page, new, lens, seed=dim + len(new), max_pages=max(1, -(-max(lens) // page)) + 2)
    caches = su.fill()
    q = dev(1.5 * su.rng.randn(sum(new), kv_heads * share, dim).astype(np.float32), dtype)
    q64 = f64(q)
    lse = true_lse(su, caches, q64, window, causal)
    before = np.abs(su.rng.randn(su.pages, kv_heads, page)).astype(np.float32)
    for b, (n, m) in enumerate(zip(new, lens)):            # what the new tokens' places hold does not count
        pg, slot = places(su, b, m)
        before[pg[max(m - n, 0):], :, slot[max(m - n, 0):]] = np.nan
    for max_len in (None, 1, 100000):
        for fresh in (False, True):
            weights, err = dev(before), torch.zeros(1, dtype=torch.int32, device="cuda")
            run_weigh(su, weights, q, dev(lse), window, causal, fresh, max_len, err)
            assert err.item() == 0
            check_weights(su, caches, q64, lse, before, weights.cpu().numpy(), window, causal, fresh)
            again = dev(before)
            run_weigh(su, again, q, dev(lse), window, causal, fresh, max_len)
            assert torch.equal(weights.view(torch.int32), again.view(torch.int32))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [5, 10, 45])               # rows of a key head: up to 16, up to 32, more
def test_weights_of_every_type_and_width(kind, dim, dtype, new):
    su = Setup(kind, 2, dim, 16, [new, 1], [300, 290], seed=dim)
    caches = su.fill()
    wide = torch.zeros(new + 1, 7, dim + 3, device="cuda", dtype=dtype)         # rows that start off 16 bytes
    q = wide[:, 1:7, 2:dim + 2]
    q.copy_(dev(1.5 * su.rng.randn(new + 1, 6, dim).astype(np.float32)))
    lse = true_lse(su, caches, f64(q), 0, True)
    before = np.zeros((su.pages, 2, 16), np.float32)
    weights = dev(before)
    run_weigh(su, weights, q, dev(lse))
    check_weights(su, caches, f64(q), lse, before, weights.cpu().numpy(), 0, True, False)
    other = dev(before)
    run_weigh(su, other, q.contiguous(), dev(lse))
    assert torch.equal(weights, other)


# name: (sequences, key heads, query heads of each, most new tokens, longest length)
FORMS = {
    "up to 16 rows, many pieces a wave": (70, 8, 4, 4, 1500),
    "up to 32 rows": (40, 8, 4, 8, 400),
    "many rows, a wave's own keys": (33, 8, 3, 70, 600),
    "many rows, a team's keys": (3, 2, 5, 70, 900),
    "many rows, heads that 64 rows do not hold whole": (2, 1, 96, 9, 500),
}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 256])
def test_weights_in_every_form(form, kind, dim):
    """Every form in which the call is launched, at sizes that select it; some sequences against the oracle."""
    batch, kv_heads, share, chunk, longest = FORMS[form]
    rng = np.random.RandomState(dim + len(form))
    lens = rng.randint(1, longest + 1, batch)
    new = np.minimum(rng.randint(1, chunk + 1, batch), lens)
    lens[0], new[0] = longest, chunk
    lens[1], new[1] = chunk - 1, chunk                     # a row that sees nothing
    page = int(rng.choice([7, 16, 48]))
    su = Setup(kind, kv_heads, dim, page, new.tolist(), lens.tolist(), seed=dim, max_pages=-(-max(longest, chunk) // page) + 1)
    gen = torch.Generator(device="cuda").manual_seed(dim)
    k, v = (torch.randn(int(lens.sum()), kv_heads, dim, device="cuda", generator=gen) for _ in range(2))
    ends = np.concatenate(([0], np.cumsum(lens)))
    wd.kv_write(su.desc, su.pool, k, v, *su.plan(starts=ends))
    sample = sorted({0, 1, batch // 2, batch - 1})
    caches = [(sv.held(k[ends[b]:ends[b + 1]].cpu().numpy(), su.kind), None) if b in sample else None for b in range(batch)]
    for dtype in (torch.bfloat16, torch.float32):
        q = (1.5 * torch.randn(int(new.sum()), kv_heads * share, dim, device="cuda", generator=gen)).to(dtype)
        q64 = f64(q)
        for window, causal in ((0, True), (29, True), (0, False)):
            _, lse = run_lse(su, q, window, causal)
            before = torch.rand(su.pages, kv_heads, page, device="cuda", generator=gen)
            weights, err = before.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
            run_weigh(su, weights, q, lse, window, causal, err=err)
            again = before.clone()
            run_weigh(su, again, q, lse, window, causal)
            assert err.item() == 0 and torch.equal(weights, again)
            old, got, lse64 = f64(before), f64(weights), f64(lse)
            for b in sample:
                a, e, m = su.starts[b], su.starts[b + 1], int(lens[b])
                see = seen(e - a, m, window, causal)
                sums, slack = ev.weigh(q64[a:e], caches[b][0], np.where(np.isfinite(lse64[a:e]), lse64[a:e], 0.0), see, 1.0 / math.sqrt(dim))
                page_at, slot = places(su, b, m)
                want = np.where((np.arange(m) >= m - (e - a))[:, None], 0.0, old[page_at, :, slot]) + sums
                bound = slack + sums * ((e - a) * share + 8) * 2.0 ** -24 + 2.0 ** -24 * np.abs(want)
                ok = bool((np.abs(got[page_at, :, slot] - want) <= bound).all())
                assert ok, (b, (np.abs(got[page_at, :, slot] - want) - bound).max())


@pytest.mark.parametrize("new", [1, 64, 200])
def test_each_row_gives_a_weight_of_one_in_all(new):
    su = Setup("fp8", 2, 128, 16, [new, 1], [700, 90], seed=41)
    su.fill()
    q = dev(su.rng.randn(new + 1, 8, 128).astype(np.float32), torch.bfloat16)
    _, lse = run_lse(su, q)
    weights = torch.full((su.pages, 2, 16), 5.0, device="cuda")
    run_weigh(su, weights, q, lse, fresh=True)
    w = weights.double().cpu().numpy()
    for b, n in ((0, new), (1, 1)):
        page, slot = places(su, b, su.lens[b])
        # the log-sum's error and the weights', each below 2^-14 for scores of this size
        assert np.allclose(w[page, :, slot].sum(0), 4 * n, rtol=2.0 ** -13)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("new", [3, 60])
def test_a_key_that_is_not_finite_spoils_its_own_weight_alone(kind, new):
    su = Setup(kind, 2, 64, 16, [new], [new + 50], seed=42)
    caches = su.fill()
    q = dev(su.rng.randn(new, 4, 64).astype(np.float32))
    lse = dev(true_lse(su, caches, f64(q), 0, True))
    clean = torch.zeros(su.pages, 2, 16, device="cuda")
    run_weigh(su, clean, q, lse)
    for at in (20, 50 + new // 2):                         # in the text; a new token's
        pool = su.pool.clone()
        bad = torch.randn(1, 2, 64, device="cuda")
        bad[0, 1, 3] = math.nan
        wd.kv_write(su.desc, su.pool, bad, bad, dev(np.array([0, 1], np.int32)), dev(np.array([at + 1], np.int32)), dev(su.table))
        got = torch.zeros_like(clean)
        run_weigh(su, got, q, lse)
        here = torch.zeros(su.pages, 2, 16, dtype=torch.bool, device="cuda")
        here[su.table[0][at // 16], :, at % 16] = True
        assert torch.equal(got[~here], clean[~here])
        assert torch.isnan(got[su.table[0][at // 16], 1, at % 16]) and torch.isfinite(got[su.table[0][at // 16], 0, at % 16])
        su.pool.copy_(pool)
    # a key that no row sees takes no harm and does none
    run_weigh(su, clean, q, lse, window=5, fresh=True)
    bad = torch.full((30, 2, 64), math.nan, device="cuda")
    wd.kv_write(su.desc, su.pool, bad, bad, dev(np.array([0, 30], np.int32)), dev(np.array([30], np.int32)), dev(su.table))
    got = torch.zeros_like(clean)
    run_weigh(su, got, q, lse, window=5, fresh=True)
    page, slot = places(su, 0, new + 50)
    assert torch.equal(got[page, :, slot], clean[page, :, slot]) and (got[page[:30], :, slot[:30]] == 0).all()


def test_weights_with_bad_arrays_are_bounded_and_counted():
    su = Setup("fp8", 2, 64, 16, [2, 2], [40, 40], seed=43)
    su.fill()
    q, lse = dev(su.rng.randn(4, 2, 64).astype(np.float32)), torch.zeros(4, 2, device="cuda")
    weights, err = torch.zeros(su.pages, 2, 16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for starts, lens in (([0, 2, 900], [40, 40]), ([-5, 2, 4], [40, 40]), ([0, 2, 4], [40, 1 << 29]), ([0, 2, 4], [40, -7]),
                         ([3, 1, 4], [40, 40])):
        err.zero_()
        run_weigh(su, weights, q, lse, err=err, plan=su.plan(starts, lens), max_chunk=4)
        assert err.item() >= 1
    for page in (-1, su.pages, 1 << 30, -(1 << 31)):
        table = su.table.copy()
        table[0, 1] = page
        plan = su.plan()[:2] + (dev(table),)
        err.zero_()
        weights.fill_(3.0)
        run_weigh(su, weights, q, lse, err=err, plan=plan, fresh=True)
        assert err.item() >= 1 and (weights[su.table[0, 1]] == 3.0).all() and (weights[su.table[0, 0]] != 3.0).all()


def run_choose(su, weights, budget, sinks, recent, err=None, lens=None, table=None):
    keep = torch.full((len(su.lens), su.kv_heads, budget), 77, dtype=torch.int32, device="cuda")
    counts = torch.full((len(su.lens),), 77, dtype=torch.int32, device="cuda")
    wd.kv_choose(su.desc, weights, su.plan(lens=lens)[1], dev(su.table if table is None else table), keep, counts, sinks=sinks,
                 recent=recent, err_count=err)
    return keep, counts


@pytest.mark.parametrize("kv_heads,page,lens,budget,sinks,recent", [
    (1, 1, [1], 1, 0, 0), (2, 16, [0, 1, 5, 6, 7, 50], 6, 1, 2), (3, 7, [300, 1023, 1024, 1025, 40], 37, 4, 9), (8, 16, [2304], 2048, 4, 512),
    (1, 64, [5000, 4096, 4097], 4096, 0, 0), (2, 48, [9000], 1, 0, 1), (2, 48, [9000], 8999, 0, 0), (1, 16, [4000], 100, 50, 50),
    (2, 128, [33000, 32768, 32769, 12], 5000, 4, 100), (1, 4096, [131000], 131, 3, 0), (1, 16, [131073, 70000], 65536, 4, 1000),
    (2, 16, [700] * 33, 64, 4, 16),
])
@pytest.mark.parametrize("what", ["spread", "ties", "odd"])
def test_choices(kv_heads, page, lens, budget, sinks, recent, what):
    su = Setup("fp8", kv_heads, 32, page, [0] * len(lens), lens, seed=len(lens) + budget)
    w = np.exp(3 * su.rng.randn(su.pages, kv_heads, page)).astype(np.float32)
    if what == "ties":
        w = su.rng.choice(np.array([0.0, -0.0, 0.5, 0.5, 1.0], np.float32), w.shape)
    elif what == "odd":
        w *= su.rng.choice([-1.0, 1.0], w.shape).astype(np.float32)
        at = su.rng.rand(*w.shape)
        w[at < 0.1], w[(at > 0.1) & (at < 0.15)], w[(at > 0.15) & (at < 0.2)], w[(at > 0.2) & (at < 0.4)] = np.nan, np.inf, -np.inf, 1e-42
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep, counts = run_choose(su, dev(w), budget, sinks, recent, err)
    got = keep.cpu().numpy()
    assert counts.tolist() == [min(m, budget) for m in lens] and err.item() == 0
    for b, m in enumerate(lens):
        page_at, slot = places(su, b, m)
        for h in range(kv_heads):
            want = ev.choose(w[page_at, h, slot], budget, sinks, recent)
            assert got[b, h].tolist() == want + [-1] * (budget - len(want))


def test_choices_from_weights_off_16_bytes():
    su = Setup("fp8", 2, 32, 16, [0, 0], [3000, 40000], seed=52)
    buffer = torch.rand(su.pages * 2 * 16 + 3, device="cuda")
    for shift in (1, 2, 3):
        view = buffer[shift:shift + su.pages * 32].view(su.pages, 2, 16)
        got, want = run_choose(su, view, 1500, 4, 100), run_choose(su, view.clone(), 1500, 4, 100)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_choices_with_bad_arrays_are_bounded_and_counted():
    su = Setup("fp8", 2, 32, 16, [0, 0], [40, 100], seed=51)
    w = dev(np.exp(su.rng.randn(su.pages, 2, 16)).astype(np.float32))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for lens in ([40, -5], [1 << 30, 100], [40, 113], [-(1 << 31), 100]):
        err.zero_()
        keep, counts = run_choose(su, w, 30, 2, 5, err, lens=lens)
        assert err.item() >= 1
        most = su.table.shape[1] * 16
        assert counts.tolist() == [min(max(m, 0), most, 30) for m in lens]
        assert ((keep >= -1) & (keep < most)).all()
    for bad in (-1, su.pages, -(1 << 31), (1 << 31) - 1):
        table = su.table.copy()
        table[1, 2] = bad                                  # its 16 weights count as the smallest
        err.zero_()
        keep, _ = run_choose(su, w, 30, 2, 5, err, table=table)
        assert err.item() >= 1 and not ((keep[1] >= 32) & (keep[1] < 48)).any()


def kept_lists(rng, lens, firsts, heads, width):
    """Ascending entries past their indexes, by sequence and head; counts."""
    counts = [min(width, m - f) for m, f in zip(lens, firsts)]
    lists = np.full((len(lens), heads, width), -1, np.int32)
    for b, (m, f) in enumerate(zip(lens, firsts)):
        for h in range(heads):
            lists[b, h, :counts[b]] = np.sort(rng.permutation(m - f)[:counts[b]])
    return lists, counts


def filled(kind, kv_heads, dim, page, new, lens, seed):
    """A pool of random bytes (a move copies whatever they are) and random weights."""
    su = Setup(kind, kv_heads, dim, page, new, lens, seed=seed)
    su.pool.copy_(dev(su.rng.randint(0, 256, su.pool.numel()).astype(np.uint8)))
    return su, su.rng.randint(0, 1 << 32, (su.pages, kv_heads, page), dtype=np.uint64).astype(np.uint32).view(np.float32)


def check_keep(su, w, lists, counts, starts=None, give_counts=True, with_weights=True):
    firsts = [0] * len(su.lens) if starts is None else [m - (starts[b + 1] - starts[b]) for b, m in enumerate(su.lens)]
    pool, weights = su.pool.cpu().numpy(), w.copy()
    ev.keep(su.lay, pool, weights if with_weights else None, su.table, su.lens, lists, counts, firsts)
    got_w, err = dev(w), torch.zeros(1, dtype=torch.int32, device="cuda")
    _, lens, table = su.plan()
    wd.kv_keep(su.desc, su.pool, dev(lists), lens, table, counts=dev(np.asarray(counts, np.int32)) if give_counts else None,
               starts=None if starts is None else dev(np.asarray(starts, np.int32)), weights=got_w if with_weights else None, err_count=err)
    assert np.array_equal(su.pool.cpu().numpy(), pool)
    assert np.array_equal(got_w.cpu().numpy().view(np.uint32), weights.view(np.uint32))
    assert err.item() == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("kv_heads,dim,page,lens,width", [
    (1, 32, 1, [1], 1), (2, 64, 16, [40, 7, 0, 200], 33), (3, 96, 7, [100, 3], 64), (2, 128, 16, [900, 700], 350), (1, 160, 48, [300], 299),
    (2, 192, 5, [77, 78], 20), (1, 256, 32, [500], 123), (4, 224, 16, [90, 20, 33], 40), (1, 128, 64, [6000], 2500),
])
def test_moves(kind, kv_heads, dim, page, lens, width):
    for every in (True, False):
        su, w = filled(kind, kv_heads, dim, page, [0] * len(lens), lens, seed=dim + width)
        lists, counts = kept_lists(su.rng, lens, [0] * len(lens), kv_heads if every else 1, width)
        check_keep(su, w, lists, counts, with_weights=every)
    # without counts: -1 moves nothing
    su, w = filled(kind, kv_heads, dim, page, [0] * len(lens), lens, seed=dim + width)
    lists, _ = kept_lists(su.rng, lens, [0] * len(lens), kv_heads, width)
    check_keep(su, w, lists, [width] * len(lens), give_counts=False)


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("fp8", 96), ("fp4", 64)])
@pytest.mark.parametrize("gap", [1, 2, 63, 300, 1025, 5000])
def test_moves_over_themselves(kind, dim, gap):
    """Long lists that move by a little: every place is read by one entry and written by another."""
    m = 12001
    su, w = filled(kind, 2, dim, 16, [0], [m], seed=gap)
    lists = np.arange(m - gap, dtype=np.int32)[None, None].repeat(2, 1)
    lists[0, 0, 5:] += gap
    lists[0, 1, 4000:] += gap
    lists = np.minimum(lists, m - 1)
    check_keep(su, w, np.ascontiguousarray(lists), [m - gap])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_moves_of_accepted_nodes(kind):
    """Places count from the first new token; one list for all heads."""
    new, lens = [20, 64, 1, 0, 9], [100, 64, 33, 12, 300]
    su, w = filled(kind, 3, 128, 16, new, lens, seed=61)
    lists = np.full((5, 1, 8), -1, np.int32)
    counts = [8, 8, 1, 0, 3]
    for b, n in enumerate(new):
        if counts[b]:
            lists[b, 0, :counts[b]] = np.concatenate(([0], 1 + np.sort(su.rng.permutation(n - 1)[:counts[b] - 1])))
    check_keep(su, w, lists, counts, starts=su.starts, with_weights=False)
    check_keep(su, w, lists, [8] * 5, starts=su.starts, give_counts=False, with_weights=True)


def test_bad_moves_are_left_out_and_counted():
    m = 100
    su, w = filled("fp8", 2, 64, 16, [0], [m], seed=62)
    _, lens, table = su.plan()
    clean = su.pool.clone()
    good = np.arange(3, 43, dtype=np.int32)
    for at, what in ((0, -2), (5, 4), (7, 9), (39, m), (39, (1 << 31) - 1), (12, -(1 << 31)), (20, 21)):
        lists = good.copy()
        lists[at] = what                                    # below its index, out of order, past the length
        fine = lists.copy()
        for i in range(40):
            if lists[i] != -1 and not (lists[i] >= i and lists[i] < m and (i == 0 or lists[i] == i or lists[i] > lists[i - 1])):
                fine[i] = -1
        su.pool.copy_(clean)
        pool, weights = clean.cpu().numpy().copy(), w.copy()
        ev.keep(su.lay, pool, weights, su.table, su.lens, fine[None, None], [40], [0])
        got, err = dev(w), torch.zeros(1, dtype=torch.int32, device="cuda")
        wd.kv_keep(su.desc, su.pool, dev(lists[None, None]), lens, table, weights=got, err_count=err)
        assert err.item() >= 1, (at, what)
        assert np.array_equal(su.pool.cpu().numpy(), pool) and np.array_equal(got.cpu().numpy().view(np.uint32), weights.view(np.uint32))
    for bad in (-1, su.pages, (1 << 31) - 1, -(1 << 31)):
        t = su.table.copy()
        t[0, 1] = bad
        su.pool.copy_(clean)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        wd.kv_keep(su.desc, su.pool, dev(good[None, None]), lens, dev(t), err_count=err)
        assert err.item() >= 1
        same = (su.pool == clean).view(su.pages, -1).all(-1).cpu().numpy()
        touched = [int(p) for p in su.table[0, [0, 2]]]
        assert all(same[p] for p in range(su.pages) if p not in touched)
    for counts, starts, lens_are in (([41], None, [m]), ([-1], None, [m]), (None, [0, -3], [m]), (None, [0, m + 1], [m]), (None, None, [1 << 20])):
        su.pool.copy_(clean)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        wd.kv_keep(su.desc, su.pool, dev(good[None, None]), dev(np.asarray(lens_are, np.int32)), table,
                   counts=None if counts is None else dev(np.asarray(counts, np.int32)),
                   starts=None if starts is None else dev(np.asarray(starts, np.int32)), err_count=err)
        assert err.item() >= 1


def test_a_pool_past_32_bits():
    su = Setup("bf16", 2, 128, 16, [3], [200], seed=63)
    pages = (5 << 30) // (2 * su.lay.block)
    su.desc, su.pages = wd.make_kv_desc(su.kind, 2, 128, 16, pages), pages
    su.pool = torch.empty(wd.kv_pool_bytes(su.desc), dtype=torch.uint8, device="cuda")
    assert su.pool.numel() > 1 << 32
    su.table[0] = pages - 1 - np.arange(su.table.shape[1])
    caches = su.fill()
    q = dev(su.rng.randn(3, 4, 128).astype(np.float32))
    lse = true_lse(su, caches, f64(q), 0, True)
    weights = torch.zeros(pages, 2, 16, device="cuda")
    run_weigh(su, weights, q, dev(lse))
    page, slot = places(su, 0, 200)
    sums, slack = ev.weigh(f64(q), caches[0][0], lse.astype(np.float64), seen(3, 200, 0, True), 1 / math.sqrt(128))
    got = weights[torch.from_numpy(page).cuda().long(), :, torch.from_numpy(slot).cuda()].double().cpu().numpy()
    assert (np.abs(got - sums) <= slack + sums * 20 * 2.0 ** -24).all()
    keep, counts = run_choose(su, weights, 100, 4, 20)
    wd.kv_keep(su.desc, su.pool, keep, su.plan()[1], su.plan()[2], counts=counts, weights=weights)
    out = torch.empty(2, 100, 2, 128, device="cuda")
    wd.kv_read(su.desc, su.pool, out[0], out[1], dev(np.array([0, 100], np.int32)), counts, dev(su.table))
    for h in range(2):
        want = ev.choose(got[:, h].astype(np.float32), 100, 4, 20)
        for x, held in zip(out, caches[0]):
            assert np.array_equal(f64(x[:, h]), held[want, h])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_a_prompt_that_is_cut_down(kind):
    """Attention, weights, choice and move together; then a new token over what is left, against a dense recomputation."""
    su = Setup(kind, 2, 64, 16, [300, 80], [300, 80], seed=64)
    caches = su.fill()
    # the short sequence keeps all of its five full pages: its next token needs a sixth
    su.table[1, 5] = min(set(range(su.pages)) - set(su.table[su.table >= 0].tolist()))
    q = dev(su.rng.randn(380, 6, 64).astype(np.float32))
    _, lse = run_lse(su, q)
    weights = torch.full((su.pages, 2, 16), math.nan, device="cuda")
    run_weigh(su, weights, q, lse)
    keep, counts = run_choose(su, weights, 100, 4, 30)
    w = weights.cpu().numpy()
    wd.kv_keep(su.desc, su.pool, keep, su.plan()[1], su.plan()[2], counts=counts, weights=weights)
    lens = counts + 1
    k, v = (torch.randn(2, 2, 64, device="cuda") for _ in range(2))
    starts = torch.arange(3, dtype=torch.int32, device="cuda")
    wd.kv_write(su.desc, su.pool, k, v, starts, lens, dev(su.table))
    one = dev(su.rng.randn(2, 6, 64).astype(np.float32))
    out, ws = torch.empty_like(one), torch.empty(wd.attn_workspace_bytes(su.desc, 6, 2, 2, 1, 101), dtype=torch.uint8, device="cuda")
    wd.attn(su.desc, su.pool, one, out, starts, lens, dev(su.table), ws, max_chunk=1, max_len=101)
    for b, m in enumerate(su.lens):
        page, slot = places(su, b, m)
        for h in range(2):
            kept = ev.choose(w[page, h, slot], 100, 4, 30)
            assert keep[b, h, :len(kept)].tolist() == kept
            new_page, new_slot = places(su, b, len(kept))
            assert np.array_equal(weights.cpu().numpy()[new_page, h, new_slot], w[page, h, slot][kept])
            kk = np.concatenate((caches[b][0][kept, h], sv.held(k[b:b + 1, h].cpu().numpy(), su.kind)))
            vv = np.concatenate((caches[b][1][kept, h], sv.held(v[b:b + 1, h].cpu().numpy(), su.kind)))
            ref, mass, spread = sv.attend(f64(one[b:b + 1, 3 * h:3 * h + 3]), kk[:, None], vv[:, None], np.array([len(kk) - 1]), 0.125)
            bound = mass * (2 * (3 * 64 + 8) * 2.0 ** -24 * spread[..., None] + (len(kk) + 64) * 2.0 ** -23)
            ok = bool((np.abs(f64(out[b:b + 1, 3 * h:3 * h + 3]) - ref) <= bound).all())
            assert ok


def test_eviction_on_another_stream_and_in_a_graph():
    su = Setup("fp8", 2, 128, 16, [1, 1], [700, 90], seed=65)
    su.fill()
    q = dev(su.rng.randn(2, 8, 128).astype(np.float32), torch.bfloat16)
    _, lens, table = su.plan()
    starts = su.plan()[0]
    out, lse = torch.empty_like(q), torch.empty(2, 8, device="cuda")
    ws = torch.empty(wd.attn_workspace_bytes(su.desc, 8, 2, 2, 1, 700), dtype=torch.uint8, device="cuda")
    weights = torch.rand(su.pages, 2, 16, device="cuda")
    keep, counts = torch.empty(2, 2, 64, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    pool0, weights0 = su.pool.clone(), weights.clone()

    def step():
        wd.attn(su.desc, su.pool, q, out, starts, lens, table, ws, max_chunk=1, max_len=700, lse=lse)
        wd.kv_weigh(su.desc, su.pool, weights, q, lse, starts, lens, table, max_chunk=1, max_len=700)
        wd.kv_choose(su.desc, weights, lens, table, keep, counts, sinks=4, recent=16)
        wd.kv_keep(su.desc, su.pool, keep, lens, table, counts=counts, weights=weights)

    def state():
        return [x.clone() for x in (out, lse, weights, keep, counts, su.pool)]

    def reset():
        su.pool.copy_(pool0)
        weights.copy_(weights0)

    step()
    want = state()
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(state(), want))
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        q.copy_(dev(su.rng.randn(2, 8, 128).astype(np.float32), torch.bfloat16))
        reset()
        step()
        want = state()
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(state(), want))
