"""Attention of drafted trees over the paged cache, on the GPU against the 64-bit oracle (oracle/trees.py), per output
within bounds that follow from its roundings, with A = sum p |v| / sum p:
* a score is a sum of D exact products of bf16 numbers (three terms a query for f32 queries) in f32: its error is below
  (3 D + 8) 2^-24 times scale * sum |q_d k_d|, and exp turns it into a relative error of p, in the numerator and in the sum of
  p: 2 A times that; v_exp_f32 and the sums over n keys add (n + 64) 2^-23 A;
* bf16 queries: the output is rounded to bf16, by 2^-8 of it at most.  Where a (sequence, key head) has more than 64 rows, p is
  rounded to bf16 in the numerator and in the sum alike: sum p d (v - out) / sum p with |d| <= 2^-8, which is at most
  2^-8 (A + |out|).  Where it has fewer, two terms of p leave |d| <= 2^-16;
* f32 queries: three bf16 terms of p leave 2^-26, below the terms above."""

import math

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from oracle import serving as sv
from oracle import trees
from test_gpu_serving import Setup, dev, f64, run_attn

pytestmark = pytest.mark.gpu


def random_tree(rng, n, wide=False):
    """Parents of n nodes; wide: several roots, long chains and stars among them."""
    if not wide:
        return [-1][:n] + [int(rng.randint((i - 1) // 3, i)) for i in range(1, n)]
    return [int(rng.choice([-1, 0 if i else -1, i - 1, rng.randint(-1, i)])) for i in range(n)]


def run_tree(su, q, parents, dtype, window=0, max_len=None, err=None, out=None, plan=None, stream=None, scale=None, max_chunk=None):
    q = q if isinstance(q, torch.Tensor) else dev(q, dtype)
    out = torch.full_like(q, 9.0) if out is None else out
    max_chunk, max_len = max(max(su.new), 1) if max_chunk is None else max_chunk, max(max(su.lens), 1) if max_len is None else max_len
    ws = torch.empty(wd.attn_workspace_bytes(su.desc, q.shape[1], q.shape[0], len(su.lens), max_chunk, max_len), dtype=torch.uint8,
                     device="cuda")
    parents = parents if isinstance(parents, torch.Tensor) else dev(np.concatenate([np.asarray(p, np.int32) for p in parents]))
    wd.attn_tree(su.desc, su.pool, q, out, *(plan or su.plan()), parents, ws, max_chunk=max_chunk, max_len=max_len, window=window,
                 err_count=err, stream=stream, scale=scale)
    return out


def check_rows(got, q64, k, v, see, dim, dtype, few):
    ref, mass, spread, _ = trees.attend(q64, k, v, see, 1.0 / math.sqrt(dim))
    bound = mass * (2 * (3 * dim + 8) * 2.0 ** -24 * spread[..., None] + (len(k) + 64) * 2.0 ** -23)
    if dtype == torch.bfloat16:
        bound = bound + (2.0 ** -16 if few else 2.0 ** -8) * (mass + np.abs(ref))
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    off = np.abs(got - ref) - bound
    ok = bool(np.isfinite(got).all() and (off <= 0).all())
    assert ok, (np.abs(got - ref).max(), off.max())


def is_few(su, heads):
    return max(su.new) * heads // su.kv_heads <= 64


def check_tree(su, caches, parents, q, out, dtype, window=0):
    q64, got = f64(q if isinstance(q, torch.Tensor) else dev(q, dtype)), f64(out)
    for b, (k, v) in enumerate(caches):
        a, e = su.starts[b], su.starts[b + 1]
        text = su.lens[b] - (e - a)
        see = trees.sees(parents[b], max(text, 0), window)
        if text < 0:      # the first nodes have no place
            see = np.zeros((e - a, su.lens[b]), bool)
            path = trees.sees(parents[b], 0)
            for i in range(e - a):
                up = [j for j in range(e - a) if path[i, j]]
                for j in up[-window:] if window else up:
                    if text + j >= 0:
                        see[i, text + j] = True
        check_rows(got[a:e], q64[a:e], k, v, see, su.dim, dtype, is_few(su, got.shape[1]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kind,kv_heads,share,dim,page,new,lens,window", [
    ("bf16", 1, 1, 32, 1, [1], [1], 0),                        # one node that sees itself
    ("fp8", 2, 1, 64, 16, [1, 16, 0, 5], [1, 63, 5, 300], 0),  # a sequence with nothing new
    ("fp4", 1, 8, 128, 16, [8, 3], [64, 513], 0),              # shared heads
    ("fp8", 3, 4, 96, 7, [16, 3, 8], [16, 130, 257], 0),       # a tree without a text, odd pages
    ("bf16", 2, 2, 160, 48, [2, 32], [2, 200], 0),
    ("fp4", 2, 5, 256, 16, [13, 1], [100, 129], 0),            # 65 rows
    ("fp8", 1, 6, 128, 64, [64, 33], [70, 201], 0),            # the most nodes
    ("fp4", 4, 1, 64, 128, [64, 64, 1], [150, 400, 128], 0),
    ("fp8", 2, 3, 128, 16, [40, 7, 1], [300, 7, 200], 9),      # windows
    ("fp4", 1, 1, 64, 48, [50], [400], 3),
    ("bf16", 2, 1, 96, 16, [5, 1], [70, 90], 1),               # each node sees itself alone
    ("fp8", 1, 4, 128, 16, [9, 2], [5, 1], 0),                 # fewer places than nodes
    ("fp4", 1, 70, 64, 16, [2, 1], [65, 1000], 0),             # more than 64 rows of one node
])
def test_attention_of_trees(kind, kv_heads, share, dim, page, new, lens, window, dtype, wide):
    su = Setup(kind, kv_heads, dim, page, new, lens, seed=dim + len(new), max_pages=max(1, -(-max(lens) // page)) + 2)
    caches = su.fill()
    parents = [random_tree(su.rng, n, wide) for n in new]
    q = su.rng.randn(sum(new), kv_heads * share, dim).astype(np.float32) * 1.5
    for max_len in (None, 1, 100000):       # the split rule: as it comes, none, many
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = run_tree(su, q, parents, dtype, window, max_len=max_len, err=err)
        check_tree(su, caches, parents, q, out, dtype, window)
        assert err.item() == 0
        assert torch.equal(out, run_tree(su, q, parents, dtype, window, max_len=max_len))


# name: (sequences, key heads, query heads of each, nodes, longest length, max_len that is told)
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
    "many rows, eight waves, split": (17, 8, 5, 64, 420, 100000),
}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 256])
def test_trees_in_every_form(form, kind, dim):
    """Every form in which attention is launched, at sizes that select it."""
    batch, kv_heads, share, chunk, longest, max_len = FORMS[form]
    seed = dim + len(form)
    rng = np.random.RandomState(seed)
    lens = rng.randint(1, longest + 1, batch)
    new = np.minimum(rng.randint(1, chunk + 1, batch), lens)
    lens[0], new[0] = longest, chunk
    lens[1], new[1] = chunk, chunk                     # no text
    page = int(rng.choice([7, 16, 48]))
    su = Setup(kind, kv_heads, dim, page, new.tolist(), lens.tolist(), seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(int(lens.sum()), kv_heads, dim, device="cuda", generator=gen) for _ in range(2))
    ends = np.concatenate(([0], np.cumsum(lens)))
    wd.kv_write(su.desc, su.pool, k, v, *su.plan(starts=ends))
    parents = [random_tree(rng, int(n), b % 2 == 1) for b, n in enumerate(new)]
    for dtype in (torch.bfloat16, torch.float32):
        q = (1.5 * torch.randn(int(new.sum()), kv_heads * share, dim, device="cuda", generator=gen)).to(dtype)
        for window in (0, 29):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = run_tree(su, q, parents, dtype, window, max_len=max_len, err=err)
            assert err.item() == 0 and torch.equal(out, run_tree(su, q, parents, dtype, window, max_len=max_len))
            q64, got = f64(q), f64(out)
            for b in sorted({0, 1, batch // 2, batch - 1}):
                a, n, m = su.starts[b], int(new[b]), int(lens[b])
                rows = sorted(set([0, n // 3, n - 2, n - 1]) & set(range(n)))
                see = trees.sees(parents[b], m - n, window)[rows]
                at = [a + r for r in rows]
                for h in sorted({0, kv_heads - 1}):
                    mine = slice(h * share, (h + 1) * share)
                    kk, vv = (sv.held(x[ends[b]:ends[b + 1], h:h + 1].cpu().numpy(), su.kind) for x in (k, v))
                    check_rows(got[at][:, mine], q64[at][:, mine], kk, vv, see, dim, dtype, is_few(su, kv_heads * share))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("share,window", [(1, 0), (1, 5), (6, 0), (6, 7)])
def test_a_chain_gives_what_causal_attention_gives(dtype, share, window):
    su = Setup("fp8", 2, 128, 16, [5, 64, 1], [200, 90, 700], seed=21)
    su.fill()
    q = su.rng.randn(70, 2 * share, 128).astype(np.float32)
    chains = [list(range(-1, n - 1)) for n in su.new]
    for max_len in (1, 100000):
        assert torch.equal(run_tree(su, q, chains, dtype, window, max_len=max_len), run_attn(su, q, dtype, window, max_len=max_len))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("share", [1, 5])
def test_a_node_that_is_not_seen_has_no_effect(kind, share):
    """A key and a value that are not finite, at a node that only its own subtree sees."""
    su = Setup(kind, 2, 64, 16, [40], [90], seed=22)
    su.fill()
    parents = random_tree(su.rng, 40)
    q = su.rng.randn(40, 2 * share, 64).astype(np.float32)
    at, text = 2, 50
    below = trees.sees(parents, text)[:, text + at]
    assert 0 < below.sum() < 40
    for max_len in (1, 100000):
        clean = run_tree(su, q, [parents], torch.bfloat16, max_len=max_len)
        pool = su.pool.clone()
        for spoil_key in (False, True):
            k, v = (torch.randn(1, 2, 64, device="cuda") for _ in range(2))
            (k if spoil_key else v)[0, 0, 7] = math.nan
            wd.kv_write(su.desc, su.pool, k, v, dev(np.array([0, 1], np.int32)), dev(np.array([text + at + 1], np.int32)), dev(su.table))
            out = run_tree(su, q, [parents], torch.bfloat16, max_len=max_len)
            see = torch.from_numpy(below).cuda()
            assert torch.equal(out[~see], clean[~see])
            assert torch.isnan(out[see][:, :share]).any(-1).all() and torch.isfinite(out[see][:, share:]).all()
            su.pool.copy_(pool)


def test_bad_parents_and_large_trees_are_bounded_and_counted():
    su = Setup("fp8", 2, 64, 16, [6, 4], [40, 44], seed=23)
    caches = su.fill()
    q = su.rng.randn(10, 4, 64).astype(np.float32)
    good = [[-1, 0, 0, 1, 2, -1], [-1, 0, 1, 2]]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (5, 900, -2, -(1 << 31), (1 << 31) - 1, 3):
        parents = np.concatenate([np.asarray(p) for p in good]).astype(np.int64)
        parents[3] = bad                                 # not an earlier node: taken as -1
        err.zero_()
        out = run_tree(su, q, dev(parents.astype(np.int32)), torch.float32, err=err)
        assert err.item() >= 1
        check_tree(su, caches, [[-1, 0, 0, -1, 2, -1], good[1]], q, out, torch.float32)
    # more nodes than a tree may have: the rows past them see the text alone (here: rows within max_chunk's blocks)
    big = Setup("fp8", 1, 64, 16, [70], [100], seed=24)
    (k, v), = big.fill()
    q = big.rng.randn(70, 2, 64).astype(np.float32)
    chain = list(range(-1, 69))
    err.zero_()
    parents = dev(np.asarray(chain, np.int32))
    ws = torch.empty(wd.attn_workspace_bytes(big.desc, 2, 64, 2, 64, 100), dtype=torch.uint8, device="cuda")
    plan = dev(np.array([0, 70, 70], np.int32)), dev(np.array([100, 1], np.int32)), dev(np.repeat(big.table, 2, 0))
    qd = dev(q)
    out = torch.full_like(qd, 9.0)
    wd.attn_tree(big.desc, big.pool, qd, out, *plan, parents, ws, max_chunk=64, max_len=100, err_count=err)
    assert err.item() >= 1
    check_rows(f64(out[:64]), f64(qd[:64]), k, v, np.pad(trees.sees(chain[:64], 30), ((0, 0), (0, 6))), 64, torch.float32, False)


def test_trees_on_another_stream_and_in_a_graph():
    su = Setup("fp8", 2, 128, 16, [33, 20], [400, 90], seed=25)
    caches = su.fill()
    parents = [random_tree(su.rng, n) for n in su.new]
    flat = dev(np.concatenate(parents).astype(np.int32))
    q = dev(su.rng.randn(53, 4, 128).astype(np.float32), torch.bfloat16)
    plan = su.plan()
    want = run_tree(su, q, flat, torch.bfloat16, plan=plan)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = run_tree(su, q, flat, torch.bfloat16, plan=plan)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    ws = torch.empty(wd.attn_workspace_bytes(su.desc, 4, 53, 2, 33, 400), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    with torch.cuda.graph(graph):
        wd.attn_tree(su.desc, su.pool, q, out, *plan, flat, ws, max_chunk=33, max_len=400)
    for i in range(3):
        q.copy_(dev(su.rng.randn(53, 4, 128).astype(np.float32), torch.bfloat16))
        want = run_tree(su, q, flat, torch.bfloat16, plan=plan)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert len(caches) == 2


def test_rows_of_no_sequence_are_left():
    su = Setup("fp8", 1, 64, 16, [5, 3], [50, 70], seed=26)
    caches = su.fill()
    parents = [random_tree(su.rng, n) for n in su.new] + [[3, -7, 0, 1]]
    q = dev(su.rng.randn(12, 2, 64).astype(np.float32))
    for max_len in (1, 100000):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = run_tree(su, q, parents, torch.float32, max_len=max_len, err=err, max_chunk=6)
        assert (out[8:] == 9.0).all() and err.item() == 0
        check_tree(su, caches, parents, q, out, torch.float32)
