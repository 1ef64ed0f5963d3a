"""The check of drafted trees on the GPU: tokens, paths and counts equal the oracle's (oracle/trees.py).  Both take S and its
products in 64 bits from the same numbers in the same order, so the decisions are the same."""

import math

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from oracle import trees
from test_gpu_serving import dev
from test_gpu_trees import random_tree

pytestmark = pytest.mark.gpu


def run_verify(target, starts, tokens, parents, uniforms, noise, width, err=None, stream=None, ws=None):
    b, v = noise.shape
    accepted = torch.full((b,), 77, dtype=torch.int32, device="cuda")
    path, out = (torch.full((b, width), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(wd.tree_workspace_bytes(b, v), dtype=torch.uint8, device="cuda") if ws is None else ws
    wd.tree_verify(target, starts, tokens, parents, uniforms, noise, accepted, path, out, ws, err_count=err, stream=stream)
    return accepted, path, out


def made(rng, sizes, vocab, dtype, peak=3.0, picked=True):
    """Trees of given sizes over targets in which a few tokens hold most of the mass; children hold their node's likely tokens."""
    n = sum(sizes)
    logits = torch.from_numpy(rng.randn(max(n, 1), vocab).astype(np.float32)) * peak
    target = torch.softmax(logits, -1).to(dtype)[:n].cuda()
    starts = np.concatenate(([0], np.cumsum(sizes))).astype(np.int32)
    parents = [random_tree(rng, s, wide=b % 3 == 2) for b, s in enumerate(sizes)]
    tokens = rng.randint(0, vocab, n).astype(np.int32)
    if picked:
        order = torch.argsort(target.float(), dim=-1, descending=True, stable=True)[:, :6].cpu().numpy()
        for b, tree in enumerate(parents):
            for i, p in enumerate(tree):
                if p >= 0:
                    tokens[starts[b] + i] = order[starts[b] + p][rng.randint(0, min(6, vocab))]     # twice the same among siblings
    flat = np.asarray(sum(parents, []), np.int32)
    uniforms = rng.rand(n).astype(np.float32)
    noise = np.maximum(rng.exponential(size=(len(sizes), vocab)).astype(np.float32), 1e-30)
    return target, starts, tokens, flat, uniforms, noise


def check(case, width, err_is=0):
    target, starts, tokens, parents, uniforms, noise = case
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_verify(target, *(dev(x) for x in (starts, tokens, parents, uniforms, noise)), width, err=err)
    want = trees.verify(target.float().cpu().numpy(), starts, tokens, parents, uniforms, noise, width)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert err.item() == err_is
    return want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,vocab,width", [
    ([1], 1, 1), ([1], 7, 3), ([16], 999, 16), ([64], 513, 64), ([64, 64], 8192, 64), ([30], 8193, 64), ([12, 0, 1, 64, 7], 1000, 9),
    ([20] * 40, 333, 20), ([5] * 600, 65, 5), ([33], 100003, 33), ([17, 40, 3], 32000, 12), ([40], 50, 2), ([9], 9, 1),
])
def test_trees_are_checked_as_the_oracle_does(sizes, vocab, width, dtype):
    rng = np.random.RandomState(vocab + len(sizes))
    longest = 0
    for peak in (0.5, 3.0, 8.0):
        longest = max(longest, check(made(rng, sizes, vocab, dtype, peak), width)[0].max())
    if len(sizes) >= 40:
        assert longest > 1          # some walk went somewhere


@pytest.mark.parametrize("drafts", [1, 4, 63])
def test_a_chain_gives_what_the_check_of_drafts_gives(drafts):
    rng = np.random.RandomState(drafts)
    b, v = 20, 500
    target = torch.softmax(torch.from_numpy(rng.randn(b, drafts + 1, v).astype(np.float32)) * 6, -1).cuda()
    tokens = target[:, :drafts].argmax(-1).int()
    uniforms = torch.from_numpy((rng.rand(b, drafts) * 0.9).astype(np.float32)).cuda()
    noise = torch.from_numpy(rng.exponential(size=(b, v)).astype(np.float32)).cuda().clamp_(min=1e-30)
    accepted, out = torch.empty(b, dtype=torch.int32, device="cuda"), torch.empty(b, drafts + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(wd.draft_workspace_bytes(b, v), dtype=torch.uint8, device="cuda")
    wd.draft_verify(target, None, tokens, uniforms, noise, accepted, out, ws)
    pad = lambda x: torch.cat((torch.zeros_like(x[:, :1]), x), 1).flatten().contiguous()  # noqa: E731
    starts = torch.arange(b + 1, device="cuda", dtype=torch.int32) * (drafts + 1)
    parents = torch.arange(-1, drafts, device="cuda", dtype=torch.int32).repeat(b)
    got = run_verify(target.flatten(0, 1), starts, pad(tokens), parents, pad(uniforms), noise, drafts + 1)
    assert torch.equal(got[0], accepted) and torch.equal(got[2], out)
    assert drafts < 4 or len(set(accepted.tolist())) > 2


def test_the_law_of_the_first_token():
    """Over many draws the first token after the root has the target's own distribution, whatever was picked."""
    rng = np.random.RandomState(3)
    b, v = 20000, 6
    p = np.array([0.4, 0.25, 0.2, 0.1, 0.05, 0.0], np.float32)
    picked = [2, 0, 2, 5]                                  # a token twice, one that cannot be
    target = torch.from_numpy(np.tile(p, (b * 5, 1))).cuda()
    starts = dev(np.arange(b + 1, dtype=np.int32) * 5)
    tokens = dev(np.tile(np.array([0] + picked, np.int32), b))
    parents = dev(np.tile(np.array([-1, 0, 0, 0, 0], np.int32), b))
    uniforms, noise = dev(rng.rand(b * 5).astype(np.float32)), dev(rng.exponential(size=(b, v)).astype(np.float32))
    _, _, out = run_verify(target, starts, tokens, parents, uniforms, noise, 5)
    seen = np.bincount(out[:, 0].cpu().numpy(), minlength=v) / b
    # five standard deviations of a share of b draws
    assert (np.abs(seen - p) <= 5 * np.sqrt(p * (1 - p) / b) + 1e-9).all(), seen


def test_nothing_left_draws_from_all():
    target = np.zeros((3, 40), np.float32)
    target[0, [3, 7]] = 0.5                                # children 3 and 7 refused: nothing else has a chance
    target[1:] = 1.0 / 40
    case = (torch.from_numpy(target).cuda(), np.array([0, 3], np.int32), np.array([0, 3, 7], np.int32), np.array([-1, 0, 0], np.int32),
            np.array([0, 0.999, 1.0], np.float32), np.random.RandomState(0).exponential(size=(1, 40)).astype(np.float32))
    # a uniform of 1 is outside [0, 1): S = 0.5 = w is refused
    got = check(case, 3)
    assert got[0][0] == 0 and got[2][0, 0] in (3, 7)


def test_odd_probabilities_and_noise():
    rng = np.random.RandomState(8)
    target, starts, tokens, parents, uniforms, noise = made(rng, [20, 20, 20, 3], 300, torch.float32)
    t = target.cpu().numpy()
    t[:20, ::3] = np.nan
    t[20:40, ::2] = -1.0
    t[60:] = 0.0
    noise[1, 5:40] = np.nan
    noise[2, 7:90] = -1.0
    noise[2, 100] = 0.0
    noise[3] = np.inf
    check((torch.from_numpy(t).cuda(), starts, tokens, parents, uniforms, noise), 20, err_is=1)     # the last has nothing to draw


def test_bad_trees_are_bounded_and_counted():
    rng = np.random.RandomState(9)
    target, starts, tokens, parents, uniforms, noise = made(rng, [10, 12], 100, torch.float32)
    for where, what in ((3, 3), (3, 60), (3, -2), (13, -(1 << 31)), (13, (1 << 31) - 1)):
        bad, fine = parents.copy(), parents.copy()
        bad[where], fine[where] = what, -1
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run_verify(target, *(dev(x) for x in (starts, tokens, bad, uniforms, noise)), 12, err=err)
        want = trees.verify(target.cpu().numpy(), starts, tokens, fine, uniforms, noise, 12)
        assert err.item() == 1 and all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(got, want))
    for what in (-1, 100, 1 << 30, -(1 << 31)):
        t = tokens.copy()
        t[parents == 0] = what
        check((target, starts, t, parents, uniforms, noise), 12, err_is=2)
    for s in ([0, 10, 500], [-4, 10, 22], [0, 30, 22], [22, 0, 22]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run_verify(target, dev(np.asarray(s, np.int32)), *(dev(x) for x in (tokens, parents, uniforms, noise)), 12, err=err)
        assert err.item() >= 1
        assert all(((x >= -1) & (x < 100)).all() for x in got)
    # more nodes than a tree may have: those past the 64th are not looked at
    target, starts, tokens, parents, uniforms, noise = made(rng, [70], 50, torch.float32)
    check((target, starts, tokens, parents, uniforms, noise), 64, err_is=1)


def test_rows_past_32_bits():
    n, v = 40, 60_000_000                                  # 2.4e9 entries of bf16
    target = torch.zeros(n, v, dtype=torch.bfloat16, device="cuda")
    chain = torch.arange(-1, n - 1, dtype=torch.int32, device="cuda")
    tokens = torch.arange(n, dtype=torch.int32, device="cuda") * 1_499_999
    target[chain[1:].long(), tokens[1:].long()] = 1.0
    target[n - 1, v - 1] = 0.5
    noise = torch.ones(1, v, device="cuda")
    accepted, path, out = run_verify(target, torch.tensor([0, n], dtype=torch.int32, device="cuda"), tokens, chain,
                                     torch.full((n,), 0.5, device="cuda"), noise, n)
    assert accepted.item() == n - 1 and path[0].tolist() == list(range(n)) and out[0].tolist() == tokens[1:].tolist() + [v - 1]


def test_in_a_graph_and_on_another_stream():
    rng = np.random.RandomState(12)
    case = made(rng, [30, 9], 32000, torch.float32)
    args = [case[0]] + [dev(x) for x in case[1:]]
    want = run_verify(*args, 30)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_verify(*args, 30)
    side.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    ws = torch.empty(wd.tree_workspace_bytes(2, 32000), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(2, dtype=torch.int32, device="cuda")] + [torch.empty(2, 30, dtype=torch.int32, device="cuda") for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wd.tree_verify(*args, *outs, ws)
    for i in range(3):
        args[4].copy_(torch.rand(39, device="cuda"))
        want = run_verify(*args, 30)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(outs, want))
    assert math.isfinite(float(args[5].sum()))
