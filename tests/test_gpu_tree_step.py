"""A decoding step with drafted trees: their keys and values are written, their nodes attend, the trees are checked, the accepted
nodes move to the end of the text, and the next step's attention is what a dense recomputation over the accepted text gives."""

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from oracle import serving as sv
from oracle import trees
from test_gpu_serving import Setup, dev, f64
from test_gpu_trees import check_rows, random_tree, run_tree

pytestmark = pytest.mark.gpu
VOCAB = 300


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_tree_decoding(kind, captured):
    texts, nodes, steps, kv_heads, share, dim = [37, 5, 120], 12, 4, 2, 3, 64
    room = [n + steps * nodes for n in texts]
    su = Setup(kind, kv_heads, dim, 16, [nodes] * 3, room, seed=71)
    rng, gen = su.rng, torch.Generator(device="cuda").manual_seed(71)
    table = dev(su.table)
    # the texts so far, and what the oracle holds of them
    k, v = (torch.randn(sum(texts), kv_heads, dim, device="cuda", generator=gen) for _ in range(2))
    ends = np.concatenate(([0], np.cumsum(texts)))
    wd.kv_write(su.desc, su.pool, k, v, dev(ends.astype(np.int32)), dev(np.asarray(texts, np.int32)), table)
    held = [[sv.held(x[ends[b]:ends[b + 1]].cpu().numpy(), su.kind) for x in (k, v)] for b in range(3)]

    # buffers of a step, the same for all steps
    n = 3 * nodes
    new = [torch.empty(n, kv_heads, dim, device="cuda") for _ in range(2)]
    q, out = torch.empty(n, kv_heads * share, dim, device="cuda"), torch.empty(n, kv_heads * share, dim, device="cuda")
    starts, lens = dev(np.arange(4, dtype=np.int32) * nodes), torch.empty(3, dtype=torch.int32, device="cuda")
    parents, tokens = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
    target, noise, uniforms = torch.empty(n, VOCAB, device="cuda"), torch.empty(3, VOCAB, device="cuda"), torch.empty(n, device="cuda")
    accepted, path, said = (torch.empty(*s, dtype=torch.int32, device="cuda") for s in ((3,), (3, nodes), (3, nodes)))
    space = torch.empty(wd.attn_workspace_bytes(su.desc, kv_heads * share, n, 3, nodes, max(room)), dtype=torch.uint8, device="cuda")
    keys = torch.empty(wd.tree_workspace_bytes(3, VOCAB), dtype=torch.uint8, device="cuda")

    def step():
        wd.kv_write(su.desc, su.pool, *new, starts, lens, table)
        wd.attn_tree(su.desc, su.pool, q, out, starts, lens, table, parents, space, max_chunk=nodes, max_len=max(room))
        wd.tree_verify(target, starts, tokens, parents, uniforms, noise, accepted, path, said, keys)
        wd.kv_keep(su.desc, su.pool, path.view(3, 1, nodes), lens, table, starts=starts)

    graph, moved = None, 0
    for i in range(steps):
        trees_now = [random_tree(rng, nodes) for _ in range(3)]
        for x in new:
            x.normal_(generator=gen)
        q.normal_(generator=gen)
        parents.copy_(dev(np.concatenate(trees_now).astype(np.int32)))
        target.copy_(torch.softmax(6 * torch.randn(n, VOCAB, device="cuda", generator=gen), -1))
        best = target.topk(3, -1).indices.cpu().numpy()
        picked = [best[b * nodes + max(p, 0)][rng.randint(0, 3)] for b in range(3) for p in trees_now[b]]
        tokens.copy_(dev(np.asarray(picked, np.int32)))
        uniforms.copy_(torch.rand(n, device="cuda", generator=gen) * 0.8)
        noise.exponential_(generator=gen).clamp_(min=1e-30)
        texts_now = [len(h[0]) for h in held]
        lens.copy_(dev(np.asarray([t + nodes for t in texts_now], np.int32)))
        if captured and graph is None:
            pool = su.pool.clone()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            su.pool.copy_(pool)
        if captured:
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        want = trees.verify(target.cpu().numpy(), starts.cpu().numpy(), tokens.cpu().numpy(), parents.cpu().numpy(), uniforms.cpu().numpy(),
                            noise.cpu().numpy(), nodes)
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip((accepted, path, said), want))
        for b in range(3):
            rows = slice(b * nodes, (b + 1) * nodes)
            both = [np.concatenate((h, sv.held(x[rows].cpu().numpy(), su.kind))) for h, x in zip(held[b], new)]
            check_rows(f64(out[rows]), f64(q[rows]), *both, trees.sees(trees_now[b], texts_now[b]), dim, torch.float32, True)
            way = [j for j in want[1][b] if j >= 0]
            moved += sum(i != j for i, j in enumerate(way))
            held[b] = [np.concatenate((x[:texts_now[b]], x[texts_now[b]:][way])) for x in both]
            # the cache holds the accepted text
            m = len(held[b][0])
            got = torch.empty(2, m, kv_heads, dim, device="cuda")
            wd.kv_read(su.desc, su.pool, got[0], got[1], dev(np.array([0, m], np.int32)), dev(np.array([m], np.int32)), table[b:b + 1])
            assert all(np.array_equal(f64(x), h) for x, h in zip(got, held[b]))
    assert moved > 3
    # one more token of each over what was accepted
    su.new, su.lens, su.starts = [1] * 3, [len(h[0]) for h in held], np.arange(4, dtype=np.int32)
    one = torch.randn(3, kv_heads * share, dim, device="cuda", generator=gen)
    plan = dev(su.starts), dev(np.asarray(su.lens, np.int32)), table
    got = run_tree(su, one, [[-1]] * 3, torch.float32, plan=plan)
    for b in range(3):
        check_rows(f64(got[b:b + 1]), f64(one[b:b + 1]), *held[b], np.ones((1, su.lens[b]), bool), dim, torch.float32, True)
