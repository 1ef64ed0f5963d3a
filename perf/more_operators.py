"""Cases for the serving operators of drafted trees and of eviction: attention of a tree of drafted tokens
over the paged cache, the check of drafted trees, the attention weight that every cached token has received, the
choice of the tokens that stay, and their move to the front of the cache.

Plain forms are written in elementary torch operations.  A cache is one uint8 pool
[pages][kv_heads][block]; a block holds, for `page` tokens of one head, the key codes [page][D * bits / 8], the value
codes, the key scales [page][D / 32] and the value scales (one byte e + 127 for 32 channels, value = code * 2^e; none in
the bf16 kind), rounded up to 16 bytes.  Weights of cached tokens are f32 [pages][kv_heads][page].  A batch is
described by starts [B + 1] (rows of each sequence's new tokens), lens [B] (tokens of each sequence, the new ones
included) and table [B][max_pages].  A tree's nodes are a sequence's new tokens; parents [rows] counts from the
sequence's first node, -1 hangs on the cached text.
"""

import math
import random

import numpy as np
import torch

own = False

BITS = {"bf16": 16, "fp8": 8, "fp4": 4}
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the drafted tree of one answer over a short context, own keys for each head: latency
        dict(name="tree_one_bf16", op="tree", kind="bf16", dtype="bfloat16", batch=1, chunk=16, kv=777, heads=32, kv_heads=32,
             head_dim=128, page=16, window=0, ragged=False),
        # a decode step of several sequences with a tree each, f32 in and out as the fused product writes
        dict(name="tree_many_fp8_f32", op="tree", kind="fp8", dtype="float32", batch=16, chunk=32, kv=4096, heads=32, kv_heads=8,
             head_dim=128, page=16, window=0, ragged=True),
        # the largest trees over long contexts, shared heads (8192 = 64 x 128)
        dict(name="tree_large_fp4", op="tree", kind="fp4", dtype="bfloat16", batch=8, chunk=64, kv=16384, heads=64, kv_heads=8,
             head_dim=128, page=48, window=0, ragged=True),
        # one sequence's tree checked: latency
        dict(name="verify_one", op="verify", dtype="float32", batch=1, chunk=16, vocab=32000, ragged=False),
        # a full batch of trees over a large odd vocabulary
        dict(name="verify_many", op="verify", dtype="float32", batch=96, chunk=32, vocab=100003, ragged=True),
        # one token's step: what each cached token got of its attention: latency
        dict(name="weigh_token_one_bf16", op="weigh", kind="bf16", dtype="bfloat16", batch=1, chunk=1, kv=777, heads=32, kv_heads=32,
             head_dim=128, page=16, window=0, ragged=False, fresh=False),
        # a decode step of many sequences with shared heads
        dict(name="weigh_tokens_many_fp8", op="weigh", kind="fp8", dtype="bfloat16", batch=64, chunk=1, kv=16384, heads=64, kv_heads=8,
             head_dim=128, page=16, window=0, ragged=True, fresh=False),
        # the last chunk of long prompts, before they are cut down: compute
        dict(name="weigh_chunk_fp8", op="weigh", kind="fp8", dtype="bfloat16", batch=2, chunk=2048, kv=8192, heads=32, kv_heads=32,
             head_dim=128, page=16, window=0, ragged=False, fresh=True),
        # one sequence that has passed its budget while decoding: latency
        dict(name="choose_one", op="choose", batch=1, kv=2304, kv_heads=8, page=16, budget=2048, ragged=False),
        # prompts cut down to an eighth
        dict(name="choose_many", op="choose", batch=32, kv=32768, kv_heads=8, page=64, budget=4096, ragged=True),
        # the accepted paths of a batch of trees: latency
        dict(name="keep_paths_bf16", op="keep", kind="bf16", batch=16, chunk=32, kv=4096, kv_heads=8, head_dim=128, page=16, budget=6,
             path=True, ragged=True),
        # long prompts cut down to a quarter, every head by its own choice, the weights moved along
        dict(name="keep_chosen_bf16", op="keep", kind="bf16", batch=8, chunk=0, kv=32768, kv_heads=8, head_dim=128, page=64, budget=8192,
             path=False, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "tree", "verify", "weigh", "weigh", "choose", "keep"))
    if op == "verify":
        return dict(op=op, dtype=rng.choice(("float32", "bfloat16")), batch=_log(rng, 1, 96), chunk=_log(rng, 1, 32),
                    vocab=_log(rng, 1000, 100003), ragged=rng.random() < 0.8)
    page = rng.choice((1, 7, 16, 16, 32, 48, 64, 128))
    kv_heads = rng.choice((1, 2, 3, 4, 8, 8, 32))
    if op == "choose":
        case = dict(op=op, batch=_log(rng, 1, 64), kv_heads=kv_heads, page=page, ragged=rng.random() < 0.8)
        case["kv"] = min(_log(rng, 16, (1 << 23) // (case["batch"] * kv_heads)), 131000)
        case["budget"] = rng.choice((max(1, case["kv"] - _log(rng, 1, case["kv"])), _log(rng, 1, case["kv"])))
        return case
    case = dict(op=op, kind=rng.choice(tuple(BITS)), page=page, head_dim=rng.choice((32, 64, 96, 128, 128, 128, 192, 256)),
                kv_heads=kv_heads, ragged=rng.random() < 0.8)
    width = case["head_dim"] * kv_heads
    if op == "keep":
        case.update(batch=_log(rng, 1, 32), path=rng.random() < 0.4)
        case["kv"] = min(_log(rng, 80, max(81, (1 << 27) // (case["batch"] * width))), 32768)
        case["chunk"] = _log(rng, 2, 64) if case["path"] else 0
        case["budget"] = _log(rng, 1, min(case["chunk"], 8)) if case["path"] else _log(rng, 1, case["kv"])
        return case
    case.update(dtype=rng.choice(("bfloat16", "bfloat16", "float32")), window=rng.choice((0, 0, 0, _log(rng, 1, 4096))),
                heads=kv_heads * rng.choice((1, 2, 4, 6, 8) if kv_heads < 32 else (1, 2)))
    if op == "tree":
        case.update(chunk=_log(rng, 1, 64), batch=_log(rng, 1, 32))
    else:
        kind = rng.choice(("token", "last", "chunk"))
        case["chunk"] = {"token": 1, "last": rng.randint(2, 64), "chunk": _log(rng, 64, 2048)}[kind]
        case["batch"] = _log(rng, 1, 4 if kind == "chunk" else 64)
        case["fresh"] = rng.random() < 0.5
    most = min((1 << 27) // (case["batch"] * width), (1 << 33) // (case["batch"] * case["heads"] * case["head_dim"] * case["chunk"]))
    case["kv"] = max(case["chunk"], min(_log(rng, 16, max(17, most)), 131000))
    return case


def _plan(case):
    """Host side of a batch: (new tokens of each sequence, lengths, max_pages)."""
    rng = random.Random("%s %s %s %s" % (case["batch"], case.get("chunk"), case.get("kv"), case.get("page")))
    b, chunk, kv = case["batch"], case.get("chunk", 0), case.get("kv", 1)
    new = [chunk if i == 0 or not case["ragged"] else rng.randint((chunk + 1) // 2, chunk) for i in range(b)]
    if "kv" not in case:
        return new, new, 0
    lens = [kv if i == 0 or not case["ragged"] else rng.randint(max(1, kv // 4), kv) for i in range(b)]
    return [min(n, m) for n, m in zip(new, lens)], lens, -(-kv // case["page"])


def _batch(case, gen):
    """starts, lens and table on the GPU, and the number of pages; pages lie in random order."""
    new, lens, max_pages = _plan(case)
    need = [-(-n // case["page"]) for n in lens]
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.tensor(np.cumsum([0] + need[:-1]), device="cuda")
    slot = torch.arange(max_pages, device="cuda")
    used = slot[None] < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(used, ids[(at[:, None] + slot[None]).clamp(max=pages - 1)], -1).contiguous()
    starts = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda")
    return starts, torch.tensor(lens, dtype=torch.int32, device="cuda"), table, pages


def _trees(case):
    """Parents of every sequence's nodes: node 0 is the root, a node's parent one of the two thirds before it."""
    rng = random.Random("trees %s %s" % (case["batch"], case["chunk"]))
    return [[-1] + [rng.randint((i - 1) // 3, i - 1) for i in range(1, n)] for n in _plan(case)[0]]


def _block(case):
    row = case["head_dim"] * BITS[case["kind"]] // 8
    groups = 0 if case["kind"] == "bf16" else case["head_dim"] // 32
    return row, groups, (2 * case["page"] * (row + groups) + 15) // 16 * 16


def _regions(case, pool):
    """Views of a pool: (codes, scales) of the keys, then of the values, [pages][kv_heads][page][...]."""
    row, groups, block = _block(case)
    p = case["page"]
    blocks = pool.view(-1, case["kv_heads"], block)
    codes = blocks[..., :2 * p * row].unflatten(-1, (2, p, row))
    scales = blocks[..., 2 * p * row:2 * p * (row + groups)].unflatten(-1, (2, p, groups)) if groups else None
    return [(codes[:, :, i], None if scales is None else scales[:, :, i]) for i in (0, 1)]


def _quantise(x, kind):
    """(codes uint8, scale bytes) of finite x [..., D]."""
    if kind == "bf16":
        return x.to(torch.bfloat16).contiguous().view(torch.uint8), None
    top, most, high = (0.875, 448.0, 119) if kind == "fp8" else (0.75, 6.0, 125)
    g = x.float().unflatten(-1, (-1, 32))
    amax = g.abs().amax(-1)
    mant, ex = torch.frexp(amax)
    e = ex - (9 if kind == "fp8" else 3) + (mant > top)
    e = torch.where(amax > 0, e, -100).clamp(-100, high)
    y = (g * torch.ldexp(torch.ones_like(amax), -e)[..., None]).clamp(-most, most).flatten(-2)
    scale = (e + 127).to(torch.uint8)
    if kind == "fp8":
        return y.to(torch.float8_e4m3fn).view(torch.uint8), scale
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + 8 * torch.signbit(y).to(torch.uint8))
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _values(codes, scale, kind):
    """The f32 values of codes [..., row] and scale bytes [..., D / 32]."""
    if kind == "bf16":
        return codes.contiguous().view(torch.bfloat16).float()
    if kind == "fp8":
        v = codes.contiguous().view(torch.float8_e4m3fn).float()
    else:
        lut = torch.tensor(FP4 + tuple(-f for f in FP4), device=codes.device)
        v = lut[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    f = torch.ldexp(torch.ones(scale.shape, device=codes.device), scale.int() - 127)
    return (v.unflatten(-1, (-1, 32)) * f[..., None]).flatten(-2)


def _held(x, kind):
    """What the cache holds for x, in 64 bits."""
    return _values(*_quantise(x, kind), kind).double()


def _positions(starts, lens, n):
    """(sequence, position) of each of n new tokens."""
    row = torch.arange(n, device="cuda")
    seq = torch.searchsorted(starts[1:].long(), row, right=True)
    return seq, lens[seq] - starts[seq + 1] + row.int()


def _tokens(n, heads, dim, gen):
    """Keys or values of n tokens: normal, with a few channels that are much larger, as keys have them."""
    x = torch.randn(n, heads, dim, generator=gen, device="cuda")
    gain = torch.rand(heads, dim, generator=gen, device="cuda")
    return (x * torch.where(gain > 0.97, 6.0, 0.5 + gain)).bfloat16()


def _exponential(shape, gen):
    return torch.empty(shape, device="cuda").exponential_(generator=gen).clamp_(min=1e-30)


def _inputs(case, seed):
    """What exists before quantisation."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "verify":
        # distributions as a model has them: one token or a few hold most of the mass; a node's children are its
        # likeliest tokens in order
        trees, v = _trees(case), case["vocab"]
        n = sum(len(t) for t in trees)
        target = torch.softmax(5.0 * torch.randn(n, v, generator=gen, device="cuda"), -1).to(getattr(torch, case["dtype"]))
        rank, above, base = [], [], 0
        for t in trees:
            rank += [sum(p == t[i] for p in t[:i]) for i in range(len(t))]
            above += [base + max(p, 0) for p in t]
            base += len(t)
        best = target.float().topk(max(rank) + 1, -1).indices
        tokens = best[torch.tensor(above, device="cuda"), torch.tensor(rank, device="cuda")].int()
        return dict(target=target, tokens=tokens, parents=torch.tensor(sum(trees, []), dtype=torch.int32, device="cuda"),
                    starts=torch.tensor(np.cumsum([0] + [len(t) for t in trees]), dtype=torch.int32, device="cuda"),
                    uniforms=torch.rand(n, generator=gen, device="cuda"), noise=_exponential((case["batch"], v), gen))
    starts, lens, table, pages = _batch(case, gen)
    new, kv, _ = _plan(case)
    made = dict(starts=starts, lens=lens, table=table, pages=pages, new=sum(new))
    b, hkv, most = case["batch"], case["kv_heads"], case["kv"]
    if case["op"] != "choose":
        made["ends"] = torch.tensor(np.cumsum([0] + kv), dtype=torch.int32, device="cuda")
        made["k"], made["v"] = (_tokens(sum(kv), hkv, case["head_dim"], gen) for _ in range(2))
    if case["op"] in ("tree", "weigh"):
        q = torch.randn(sum(new), case["heads"], case["head_dim"], generator=gen, device="cuda")
        made["q"] = (1.5 * q).to(getattr(torch, case["dtype"]))
    if case["op"] == "tree":
        made["parents"] = torch.tensor(sum(_trees(case), []), dtype=torch.int32, device="cuda")
    if case["op"] in ("weigh", "choose") or (case["op"] == "keep" and not case["path"]):
        # a few tokens hold most of the weight; some have never been seen
        shape = (pages, hkv, case["page"])
        w = torch.exp(2.0 * torch.randn(shape, generator=gen, device="cuda"))
        made["weights"] = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.05, 0.0, w)
    if case["op"] == "keep" and case["path"]:
        rng = random.Random("path %s" % seed)
        keep = torch.full((b, 1, case["budget"]), -1, dtype=torch.int32)
        for i, n in enumerate(new):
            path = [0] + sorted(rng.sample(range(1, n), min(rng.randint(0, case["budget"] - 1), n - 1)))
            keep[i, 0, :len(path)] = torch.tensor(path[:case["budget"]], dtype=torch.int32)
        made["keep"] = keep.cuda()
        made["counts"] = (made["keep"][:, 0] >= 0).sum(-1).int()
    elif case["op"] == "keep":
        at = torch.arange(most, device="cuda")
        rank = torch.rand(b, hkv, most, generator=gen, device="cuda")
        rank = torch.where((at >= lens[:, None, None] - case["budget"] // 4) | (at < 4), 2.0, rank)
        rank = torch.where(at < lens[:, None, None], rank, -1.0)
        keep = rank.topk(case["budget"], -1).indices.sort(-1).values.int()
        made["keep"] = torch.where(keep < lens[:, None, None], keep, -1).contiguous()
        made["counts"] = lens.clamp(max=case["budget"])
    return made


def _store(case, pool, k, v, starts, lens, table):
    seq, pos = _positions(starts, lens, k.shape[0])
    page, slot = table[seq, pos // case["page"]].long(), (pos % case["page"]).long()
    for x, (codes, scales) in zip((k, v), _regions(case, pool)):
        c, s = _quantise(x, case["kind"])
        codes[page, :, slot] = c
        if s is not None:
            scales[page, :, slot] = s


def prepare(case, seed):
    made = _inputs(case, seed)
    made["case"] = case
    if case["op"] in ("verify", "choose"):
        return made
    pool = torch.zeros(made["pages"] * case["kv_heads"] * _block(case)[2], dtype=torch.uint8, device="cuda")
    _store(case, pool, made.pop("k"), made.pop("v"), made.pop("ends"), made["lens"], made["table"])
    made["pool"] = pool
    if case["op"] == "weigh":
        # the attention of the same rows has given their log-sums before
        made["lse"] = _row_sums(*_scores(made))
    return made


def _cached(state, which):
    """Keys or values [B][kv_heads][kv][D] in f32, zero past a sequence's end."""
    case, lens = state["case"], state["lens"]
    key = torch.arange(case["kv"], device="cuda")
    page = state["table"][:, key // case["page"]].clamp(min=0).long()
    c, s = _regions(case, state["pool"])[which]
    x = _values(c[page, :, key % case["page"]], None if s is None else s[page, :, key % case["page"]], case["kind"])
    return x.masked_fill(key[None, :, None, None] >= lens[:, None, None, None], 0.0).transpose(1, 2).contiguous()


def _ancestors(state, chunk):
    """[B][chunk][chunk]: whether node j is node i or above it; and the depth of each node."""
    starts, b = state["starts"].long(), state["case"]["batch"]
    step = torch.arange(chunk, device="cuda")
    row = starts[:-1, None] + step[None]
    there = row < starts[1:, None]
    parent = torch.where(there, state["parents"][row.clamp(max=state["new"] - 1)].long(), -1)
    at = step[None].expand(b, -1).clone()
    above = torch.zeros(b, chunk, chunk, dtype=torch.bool, device="cuda")
    for _ in range(chunk):
        above |= (at[..., None] == step) & (at >= 0)[..., None]
        at = torch.where(at >= 0, parent.gather(1, at.clamp(min=0)), -1)
    return above, above.sum(-1) - 1


def _scores(state):
    """Scaled scores [B][kv_heads][share][chunk][kv] in f32, minus infinity where a row does not see the key."""
    case = state["case"]
    starts, lens, q = state["starts"], state["lens"], state["q"]
    b, hkv, d, chunk, kv = case["batch"], case["kv_heads"], case["head_dim"], case["chunk"], case["kv"]
    share = case["heads"] // hkv
    key, step = torch.arange(kv, device="cuda"), torch.arange(chunk, device="cuda")
    new = starts[1:] - starts[:-1]
    row = (starts[:-1, None] + step[None]).clamp(max=q.shape[0] - 1).long()
    qs = q.float()[row].view(b, chunk, hkv, share, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, share * chunk, d)
    s = torch.matmul(qs, _cached(state, 0).transpose(-1, -2)).view(b, hkv, share, chunk, kv) * (1.0 / math.sqrt(d))
    text = (lens - new)[:, None, None]
    if case["op"] == "tree":
        above, depth = _ancestors(state, chunk)
        node = (key[None, None] - text).clamp(0, chunk - 1).expand(b, chunk, kv)
        seen = torch.where(key < text, True, above.gather(2, node) & (key < lens[:, None, None]))
        place = torch.where(key < text, key, text + depth.gather(1, node[:, 0])[:, None])
        pos = text + depth[..., None]
    else:
        place, pos = key, text + step[:, None]
        seen = (place <= pos) & (key < lens[:, None, None])
    if case["window"]:
        seen = seen & (place > pos - case["window"])
    seen = seen & (step[None] < new[:, None])[..., None]
    return s.masked_fill(~seen[:, None, None], -math.inf), seen


def _row_sums(s, seen):
    """log sum_j exp(s_j) of the real rows, [rows][heads]."""
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    lse = (torch.log(torch.exp(s - top).sum(-1, keepdim=True)) + top)[..., 0]
    b, hkv, share, chunk = lse.shape
    real = seen.any(-1)
    return lse.permute(0, 3, 1, 2).reshape(b, chunk, hkv * share)[real].contiguous()


def _by_row(x, state):
    """[B][chunk][...] -> [rows][...]."""
    at = torch.arange(state["new"], device="cuda")
    seq = torch.searchsorted(state["starts"][1:].long(), at, right=True)
    return x[seq, at - state["starts"][seq]]


def _plain_tree(state):
    case = state["case"]
    s, _ = _scores(state)
    b, hkv, share, chunk, kv = s.shape
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul((p / torch.where(total > 0, total, 1.0)).view(b, hkv, share * chunk, kv), _cached(state, 1))
    o = o.view(b, hkv, share, chunk, -1).permute(0, 3, 1, 2, 4).reshape(b, chunk, case["heads"], -1)
    return _by_row(o, state).to(state["q"].dtype)


def _plain_weigh(state):
    case, lens, weights = state["case"], state["lens"], state["weights"]
    s, _ = _scores(state)
    b, hkv, share, chunk, kv = s.shape
    step = torch.arange(chunk, device="cuda")
    row = (state["starts"][:-1, None] + step[None]).clamp(max=state["new"] - 1).long()
    lse = state["lse"][row].view(b, chunk, hkv, share).permute(0, 2, 3, 1)
    got = torch.exp(s - lse[..., None]).sum((2, 3))
    key = torch.arange(kv, device="cuda")
    seq, at = torch.nonzero(key[None] < lens[:, None], as_tuple=True)
    page, slot = state["table"][seq, at // case["page"]].long(), at % case["page"]
    old = weights[page, :, slot]
    first = lens - (state["starts"][1:] - state["starts"][:-1])
    keeps = (at < first[seq]) & (not case["fresh"])
    weights[page, :, slot] = torch.where(keeps[:, None], old, 0.0) + got[seq, :, at]
    return weights


def _first_best(weight, noise):
    """argmax of weight / noise over the entries of positive weight, ties to the lowest index; (index, any)."""
    score = torch.where((weight > 0) & (noise >= 0), weight / noise, -1.0)
    best = score.amax(-1, keepdim=True)
    at = torch.arange(score.shape[-1], device="cuda")
    return torch.where(score == best, at, score.shape[-1]).amin(-1), best[:, 0] >= 0


def _plain_verify(state):
    target, starts, parents, tokens = state["target"], state["starts"].long(), state["parents"], state["tokens"]
    b, chunk = state["case"]["batch"], state["case"]["chunk"]
    n, each = starts[1:] - starts[:-1], torch.arange(b, device="cuda")
    current = torch.zeros(b, dtype=torch.long, device="cuda")
    left = torch.ones(b, dtype=torch.float64, device="cuda")
    fallen = torch.zeros(b, chunk, dtype=torch.bool, device="cuda")      # unaccepted children of the current node
    path = torch.full((b, chunk), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    done = torch.zeros(b, dtype=torch.long, device="cuda")
    node_tokens = tokens[(starts[:-1, None] + torch.arange(chunk, device="cuda")).clamp(max=tokens.numel() - 1)]
    for i in range(1, chunk):
        row = (starts[:-1] + i).clamp(max=tokens.numel() - 1)
        child = (i < n) & (parents[row] == current)
        again = (fallen & (node_tokens == tokens[row][:, None])).any(-1)
        w = torch.where(again, 0.0, target[starts[:-1] + current, tokens[row].long()].double())
        ok = child & (state["uniforms"][row].double() * left.clamp(min=0.0) < w)
        left = torch.where(ok, 1.0, torch.where(child, left - w, left))
        fallen[:, i] = child
        fallen &= ~ok[:, None]
        current = torch.where(ok, i, current)
        done = done + ok
        path[each, done] = torch.where(ok, i, path[each, done])
    out = torch.where(path > 0, node_tokens.gather(1, path.clamp(min=0).long()), -1)
    out = torch.cat((out[:, 1:], torch.full((b, 1), -1, dtype=torch.int32, device="cuda")), 1)
    p = target[starts[:-1] + current].float()
    dropped = torch.zeros(b, p.shape[1], dtype=torch.int32, device="cuda")
    dropped.scatter_reduce_(1, node_tokens.long(), fallen.int(), "amax")
    first, some = _first_best(p.masked_fill(dropped > 0, 0.0), state["noise"])
    other, any_ = _first_best(p, state["noise"])
    out.scatter_(1, done[:, None], torch.where(some, first, torch.where(any_, other, -1)).int()[:, None])
    return [done.int(), path, out]


def _plain_choose(state):
    case, lens = state["case"], state["lens"][:, None, None]
    key, budget = torch.arange(case["kv"], device="cuda"), case["budget"]
    sinks, recent = _protected(case)
    page = state["table"][:, key // case["page"]].clamp(min=0).long()
    w = state["weights"][page, :, key % case["page"]].transpose(1, 2)
    w = torch.where((key < sinks) | (key >= lens - recent), math.inf, w)
    w = torch.where(key < lens, w, -math.inf)
    order = w.sort(stable=True, dim=-1, descending=True).indices[..., :budget]
    keep = torch.where(torch.arange(budget, device="cuda") < lens, order, case["kv"]).sort(-1).values
    return [torch.where(keep < case["kv"], keep, -1).int(), state["lens"].clamp(max=budget)]


def _protected(case):
    """First and last tokens that always stay."""
    sinks = min(4, case["budget"] // 4)
    return sinks, (case["budget"] - sinks) // 4


def _plain_keep(state):
    case, keep, counts = state["case"], state["keep"].long(), state["counts"].long()
    lens, table = state["lens"].long(), state["table"].long()
    first = (lens - (state["starts"][1:] - state["starts"][:-1]))[:, None, None] if case["path"] else 0
    keep = keep.expand(-1, case["kv_heads"], -1)
    to = torch.arange(keep.shape[-1], device="cuda")
    seq, head, i = torch.nonzero((to < counts[:, None, None]) & (keep >= 0), as_tuple=True)
    src = (first + keep)[seq, head, i]
    dst = (first + to.expand_as(keep))[seq, head, i]
    page, slot = table[seq, src // case["page"]], src % case["page"]
    new_page, new_slot = table[seq, dst // case["page"]], dst % case["page"]
    parts = [x for pair in _regions(case, state["pool"]) for x in pair if x is not None]
    if "weights" in state:
        parts.append(state["weights"])
    for x in parts:
        x[new_page, head, new_slot] = x[page, head, slot]


def _kept_rows(state):
    """starts and lens of the tokens that stand in their new places."""
    if "kept" not in state:
        counts = state["counts"]
        starts = torch.cat((counts.new_zeros(1), counts.cumsum(0).int()))
        first = state["lens"] - (state["starts"][1:] - state["starts"][:-1]) if state["case"]["path"] else 0
        state["kept"] = starts, first + counts, int(starts[-1])
    return state["kept"]


def _moved(state, k, v):
    """What a pass of the move gives back: the pool's values in the bf16 kind, else the kept tokens read back."""
    pool = [state["pool"].view(torch.bfloat16)] if k is None else [k, v]
    return pool + ([state["weights"]] if "weights" in state else [])


def _own(state):
    import weight_decompression_amd as wd
    case = state["case"]
    if case["op"] == "verify":
        b, v, n = case["batch"], case["vocab"], case["chunk"]
        accepted = torch.empty(b, dtype=torch.int32, device="cuda")
        path, out = (torch.empty(b, n, dtype=torch.int32, device="cuda") for _ in range(2))
        if "workspace" not in state:
            state["workspace"] = torch.empty(wd.tree_workspace_bytes(b, v), dtype=torch.uint8, device="cuda")
        wd.tree_verify(state["target"], state["starts"], state["tokens"], state["parents"], state["uniforms"], state["noise"],
                       accepted, path, out, state["workspace"])
        return [accepted, path, out]
    starts, lens, table = state["starts"], state["lens"], state["table"]
    if "desc" not in state:
        kind = {"bf16": wd.KV_BF16, "fp8": wd.KV_FP8, "fp4": wd.KV_FP4}[case.get("kind", "fp8")]
        state["desc"] = wd.make_kv_desc(kind, case["kv_heads"], case.get("head_dim", 128), case["page"], state["pages"])
    desc = state["desc"]
    if case["op"] == "tree":
        out = torch.empty_like(state["q"])
        if "workspace" not in state:
            size = wd.attn_workspace_bytes(desc, case["heads"], state["new"], case["batch"], case["chunk"], case["kv"])
            state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        wd.attn_tree(desc, state["pool"], state["q"], out, starts, lens, table, state["parents"], state["workspace"],
                     max_chunk=case["chunk"], max_len=case["kv"], window=case["window"])
        return [out]
    if case["op"] == "weigh":
        wd.kv_weigh(desc, state["pool"], state["weights"], state["q"], state["lse"], starts, lens, table, max_chunk=case["chunk"],
                    max_len=case["kv"], window=case["window"], fresh=case["fresh"])
        return [state["weights"]]
    if case["op"] == "choose":
        keep = torch.empty(case["batch"], case["kv_heads"], case["budget"], dtype=torch.int32, device="cuda")
        counts = torch.empty(case["batch"], dtype=torch.int32, device="cuda")
        sinks, recent = _protected(case)
        wd.kv_choose(desc, state["weights"], lens, table, keep, counts, sinks=sinks, recent=recent)
        return [keep, counts]
    wd.kv_keep(desc, state["pool"], state["keep"], lens, table, counts=state["counts"], starts=starts if case["path"] else None,
               weights=state.get("weights"))
    if case["kind"] == "bf16":
        return _moved(state, None, None)
    kept, ends, n = _kept_rows(state)
    k, v = (torch.empty(n, case["kv_heads"], case["head_dim"], dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wd.kv_read(desc, state["pool"], k, v, kept, ends, table)
    return _moved(state, k, v)


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "verify":
        return _plain_verify(state)
    if case["op"] == "tree":
        return [_plain_tree(state)]
    if case["op"] == "weigh":
        return [_plain_weigh(state)]
    if case["op"] == "choose":
        return _plain_choose(state)
    _plain_keep(state)
    if case["kind"] == "bf16":
        return _moved(state, None, None)
    starts, lens, n = _kept_rows(state)
    seq, pos = _positions(starts, lens, n)
    page, slot = state["table"][seq, pos // case["page"]].long(), (pos % case["page"]).long()
    return _moved(state, *[_values(c[page, :, slot], None if s is None else s[page, :, slot], case["kind"]).bfloat16()
                           for c, s in _regions(case, state["pool"])])


def work(case):
    new, lens, _ = _plan(case)
    if case["op"] == "verify":
        size = 4 if case["dtype"] == "float32" else 2
        # the row that each sequence draws from, its noise, a probability and four numbers a node, three numbers out
        return {"bytes": case["batch"] * (case["vocab"] * (size + 4) + 8 * case["chunk"]) + sum(new) * (size + 12),
                "flops": case["batch"] * case["vocab"]}
    if case["op"] == "choose":
        kept = sum(min(m, case["budget"]) for m in lens)
        return {"bytes": 4 * case["kv_heads"] * (sum(lens) + kept), "flops": case["kv_heads"] * sum(lens)}
    row, groups, _ = _block(case)
    token = 2 * case["kv_heads"] * (row + groups)
    if case["op"] == "keep":
        # tokens that change places: on a path about half of those that fit; of a choice all but the first four
        moved = sum(min(m, (case["budget"] - 1) / 2 if case["path"] else max(case["budget"] - 4, 0)) for m in lens)
        wide = 0 if case["path"] else 4 * case["kv_heads"]
        back = 0
        if case["kind"] != "bf16":
            kept = sum(min(m, (case["budget"] + 1) / 2 if case["path"] else case["budget"]) for m in lens)
            back = kept * (token + 4 * case["kv_heads"] * case["head_dim"])
        return {"bytes": int(moved * 2 * (token + wide) + back) + 4, "flops": 0}
    size = 4 if case["dtype"] == "float32" else 2
    pairs, keys = 0, 0
    trees = _trees(case) if case["op"] == "tree" else None
    for b, (n, m) in enumerate(zip(new, lens)):
        w = case["window"] or m
        if trees is not None:
            depth = []
            for p in trees[b]:
                depth.append(0 if p < 0 else depth[p] + 1)
            pairs += sum(min(d + 1, w) + min(m - n, max(w - d - 1, 0)) for d in depth)
            keys += min(m - n, w - 1) + n
        else:
            pairs += int(np.minimum(np.arange(m - n, m) + 1, w).sum())
            keys += min(m, n + w - 1)
    rows = sum(new) * case["heads"]
    if case["op"] == "tree":
        return {"bytes": keys * token + 2 * rows * case["head_dim"] * size, "flops": 4 * pairs * case["heads"] * case["head_dim"]}
    times = sum(lens) if case["fresh"] else 2 * keys - sum(new)
    return {"bytes": keys * token // 2 + rows * (case["head_dim"] * size + 4) + 4 * case["kv_heads"] * times,
            "flops": 2 * pairs * case["heads"] * case["head_dim"]}


def _exact_keep(case, seed):
    state, made = prepare(case, seed), _inputs(case, seed)
    new, lens, _ = _plan(case)
    page, hkv, table = case["page"], case["kv_heads"], state["table"].long()
    weights = state["weights"].double() if "weights" in state else None
    k, v, end, kept = _held(made["k"], case["kind"]), _held(made["v"], case["kind"]), 0, []
    cache = state["pool"].view(torch.bfloat16).double().view(-1, hkv, 2, page, case["head_dim"]) if case["kind"] == "bf16" else None
    for b, (n, m) in enumerate(zip(new, lens)):
        count, first, rows = int(state["counts"][b]), m - n if case["path"] else 0, []
        dst = torch.arange(first, first + count, device="cuda")
        for h in range(hkv):
            src = first + state["keep"][b, h % state["keep"].shape[1], :count].long()
            rows.append(torch.stack((k[end + src, h], v[end + src, h])))
            old, there = (table[b, src // page], h), (table[b, dst // page], h)
            if weights is not None:
                weights[there + (dst % page,)] = weights[old + (src % page,)]
            if cache is not None:
                cache[there[0], h, :, dst % page] = rows[-1].transpose(0, 1)
        kept.append(torch.stack(rows, 2))
        end += m
    kept = torch.cat(kept, 1)
    return ([kept[0], kept[1]] if cache is None else [cache.flatten()]) + ([] if weights is None else [weights])


def exact(case, seed):
    if case["op"] == "keep":
        return _exact_keep(case, seed)
    if case["op"] not in ("tree", "weigh"):
        return None
    state = prepare(case, seed)
    made = _inputs(case, seed)
    new, lens, _ = _plan(case)
    hkv, d = case["kv_heads"], case["head_dim"]
    share, first, end, outs = case["heads"] // hkv, 0, 0, []
    weights = state["weights"].double() if case["op"] == "weigh" else None
    for b, (n, m) in enumerate(zip(new, lens)):
        at = torch.arange(m, device="cuda")
        if case["op"] == "tree":
            parent = _trees(case)[b]
            seen, place = np.zeros((n, m), bool), np.arange(m)
            for i in range(n):
                up = []
                j = i
                while j >= 0:
                    up.append(j)
                    j = parent[j]
                place[m - n + i] = m - n + len(up) - 1
                seen[i, :m - n] = True
                seen[i, [m - n + j for j in up]] = True
            if case["window"]:
                seen &= place[None, :] > place[m - n:, None] - case["window"]
            seen = torch.tensor(seen, device="cuda")
        else:
            gap = torch.arange(m - n, m, device="cuda")[:, None] - at[None]
            seen = (gap >= 0) & (gap < (case["window"] or m))
        got = torch.zeros(m, hkv, dtype=torch.float64, device="cuda")
        out = torch.empty(n, hkv, share, d, dtype=torch.float64, device="cuda")
        for h in range(hkv):
            q = made["q"][first:first + n, h * share:(h + 1) * share].double()
            keys = _held(made["k"][end:end + m, h], case["kind"])
            s = (q.reshape(n * share, d) @ keys.t()).view(n, share, m) / math.sqrt(d)
            s = s.masked_fill(~seen[:, None], -math.inf)
            if case["op"] == "tree":
                p = torch.softmax(s, -1).view(n * share, m)
                out[:, h] = (p @ _held(made["v"][end:end + m, h], case["kind"])).view(n, share, d)
            else:
                lse = state["lse"][first:first + n, h * share:(h + 1) * share].double()
                got[:, h] = torch.exp(s - lse[..., None]).sum((0, 1))
        if weights is None:
            outs.append(out.flatten(1, 2))
        else:
            page, slot = state["table"][b, at // case["page"]].long(), at % case["page"]
            stays = (at < m - n) & (not case["fresh"])
            weights[page, :, slot] = torch.where(stays[:, None], weights[page, :, slot], 0.0) + got
        first, end = first + n, end + m
    return [torch.cat(outs)] if weights is None else [weights]
