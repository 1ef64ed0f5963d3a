"""Cases for the serving operators: the paged key/value cache (written and read back),
the attention that reads it, and the check of drafted tokens.

Plain forms are written in elementary torch operations in 32 bits.  A cache is one uint8
pool [pages][kv_heads][block]; a block holds, for `page` tokens of one head, the key codes
[page][D * bits / 8], the value codes, the key scales [page][D / 32] and the value scales
(one byte e + 127 for 32 channels, value = code * 2^e; none in the bf16 kind), rounded up to
16 bytes.  A batch is described by starts [B + 1] (rows of each sequence's new tokens), lens
[B] (tokens of each sequence, the new ones included) and table [B][max_pages].
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
        # one new token in each of 16 sequences: the cache's part of a decode step (latency)
        dict(name="cache_write_tokens_fp8", op="write", kind="fp8", dtype="float32", batch=16, chunk=1, kv=900,
             kv_heads=8, head_dim=128, page=16, ragged=True),
        # prompts of several sequences written at once, keys and values of a 4096-wide layer
        dict(name="cache_write_prompt_fp4", op="write", kind="fp4", dtype="bfloat16", batch=5, chunk=4099, kv=6001,
             kv_heads=32, head_dim=128, page=32, ragged=True),
        # a whole cache read back, for a layer that is moved or attended elsewhere
        dict(name="cache_read_all_fp8", op="read", kind="fp8", dtype="bfloat16", batch=12, chunk=0, kv=16384,
             kv_heads=8, head_dim=128, page=64, ragged=True),
        # one answer, one token, a short context: every microsecond is latency
        dict(name="attn_token_one_bf16", op="attn", kind="bf16", dtype="bfloat16", batch=1, chunk=1, kv=777,
             heads=32, kv_heads=32, head_dim=128, page=16, window=0, ragged=False),
        # a decode step of many sequences with shared heads (8192 = 64 x 128)
        dict(name="attn_tokens_many_fp8", op="attn", kind="fp8", dtype="bfloat16", batch=64, chunk=1, kv=16384,
             heads=64, kv_heads=8, head_dim=128, page=16, window=0, ragged=True),
        # a decode step over few long contexts: the axis has to be split
        dict(name="attn_tokens_long_fp4", op="attn", kind="fp4", dtype="bfloat16", batch=3, chunk=1, kv=131000,
             heads=32, kv_heads=8, head_dim=128, page=64, window=0, ragged=True),
        # a step that checks drafted tokens: up to 8 new tokens a sequence, f32 in and out as the fused product writes
        dict(name="attn_drafts_fp8_f32", op="attn", kind="fp8", dtype="float32", batch=16, chunk=8, kv=4096,
             heads=32, kv_heads=32, head_dim=128, page=16, window=0, ragged=True),
        # a chunk of a long prompt over what is cached already (4096 = 32 x 128): compute
        dict(name="attn_chunk_fp8", op="attn", kind="fp8", dtype="bfloat16", batch=2, chunk=2048, kv=8192,
             heads=32, kv_heads=32, head_dim=128, page=16, window=0, ragged=False),
        # ragged chunks, shared heads, a sliding window, narrow heads, pages that no tile divides
        dict(name="attn_chunk_window_fp4", op="attn", kind="fp4", dtype="bfloat16", batch=7, chunk=1021, kv=5003,
             heads=24, kv_heads=4, head_dim=64, page=48, window=1000, ragged=True),
        # wide heads on the unquantised cache
        dict(name="attn_chunk_wide_bf16", op="attn", kind="bf16", dtype="bfloat16", batch=3, chunk=700, kv=3500,
             heads=16, kv_heads=4, head_dim=256, page=16, window=0, ragged=True),
        # one sequence's drafts checked (latency)
        dict(name="verify_one", op="verify", dtype="float32", batch=1, drafts=4, vocab=32000),
        # a full batch over a large odd vocabulary
        dict(name="verify_many", op="verify", dtype="float32", batch=96, drafts=7, vocab=100003),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "attn", "attn", "attn", "verify"))
    if op == "verify":
        return dict(op=op, dtype=rng.choice(("float32", "bfloat16")), batch=_log(rng, 1, 96), drafts=rng.randint(1, 8),
                    vocab=_log(rng, 1000, 100003))
    case = dict(op=op, kind=rng.choice(tuple(BITS)), dtype=rng.choice(("bfloat16", "bfloat16", "float32")),
                page=rng.choice((1, 7, 16, 16, 32, 48, 64, 128)), head_dim=rng.choice((32, 64, 96, 128, 128, 128, 192, 256)),
                kv_heads=rng.choice((1, 2, 3, 4, 8, 8, 32)), ragged=rng.random() < 0.8)
    if op != "attn":
        case.update(batch=_log(rng, 1, 32))
        case["kv"] = _log(rng, 16, max(16, (1 << 27) // (case["batch"] * case["kv_heads"] * case["head_dim"])))
        case["kv"] = min(case["kv"], 32768)
        case["chunk"] = 0 if op == "read" else _log(rng, 1, min(case["kv"], 8192))
        return case
    case["window"] = rng.choice((0, 0, 0, _log(rng, 1, 4096)))
    case["heads"] = case["kv_heads"] * rng.choice((1, 2, 4, 6, 8) if case["kv_heads"] < 32 else (1, 2))
    kind = rng.choice(("token", "drafts", "chunk"))
    case["chunk"] = {"token": 1, "drafts": rng.randint(2, 12), "chunk": _log(rng, 13, 2048)}[kind]
    case["batch"] = _log(rng, 1, 4 if kind == "chunk" else 64)
    width = case["batch"] * case["head_dim"]
    most = (1 << 27) // (width * case["kv_heads"])
    if kind == "chunk":
        most = min(most, (1 << 33) // (width * case["heads"] * case["chunk"]))
    case["kv"] = max(case["chunk"], min(_log(rng, 16, max(17, most)), 131000))
    return case


def _plan(case):
    """Host side of a batch: (new tokens of each sequence, lengths, max_pages)."""
    rng = random.Random("%s %s %s %s" % (case["batch"], case["chunk"], case["kv"], case["page"]))
    b, kv, chunk = case["batch"], case["kv"], case["chunk"]
    lens = [kv if i == 0 or not case["ragged"] else rng.randint(max(1, kv // 4), kv) for i in range(b)]
    if case["op"] == "read":
        new = list(lens)
    else:
        new = [chunk if i == 0 or not case["ragged"] else rng.randint((chunk + 1) // 2, chunk) for i in range(b)]
        new = [min(n, m) for n, m in zip(new, lens)]
    return new, lens, -(-kv // case["page"])


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
    """(codes uint8, scale bytes) of x [..., D]."""
    if kind == "bf16":
        return x.to(torch.bfloat16).contiguous().view(torch.uint8), None
    top, most, high = (0.875, 448.0, 119) if kind == "fp8" else (0.75, 6.0, 125)
    g = x.float().unflatten(-1, (-1, 32))
    amax = g.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    mant, ex = torch.frexp(amax.masked_fill(bad, 1.0))
    e = ex - (9 if kind == "fp8" else 3) + (mant > top)
    e = torch.where(amax > 0, e, -100).clamp(-100, high)
    y = (g * torch.ldexp(torch.ones_like(amax), -e)[..., None]).clamp(-most, most).masked_fill(bad[..., None], 0.0).flatten(-2)
    scale = torch.where(bad, 255, e + 127).to(torch.uint8)
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
    f = torch.where(scale == 255, math.nan, f)
    return (v.unflatten(-1, (-1, 32)) * f[..., None]).flatten(-2)


def _positions(starts, lens, n):
    """(sequence, position) of each of n new tokens."""
    row = torch.arange(n, device="cuda")
    seq = torch.searchsorted(starts[1:].long(), row, right=True)
    return seq, lens[seq] - starts[seq + 1] + row.int()


def _rows(case, n, gen, heads):
    """Keys or values of n tokens: normal, with a few channels that are much larger, as keys have them."""
    x = torch.randn(n, heads, case["head_dim"], generator=gen, device="cuda")
    gain = torch.rand(heads, case["head_dim"], generator=gen, device="cuda")
    return x * torch.where(gain > 0.97, 6.0, 0.5 + gain)


def _inputs(case, seed):
    """What exists before quantisation."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = getattr(torch, case["dtype"])
    if case["op"] == "verify":
        b, s, v = case["batch"], case["drafts"], case["vocab"]
        logits = 2.5 * torch.randn(b, s + 1, v, generator=gen, device="cuda")
        draft = torch.softmax(logits[:, :s] + 0.6 * torch.randn(b, s, v, generator=gen, device="cuda"), -1).to(dtype)
        target = torch.softmax(logits, -1).to(dtype)
        noise = torch.empty(b, v, device="cuda").exponential_(generator=gen).clamp_(min=1e-30)
        race = draft.float() / torch.empty(b, s, v, device="cuda").exponential_(generator=gen).clamp_(min=1e-30)
        counts = torch.randint(0, s + 1, (b,), generator=gen, device="cuda", dtype=torch.int32)
        counts[0] = s
        return dict(target=target, draft=draft, noise=noise, tokens=race.argmax(-1).int(), counts=counts,
                    uniforms=torch.rand(b, s, generator=gen, device="cuda"))
    starts, lens, table, pages = _batch(case, gen)
    new, kv, _ = _plan(case)
    n = sum(new)
    made = dict(starts=starts, lens=lens, table=table, pages=pages, new=n)
    if case["op"] == "write":
        # keys and values as slices of one fused projection's output
        qkv = torch.cat([_rows(case, n, gen, case["kv_heads"]) for _ in range(2)], 1).to(dtype)
        made.update(k=qkv[:, :case["kv_heads"]], v=qkv[:, case["kv_heads"]:])
        return made
    total = sum(kv)
    made.update(k=_rows(case, total, gen, case["kv_heads"]).bfloat16(), v=_rows(case, total, gen, case["kv_heads"]).bfloat16())
    made["ends"] = torch.tensor(np.cumsum([0] + kv), dtype=torch.int32, device="cuda")
    if case["op"] == "attn":
        q = torch.randn(n, case["heads"], case["head_dim"], generator=gen, device="cuda")
        made["q"] = (q * 1.5).to(dtype)
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
    if case["op"] == "verify":
        return made
    pool = torch.zeros(made["pages"] * case["kv_heads"] * _block(case)[2], dtype=torch.uint8, device="cuda")
    if case["op"] != "write":
        _store(case, pool, made.pop("k"), made.pop("v"), made["ends"], made["lens"], made["table"])
    made["pool"] = pool
    return made


def _plain_read(state, dtype):
    case = state["case"]
    seq, pos = _positions(state["starts"], state["lens"], state["new"])
    page, slot = state["table"][seq, pos // case["page"]].long(), (pos % case["page"]).long()
    return [_values(c[page, :, slot], None if s is None else s[page, :, slot], case["kind"]).to(dtype)
            for c, s in _regions(case, state["pool"])]


def _plain_attn(state):
    case = state["case"]
    starts, lens, table, q = state["starts"], state["lens"], state["table"], state["q"]
    b, hkv, d, chunk, kv = case["batch"], case["kv_heads"], case["head_dim"], case["chunk"], case["kv"]
    share = case["heads"] // hkv
    key = torch.arange(kv, device="cuda")
    page = table[:, key // case["page"]].clamp(min=0).long()
    inside = key[None] < lens[:, None]
    k, v = (_values(c[page, :, key % case["page"]], None if s is None else s[page, :, key % case["page"]], case["kind"])
            .masked_fill(~inside[:, :, None, None], 0.0).transpose(1, 2).contiguous() for c, s in _regions(case, state["pool"]))
    step = torch.arange(chunk, device="cuda")
    new = starts[1:] - starts[:-1]
    row = (starts[:-1, None] + step[None]).clamp(max=q.shape[0] - 1).long()
    qs = q.float()[row].view(b, chunk, hkv, share, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, share * chunk, d)
    s = torch.matmul(qs, k.transpose(-1, -2)).view(b, hkv, share, chunk, kv) * (1.0 / math.sqrt(d))
    pos = (lens - new)[:, None] + step[None]
    seen = inside[:, None] & (key[None, None] <= pos[..., None])
    if case["window"]:
        seen = seen & (key[None, None] > pos[..., None] - case["window"])
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul((p / torch.where(total > 0, total, 1.0)).view(b, hkv, share * chunk, kv), v)
    o = o.view(b, hkv, share, chunk, d).permute(0, 3, 1, 2, 4).reshape(b, chunk, case["heads"], d)
    seq = torch.searchsorted(starts[1:].long(), torch.arange(q.shape[0], device="cuda"), right=True)
    return o[seq, torch.arange(q.shape[0], device="cuda") - starts[seq]].to(q.dtype)


def _first_best(weight, noise):
    """argmax of weight / noise over the entries of positive weight, ties to the lowest index; (index, any)."""
    score = torch.where((weight > 0) & (noise >= 0), weight / noise, -1.0)
    best = score.amax(-1, keepdim=True)
    at = torch.arange(score.shape[-1], device="cuda")
    return torch.where(score == best, at, score.shape[-1]).amin(-1), best[:, 0] >= 0


def _plain_verify(state):
    target, draft, tokens, counts = state["target"], state["draft"], state["tokens"].long(), state["counts"]
    b, s, _ = draft.shape
    at = torch.arange(s, device="cuda")
    p = target[:, :s].gather(-1, tokens[..., None])[..., 0].float()
    q = draft.gather(-1, tokens[..., None])[..., 0].float()
    ok = (state["uniforms"] * q < p) & (at[None] < counts[:, None])
    accepted = ok.int().cumprod(-1).sum(-1)
    each = torch.arange(b, device="cuda")
    whole = accepted >= counts
    row = target[each, accepted].float()
    rest = row - torch.where(whole[:, None], 0.0, draft[each, accepted.clamp(max=s - 1)].float())
    first, some = _first_best(rest, state["noise"])
    other, any_ = _first_best(row, state["noise"])
    last = torch.where(some, first, torch.where(any_, other, -1)).int()
    out = torch.where(at[None] < accepted[:, None], state["tokens"], -1)
    out = torch.cat((out, torch.full((b, 1), -1, dtype=torch.int32, device="cuda")), 1)
    out.scatter_(1, accepted[:, None], last[:, None])
    return [accepted.int(), out]


def _own(state):
    import weight_decompression_amd as wd
    case = state["case"]
    if case["op"] == "verify":
        b, s, v = state["draft"].shape
        accepted = torch.empty(b, dtype=torch.int32, device="cuda")
        out = torch.empty(b, s + 1, dtype=torch.int32, device="cuda")
        if "workspace" not in state:
            state["workspace"] = torch.empty(wd.draft_workspace_bytes(b, v), dtype=torch.uint8, device="cuda")
        wd.draft_verify(state["target"], state["draft"], state["tokens"], state["uniforms"], state["noise"], accepted, out,
                        state["workspace"], counts=state["counts"])
        return [accepted, out]
    if "desc" not in state:
        kind = {"bf16": wd.KV_BF16, "fp8": wd.KV_FP8, "fp4": wd.KV_FP4}[case["kind"]]
        state["desc"] = wd.make_kv_desc(kind, case["kv_heads"], case["head_dim"], case["page"], state["pages"])
    desc, pool, plan = state["desc"], state["pool"], (state["starts"], state["lens"], state["table"])
    if case["op"] == "attn":
        out = torch.empty_like(state["q"])
        if "workspace" not in state:
            size = wd.attn_workspace_bytes(desc, case["heads"], state["new"], case["batch"], case["chunk"], case["kv"])
            state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        wd.attn(desc, pool, state["q"], out, *plan, state["workspace"], max_chunk=case["chunk"], max_len=case["kv"],
                window=case["window"])
        return [out]
    if case["op"] == "write":
        wd.kv_write(desc, pool, state["k"], state["v"], *plan)
    shape = (state["new"], case["kv_heads"], case["head_dim"])
    k, v = (torch.empty(shape, dtype=getattr(torch, case["dtype"]), device="cuda") for _ in range(2))
    wd.kv_read(desc, pool, k, v, *plan)
    return [k, v]


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "verify":
        return _plain_verify(state)
    if case["op"] == "attn":
        return [_plain_attn(state)]
    if case["op"] == "write":
        _store(case, state["pool"], state["k"], state["v"], state["starts"], state["lens"], state["table"])
    return _plain_read(state, getattr(torch, case["dtype"]))


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "verify":
        b, s, v = case["batch"], case["drafts"], case["vocab"]
        return {"bytes": b * v * (2 * size + 4) + b * s * (2 * size + 8) + 4 * b * (s + 3), "flops": 2 * b * v}
    new, lens, _ = _plan(case)
    row, groups, _ = _block(case)
    token = 2 * case["kv_heads"] * (row + groups)
    wide = 2 * case["kv_heads"] * case["head_dim"] * size
    if case["op"] != "attn":
        # a write reads the new keys and values, writes their codes, and gives the values back from them
        times = 2 if case["op"] == "write" else 1
        return {"bytes": sum(new) * (wide + token) * times, "flops": 2 * sum(new) * case["kv_heads"] * case["head_dim"] * times}
    pairs, keys = 0, 0
    for n, m in zip(new, lens):
        w = case["window"] or m
        at = np.arange(m - n, m)
        pairs += int(np.minimum(at + 1, w).sum())
        keys += min(m, n + w - 1)
    return {"bytes": keys * token + 2 * sum(new) * case["heads"] * case["head_dim"] * size,
            "flops": 4 * pairs * case["heads"] * case["head_dim"]}


def _nearest(x, grid):
    """The nearest of the sorted values `grid` to each x >= 0, ties to the entry of even index."""
    hi = torch.searchsorted(grid, x).clamp(1, grid.numel() - 1)
    low, up = x - grid[hi - 1], grid[hi] - x
    down = (low < up) | ((low == up) & (hi % 2 == 1))
    return grid[torch.where(down, hi - 1, hi)]


def _held(x, kind):
    """What the cache holds for x, in 64 bits: each group divided by its power of two, rounded to the code's values."""
    if kind == "bf16":
        # 8 significant bits, down to the step of the subnormals
        x = x.double()
        step = torch.exp2((torch.floor(torch.log2(x.abs().clamp(min=1e-300))) - 7).clamp(min=-133))
        return torch.round(x / step) * step
    grid = torch.tensor(FP4 if kind == "fp4" else [f * 2.0 ** -9 for f in range(8)]
                        + [(8 + m) * 2.0 ** (x - 10) for x in range(1, 16) for m in range(8)][:-1], dtype=torch.float64, device="cuda")
    g = x.double().unflatten(-1, (-1, 32))
    amax = g.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax / grid[-1]))
    e = torch.where(amax > 0, e, -100.0).clamp(-100, 119 if kind == "fp8" else 125)
    unit = torch.exp2(e)
    return (torch.sign(g) * _nearest(g.abs() / unit, grid) * unit).flatten(-2)


def exact(case, seed):
    if case["op"] == "verify":
        return None
    made = _inputs(case, seed)
    k, v = _held(made["k"], case["kind"]), _held(made["v"], case["kind"])
    if case["op"] == "write":
        return [k, v]
    new, lens, _ = _plan(case)
    if case["op"] == "read":
        return [k, v]
    share, first = case["heads"] // case["kv_heads"], 0
    out, end = [], 0
    for n, m in zip(new, lens):
        q = made["q"][first:first + n].double().unflatten(1, (case["kv_heads"], share)).permute(1, 2, 0, 3)
        keys, vals = (x[end:end + m].permute(1, 0, 2) for x in (k, v))
        s = (q.reshape(case["kv_heads"], share * n, -1) @ keys.transpose(1, 2)).view(case["kv_heads"], share, n, m) / math.sqrt(case["head_dim"])
        gap = torch.arange(m - n, m, device="cuda")[:, None] - torch.arange(m, device="cuda")[None]
        seen = (gap >= 0) & (gap < (case["window"] or m))
        p = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
        out.append((p.view(case["kv_heads"], share * n, m) @ vals).view(case["kv_heads"], share, n, -1).permute(2, 0, 1, 3).flatten(1, 2))
        first, end = first + n, end + m
    return [torch.cat(out)]
