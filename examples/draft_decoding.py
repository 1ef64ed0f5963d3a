"""Draft decoding on 2-bit weights and an e4m3 (or e2m1) paged cache, the calls as a serving loop makes them.

A small decoder with random weights stands for a model: every matrix is quantised with
llvq_quantize and multiplied with llvq_gemv (llvq_decode and a library product for a prompt).  Several
sequences decode at once.  In each round a draft model (the target's first layers) proposes a few tokens
for each sequence, one at a time; the target then takes all of them in one batch: its new keys and values go into the
paged cache (llvq_kv_write), the new tokens attend to their sequences (llvq_attn), and
llvq_draft_verify says which drafts stand and draws the token after them.  What was cached for drafts that fell is simply overwritten: lengths are the only state.

    python examples/draft_decoding.py [--rounds 8] [--drafts 4] [--kind fp8]
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import weight_decompression_amd as wd  # noqa: E402
from weight_decompression_amd import synth  # noqa: E402

KINDS = {"bf16": wd.KV_BF16, "fp8": wd.KV_FP8, "fp4": wd.KV_FP4}


class Packed:
    """A matrix [rows][cols] at 2 bits a weight."""

    def __init__(self, rows, cols, gen, std):
        self.desc = wd.make_desc(wd.MODE_SHAPEGAIN, rows, cols, max_shell=10, shape_bits=44, gain_bits=4)
        w = torch.randn(rows, cols, generator=gen, device="cuda") * std
        self.gains = torch.from_numpy((std * synth.chi_gain_table(16)).astype(np.float16)).cuda()
        self.packed = torch.empty(wd.packed_bytes(self.desc), dtype=torch.uint8, device="cuda")
        ws = torch.empty(wd.quantize_workspace_bytes(self.desc), dtype=torch.uint8, device="cuda")
        wd.quantize(self.desc, w, self.gains, self.packed, ws)

    def dense(self):
        out = torch.empty(self.desc.rows, self.desc.cols, dtype=torch.bfloat16, device="cuda")
        wd.decode(self.desc, self.packed, self.gains, wd.OUT_BF16, out)
        return out

    def __call__(self, x):
        x = x.bfloat16()
        if x.shape[0] > wd.MAX_BATCH:            # a prompt: decode once, one library product
            return (x @ self.dense().t()).float()
        y = torch.empty(x.shape[0], self.desc.rows, device="cuda")
        wd.gemv(self.desc, self.packed, self.gains, x.contiguous(), y)
        return y


class Cache:
    """One layer's paged cache."""

    def __init__(self, model, pages):
        self.desc = wd.make_kv_desc(model.kind, model.kv_heads, model.dim, model.page, pages)
        self.pool = torch.zeros(wd.kv_pool_bytes(self.desc), dtype=torch.uint8, device="cuda")


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Model:
    def __init__(self, kind="fp8", layers=3, hidden=256, heads=8, kv_heads=2, dim=64, inner=512, vocab=999, page=16, max_len=512, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.kind, self.heads, self.kv_heads, self.dim, self.page, self.vocab = KINDS[kind], heads, kv_heads, dim, page, vocab
        self.max_len = max_len
        self.embed = torch.randn(vocab, hidden, generator=gen, device="cuda")
        self.place = 0.3 * torch.randn(max_len, hidden, generator=gen, device="cuda")
        width = (heads + 2 * kv_heads) * dim
        self.layers = [(Packed(width, hidden, gen, hidden ** -0.5), Packed(hidden, heads * dim, gen, (heads * dim) ** -0.5),
                        Packed(inner, hidden, gen, hidden ** -0.5), Packed(hidden, inner, gen, inner ** -0.5)) for _ in range(layers)]
        self.head = Packed(vocab, hidden, gen, 2.0 * hidden ** -0.5)

    def caches(self, pages, layers=None):
        return [Cache(self, pages) for _ in range(layers or len(self.layers))]

    def __call__(self, tokens, positions, caches, plan, max_chunk, max_len):
        """Logits of new tokens (rows of all sequences, packed); their keys and values go into the caches.  The
        first len(caches) layers run."""
        x = self.embed[tokens] + self.place[positions]
        n, h, kv, d = x.shape[0], self.heads, self.kv_heads, self.dim
        for (wqkv, wo, up, down), cache in zip(self.layers, caches):
            qkv = wqkv(norm(x)).view(n, h + 2 * kv, d)
            wd.kv_write(cache.desc, cache.pool, qkv[:, h:h + kv], qkv[:, h + kv:], *plan)
            out = torch.empty(n, h, d, device="cuda")
            size = wd.attn_workspace_bytes(cache.desc, h, n, plan[1].numel(), max_chunk, max_len)
            ws = torch.empty(size, dtype=torch.uint8, device="cuda")
            wd.attn(cache.desc, cache.pool, qkv[:, :h], out, *plan, ws, max_chunk=max_chunk, max_len=max_len)
            x = x + wo(out.view(n, h * d))
            x = x + down(torch.nn.functional.silu(up(norm(x))))
        return self.head(norm(x))


class Decoder:
    """Sequences that share a target and a draft model's caches."""

    def __init__(self, model, prompts, draft_layers=1, seed=1):
        self.model, self.gen = model, torch.Generator(device="cuda").manual_seed(seed)
        b, per = len(prompts), -(-model.max_len // model.page)
        self.table = torch.randperm(b * per, device="cuda", generator=self.gen).to(torch.int32).view(b, per)
        self.target, self.draft = model.caches(b * per), model.caches(b * per, draft_layers)
        self.text = [list(p) for p in prompts]
        # a cache holds all of a text but its last token
        rows = [p[:-1] for p in prompts]
        for caches in (self.target, self.draft):
            self.forward(rows, [len(r) for r in rows], caches)
        self.accepted = self.proposed = 0

    def forward(self, rows, lens, caches):
        """The model on new tokens rows[b], the last of lens[b] cached ones."""
        if max(lens) > self.model.max_len:
            raise ValueError(f"a text of {max(lens)} tokens passes the model's {self.model.max_len} places")
        starts = np.concatenate(([0], np.cumsum([len(r) for r in rows])))
        positions = np.concatenate([np.arange(n - len(r), n) for r, n in zip(rows, lens)])
        dev = lambda x, t: torch.tensor(np.asarray(x), dtype=t, device="cuda")  # noqa: E731
        plan = dev(starts, torch.int32), dev(lens, torch.int32), self.table
        tokens = dev([t for r in rows for t in r], torch.int64)
        return self.model(tokens, dev(positions, torch.int64), caches, plan, max(map(len, rows)), max(lens))

    def noise(self, *shape):
        return torch.empty(*shape, device="cuda").exponential_(generator=self.gen).clamp_(min=1e-30)

    def round(self, drafts):
        """One round: drafts tokens a sequence proposed, checked and taken over."""
        base = [len(t) for t in self.text]
        if max(base) + drafts > self.model.max_len:
            raise ValueError(f"{drafts} drafts after a text of {max(base)} tokens pass the model's {self.model.max_len} places")
        b, v = len(self.text), self.model.vocab
        probs = torch.empty(b, drafts, v, device="cuda")
        rows = [[t[-1]] for t in self.text]
        tokens = torch.empty(b, drafts, dtype=torch.int32, device="cuda")
        for i in range(drafts):
            logits = self.forward(rows, [n + i for n in base], self.draft)
            probs[:, i] = torch.softmax(logits, -1)
            tokens[:, i] = (probs[:, i] / self.noise(b, v)).argmax(-1)
            rows = [[t] for t in tokens[:, i].tolist()]
        rows = [[t[-1]] + d for t, d in zip(self.text, tokens.tolist())]
        logits = self.forward(rows, [n + drafts for n in base], self.target)
        target = torch.softmax(logits, -1).view(b, drafts + 1, v)
        accepted = torch.empty(b, dtype=torch.int32, device="cuda")
        out = torch.empty(b, drafts + 1, dtype=torch.int32, device="cuda")
        ws = torch.empty(wd.draft_workspace_bytes(b, v), dtype=torch.uint8, device="cuda")
        uniforms = torch.rand(b, drafts, generator=self.gen, device="cuda")
        wd.draft_verify(target, probs, tokens, uniforms, self.noise(b, v), accepted, out, ws)
        last = [[t[-1], d[-1]] if len(t) else [] for t, d in zip(self.text, rows)]
        for text, new in zip(self.text, out.tolist()):
            text += [t for t in new if t >= 0]
        # the draft model has not seen its own last token yet; if that one stood, it is cached now
        if any(n == drafts for n in accepted.tolist()):
            self.forward([[pair[1]] for pair in last], [n + drafts for n in base], self.draft)
        self.accepted += int(accepted.sum())
        self.proposed += b * drafts
        return logits


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rounds", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--kind", choices=sorted(KINDS), default="fp8")
    a = ap.parse_args()
    rng = np.random.RandomState(0)
    model = Model(a.kind)
    prompts = [rng.randint(0, model.vocab, n).tolist() for n in (37, 5, 120)]
    run = Decoder(model, prompts)
    rounds = 0
    while rounds < a.rounds and max(map(len, run.text)) + a.drafts <= model.max_len:
        run.round(a.drafts)
        rounds += 1
    for p, t in zip(prompts, run.text):
        print(f"{len(p)} tokens of prompt, then {t[len(p):]}")
    new = sum(map(len, run.text)) - sum(map(len, prompts))
    print(f"{run.accepted} of {run.proposed} drafts accepted, {new / max(rounds * len(prompts), 1):.2f} tokens a sequence and round")


if __name__ == "__main__":
    main()
