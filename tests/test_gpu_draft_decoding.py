"""The example of draft decoding: the serving calls together, against a dense recomputation."""

import os
import sys

import numpy as np
import pytest
import torch

from oracle import serving as sv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def dense_logits(ex, model, text, kind, layers=None):
    """Logits of every position of one sequence in f64 on the CPU, on the decoded weights and the cached values."""
    x = model.embed[text].double().cpu() + model.place[:len(text)].double().cpu()
    n, h, kv, d = len(text), model.heads, model.kv_heads, model.dim
    held = lambda t: torch.from_numpy(sv.held(t.float().numpy(), model.kind))  # noqa: E731
    norm = lambda t: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    mul = lambda w, t: t.bfloat16().double() @ w.dense().double().cpu().t()  # noqa: E731
    for wqkv, wo, up, down in model.layers[:layers]:
        qkv = mul(wqkv, norm(x)).view(n, h + 2 * kv, d)
        out, _, _ = sv.attend(qkv[:, :h].numpy(), held(qkv[:, h:h + kv]).numpy(), held(qkv[:, h + kv:]).numpy(), np.arange(n), d ** -0.5)
        x = x + mul(wo, torch.from_numpy(out).reshape(n, h * d))
        x = x + mul(down, torch.nn.functional.silu(mul(up, norm(x))))
    return mul(model.head, norm(x)).numpy()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_rounds_of_draft_decoding(kind):
    import draft_decoding as ex
    rng = np.random.RandomState(1)
    model = ex.Model(kind, layers=2, vocab=200)
    prompts = [rng.randint(0, model.vocab, n).tolist() for n in (20, 2, 33)]
    run = ex.Decoder(model, prompts)
    for _ in range(3):
        before = [list(t) for t in run.text]
        logits = run.round(4).view(3, 5, -1).double().cpu().numpy()
        for b in range(3):
            new = run.text[b][len(before[b]):]
            assert 1 <= len(new) <= 5 and all(0 <= t < model.vocab for t in new)
            # the first of the round's logits belongs to the text before it
            want = dense_logits(ex, model, before[b], kind)[-1]
            # Two roundings to bf16 of each product's input (2^-8 relative at most, 2^-9 on average, over
            # sqrt(K) terms: relative 2^-9 of the result's size) and a code's step where a key or value lies near a tie
            # (a group's step is 2^-3 or 2^-1 of its values, met by few of them): the logits agree to a few percent
            # of their spread, a wrong place or mask changes them by all of it.
            assert np.abs(logits[b, 0] - want).max() < 0.25 * want.std(), kind
    assert run.proposed == 36


def test_a_draft_that_is_the_target_is_accepted():
    import draft_decoding as ex
    model = ex.Model("fp8", layers=2, vocab=300)
    rng = np.random.RandomState(2)
    run = ex.Decoder(model, [rng.randint(0, 300, n).tolist() for n in (9, 14)], draft_layers=2)
    for _ in range(4):
        run.round(4)
    # u q < p with p = q up to roundings of different product orders fails for few u
    assert run.accepted >= 0.8 * run.proposed
