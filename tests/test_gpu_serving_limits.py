"""The serving calls at the ends of what they accept."""

import pytest
import torch

from test_gpu_serving import run_draft

pytestmark = pytest.mark.gpu


def test_drafts_over_the_largest_vocabulary():
    """Entries up to 2^31 - 2: a rejected draft is replaced from the rest, whose only entry is near the end."""
    vocab = (1 << 31) - 1
    target = torch.zeros(1, 2, vocab, dtype=torch.bfloat16, device="cuda")
    draft = torch.zeros(1, 1, vocab, dtype=torch.bfloat16, device="cuda")
    noise = torch.ones(1, vocab, device="cuda")
    target[0, 0, 5] = target[0, 0, vocab - 2] = 0.5
    draft[0, 0, 5] = 0.75
    tokens = torch.full((1, 1), 5, dtype=torch.int32, device="cuda")
    for u, want in ((0.9, (0, [vocab - 2, -1])), (0.5, (1, [5, vocab - 1]))):
        target[0, 1, vocab - 1] = 1.0
        acc, out = run_draft(target, draft, tokens, torch.full((1, 1), u, device="cuda"), noise)
        assert (acc[0], out[0].tolist()) == want
