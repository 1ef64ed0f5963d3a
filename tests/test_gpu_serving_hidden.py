"""What a row does not see has no effect on it, to the bit: keys whose scores pass all others'."""

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from test_gpu_serving import Setup, run_attn

pytestmark = pytest.mark.gpu
BOTH = [torch.bfloat16, torch.float32]


class Hidden:
    """One sequence of `new` rows after `old` tokens; the token in the middle of the new ones is for the tests to
    change: rows 0..first - 1 do not see it."""

    def __init__(self, kind, dim, new, old, seed):
        self.su = su = Setup(kind, 2, dim, 16, [new], [new + old], seed=seed)
        su.fill()
        self.q = su.rng.randn(new, 4, dim).astype(np.float32)
        self.first = new // 2
        at = old + self.first
        self.place = int(su.table[0][at // 16]), at % 16
        self.plan = su.plan(starts=[0, 1], lens=[at + 1])       # of that token alone


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("max_len", [1, 100000])
@pytest.mark.parametrize("new", [6, 140])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_a_large_key_that_a_row_does_not_see(kind, new, max_len, dtype):
    h = Hidden(kind, 128, new, 370, seed=new)
    su, first = h.su, h.first
    clean = run_attn(su, h.q, dtype, max_len=max_len)
    k = torch.full((1, 2, 128), 40.0, device="cuda") * dev_sign(h.q)
    wd.kv_write(su.desc, su.pool, k, torch.zeros_like(k), *h.plan)
    out = run_attn(su, h.q, dtype, max_len=max_len)
    assert torch.equal(out[:first], clean[:first])
    assert not torch.equal(out[first:], clean[first:])


def dev_sign(q):
    """The signs of the last row's queries, a head of each pair: its score with such a key is large."""
    return torch.from_numpy(np.sign(q[-1:, ::2])).cuda()
