"""What a row does not see has no effect on it, whatever bytes lie there: bytes that no write leaves (codes and
scales that stand for values that are not finite), and keys whose scores pass all others'."""

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

    def poke(self, head, is_v, codes, scales):
        """Bytes of the token's key or value: {offset: byte} of its codes and of its scales."""
        lay = self.su.lay
        for at, these in ((lay.codes, codes), (lay.scales, scales)):
            for offset, byte in these.items():
                self.su.pool[at(self.place[0], head, self.place[1], is_v) + offset] = byte

    def read(self):
        out = torch.empty(2, 1, 2, self.su.dim, device="cuda")
        wd.kv_read(self.su.desc, self.su.pool, out[0], out[1], *self.plan)
        return out[1, 0]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("max_len", [1, 100000])
@pytest.mark.parametrize("new", [6, 140])
@pytest.mark.parametrize("dim", [64, 128, 160, 256])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_values_of_bytes_that_no_write_leaves(kind, dim, new, max_len, dtype):
    h = Hidden(kind, dim, new, 50, seed=dim + new)
    su, first = h.su, h.first
    clean = run_attn(su, h.q, dtype, max_len=max_len)
    was = su.pool.clone()
    ch = dim - 27                                    # a channel of the last group, in the second half of wide heads
    group = ch // 32
    last = 246 if kind == "fp8" else 252             # the last scale byte that stands for a power of two
    cases = [({}, {group: byte}) for byte in (255, 254, last + 1)]
    if kind == "fp8":
        cases += [({ch: 0x7F}, {}), ({ch: 0xFF}, {})]
    for codes, scales in cases:
        su.pool.copy_(was)
        h.poke(1, 1, codes, scales)
        nan = torch.zeros(2, dim, dtype=torch.bool, device="cuda")
        nan[1, ch if codes else slice(32 * group, 32 * group + 32)] = True
        assert torch.equal(torch.isnan(h.read()), nan)
        out = run_attn(su, h.q, dtype, max_len=max_len)
        assert torch.equal(out[:first], clean[:first])
        # the rows that see it: NaN there, and the rest as it was
        rows = nan.repeat_interleave(2, 0).expand(new - first, 4, dim)
        assert torch.equal(torch.isnan(out[first:]), rows)
        assert torch.equal(out[first:][~rows], clean[first:][~rows])
    # any bytes at all, keys among them
    for seed in range(3):
        su.pool.copy_(was)
        noise = np.random.RandomState(seed).randint(0, 256, (2, 2, 2, 512))
        for head in range(2):
            for is_v in range(2):
                h.poke(head, is_v, dict(enumerate(noise[head, is_v, 0, :su.lay.row].tolist())),
                       dict(enumerate(noise[head, is_v, 1, :su.lay.groups].tolist())))
        assert torch.equal(run_attn(su, h.q, dtype, max_len=max_len)[:first], clean[:first])


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("max_len", [1, 100000])
@pytest.mark.parametrize("new", [6, 140])
@pytest.mark.parametrize("dim", [64, 128, 160, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_written_values_that_are_not_finite(kind, dim, new, max_len, dtype):
    h = Hidden(kind, dim, new, 50, seed=dim + new)
    su, first = h.su, h.first
    clean = run_attn(su, h.q, dtype, max_len=max_len)
    k, v = torch.randn(2, 1, 2, dim, device="cuda")
    v[0, 0, dim - 1], v[0, 1, 3] = float("-inf"), float("nan")
    wd.kv_write(su.desc, su.pool, k, v, *h.plan)
    held = h.read()
    odd = ~torch.isfinite(held)
    assert odd.sum() == (2 if kind == "bf16" else 64)
    out = run_attn(su, h.q, dtype, max_len=max_len)
    assert torch.equal(out[:first], clean[:first])
    rows = odd.repeat_interleave(2, 0).expand(new - first, 4, dim)
    assert torch.equal(~torch.isfinite(out[first:]), rows)
    if kind == "bf16":
        assert (out[first:, :2, dim - 1] == float("-inf")).all()


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


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("max_len", [1, 100000])
@pytest.mark.parametrize("new", [9, 150])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_a_padded_chunk_over_places_never_written(kind, new, max_len, dtype):
    """A chunk padded to a fixed length in a pool of arbitrary bytes: the rows before the padding are those of the
    unpadded chunk."""
    pad = new // 3
    su = Setup(kind, 2, 128, 16, [new], [new + 40], seed=new)
    su.pool.copy_(torch.from_numpy(su.rng.randint(0, 256, su.pool.numel()).astype(np.uint8)))
    total = new + 40 - pad
    k, v = torch.randn(2, total, 2, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(new))
    wd.kv_write(su.desc, su.pool, k, v, *su.plan(starts=[0, total], lens=[total]))
    q = torch.from_numpy(su.rng.randn(new, 4, 128).astype(np.float32)).cuda().to(dtype)
    padded = run_attn(su, q, dtype, max_len=max_len)
    short = run_attn(su, q[:new - pad].contiguous(), dtype, max_len=max_len, max_chunk=new,
                     plan=su.plan(starts=[0, new - pad], lens=[total]))
    assert torch.isfinite(short).all() and torch.equal(padded[:new - pad], short)
