"""A window counts cached places, so after a cut it reaches kept tokens that lie farther back in the text, unless the newest
`recent` tokens fill it: then the next tokens see what they would have seen uncut.  Bounds as in the tests of attention."""

import math

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from oracle import serving as sv
from test_gpu_eviction import run_choose, run_weigh
from test_gpu_attn_lse import run_lse
from test_gpu_serving import Setup, dev, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("recent,window", [(39, 40), (40, 12), (20, 40), (0, 30)])
def test_windows_over_a_cut_sequence(kind, recent, window):
    su = Setup(kind, 2, 64, 16, [200], [200], seed=91 + recent + window)
    (keys, values), = su.fill()
    weights = torch.full((su.pages, 2, 16), math.nan, device="cuda")
    q = dev(su.rng.randn(200, 6, 64).astype(np.float32))
    run_weigh(su, weights, q, run_lse(su, q)[1])
    keep, counts = run_choose(su, weights, 60, 4, recent)
    _, lens, table = su.plan()
    wd.kv_keep(su.desc, su.pool, keep, lens, table, counts=counts, weights=weights)
    # three more tokens, one after the other
    k, v, one = (torch.randn(3, h, 64, device="cuda") for h in (2, 2, 6))
    starts, out = torch.arange(2, dtype=torch.int32, device="cuda"), torch.empty(1, 6, 64, device="cuda")
    new = [sv.held(x.cpu().numpy(), su.kind) for x in (k, v)]
    for i in range(3):
        m = counts + 1 + i
        wd.kv_write(su.desc, su.pool, k[i:i + 1], v[i:i + 1], starts, m, table)
        ws = torch.empty(wd.attn_workspace_bytes(su.desc, 6, 1, 1, 1, 64), dtype=torch.uint8, device="cuda")
        wd.attn(su.desc, su.pool, one[i:i + 1], out, starts, m, table, ws, max_chunk=1, max_len=64, window=window)
        for h in range(2):
            kept = keep[0, h].tolist()
            held = [np.concatenate((x[:, h][kept], y[:i + 1, h])) for x, y in zip((keys, values), new)]
            whole = [np.concatenate((x[:, h], y[:i + 1, h])) for x, y in zip((keys, values), new)]
            seen = [x[-window:] for x in held]
            # whether what is seen is what the text's own window holds
            assert all(np.array_equal(a, b[-window:]) for a, b in zip(seen, whole)) == (recent >= window - 1 - i)
            at = np.array([len(seen[0]) - 1])
            ref, mass, spread = sv.attend(f64(one[i:i + 1, 3 * h:3 * h + 3]), seen[0][:, None], seen[1][:, None], at, 0.125)
            bound = mass * (2 * (3 * 64 + 8) * 2.0 ** -24 * spread[..., None] + (len(seen[0]) + 64) * 2.0 ** -23)
            ok = bool((np.abs(f64(out[:, 3 * h:3 * h + 3]) - ref) <= bound).all())
            assert ok
