"""Trees of more nodes than a tree may have, where the launched rows hold the nodes past the last one: counted for their number
alone, those nodes see the text and are seen by none.  (Forms for up to 64 rows hold no row of such a node.)"""

import numpy as np
import pytest
import torch

import weight_decompression_amd as wd
from oracle import trees
from test_gpu_serving import Setup, dev, f64
from test_gpu_trees import check_rows, random_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind,kv_heads,dim", [("fp8", 2, 64), ("bf16", 1, 128), ("fp4", 1, 256), ("fp8", 130, 128)])     # (the last: eight waves)
@pytest.mark.parametrize("window", [0, 9])
@pytest.mark.parametrize("max_len", [1, 100000])
def test_nodes_past_the_last_see_the_text_alone(kind, kv_heads, dim, dtype, window, max_len):
    # 3 rows a node and a max_chunk of 64: 192 rows, in blocks of 128 or 256 that reach to node 84
    n, text = 70, 50
    su = Setup(kind, kv_heads, dim, 16, [n, 0], [text + n, 3], seed=111)
    (k, v), _ = su.fill()
    q = dev(su.rng.randn(n, 3 * kv_heads, dim).astype(np.float32), dtype)
    parents = random_tree(su.rng, 64, True) + [3, -1, 900, -7, 64, 68]
    starts, lens, table = su.plan()
    ws = torch.empty(wd.attn_workspace_bytes(su.desc, 3 * kv_heads, n, 2, 64, max_len), dtype=torch.uint8, device="cuda")

    def run(first, rows, length):
        out, err = torch.full_like(q, 9.0), torch.zeros(1, dtype=torch.int32, device="cuda")
        wd.attn_tree(su.desc, su.pool, q[:rows], out[:rows], dev(np.array([0, rows, rows], np.int32)), dev(np.array([length, 3], np.int32)),
                     table, dev(np.asarray(first, np.int32)), ws, max_chunk=64, max_len=max_len, window=window, err_count=err)
        return out, err.item()

    out, err = run(parents, n, text + n)
    assert err >= 1
    see = np.zeros((n, text + n), bool)
    see[:64, :text + 64] = trees.sees(parents[:64], text, window)
    see[64:, max(text - window + 1, 0) if window else 0:text] = True
    for h in sorted({0, kv_heads - 1}):
        mine = slice(3 * h, 3 * h + 3)
        check_rows(f64(out[:, mine]), f64(q[:, mine]), k[:, h:h + 1], v[:, h:h + 1], see, dim, dtype, False)
    # the same without them: not counted, and the same rows
    fewer, err = run(parents[:64], 64, text + 64)
    assert err == 0 and (fewer[64:] == 9.0).all()
    check_rows(f64(fewer[:64, :3]), f64(q[:64, :3]), k[:text + 64, :1], v[:text + 64, :1], see[:64, :text + 64], dim, dtype, False)
