"""A workspace sized once for the largest step serves every smaller one (without a GPU)."""

import os
import subprocess

import pytest

import weight_decompression_amd as wd
from weight_decompression_amd import build_lib

HERE = os.path.dirname(os.path.abspath(__file__))


def test_one_workspace_for_all_smaller_calls(tmp_path):
    try:
        hipcc = build_lib.hipcc_path()
    except RuntimeError:
        pytest.skip("needs hipcc")
    if not os.path.exists(wd.LIB_PATH):
        pytest.fail("libllvq.so is not built (run __graft_entry__.build())")
    exe, (place, name) = str(tmp_path / "serve_workspace_host"), os.path.split(os.path.abspath(wd.LIB_PATH))
    subprocess.run([hipcc, f"--offload-arch={build_lib.OFFLOAD_ARCH}", "-O1", "-std=c++17", "-I", build_lib.INCLUDE, "-o", exe,
                    os.path.join(HERE, "host_build", "serve_workspace_host.cpp"), "-L" + place, "-l:" + name, "-Wl,-rpath," + place],
                   check=True, capture_output=True)
    # no device is to be seen, wherever this runs
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")
    p = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert p.returncode == 0 and p.stdout.startswith("ok "), p.stdout[-1000:] + p.stderr[-3000:]


def test_sizes_do_not_shrink_as_the_batch_grows():
    d = wd.make_kv_desc(wd.KV_FP8, 32, 128, 16, 1 << 16)
    sizes = [wd.attn_workspace_bytes(d, 32, b, b, 1, 4096) for b in range(1, 65)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    drafts = [wd.draft_workspace_bytes(b, 100003) for b in range(1, 700)]
    assert drafts == sorted(drafts)
