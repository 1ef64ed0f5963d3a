"""Refusals of the calls for drafted trees and eviction, without a GPU: the C entries reject bad arguments before any launch, and
the binding refuses wrong dtypes, shapes, devices and short buffers before the library is reached."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import weight_decompression_amd as wd
from test_serving_checks import BAD_BATCHES, BAD_DESCS, ODD, P, attn_args, batch, desc, g, i32, lib, other  # noqa: F401
from weight_decompression_amd import build_lib

HERE = os.path.dirname(os.path.abspath(__file__))
TWO = ctypes.c_void_p(0x10002)
BAD_LISTS = [b for b in BAD_BATCHES if set(b) <= {"lens", "table", "batch", "max_pages"}]


def attn_form(lib, name, extra, d=None, pool=P, q=P, qs=(512, 64), out=P, os_=(512, 64), dtype=1, heads=8, n=None, max_chunk=2,  # noqa: F811
              max_len=4000, scale=0.1, causal=1, window=0, ws=P, size=1 << 30, err=None):
    d, n = desc() if d is None else d, batch() if n is None else n
    head = (ctypes.byref(d), pool, q, *qs, out, *os_, dtype, heads, ctypes.byref(n))
    if name == "llvq_attn_tree":
        return lib.llvq_attn_tree(*head, extra, max_chunk, max_len, scale, window, ws, size, err, None)
    return lib.llvq_attn_lse(*head, max_chunk, max_len, scale, causal, window, extra, ws, size, err, None)


@pytest.mark.parametrize("name", ["llvq_attn_tree", "llvq_attn_lse"])
def test_attn_form_refusals(lib, name):  # noqa: F811
    for bad in BAD_DESCS:
        assert attn_form(lib, name, P, d=desc(**bad)) == -1, bad
    for bad in BAD_BATCHES:
        assert attn_form(lib, name, P, n=batch(**bad)) == -1, bad
    for extra in (None, TWO):
        assert attn_form(lib, name, extra) == -1
    for bad in (dict(pool=None), dict(q=None), dict(out=None), dict(out=ODD), dict(dtype=2), dict(heads=7), dict(max_chunk=1), dict(max_chunk=0),
                dict(max_len=0), dict(scale=0.0), dict(scale=float("inf")), dict(window=-1), dict(ws=None), dict(size=0), dict(qs=(-1, 64)),
                dict(err=TWO)):
        assert attn_form(lib, name, P, **bad) == -1, bad
    if name == "llvq_attn_tree":
        assert attn_form(lib, name, P, max_chunk=65) == -1
    assert attn_form(lib, name, None, q=None, out=None, ws=None, n=batch(tokens=0)) == 0


def verify(lib, target=P, dtype=0, starts=P, tokens=P, parents=P, uni=P, noise=P, b=2, n=9, v=100, width=5, acc=P, path=P, out=P, ws=P,  # noqa: F811
           size=1 << 20, err=None):
    return lib.llvq_tree_verify(target, dtype, starts, tokens, parents, uni, noise, b, n, v, width, acc, path, out, ws, size, err, None)


def test_verify_refusals(lib):  # noqa: F811
    for name in ("target", "starts", "tokens", "parents", "uni", "noise", "acc", "path", "out", "ws"):
        assert verify(lib, **{name: None}) == -1, name
        assert verify(lib, **{name: TWO}) == -1, name
    for bad in (dict(dtype=2), dict(b=-1), dict(b=32769), dict(n=-1), dict(n=(1 << 27) + 1), dict(v=0), dict(width=0), dict(width=65),
                dict(ws=ODD), dict(size=15), dict(err=TWO), dict(dtype=1, target=ctypes.c_void_p(0x10001))):
        assert verify(lib, **bad) == -1, bad
    assert verify(lib, b=0, target=None, starts=None, noise=None, acc=None, path=None, out=None, ws=None) == 0
    assert lib.llvq_tree_workspace_bytes(-1, 10) == -1 and lib.llvq_tree_workspace_bytes(1, 0) == -1
    sizes = [wd.tree_workspace_bytes(b, 100003) for b in range(1, 700)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def weigh(lib, d=None, pool=P, w=P, q=P, qs=(512, 64), dtype=1, heads=8, lse=P, n=None, max_chunk=2, max_len=4000, scale=0.1, causal=1,  # noqa: F811
          window=0, fresh=0, err=None):
    d, n = desc() if d is None else d, batch() if n is None else n
    return lib.llvq_kv_weigh(ctypes.byref(d), pool, w, q, *qs, dtype, heads, lse, ctypes.byref(n), max_chunk, max_len, scale, causal, window,
                             fresh, err, None)


def test_weigh_refusals(lib):  # noqa: F811
    for bad in BAD_DESCS:
        assert weigh(lib, d=desc(**bad)) == -1, bad
    for bad in BAD_BATCHES:
        assert weigh(lib, n=batch(**bad)) == -1, bad
    for bad in (dict(pool=None), dict(pool=ODD), dict(w=None), dict(w=TWO), dict(q=None), dict(q=ctypes.c_void_p(0x10001)), dict(lse=None),
                dict(lse=TWO), dict(dtype=2), dict(heads=0), dict(heads=7), dict(max_chunk=1), dict(max_chunk=0), dict(max_len=0),
                dict(max_len=(1 << 30) + 1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=2.4e38), dict(window=-1),
                dict(window=(1 << 30) + 1), dict(qs=(-1, 64)), dict(qs=(512, -64)), dict(err=TWO)):
        assert weigh(lib, **bad) == -1, bad
    for empty in (dict(tokens=0), dict(batch=0)):
        assert weigh(lib, pool=None, w=None, q=None, lse=None, n=batch(starts=None, lens=None, table=None, **dict(dict(tokens=0), **empty))) == 0
    # more (sequence, key head) pairs than a launch takes
    assert weigh(lib, d=desc(kv_heads=1024, pages=1), heads=1024, n=batch(batch=32768, tokens=3)) == -1


def choose(lib, d=None, w=P, n=None, budget=10, sinks=2, recent=3, keep=P, counts=P, err=None):  # noqa: F811
    d, n = desc() if d is None else d, batch() if n is None else n
    return lib.llvq_kv_choose(ctypes.byref(d), w, ctypes.byref(n), budget, sinks, recent, keep, counts, err, None)


def keep_call(lib, d=None, pool=P, w=P, n=None, keep=P, lists=2, width=4, counts=P, err=None):  # noqa: F811
    d, n = desc() if d is None else d, batch() if n is None else n
    return lib.llvq_kv_keep(ctypes.byref(d), pool, w, ctypes.byref(n), keep, lists, width, counts, err, None)


def test_choose_and_keep_refusals(lib):  # noqa: F811
    for call in (choose, keep_call):
        for bad in BAD_DESCS:
            assert call(lib, d=desc(**bad)) == -1, bad
        for bad in BAD_LISTS:
            assert call(lib, n=batch(**bad)) == -1, bad
        assert call(lib, n=batch(starts=0x10002)) == -1
        assert call(lib, err=TWO) == -1
    assert len(BAD_LISTS) > 5
    for bad in (dict(w=None), dict(w=TWO), dict(keep=None), dict(keep=TWO), dict(counts=None), dict(counts=TWO), dict(budget=0), dict(budget=-1),
                dict(budget=(1 << 30) + 1), dict(sinks=-1), dict(recent=-1), dict(sinks=8), dict(sinks=(1 << 31) - 1, recent=(1 << 31) - 1)):
        assert choose(lib, **bad) == -1, bad
    for bad in (dict(pool=None), dict(pool=ODD), dict(w=TWO), dict(keep=None), dict(keep=TWO), dict(counts=TWO), dict(lists=0), dict(lists=3),
                dict(width=-1), dict(width=(1 << 30) + 1)):
        assert keep_call(lib, **bad) == -1, bad
    assert choose(lib, n=batch(batch=0, lens=None, table=None), w=None, keep=None, counts=None) == 0
    assert keep_call(lib, n=batch(batch=0, lens=None, table=None), pool=None, keep=None) == 0
    assert keep_call(lib, width=0, keep=None) == 0
    big = dict(d=desc(kv_heads=1024, pages=1), n=batch(batch=32768))
    assert choose(lib, **big) == -1 and keep_call(lib, lists=1024, **big) == -1


class _Entries:
    """A library whose entries answer -1 to whatever passes the binding's checks."""

    def __getattr__(self, name):
        return lambda *a: 64 if name.endswith("bytes") else -1


@pytest.fixture
def refusing(monkeypatch):
    monkeypatch.setattr(wd, "load_library", lambda *a: _Entries())
    monkeypatch.setattr(wd, "_launch", lambda function, device, stream, *a: function(*a))


def test_checks_of_lse_and_parents(refusing):
    with pytest.raises(wd.LlvqError):
        wd.attn(**attn_args(lse=g(torch.zeros(5, 6))))
    for bad in (torch.zeros(5, 6), g(torch.zeros(5, 5)), g(torch.zeros(5, 6).half()), g(torch.zeros(6, 5)).t(), 3.0, other(torch.zeros(5, 6))):
        with pytest.raises((ValueError, TypeError)):
            wd.attn(**attn_args(lse=bad))
    with pytest.raises(wd.LlvqError):
        wd.attn_tree(**attn_args(parents=i32(5)))
    for bad in (None, i32(4), i32(5, 1), torch.zeros(5, dtype=torch.int32), g(torch.zeros(5, dtype=torch.int64)), i32(10)[::2],
                other(torch.zeros(5, dtype=torch.int32))):
        with pytest.raises((ValueError, TypeError)):
            wd.attn_tree(**attn_args(parents=bad))
    for bad in (dict(q=None), dict(q=g(torch.zeros(5, 5, 64))), dict(out=torch.zeros(5, 6, 64)), dict(table=i32(2, 2)),
                dict(workspace=torch.zeros(64, dtype=torch.uint8))):
        with pytest.raises((ValueError, TypeError)):
            wd.attn_tree(**attn_args(parents=i32(5), **bad))


def verify_args(**over):
    a = dict(target=g(torch.zeros(9, 10)), starts=i32(3), tokens=i32(9), parents=i32(9), uniforms=g(torch.zeros(9)), noise=g(torch.zeros(2, 10)),
             accepted=i32(2), path=i32(2, 5), out=i32(2, 5), workspace=g(torch.zeros(64, dtype=torch.uint8)))
    a.update(over)
    return a


def test_verify_binding(refusing):
    for fine in (dict(), dict(target=g(torch.zeros(9, 10).bfloat16())), dict(err_count=i32(1))):
        with pytest.raises(wd.LlvqError):
            wd.tree_verify(**verify_args(**fine))
    with pytest.raises(ValueError, match="workspace"):
        wd.tree_verify(**verify_args(workspace=g(torch.zeros(63, dtype=torch.uint8))))
    for bad in (dict(target=g(torch.zeros(9, 2, 5))), dict(target=g(torch.zeros(9, 10).half())), dict(target=torch.zeros(9, 10)), dict(target=None),
                dict(starts=i32(2)), dict(starts=g(torch.zeros(3, dtype=torch.int64))), dict(tokens=i32(8)), dict(parents=i32(9, 1)),
                dict(uniforms=g(torch.zeros(8))), dict(uniforms=i32(9)), dict(noise=g(torch.zeros(2, 9))), dict(noise=g(torch.zeros(10, 2)).t()),
                dict(accepted=i32(3)), dict(path=i32(10)), dict(path=i32(5, 2).t()), dict(out=i32(2, 4)), dict(out=None), dict(workspace=None),
                dict(noise=other(torch.zeros(2, 10))), dict(workspace=torch.zeros(64, dtype=torch.uint8)), dict(parents=i32(18)[::2]),
                dict(err_count=g(torch.zeros(1)))):
        with pytest.raises((ValueError, TypeError)):
            wd.tree_verify(**verify_args(**bad))


def weigh_args(**over):
    a = dict(desc=desc(), pool=g(torch.zeros(8 * 2 * 16 * 132, dtype=torch.uint8)), weights=g(torch.zeros(8, 2, 16)), q=g(torch.zeros(5, 6, 64)),
             lse=g(torch.zeros(5, 6)), starts=i32(4), lens=i32(3), table=i32(3, 2), max_chunk=3, max_len=32)
    a.update(over)
    return a


def test_weigh_binding(refusing):
    for fine in (dict(), dict(q=g(torch.zeros(5, 9, 80))[:, 1:7, 8:72]), dict(q=g(torch.zeros(5, 6, 64).bfloat16())), dict(err_count=i32(1))):
        with pytest.raises(wd.LlvqError):
            wd.kv_weigh(**weigh_args(**fine))
    for bad in (dict(weights=g(torch.zeros(8, 16, 2)).transpose(1, 2)), dict(weights=g(torch.zeros(7, 2, 16))), dict(weights=g(torch.zeros(8, 2, 16).half())),
                dict(weights=torch.zeros(8, 2, 16)), dict(q=g(torch.zeros(5, 5, 64))), dict(q=g(torch.zeros(5, 6, 64).half())), dict(q=None),
                dict(q=g(torch.zeros(5, 64, 6)).transpose(1, 2)), dict(lse=g(torch.zeros(6, 5))), dict(lse=g(torch.zeros(5, 6).bfloat16())),
                dict(lse=None), dict(pool=None), dict(table=i32(2, 2)), dict(starts=i32(3)), dict(weights=other(torch.zeros(8, 2, 16))),
                dict(lse=other(torch.zeros(5, 6))), dict(err_count=other(torch.zeros(1, dtype=torch.int32)))):
        with pytest.raises((ValueError, TypeError)):
            wd.kv_weigh(**weigh_args(**bad))


def choose_args(**over):
    a = dict(desc=desc(), weights=g(torch.zeros(8, 2, 16)), lens=i32(3), table=i32(3, 2), keep=i32(3, 2, 7), counts=i32(3), sinks=1, recent=2)
    a.update(over)
    return a


def keep_args(**over):
    a = dict(desc=desc(), pool=g(torch.zeros(8 * 2 * 16 * 132, dtype=torch.uint8)), keep=i32(3, 2, 7), lens=i32(3), table=i32(3, 2))
    a.update(over)
    return a


def test_choose_and_keep_binding(refusing):
    for fine in (dict(), dict(err_count=i32(1))):
        with pytest.raises(wd.LlvqError):
            wd.kv_choose(**choose_args(**fine))
    for fine in (dict(), dict(keep=i32(3, 1, 7)), dict(counts=i32(3)), dict(starts=i32(4)), dict(weights=g(torch.zeros(8, 2, 16)))):
        with pytest.raises(wd.LlvqError):
            wd.kv_keep(**keep_args(**fine))
    common = (dict(keep=i32(3, 3, 7)), dict(keep=i32(2, 2, 7)), dict(keep=i32(3, 14)), dict(keep=None), dict(keep=g(torch.zeros(3, 2, 7))),
              dict(keep=i32(3, 7, 2).transpose(1, 2)), dict(lens=i32(3, 1)), dict(lens=None), dict(lens=g(torch.zeros(3))), dict(table=i32(6)),
              dict(table=i32(2, 3).t()), dict(counts=i32(2)), dict(counts=torch.zeros(3, dtype=torch.int32)), dict(weights=g(torch.zeros(8, 2, 15))),
              dict(table=other(torch.zeros(3, 2, dtype=torch.int32))), dict(err_count=g(torch.zeros(1))))
    for bad in common:
        with pytest.raises((ValueError, TypeError)):
            wd.kv_choose(**choose_args(**bad))
        with pytest.raises((ValueError, TypeError)):
            wd.kv_keep(**keep_args(**bad))
    for bad in (dict(pool=None), dict(pool=g(torch.zeros(8 * 2 * 16 * 132 - 1, dtype=torch.uint8))), dict(starts=i32(3)), dict(starts=g(torch.zeros(4)))):
        with pytest.raises((ValueError, TypeError)):
            wd.kv_keep(**keep_args(**bad))
    with pytest.raises((ValueError, TypeError)):
        wd.kv_choose(**choose_args(weights=None))


def test_largest_sizes_are_clean_under_sanitizers(tmp_path):
    """The host side of the calls at the largest sizes they accept, without a device."""
    try:
        hipcc = build_lib.hipcc_path()
    except RuntimeError:
        pytest.skip("needs hipcc")
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path / "evict_largest_host")
    san = [a for f in ("-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer")
           for a in ("-Xarch_host", f)]
    subprocess.run([hipcc, f"--offload-arch={build_lib.OFFLOAD_ARCH}", "-O1", "-g", "-std=c++17", "-Xarch_device", "-O1", *san, "-parallel-jobs=2",
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", build_lib.INCLUDE, "-o", exe,
                    *[os.path.join(build_lib.CSRC_SERVE, unit) for unit in ("llvq_tree.hip", "llvq_evict.hip")],
                    os.path.join(HERE, "host_build", "evict_largest_host.cpp")], check=True, capture_output=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1",
               HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")
    p = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert p.returncode == 0, p.stdout[-1000:] + p.stderr[-3000:]
    assert "runtime error" not in p.stderr and "AddressSanitizer" not in p.stderr, p.stderr[-3000:]
    assert p.stdout.startswith("ok ")
