"""Refusals of the serving calls, without a GPU: the C entries reject bad arguments before any launch, and the
binding refuses host tensors, wrong dtypes, shapes, strides and short buffers before the library
is reached."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import weight_decompression_amd as wd
from weight_decompression_amd import build_lib

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10004)
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(wd.LIB_PATH):
        pytest.fail("libllvq.so is not built (run __graft_entry__.build())")
    return wd.load_library()


def desc(**over):
    a = dict(kind=wd.KV_FP8, kv_heads=2, head_dim=64, page_tokens=16, pages=8)
    a.update(over)
    return wd.make_kv_desc(**a)


def batch(**over):
    a = dict(starts=P.value, lens=P.value, table=P.value, batch=2, max_pages=4, tokens=3)
    a.update(over)
    return wd.Batch(*(a[n] for n in ("starts", "lens", "table", "batch", "max_pages", "tokens")))


BAD_DESCS = [dict(kind=3), dict(kind=-1), dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=48), dict(head_dim=0),
             dict(head_dim=288), dict(page_tokens=0), dict(page_tokens=4097), dict(pages=0), dict(pages=-1)]
BAD_BATCHES = [dict(starts=None), dict(lens=None), dict(table=None), dict(starts=0x10002), dict(lens=0x10001), dict(table=0x10003),
               dict(batch=-1), dict(batch=32769), dict(max_pages=-1), dict(tokens=-1), dict(tokens=(1 << 27) + 1)]


def kv(lib, name, d=None, pool=P, k=P, ks=(128, 64), v=P, vs=(128, 64), dtype=0, n=None, err=None):
    d, n = desc() if d is None else d, batch() if n is None else n
    return getattr(lib, name)(ctypes.byref(d), pool, k, *ks, v, *vs, dtype, ctypes.byref(n), err, None)


def test_pool_bytes(lib):
    for kind, token in ((wd.KV_BF16, 4 * 96), (wd.KV_FP8, 2 * 96 + 6), (wd.KV_FP4, 96 + 6)):
        d = wd.make_kv_desc(kind, 3, 96, 7, 11)
        assert wd.kv_pool_bytes(d) == 11 * 3 * (-(-7 * token // 16) * 16) == wd._pool_nbytes(d)
    big = desc(kv_heads=1024, head_dim=256, page_tokens=4096, pages=(1 << 31) - 1, kind=wd.KV_BF16)
    assert wd.kv_pool_bytes(big) == ((1 << 31) - 1) * 1024 * 4096 * 1024
    for bad in BAD_DESCS:
        assert lib.llvq_kv_pool_bytes(ctypes.byref(desc(**bad))) == -1, bad
    assert lib.llvq_kv_pool_bytes(None) == -1


@pytest.mark.parametrize("name", ["llvq_kv_write", "llvq_kv_read"])
def test_kv_refusals(lib, name):
    for bad in BAD_DESCS:
        assert kv(lib, name, d=desc(**bad)) == -1, bad
    for bad in BAD_BATCHES:
        assert kv(lib, name, n=batch(**bad)) == -1, bad
    for bad in (dict(pool=None), dict(pool=ODD), dict(k=None), dict(v=None), dict(k=ctypes.c_void_p(0x10002)), dict(dtype=2),
                dict(dtype=1, v=ctypes.c_void_p(0x10001)), dict(ks=(-128, 64)), dict(vs=(128, -1)), dict(err=ctypes.c_void_p(0x10002))):
        assert kv(lib, name, **bad) == -1, bad
    assert getattr(lib, name)(None, P, P, 1, 1, P, 1, 1, 0, ctypes.byref(batch()), None, None) == -1
    assert getattr(lib, name)(ctypes.byref(desc()), P, P, 1, 1, P, 1, 1, 0, None, None, None) == -1
    # nothing to do: nothing is needed
    for empty in (dict(tokens=0), dict(batch=0)):
        assert kv(lib, name, pool=None, k=None, v=None, n=batch(starts=None, lens=None, table=None, **empty)) == 0


def attn(lib, d=None, pool=P, q=P, qs=(512, 64), out=P, os_=(512, 64), dtype=1, heads=8, n=None, max_chunk=2, max_len=4000,
         scale=0.1, causal=1, window=0, ws=P, size=1 << 30, err=None):
    d, n = desc() if d is None else d, batch() if n is None else n
    return lib.llvq_attn(ctypes.byref(d), pool, q, *qs, out, *os_, dtype, heads, ctypes.byref(n), max_chunk, max_len, scale, causal,
                         window, ws, size, err, None)


def test_attn_refusals(lib):
    for bad in BAD_DESCS:
        assert attn(lib, d=desc(**bad)) == -1, bad
    for bad in BAD_BATCHES:
        assert attn(lib, n=batch(**bad)) == -1, bad
    for bad in (dict(pool=None), dict(pool=ODD), dict(q=None), dict(out=None), dict(q=ctypes.c_void_p(0x10001)), dict(out=ODD),
                dict(dtype=0, out=ctypes.c_void_p(0x10008)), dict(dtype=2), dict(heads=0), dict(heads=7), dict(heads=1), dict(max_chunk=1),
                dict(qs=(-1, 64)), dict(os_=(510, 64)), dict(os_=(512, 62)), dict(os_=(-4, 64)), dict(max_chunk=0), dict(max_len=0),
                dict(max_len=(1 << 30) + 1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
                dict(window=-1), dict(window=(1 << 30) + 1), dict(ws=None), dict(ws=ODD), dict(size=0), dict(size=wd.attn_workspace_bytes(desc(), 8, 3, 2, 2, 4000) - 1),
                dict(err=ctypes.c_void_p(0x10002))):
        assert attn(lib, **bad) == -1, bad
    assert attn(lib, q=None, out=None, ws=None, n=batch(tokens=0)) == 0
    for args in ((7, 10, 2, 2, 100), (8, -1, 2, 2, 100), (8, 10, -1, 2, 100), (8, 10, 2, 0, 100), (8, 10, 2, 2, 0),
                 (8, 1 << 31, 2, 2, 100), (8, 10, 32769, 2, 100), (8, 5, 2, 2, 100), (8, 4, 32768, 1 << 20, 100)):
        assert lib.llvq_attn_workspace_bytes(ctypes.byref(desc()), *args) == -1, args
    assert wd.attn_workspace_bytes(desc(), 8, 4, 2, 2, 100) == 0               # a short axis is not split
    many = wd.attn_workspace_bytes(desc(), 8, 4, 2, 2, 100000)
    assert many > 0 and many % (4 * 8 * (64 + 2) * 4) == 0


def draft(lib, target=P, q=P, dtype=0, tokens=P, counts=P, uni=P, noise=P, b=2, s=3, vocab=100, acc=P, out=P, ws=P, size=1 << 20, err=None):
    return lib.llvq_draft_verify(target, q, dtype, tokens, counts, uni, noise, b, s, vocab, acc, out, ws, size, err, None)


def test_draft_refusals(lib):
    two = ctypes.c_void_p(0x10002)
    for bad in (dict(target=None), dict(target=two), dict(q=two), dict(dtype=2), dict(tokens=None), dict(tokens=two), dict(counts=two),
                dict(uni=None), dict(uni=two), dict(noise=None), dict(noise=two), dict(b=-1), dict(b=32769), dict(s=-1), dict(s=64),
                dict(vocab=0), dict(acc=None), dict(acc=two), dict(out=None), dict(out=two), dict(ws=None), dict(ws=ODD),
                dict(size=15), dict(err=two), dict(dtype=1, target=ctypes.c_void_p(0x10001))):
        assert draft(lib, **bad) == -1, bad
    assert draft(lib, b=0, target=None, noise=None, acc=None, out=None, ws=None) == 0
    assert lib.llvq_draft_workspace_bytes(-1, 10) == -1 and lib.llvq_draft_workspace_bytes(1, 0) == -1
    assert wd.draft_workspace_bytes(3, 8192) == 24 and wd.draft_workspace_bytes(3, 8193) == 5 * 24


def test_serving_host_code_is_clean_under_sanitizers(tmp_path):
    """The host side of the serving calls with address and undefined-behaviour checks: sizes at
    their limits and refusals."""
    try:
        hipcc = build_lib.hipcc_path()
    except RuntimeError:
        pytest.skip("needs hipcc")
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path / "serve_host")
    san = [a for f in ("-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer")
           for a in ("-Xarch_host", f)]
    subprocess.run([hipcc, f"--offload-arch={build_lib.OFFLOAD_ARCH}", "-O1", "-g", "-std=c++17", "-Xarch_device", "-O1", *san,
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", build_lib.INCLUDE, "-o", exe,
                    os.path.join(build_lib.CSRC_SERVE, "llvq_serve.hip"), os.path.join(HERE, "host_build", "serve_host.cpp")],
                   check=True, capture_output=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    p = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert p.returncode == 0, p.stdout[-1000:] + p.stderr[-3000:]
    assert "runtime error" not in p.stderr and "AddressSanitizer" not in p.stderr, p.stderr[-3000:]
    assert p.stdout.startswith("ok ")


# the binding

class _OnGpu(torch.Tensor):
    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return 0


def g(t):
    return torch.Tensor._make_subclass(_OnGpu, t)


class _Reached(Exception):
    pass


@pytest.fixture
def no_library(monkeypatch):
    def sentinel(*a, **k):
        raise _Reached()
    monkeypatch.setattr(wd, "load_library", sentinel)


class _OnOther(_OnGpu):
    def get_device(self):
        return 1


def other(t):
    return torch.Tensor._make_subclass(_OnOther, t)


def test_tensors_on_several_devices_are_refused(no_library):
    for over in (dict(v=other(torch.zeros(5, 2, 64))), dict(pool=other(torch.zeros(1 << 16, dtype=torch.uint8))),
                 dict(table=other(torch.zeros(3, 2, dtype=torch.int32))), dict(err_count=other(torch.zeros(1, dtype=torch.int32)))):
        with pytest.raises(ValueError, match="devices"):
            wd.kv_write(**kv_args(**over))
    for over in (dict(out=other(torch.zeros(5, 6, 64))), dict(workspace=other(torch.zeros(64, dtype=torch.uint8)))):
        with pytest.raises(ValueError, match="devices"):
            wd.attn(**attn_args(**over))
    for over in (dict(noise=other(torch.zeros(2, 10))), dict(workspace=other(torch.zeros(64, dtype=torch.uint8)))):
        with pytest.raises(ValueError, match="devices"):
            wd.draft_verify(**draft_args(**over))


def i32(*shape):
    return g(torch.zeros(*shape, dtype=torch.int32))


def kv_args(**over):
    a = dict(desc=desc(), pool=g(torch.zeros(8 * 2 * 16 * 132, dtype=torch.uint8)), k=g(torch.zeros(5, 2, 64)), v=g(torch.zeros(5, 2, 64)),
             starts=i32(4), lens=i32(3), table=i32(3, 2), err_count=i32(1))
    a.update(over)
    return a


@pytest.mark.parametrize("call", ["kv_write", "kv_read"])
def test_kv_binding(no_library, call):
    f = getattr(wd, call)
    with pytest.raises(_Reached):
        f(**kv_args())
    with pytest.raises(_Reached):          # slices of a wider tensor
        f(**kv_args(k=g(torch.zeros(5, 9, 80))[:, 1:3, :64], v=g(torch.zeros(5, 9, 80))[:, 4:6, 8:72], err_count=None))
    for bad in (dict(pool=g(torch.zeros(8 * 2 * 16 * 132 - 1, dtype=torch.uint8))), dict(pool=torch.zeros(1 << 16, dtype=torch.uint8)),
                dict(pool=g(torch.zeros(1 << 16, dtype=torch.int8))), dict(k=g(torch.zeros(5, 2, 32))), dict(k=g(torch.zeros(4, 2, 64))),
                dict(k=g(torch.zeros(5, 2, 64).half())), dict(v=g(torch.zeros(5, 2, 64).bfloat16())), dict(v=torch.zeros(5, 2, 64)),
                dict(k=g(torch.zeros(5, 64, 2)).transpose(1, 2)), dict(k=[1.0]), dict(starts=i32(3)), dict(lens=i32(3, 1)),
                dict(table=i32(6)), dict(table=i32(4, 2)), dict(starts=g(torch.zeros(4, dtype=torch.int64))), dict(table=i32(2, 3).t()),
                dict(err_count=g(torch.zeros(1))), dict(desc=desc(kind=7)), dict(desc=desc(pages=0))):
        with pytest.raises((ValueError, TypeError)):
            f(**kv_args(**bad))


def test_outputs_that_overlap_are_refused(no_library):
    for view in (g(torch.zeros(1, 2, 64)).expand(5, 2, 64), g(torch.zeros(5, 1, 64)).expand(5, 2, 64),
                 g(torch.zeros(5 * 64 + 64)).as_strided((5, 2, 64), (64, 64, 1))):
        with pytest.raises(ValueError):
            wd.kv_read(**kv_args(k=view))
        with pytest.raises(_Reached):      # as an input it is fine
            wd.kv_write(**kv_args(k=view))
    with pytest.raises(_Reached):          # head-major outputs are fine
        wd.kv_read(**kv_args(k=g(torch.zeros(2, 5, 64)).transpose(0, 1)))


def attn_args(**over):
    a = dict(desc=desc(), pool=g(torch.zeros(8 * 2 * 16 * 132, dtype=torch.uint8)), q=g(torch.zeros(5, 6, 64)), out=g(torch.zeros(5, 6, 64)),
             starts=i32(4), lens=i32(3), table=i32(3, 2), workspace=g(torch.zeros(64, dtype=torch.uint8)), max_chunk=3, max_len=32)
    a.update(over)
    return a


def test_attn_binding(no_library):
    with pytest.raises(_Reached):
        wd.attn(**attn_args())
    for bad in (dict(q=g(torch.zeros(5, 5, 64))), dict(q=g(torch.zeros(5, 6, 32))), dict(q=g(torch.zeros(5, 384))), dict(q=None),
                dict(out=g(torch.zeros(5, 6, 64).bfloat16())), dict(out=g(torch.zeros(4, 6, 64))), dict(out=torch.zeros(5, 6, 64)),
                dict(out=g(torch.zeros(1, 6, 64)).expand(5, 6, 64)), dict(workspace=torch.zeros(64, dtype=torch.uint8)),
                dict(workspace=7), dict(starts=None), dict(pool=None), dict(table=i32(2, 2))):
        with pytest.raises((ValueError, TypeError)):
            wd.attn(**attn_args(**bad))


def draft_args(**over):
    a = dict(target=g(torch.zeros(2, 4, 10)), draft=g(torch.zeros(2, 3, 10)), tokens=i32(2, 3), uniforms=g(torch.zeros(2, 3)),
             noise=g(torch.zeros(2, 10)), accepted=i32(2), out=i32(2, 4), workspace=g(torch.zeros(64, dtype=torch.uint8)), counts=i32(2))
    a.update(over)
    return a


def test_draft_binding(no_library):
    for fine in (dict(), dict(draft=None), dict(counts=None)):
        with pytest.raises(_Reached):
            wd.draft_verify(**draft_args(**fine))
    for bad in (dict(target=g(torch.zeros(2, 10))), dict(target=g(torch.zeros(2, 4, 10).half())), dict(draft=g(torch.zeros(2, 4, 10))),
                dict(draft=g(torch.zeros(2, 3, 10).bfloat16())), dict(tokens=g(torch.zeros(2, 3, dtype=torch.int64))), dict(tokens=i32(3, 2)),
                dict(uniforms=g(torch.zeros(2, 4))), dict(noise=g(torch.zeros(10))), dict(accepted=i32(3)), dict(out=i32(2, 3)),
                dict(counts=i32(3)), dict(workspace=torch.zeros(64, dtype=torch.uint8)), dict(workspace=None), dict(target=torch.zeros(2, 4, 10)),
                dict(noise=g(torch.zeros(10, 2)).t())):
        with pytest.raises((ValueError, TypeError)):
            wd.draft_verify(**draft_args(**bad))
