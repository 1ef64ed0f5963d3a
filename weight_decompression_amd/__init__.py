"""LLVQ (Leech-lattice vector quantization) decode and fused dequant-GEMV for MI355X.

Thin ctypes binding over the C ABI in include/llvq.h (libllvq.so, built in-tree by
weight_decompression_amd/build_lib.py).  Every computation runs in the HIP kernels;
this module only marshals arguments: torch tensors provide device memory and the
current HIP stream.  There is no CPU fallback: a call without the built library raises.
"""

import ctypes
import os

from .synth import MODE_EUCLID, MODE_SHAPEGAIN  # noqa: F401  (re-exported constants)

OUT_POINTS_I8 = 0
OUT_BF16 = 1
X_F32 = 0
X_BF16 = 1
SEARCH_ANGULAR = 0
SEARCH_EUCLID = 1
MAX_BATCH = 16
KV_BF16 = 0
KV_FP8 = 1
KV_FP4 = 2
MAX_DRAFTS = 63
MAX_NODES = 64

_ERRORS = {0: "ok", -1: "invalid argument", -2: "unsupported request", -3: "HIP launch error",
           -4: "request larger than the library's fixed workspace"}

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libllvq.so")
CHECKS_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libllvq_checks.so")

EXPORTED_SYMBOLS = ("llvq_index_count", "llvq_packed_bytes", "llvq_error_string",
                    "llvq_decode", "llvq_gemv", "llvq_encode_ref", "llvq_search", "llvq_quantize_workspace_bytes",
                    "llvq_quantize", "llvq_pack_fields", "llvq_decode_many",
                    "llvq_index_count_wide", "llvq_encode_wide", "llvq_quantize_noalloc",
                    "llvq_quantize_noalloc_max_blocks", "llvq_gptq_workspace_bytes", "llvq_gptq_factor",
                    "llvq_gptq_begin", "llvq_gptq_column", "llvq_device_checks", "llvq_kv_pool_bytes",
                    "llvq_kv_write", "llvq_kv_read", "llvq_attn", "llvq_attn_workspace_bytes",
                    "llvq_draft_verify", "llvq_draft_workspace_bytes", "llvq_attn_lse", "llvq_attn_tree",
                    "llvq_tree_verify", "llvq_tree_workspace_bytes", "llvq_kv_weigh", "llvq_kv_choose", "llvq_kv_keep")


class LlvqError(RuntimeError):
    def __init__(self, code, call):
        super().__init__(f"{call} failed: {_ERRORS.get(code, 'unknown')} ({code})")
        self.code = code


class Desc(ctypes.Structure):
    """llvq_desc: one packed weight tensor [rows][cols]."""
    _fields_ = [("mode", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("max_shell", ctypes.c_int32), ("shape_bits", ctypes.c_int32), ("gain_bits", ctypes.c_int32)]

    def __repr__(self):
        return (f"Desc(mode={self.mode}, rows={self.rows}, cols={self.cols}, max_shell={self.max_shell}, "
                f"shape_bits={self.shape_bits}, gain_bits={self.gain_bits})")


class KvDesc(ctypes.Structure):
    """llvq_kv_desc: the paged key/value cache of one layer."""
    _fields_ = [("kind", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("pages", ctypes.c_int32)]

    def __repr__(self):
        return (f"KvDesc(kind={self.kind}, kv_heads={self.kv_heads}, head_dim={self.head_dim}, "
                f"page_tokens={self.page_tokens}, pages={self.pages})")


class Batch(ctypes.Structure):
    """llvq_batch: rows of new tokens and where their sequences' caches lie."""
    _fields_ = [("starts", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("tokens", ctypes.c_int32)]


_libs = {}


def load_library(path=LIB_PATH):
    """Load libllvq.so (raises if it has not been built).

    torch is imported first: PyTorch wheels carry their own HIP runtime, and the
    library must bind to the same runtime as the streams and device pointers it is
    handed (loaded first, it would bind to the system runtime and every launch on a
    torch stream would fail)."""
    if path in _libs:
        return _libs[path]
    path = os.path.abspath(path)
    if path in _libs:
        return _libs[path]
    import torch  # noqa: F401  (selects the process's HIP runtime)
    if not os.path.exists(path):
        raise RuntimeError(f"LLVQ HIP library not found at {path}; build it with "
                           f"`python -m weight_decompression_amd.build_lib` (no CPU fallback exists)")
    lib = ctypes.CDLL(path)
    vp, i32, i64, u64p = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(ctypes.c_uint64)
    dp = ctypes.POINTER(Desc)
    lib.llvq_index_count.argtypes = [i32, u64p]
    lib.llvq_index_count.restype = ctypes.c_int
    lib.llvq_index_count_wide.argtypes = [i32, u64p, u64p]
    lib.llvq_index_count_wide.restype = ctypes.c_int
    lib.llvq_packed_bytes.argtypes = [dp]
    lib.llvq_packed_bytes.restype = i64
    lib.llvq_error_string.argtypes = [ctypes.c_int]
    lib.llvq_error_string.restype = ctypes.c_char_p
    lib.llvq_decode.argtypes = [dp, vp, vp, i32, vp, vp, vp]
    lib.llvq_decode.restype = ctypes.c_int
    lib.llvq_gemv.argtypes = [dp, vp, vp, vp, i32, i32, vp, vp, vp]
    lib.llvq_gemv.restype = ctypes.c_int
    lib.llvq_encode_ref.argtypes = [vp, i64, i32, vp, vp, vp]
    lib.llvq_encode_ref.restype = ctypes.c_int
    lib.llvq_encode_wide.argtypes = [vp, i64, i32, vp, vp, vp]
    lib.llvq_encode_wide.restype = ctypes.c_int
    lib.llvq_search.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp]
    lib.llvq_search.restype = ctypes.c_int
    lib.llvq_quantize_workspace_bytes.argtypes = [dp]
    lib.llvq_quantize_workspace_bytes.restype = i64
    lib.llvq_quantize.argtypes = [dp, vp, vp, vp, vp, vp, vp]
    lib.llvq_quantize.restype = ctypes.c_int
    lib.llvq_quantize_noalloc.argtypes = [dp, vp, vp, vp, vp, vp]
    lib.llvq_quantize_noalloc.restype = ctypes.c_int
    lib.llvq_quantize_noalloc_max_blocks.argtypes = []
    lib.llvq_quantize_noalloc_max_blocks.restype = i64
    lib.llvq_gptq_workspace_bytes.argtypes = [i32]
    lib.llvq_gptq_workspace_bytes.restype = i64
    lib.llvq_gptq_factor.argtypes = [i32, vp, ctypes.c_double, vp, vp, vp, vp]
    lib.llvq_gptq_factor.restype = ctypes.c_int
    lib.llvq_gptq_begin.argtypes = [i32, i32, vp, vp, vp, vp]
    lib.llvq_gptq_begin.restype = ctypes.c_int
    lib.llvq_gptq_column.argtypes = [dp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.llvq_gptq_column.restype = ctypes.c_int
    lib.llvq_device_checks.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
    lib.llvq_device_checks.restype = ctypes.c_int
    lib.llvq_pack_fields.argtypes = [dp, vp, vp, vp]
    lib.llvq_pack_fields.restype = ctypes.c_int
    lib.llvq_decode_many.argtypes = [vp, i32, vp, vp, i32, vp, vp, vp]
    lib.llvq_decode_many.restype = ctypes.c_int
    kp, bp, f32 = ctypes.POINTER(KvDesc), ctypes.POINTER(Batch), ctypes.c_float
    lib.llvq_kv_pool_bytes.argtypes = [kp]
    lib.llvq_kv_pool_bytes.restype = i64
    for name in ("llvq_kv_write", "llvq_kv_read"):
        getattr(lib, name).argtypes = [kp, vp, vp, i64, i64, vp, i64, i64, i32, bp, vp, vp]
        getattr(lib, name).restype = ctypes.c_int
    lib.llvq_attn.argtypes = [kp, vp, vp, i64, i64, vp, i64, i64, i32, i32, bp, i32, i32, f32, i32, i32, vp, i64, vp, vp]
    lib.llvq_attn.restype = ctypes.c_int
    lib.llvq_attn_lse.argtypes = [kp, vp, vp, i64, i64, vp, i64, i64, i32, i32, bp, i32, i32, f32, i32, i32, vp, vp, i64, vp, vp]
    lib.llvq_attn_lse.restype = ctypes.c_int
    lib.llvq_attn_tree.argtypes = [kp, vp, vp, i64, i64, vp, i64, i64, i32, i32, bp, vp, i32, i32, f32, i32, vp, i64, vp, vp]
    lib.llvq_attn_tree.restype = ctypes.c_int
    lib.llvq_attn_workspace_bytes.argtypes = [kp, i32, i64, i32, i32, i32]
    lib.llvq_attn_workspace_bytes.restype = i64
    lib.llvq_draft_verify.argtypes = [vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, i64, vp, vp]
    lib.llvq_draft_verify.restype = ctypes.c_int
    lib.llvq_draft_workspace_bytes.argtypes = [i32, i32]
    lib.llvq_draft_workspace_bytes.restype = i64
    lib.llvq_tree_verify.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, i64, vp, vp]
    lib.llvq_tree_verify.restype = ctypes.c_int
    lib.llvq_tree_workspace_bytes.argtypes = [i32, i32]
    lib.llvq_tree_workspace_bytes.restype = i64
    lib.llvq_kv_weigh.argtypes = [kp, vp, vp, vp, i64, i64, i32, i32, vp, bp, i32, i32, f32, i32, i32, i32, vp, vp]
    lib.llvq_kv_weigh.restype = ctypes.c_int
    lib.llvq_kv_choose.argtypes = [kp, vp, bp, i32, i32, i32, vp, vp, vp, vp]
    lib.llvq_kv_choose.restype = ctypes.c_int
    lib.llvq_kv_keep.argtypes = [kp, vp, vp, bp, vp, i32, i32, vp, vp, vp]
    lib.llvq_kv_keep.restype = ctypes.c_int
    _libs[path] = lib
    return lib


def _check(code, call):
    if code != 0:
        raise LlvqError(code, call)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(stream)
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _launch(function, device, stream, *args):
    """Calls a C entry (its last argument the stream) with a device current: on `stream`, or on torch's
    current stream of that device, whose handle is taken without a Stream object (which costs 3 us, as much
    as a launch)."""
    import torch
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _launch(function, device, stream, *args)
    return function(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else stream)


# ---------------------------------------------------------------------------
# argument checks: every tensor handed to the library is a contiguous device tensor of
# the right dtype and at least the size the call will touch, checked here before the
# library is loaded or a kernel launched (a short, strided or host buffer would
# otherwise become an out-of-bounds device access)

def _tensor(t, name, dtypes=None, min_bytes=0, nullable=False):
    import torch
    if t is None:
        if nullable:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (got device {t.device})")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    nbytes = t.numel() * t.element_size()
    if nbytes < min_bytes:
        raise ValueError(f"{name} holds {nbytes} bytes; the call needs at least {min_bytes}")


def _blocks(desc):
    if desc.rows <= 0 or desc.cols <= 0:
        raise ValueError(f"descriptor needs rows > 0 and cols > 0: {desc!r}")
    return desc.rows * ((desc.cols + 23) // 24)


def _packed_nbytes(desc):
    """Bytes of the packed stream (the layout of include/llvq.h: fields rounded up to a
    16-byte multiple, plus 16 bytes that kernels may over-read)."""
    from .synth import packed_nbytes
    return packed_nbytes(_blocks(desc), desc.shape_bits + desc.gain_bits)


def _scales_count(desc):
    return desc.rows if desc.mode == MODE_EUCLID else (1 << max(desc.gain_bits, 0))


def _check_decode_args(desc, packed, scales, out_kind, out, err_count, what="llvq_decode"):
    import torch
    _tensor(packed, f"{what}: packed", (torch.uint8, torch.int8), _packed_nbytes(desc))
    _tensor(err_count, f"{what}: err_count", (torch.int32,), 4, nullable=True)
    if out_kind == OUT_POINTS_I8:
        _tensor(out, f"{what}: out", (torch.int8,), _blocks(desc) * 24)
        _tensor(scales, f"{what}: scales", (torch.float16,), 0, nullable=True)
    elif out_kind == OUT_BF16:
        _tensor(out, f"{what}: out", (torch.bfloat16,), 2 * desc.rows * desc.cols)
        _tensor(scales, f"{what}: scales", (torch.float16,), 2 * _scales_count(desc))
    else:
        raise ValueError(f"{what}: out_kind must be OUT_POINTS_I8 or OUT_BF16, got {out_kind}")


def make_desc(mode, rows, cols, max_shell, shape_bits, gain_bits) -> Desc:
    return Desc(mode, rows, cols, max_shell, shape_bits, gain_bits)


def index_count(max_shell: int) -> int:
    """C_M as a Python integer (shells 2..42; past shell 33 it exceeds 64 bits)."""
    lo, hi = ctypes.c_uint64(), ctypes.c_uint64()
    _check(load_library().llvq_index_count_wide(max_shell, ctypes.byref(lo), ctypes.byref(hi)),
           "llvq_index_count_wide")
    return lo.value | (hi.value << 64)


def packed_bytes(desc: Desc) -> int:
    n = load_library().llvq_packed_bytes(ctypes.byref(desc))
    if n < 0:
        raise LlvqError(int(n), "llvq_packed_bytes")
    return n


def decode(desc, packed, scales, out_kind, out, err_count=None, stream=None):
    """Decode all blocks into `out` (int8 points [rows][Kb*24] or bf16 [rows][cols])."""
    _check_decode_args(desc, packed, scales, out_kind, out, err_count)
    _check(load_library().llvq_decode(ctypes.byref(desc), _ptr(packed), _ptr(scales), out_kind, _ptr(out),
                                      _ptr(err_count), _stream(stream)), "llvq_decode")


def gemv(desc, packed, scales, x, y, err_count=None, stream=None):
    """y[b][r] = sum_k W_hat[r][k] x[b][k]; x is fp32 or bf16 [batch][cols], y fp32 [batch][rows]."""
    import torch
    _tensor(x, "llvq_gemv: x", (torch.float32, torch.bfloat16))
    xd = X_BF16 if x.dtype == torch.bfloat16 else X_F32
    if x.dim() not in (1, 2) or x.shape[-1] != desc.cols:
        raise ValueError(f"llvq_gemv: x must be [batch][{desc.cols}] or [{desc.cols}], got {tuple(x.shape)}")
    batch = 1 if x.dim() == 1 else x.shape[0]
    if not 1 <= batch <= MAX_BATCH:
        raise ValueError(f"llvq_gemv: batch must be 1..{MAX_BATCH}, got {batch}")
    _tensor(packed, "llvq_gemv: packed", (torch.uint8, torch.int8), _packed_nbytes(desc))
    _tensor(scales, "llvq_gemv: scales", (torch.float16,), 2 * _scales_count(desc))
    _tensor(y, "llvq_gemv: y", (torch.float32,), 4 * batch * desc.rows)
    _tensor(err_count, "llvq_gemv: err_count", (torch.int32,), 4, nullable=True)
    _check(load_library().llvq_gemv(ctypes.byref(desc), _ptr(packed), _ptr(scales), _ptr(x), xd, batch, _ptr(y),
                                    _ptr(err_count), _stream(stream)), "llvq_gemv")


def _check_points(points, indices, err_count, words, what):
    import torch
    _tensor(points, f"{what}: points", (torch.int8,))
    if points.numel() % 24:
        raise ValueError(f"{what}: points must hold whole 24-vectors, got {points.numel()} values")
    n = points.numel() // 24
    _tensor(indices, f"{what}: indices", (torch.int64,), 8 * words * n)
    _tensor(err_count, f"{what}: err_count", (torch.int32,), 4, nullable=True)
    return n


def encode_ref(points, max_shell, indices, err_count=None, stream=None):
    """Rank int8 lattice points [n][24] into uint64 shape indices [n] (int64 tensor)."""
    n = _check_points(points, indices, err_count, 1, "llvq_encode_ref")
    _check(load_library().llvq_encode_ref(_ptr(points), n, max_shell, _ptr(indices), _ptr(err_count),
                                          _stream(stream)), "llvq_encode_ref")


def search(x, max_shell, objective, points, indices, err_count=None, stream=None):
    """Nearest point of shells 2..max_shell to each fp32 24-vector x [n][24]
    (SEARCH_ANGULAR or SEARCH_EUCLID): int8 points [n][24] and uint64 indices [n]
    (int64 tensor) are written."""
    import torch
    _tensor(x, "llvq_search: x", (torch.float32,))
    if x.numel() % 24:
        raise ValueError(f"llvq_search: x must hold whole 24-blocks, got {x.numel()} values")
    n = x.numel() // 24
    _tensor(points, "llvq_search: points", (torch.int8,), 24 * n)
    _tensor(indices, "llvq_search: indices", (torch.int64,), 8 * n)
    _tensor(err_count, "llvq_search: err_count", (torch.int32,), 4, nullable=True)
    _check(load_library().llvq_search(_ptr(x), n, max_shell, objective, _ptr(points), _ptr(indices),
                                      _ptr(err_count), _stream(stream)), "llvq_search")


def quantize_workspace_bytes(desc: Desc) -> int:
    n = load_library().llvq_quantize_workspace_bytes(ctypes.byref(desc))
    if n < 0:
        raise LlvqError(int(n), "llvq_quantize_workspace_bytes")
    return n


def quantize(desc, w, scales, packed, workspace, err_count=None, stream=None):
    """Quantise fp32 weights w [rows][cols] into the packed stream (uint8 tensor of
    packed_bytes(desc) bytes); workspace: quantize_workspace_bytes(desc) bytes of device memory."""
    import torch
    n = _blocks(desc)
    _tensor(w, "llvq_quantize: w", (torch.float32,), 4 * desc.rows * desc.cols)
    _tensor(scales, "llvq_quantize: scales", (torch.float16,), 2 * _scales_count(desc))
    _tensor(packed, "llvq_quantize: packed", (torch.uint8, torch.int8), _packed_nbytes(desc))
    _tensor(workspace, "llvq_quantize: workspace", None, (24 * n + 7) // 8 * 8 + 8 * n)
    _tensor(err_count, "llvq_quantize: err_count", (torch.int32,), 4, nullable=True)
    _check(load_library().llvq_quantize(ctypes.byref(desc), _ptr(w), _ptr(scales), _ptr(packed), _ptr(workspace),
                                        _ptr(err_count), _stream(stream)), "llvq_quantize")


def quantize_noalloc(desc, w, scales, packed, err_count=None, stream=None):
    """quantize() without a workspace argument: the library's own fixed device array is used
    (at most quantize_noalloc_max_blocks() blocks; calls that overlap on one GPU race)."""
    import torch
    _tensor(w, "llvq_quantize_noalloc: w", (torch.float32,), 4 * desc.rows * desc.cols)
    _tensor(scales, "llvq_quantize_noalloc: scales", (torch.float16,), 2 * _scales_count(desc))
    _tensor(packed, "llvq_quantize_noalloc: packed", (torch.uint8, torch.int8), _packed_nbytes(desc))
    _tensor(err_count, "llvq_quantize_noalloc: err_count", (torch.int32,), 4, nullable=True)
    _check(load_library().llvq_quantize_noalloc(ctypes.byref(desc), _ptr(w), _ptr(scales), _ptr(packed),
                                                _ptr(err_count), _stream(stream)), "llvq_quantize_noalloc")


def quantize_noalloc_max_blocks() -> int:
    return int(load_library().llvq_quantize_noalloc_max_blocks())


def pack_fields(desc, fields, packed, stream=None):
    """Write uint64 fields [rows * Kb] (int64 tensor) as the packed stream of desc."""
    import torch
    _tensor(fields, "llvq_pack_fields: fields", (torch.int64,), 8 * _blocks(desc))
    _tensor(packed, "llvq_pack_fields: packed", (torch.uint8, torch.int8), _packed_nbytes(desc))
    _check(load_library().llvq_pack_fields(ctypes.byref(desc), _ptr(fields), _ptr(packed), _stream(stream)),
           "llvq_pack_fields")


def decode_many(descs, packed, scales, out_kind, outs, err_count=None, stream=None):
    """llvq_decode of several tensors in one call (equal widths and shell range)."""
    n = len(descs)
    if not (len(packed) == len(outs) == n and (scales is None or len(scales) == n)):
        raise ValueError("llvq_decode_many: descs, packed, scales and outs need one entry per tensor")
    for i in range(n):
        _check_decode_args(descs[i], packed[i], None if scales is None else scales[i], out_kind, outs[i],
                           err_count, f"llvq_decode_many[{i}]")
    darr = (Desc * n)(*descs)
    parr = (ctypes.c_void_p * n)(*[p.data_ptr() for p in packed])
    sarr = None if scales is None else (ctypes.c_void_p * n)(*[x.data_ptr() for x in scales])
    oarr = (ctypes.c_void_p * n)(*[o.data_ptr() for o in outs])
    _check(load_library().llvq_decode_many(ctypes.cast(darr, ctypes.c_void_p), n, ctypes.cast(parr, ctypes.c_void_p),
                                           None if sarr is None else ctypes.cast(sarr, ctypes.c_void_p), out_kind,
                                           ctypes.cast(oarr, ctypes.c_void_p), _ptr(err_count), _stream(stream)),
           "llvq_decode_many")


def encode_wide(points, max_shell, indices, err_count=None, stream=None):
    """llvq_encode_wide: int8 points [n][24] -> 128-bit indices as int64 pairs [n][2] (lo, hi)."""
    n = _check_points(points, indices, err_count, 2, "llvq_encode_wide")
    _check(load_library().llvq_encode_wide(_ptr(points), n, max_shell, _ptr(indices),
                                           _ptr(err_count), _stream(stream)), "llvq_encode_wide")


# ---------------------------------------------------------------------------
# serving: the paged key/value cache, the attention over it, the check of drafts

def make_kv_desc(kind, kv_heads, head_dim, page_tokens, pages) -> KvDesc:
    return KvDesc(kind, kv_heads, head_dim, page_tokens, pages)


def kv_pool_bytes(desc: KvDesc) -> int:
    """Bytes of the pool [pages][kv_heads][block] (include/llvq.h gives a block's layout)."""
    n = load_library().llvq_kv_pool_bytes(ctypes.byref(desc))
    if n < 0:
        raise LlvqError(int(n), "llvq_kv_pool_bytes")
    return n


def _pool_nbytes(desc):
    kind, heads, dim, page, pages = desc.kind, desc.kv_heads, desc.head_dim, desc.page_tokens, desc.pages
    if kind not in (KV_BF16, KV_FP8, KV_FP4) or pages < 1 or heads < 1 or dim < 1 or page < 1:
        raise ValueError(f"invalid cache descriptor: {desc!r}")
    token = 2 * dim if kind == KV_BF16 else (dim if kind == KV_FP8 else dim // 2) + dim // 32
    return pages * heads * ((2 * page * token + 15) // 16 * 16)


# These calls run many times a token, and a call's checks cost as much as its launch (3 us): the ordinary case
# is one expression over all of a call's tensors, and only where it fails is each looked at for the message.

def _buffer(t, call, name, dtype=None, nbytes=0):
    """Checks a contiguous device buffer (dtype None: any); returns its address."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{call}: {name} must be a torch tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{call}: {name} must be a GPU tensor (got device {t.device})")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{call}: {name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{call}: {name} must be contiguous")
    if nbytes and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{call}: {name} holds {t.numel() * t.element_size()} bytes; the call needs at least {nbytes}")
    return t.data_ptr()


def _count(err_count, device, call):
    import torch
    at = _buffer(err_count, call, "err_count", torch.int32, 4)
    _one_device(call, device, err_count)
    return at


def _space(workspace, device, call):
    """A workspace's address and bytes."""
    at = _buffer(workspace, call, "workspace")
    _one_device(call, device, workspace)
    return at, workspace.numel() * workspace.element_size()


def _rows(t, call, name, heads, dim):
    """Checks rows [tokens][heads][dim] of fp32 or bf16 with contiguous channels; returns the address
    and the (token, head) strides in elements."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{call}: {name} must be a torch tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{call}: {name} must be a GPU tensor (got device {t.device})")
    if t.dtype is not torch.bfloat16 and t.dtype is not torch.float32:
        raise TypeError(f"{call}: {name} must have dtype torch.float32 or torch.bfloat16, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{call}: {name} must be [tokens][{heads}][{dim}], got {tuple(shape)}")
    if stride[2] != 1 and shape[0]:
        raise ValueError(f"{call}: {name} must have contiguous channels (strides {stride})")
    return t.data_ptr(), stride[0], stride[1]


def _apart(t, call, name):
    """Refuses an output whose rows lie over each other (a broadcast or overlapping view)."""
    if t.is_contiguous():
        return
    (n, heads, dim), (token, head, _) = t.shape, t.stride()
    lo, hi = sorted(((token, n), (head, heads)))
    if n and not ((heads == 1 or head >= dim) and (n == 1 or token >= dim) and
                  (n == 1 or heads == 1 or hi[0] >= (lo[1] - 1) * lo[0] + dim)):
        raise ValueError(f"{call}: {name} has rows that overlap (strides {t.stride()})")


def _one_device(call, device, *tensors):
    if any(t.get_device() != device for t in tensors):
        raise ValueError(f"{call}: tensors on several devices")


def _paged(desc, pool, starts, lens, table, tokens, device, call):
    """The pool's address and llvq_batch from starts [B + 1], lens [B] and table [B][max_pages] (int32)."""
    import torch
    i32 = torch.int32
    need = _pool_nbytes(desc)
    try:
        good = (pool.get_device() == starts.get_device() == lens.get_device() == table.get_device() == device and
                pool.dtype is torch.uint8 and
                starts.dtype is i32 and lens.dtype is i32 and table.dtype is i32 and pool.is_contiguous() and
                starts.is_contiguous() and lens.is_contiguous() and table.is_contiguous() and pool.numel() >= need)
    except AttributeError:
        good = False
    if not good:
        _buffer(pool, call, "pool", torch.uint8, need)
        for t, name in ((starts, "starts"), (lens, "lens"), (table, "table")):
            _buffer(t, call, name, i32)
        _one_device(call, device, pool, starts, lens, table)
    n, shape = lens.shape, table.shape
    if len(n) != 1 or len(shape) != 2 or shape[0] != n[0] or starts.shape != (n[0] + 1,):
        raise ValueError(f"{call}: starts, lens and table must be [B + 1], [B] and [B][max_pages], got "
                         f"{tuple(starts.shape)}, {tuple(n)} and {tuple(shape)}")
    return pool.data_ptr(), Batch(starts.data_ptr(), lens.data_ptr(), table.data_ptr(), n[0], shape[1], tokens)


def _pair(call, a, b, names, heads, dim):
    """Checks two tensors of rows of one shape and dtype; (address, strides) of each and the dtype code."""
    import torch
    try:
        shape, sa, sb, dtype = a.shape, a.stride(), b.stride(), a.dtype
        good = (0 <= a.get_device() == b.get_device() and (dtype is torch.bfloat16 or dtype is torch.float32) and b.dtype is dtype and
                b.shape == shape and len(shape) == 3 and shape[1] == heads and shape[2] == dim and sa[2] == 1 and sb[2] == 1)
    except (AttributeError, IndexError):
        good = False
    if not good:
        _rows(a, call, names[0], heads, dim)
        _rows(b, call, names[1], heads, dim)
        if a.shape != b.shape or a.dtype is not b.dtype:
            raise ValueError(f"{call}: {names[0]} and {names[1]} must have one shape and dtype, got {tuple(a.shape)} {a.dtype} and "
                             f"{tuple(b.shape)} {b.dtype}")
        _one_device(call, a.get_device(), b)
        sa, sb, dtype = a.stride(), b.stride(), a.dtype
    return a.data_ptr(), sa[0], sa[1], b.data_ptr(), sb[0], sb[1], X_F32 if dtype is torch.float32 else X_BF16


def _kv_call(call, desc, pool, k, v, starts, lens, table, err_count, stream):
    rows = _pair(call, k, v, "kv", desc.kv_heads, desc.head_dim)
    if call == "llvq_kv_read":
        _apart(k, call, "k")
        _apart(v, call, "v")
    device = k.get_device()
    at, batch = _paged(desc, pool, starts, lens, table, k.shape[0], device, call)
    err = None if err_count is None else _count(err_count, device, call)
    code = _launch(getattr(load_library(), call), device, stream, desc, at, *rows, batch, err)
    if code:
        raise LlvqError(code, call)


def kv_write(desc, pool, k, v, starts, lens, table, err_count=None, stream=None):
    """Quantise the new tokens' keys and values [tokens][kv_heads][head_dim] (fp32 or bf16, any token and
    head strides) into the pool: sequence b's rows are starts[b]..starts[b + 1] and the last of its
    lens[b] cached tokens; table [B][max_pages] names its pages."""
    _kv_call("llvq_kv_write", desc, pool, k, v, starts, lens, table, err_count, stream)


def kv_read(desc, pool, k, v, starts, lens, table, err_count=None, stream=None):
    """Read the same rows back into k and v (fp32 or bf16; apart from each other and the pool), as the values they stand
    for."""
    _kv_call("llvq_kv_read", desc, pool, k, v, starts, lens, table, err_count, stream)


def attn_workspace_bytes(desc, heads, tokens, batch, max_chunk, max_len) -> int:
    """Bytes of a workspace for every attn call of no more tokens, sequences, new tokens of one and keys than these."""
    n = load_library().llvq_attn_workspace_bytes(desc, heads, tokens, batch, max_chunk, max_len)
    if n < 0:
        raise LlvqError(int(n), "llvq_attn_workspace_bytes")
    return n


def _attn_call(call, desc, pool, q, out, starts, lens, table, workspace, max_chunk, max_len, err_count, stream, between):
    """The checks and the call that attn's forms share; between: the C entry's arguments from the batch to the workspace, or a
    function of the device and [tokens, heads] that checks and gives them."""
    import torch
    heads = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
    if heads < 1 or desc.kv_heads < 1 or heads % desc.kv_heads:
        raise ValueError(f"{call}: q must be [tokens][heads][{desc.head_dim}] with a multiple of {desc.kv_heads} heads")
    *rows, dtype = _pair(call, q, out, ("q", "out"), heads, desc.head_dim)
    _apart(out, call, "out")
    device = q.get_device()
    at, batch = _paged(desc, pool, starts, lens, table, q.shape[0], device, call)
    ws, size = (None, 0) if workspace is None else _space(workspace, device, call)
    err = None if err_count is None else _count(err_count, device, call)
    code = _launch(getattr(load_library(), call), device, stream, desc, at, *rows, dtype, heads, batch,
                   *(between if type(between) is tuple else between(device, (q.shape[0], heads))), ws, size, err)
    if code:
        need = attn_workspace_bytes(desc, heads, q.shape[0], batch.batch, max_chunk, max_len)
        if size < need:
            raise ValueError(f"{call}: invalid argument, or the workspace is short: it holds {size} bytes, {need} are enough")
        raise LlvqError(code, call)


def _vector(t, call, name, dtype, shape, device):
    """Checks a contiguous device tensor of that shape; returns its address."""
    import torch
    if not (isinstance(t, torch.Tensor) and t.get_device() == device and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        _buffer(t, call, name, dtype)
        _one_device(call, device, t)
        raise ValueError(f"{call}: {name} must be {list(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def attn(desc, pool, q, out, starts, lens, table, workspace, max_chunk, max_len, scale=None, causal=True, window=0,
         err_count=None, stream=None, lse=None):
    """out[i][h] = softmax(scale * q[i][h] . K) V over the cached tokens that new token i sees.
    q and out: [tokens][heads][head_dim], fp32 or bf16; scale: 1 / sqrt(head_dim) if None; max_chunk: at least any
    sequence's new tokens; max_len: about the longest length (decides only how the keys are split); out overlaps neither q
    nor the pool; workspace: attn_workspace_bytes(...) bytes for these or larger arguments (None if that is 0); lse: if given,
    fp32 [tokens][heads], receives log sum exp(scale * q[i][h] . K) of each row."""
    import torch
    scale = desc.head_dim ** -0.5 if scale is None else scale
    if lse is None:
        _attn_call("llvq_attn", desc, pool, q, out, starts, lens, table, workspace, max_chunk, max_len, err_count, stream,
                   (max_chunk, max_len, scale, 1 if causal else 0, window))
    else:
        _attn_call("llvq_attn_lse", desc, pool, q, out, starts, lens, table, workspace, max_chunk, max_len, err_count, stream,
                   lambda device, shape: (max_chunk, max_len, scale, 1 if causal else 0, window,
                                          _vector(lse, "llvq_attn_lse", "lse", torch.float32, shape, device)))


def attn_tree(desc, pool, q, out, starts, lens, table, parents, workspace, max_chunk, max_len, scale=None, window=0,
              err_count=None, stream=None):
    """attn for trees of drafted tokens: a sequence's new tokens are the nodes of a tree, parents [tokens] (int32) gives each
    node's parent among them (-1: it follows the text), and a node sees the text, the nodes above it and itself.  At most
    MAX_NODES new tokens a sequence; the workspace is attn's."""
    import torch
    call = "llvq_attn_tree"
    scale = desc.head_dim ** -0.5 if scale is None else scale
    _attn_call(call, desc, pool, q, out, starts, lens, table, workspace, max_chunk, max_len, err_count, stream,
               lambda device, shape: (_vector(parents, call, "parents", torch.int32, shape[:1], device), max_chunk, max_len, scale,
                                      window))


def draft_workspace_bytes(batch, vocab) -> int:
    """Bytes of a workspace for every draft_verify call of no more sequences and entries than these."""
    n = load_library().llvq_draft_workspace_bytes(batch, vocab)
    if n < 0:
        raise LlvqError(int(n), "llvq_draft_workspace_bytes")
    return n


def draft_verify(target, draft, tokens, uniforms, noise, accepted, out, workspace, counts=None, err_count=None,
                 stream=None):
    """Check drafts tokens [B][S] against target [B][S + 1][V] (fp32 or bf16 probabilities; draft [B][S][V] or None for
    certain drafts) with uniforms [B][S] and exponential noise [B][V]: accepted [B] and out [B][S + 1]
    (accepted tokens, one drawn token, then -1), int32."""
    import torch
    call = "llvq_draft_verify"
    i32, f32 = torch.int32, torch.float32
    dtype = target.dtype if isinstance(target, torch.Tensor) else None
    at = _buffer(target, call, "target")
    if dtype is not f32 and dtype is not torch.bfloat16:
        raise TypeError(f"{call}: target must have dtype torch.float32 or torch.bfloat16, got {dtype}")
    if target.dim() != 3 or target.shape[1] < 1:
        raise ValueError(f"{call}: target must be [B][drafts + 1][vocab], got {tuple(target.shape)}")
    b, s, v = target.shape
    s -= 1
    each = ((tokens, "tokens", i32, (b, s)), (uniforms, "uniforms", f32, (b, s)), (noise, "noise", f32, (b, v)),
            (accepted, "accepted", i32, (b,)), (out, "out", i32, (b, s + 1)))
    if draft is not None:
        each += ((draft, "draft", dtype, (b, s, v)),)
    if counts is not None:
        each += ((counts, "counts", i32, (b,)),)
    device = target.get_device()
    for t, name, kind, shape in each:
        if not (isinstance(t, torch.Tensor) and t.get_device() == device and t.dtype is kind and t.shape == shape and t.is_contiguous()):
            _buffer(t, call, name, kind)
            _one_device(call, device, t)
            raise ValueError(f"{call}: {name} must be {list(shape)}, got {tuple(t.shape)}")
    ws, size = _space(workspace, device, call)
    err = None if err_count is None else _count(err_count, device, call)
    code = _launch(load_library().llvq_draft_verify, device, stream, at, None if draft is None else draft.data_ptr(),
                   X_F32 if dtype is f32 else X_BF16, tokens.data_ptr(), None if counts is None else counts.data_ptr(),
                   uniforms.data_ptr(), noise.data_ptr(), b, s, v, accepted.data_ptr(), out.data_ptr(), ws, size, err)
    if code:
        need = draft_workspace_bytes(b, v)
        if size < need:
            raise ValueError(f"{call}: invalid argument, or the workspace is short: it holds {size} bytes, {need} are enough")
        raise LlvqError(code, call)


def tree_workspace_bytes(batch, vocab) -> int:
    """Bytes of a workspace for every tree_verify call of no more sequences and entries than these."""
    n = load_library().llvq_tree_workspace_bytes(batch, vocab)
    if n < 0:
        raise LlvqError(int(n), "llvq_tree_workspace_bytes")
    return n


def tree_verify(target, starts, tokens, parents, uniforms, noise, accepted, path, out, workspace, err_count=None, stream=None):
    """Check trees of drafts that were picked: target [nodes][V] (fp32 or bf16 probabilities after each node), starts [B + 1],
    tokens and parents [nodes] (int32; node 0 of a sequence is the last token of its text), uniforms [nodes] and exponential
    noise [B][V] (fp32).  accepted [B]; path [B][W]: the accepted nodes from 0 on, then -1; out [B][W]: the accepted tokens, one
    drawn token, then -1 (int32); at most W - 1 drafts are accepted."""
    import torch
    call = "llvq_tree_verify"
    i32, f32 = torch.int32, torch.float32
    try:
        (n, v), (b, width), dtype, device = target.shape, path.shape, target.dtype, target.get_device()
        good = (0 <= device == starts.get_device() == tokens.get_device() == parents.get_device() == uniforms.get_device() ==
                noise.get_device() == accepted.get_device() == path.get_device() == out.get_device() == workspace.get_device() and
                (dtype is f32 or dtype is torch.bfloat16) and starts.dtype is i32 and tokens.dtype is i32 and parents.dtype is i32 and
                uniforms.dtype is f32 and noise.dtype is f32 and accepted.dtype is i32 and path.dtype is i32 and out.dtype is i32 and
                starts.shape == (b + 1,) and tokens.shape == parents.shape == uniforms.shape == (n,) and noise.shape == (b, v) and
                accepted.shape == (b,) and out.shape == (b, width) and target.is_contiguous() and starts.is_contiguous() and
                tokens.is_contiguous() and parents.is_contiguous() and uniforms.is_contiguous() and noise.is_contiguous() and
                accepted.is_contiguous() and path.is_contiguous() and out.is_contiguous() and workspace.is_contiguous())
    except (AttributeError, ValueError):
        good = False
    if not good:
        dtype = target.dtype if isinstance(target, torch.Tensor) else None
        _buffer(target, call, "target")
        if dtype is not f32 and dtype is not torch.bfloat16:
            raise TypeError(f"{call}: target must have dtype torch.float32 or torch.bfloat16, got {dtype}")
        _buffer(noise, call, "noise", f32)
        _buffer(path, call, "path", i32)
        if target.dim() != 2 or noise.dim() != 2 or path.dim() != 2:
            raise ValueError(f"{call}: target, noise and path must be [nodes][vocab], [B][vocab] and [B][width], got "
                             f"{tuple(target.shape)}, {tuple(noise.shape)} and {tuple(path.shape)}")
        (n, v), (b, width), device = target.shape, path.shape, target.get_device()
        for t, name, kind, shape in (
                (starts, "starts", i32, (b + 1,)), (tokens, "tokens", i32, (n,)), (parents, "parents", i32, (n,)),
                (uniforms, "uniforms", f32, (n,)), (noise, "noise", f32, (b, v)), (accepted, "accepted", i32, (b,)),
                (path, "path", i32, (b, width)), (out, "out", i32, (b, width))):
            _vector(t, call, name, kind, shape, device)
        _space(workspace, device, call)
    size = workspace.numel() * workspace.element_size()
    err = None if err_count is None else _count(err_count, device, call)
    code = _launch(load_library().llvq_tree_verify, device, stream, target.data_ptr(), X_F32 if dtype is f32 else X_BF16,
                   starts.data_ptr(), tokens.data_ptr(), parents.data_ptr(), uniforms.data_ptr(), noise.data_ptr(), b, n, v, width,
                   accepted.data_ptr(), path.data_ptr(), out.data_ptr(), workspace.data_ptr(), size, err)
    if code:
        need = tree_workspace_bytes(b, v)
        if size < need:
            raise ValueError(f"{call}: invalid argument, or the workspace is short: it holds {size} bytes, {need} are enough")
        raise LlvqError(code, call)


# ---------------------------------------------------------------------------
# eviction: what cached tokens have received, which of them stay, their move to the front

def _weights(desc, weights, device, call):
    import torch
    return _vector(weights, call, "weights", torch.float32, (desc.pages, desc.kv_heads, desc.page_tokens), device)


def _lists(lens, table, starts, device, call):
    """llvq_batch of lens [B], table [B][max_pages] and, if any, starts [B + 1] (int32)."""
    import torch
    i32 = torch.int32
    try:
        good = (lens.get_device() == table.get_device() == device and lens.dtype is i32 and table.dtype is i32 and
                lens.is_contiguous() and table.is_contiguous() and
                (starts is None or (starts.get_device() == device and starts.dtype is i32 and starts.is_contiguous())))
    except AttributeError:
        good = False
    if not good:
        _buffer(lens, call, "lens", i32)
        _buffer(table, call, "table", i32)
        if starts is not None:
            _buffer(starts, call, "starts", i32)
        _one_device(call, device, lens, table, *(() if starts is None else (starts,)))
    n, shape = lens.shape, table.shape
    if len(n) != 1 or len(shape) != 2 or shape[0] != n[0] or (starts is not None and starts.shape != (n[0] + 1,)):
        raise ValueError(f"{call}: lens, table and starts must be [B], [B][max_pages] and [B + 1] or None, got {tuple(n)}, {tuple(shape)} "
                         f"and {None if starts is None else tuple(starts.shape)}")
    return Batch(None if starts is None else starts.data_ptr(), lens.data_ptr(), table.data_ptr(), n[0], shape[1], 0)


def kv_weigh(desc, pool, weights, q, lse, starts, lens, table, max_chunk, max_len, scale=None, causal=True, window=0, fresh=False,
             err_count=None, stream=None):
    """weights[j] += sum of exp(scale * q[i][h] . K_j - lse[i][h]) over the new tokens i and heads h of a key head that see the
    cached token j.  weights: fp32 [pages][kv_heads][page_tokens], at the tokens' places; those of the new tokens start from
    zero, with fresh=True those of all (needed once where tokens came in that no call has weighed).  q: [tokens][heads][head_dim],
    fp32 or bf16; lse: fp32 [tokens][heads], as attn gives it for the same rows, scale and mask; max_chunk: at least any sequence's
    new tokens; max_len: about the longest length."""
    import torch
    call, f32 = "llvq_kv_weigh", torch.float32
    try:
        shape, stride, dtype, device = q.shape, q.stride(), q.dtype, q.get_device()
        heads, kv_heads = shape[1], desc.kv_heads
        good = (0 <= device == weights.get_device() == lse.get_device() and len(shape) == 3 and heads >= 1 and kv_heads >= 1 and
                heads % kv_heads == 0 and shape[2] == desc.head_dim and stride[2] == 1 and (dtype is torch.bfloat16 or dtype is f32) and
                weights.dtype is f32 and lse.dtype is f32 and weights.shape == (desc.pages, kv_heads, desc.page_tokens) and
                lse.shape == (shape[0], heads) and weights.is_contiguous() and lse.is_contiguous())
    except (AttributeError, IndexError):
        good = False
    if not good:
        heads = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
        if heads < 1 or desc.kv_heads < 1 or heads % desc.kv_heads:
            raise ValueError(f"{call}: q must be [tokens][heads][{desc.head_dim}] with a multiple of {desc.kv_heads} heads")
        _rows(q, call, "q", heads, desc.head_dim)
        shape, stride, dtype, device = q.shape, q.stride(), q.dtype, q.get_device()
        _vector(weights, call, "weights", f32, (desc.pages, desc.kv_heads, desc.page_tokens), device)
        _vector(lse, call, "lse", f32, (shape[0], heads), device)
    at, batch = _paged(desc, pool, starts, lens, table, shape[0], device, call)
    err = None if err_count is None else _count(err_count, device, call)
    code = _launch(load_library().llvq_kv_weigh, device, stream, desc, at, weights.data_ptr(), q.data_ptr(), stride[0], stride[1],
                   X_F32 if dtype is f32 else X_BF16, heads, lse.data_ptr(), batch, max_chunk, max_len,
                   desc.head_dim ** -0.5 if scale is None else scale, 1 if causal else 0, window, 1 if fresh else 0, err)
    if code:
        raise LlvqError(code, call)


def kv_choose(desc, weights, lens, table, keep, counts, sinks=0, recent=0, err_count=None, stream=None):
    """keep [B][kv_heads][budget] (int32): the positions that stay of each sequence and key head, ascending, then -1: the first
    `sinks`, the last `recent`, and between them the largest weights, the lowest position of equals.  counts [B] (int32): how many.
    A window counts cached places: where attention has one, recent >= window - 1 keeps what later rows see as it was."""
    import torch
    call, i32, f32 = "llvq_kv_choose", torch.int32, torch.float32
    try:
        shape, device, (n, pages), heads = keep.shape, keep.get_device(), table.shape, desc.kv_heads
        good = (0 <= device == lens.get_device() == table.get_device() == counts.get_device() == weights.get_device() and
                keep.dtype is i32 and lens.dtype is i32 and table.dtype is i32 and counts.dtype is i32 and weights.dtype is f32 and
                len(shape) == 3 and shape[0] == n and shape[1] == heads and lens.shape == counts.shape == (n,) and
                weights.shape == (desc.pages, heads, desc.page_tokens) and keep.is_contiguous() and lens.is_contiguous() and
                table.is_contiguous() and counts.is_contiguous() and weights.is_contiguous())
    except (AttributeError, ValueError):
        good = False
    if good:
        batch = Batch(None, lens.data_ptr(), table.data_ptr(), n, pages, 0)
    else:
        _buffer(keep, call, "keep", i32)
        device = keep.get_device()
        batch = _lists(lens, table, None, device, call)
        if keep.dim() != 3 or keep.shape[:2] != (batch.batch, desc.kv_heads):
            raise ValueError(f"{call}: keep must be [{batch.batch}][{desc.kv_heads}][budget], got {tuple(keep.shape)}")
        shape = keep.shape
        _weights(desc, weights, device, call)
        _vector(counts, call, "counts", i32, (batch.batch,), device)
    err = None if err_count is None else _count(err_count, device, call)
    code = _launch(load_library().llvq_kv_choose, device, stream, desc, weights.data_ptr(), batch, shape[2], sinks, recent,
                   keep.data_ptr(), counts.data_ptr(), err)
    if code:
        raise LlvqError(code, call)


def kv_keep(desc, pool, keep, lens, table, counts=None, starts=None, weights=None, err_count=None, stream=None):
    """Move the cached token at place keep[b][h][i] of sequence b and key head h to place i, in place, for i < counts[b] (all
    entries without counts; -1 moves nothing).  keep: int32 [B][kv_heads][N], or [B][1][N] for all heads alike, ascending.  With
    starts [B + 1], places count from the sequence's first new token, so that tree_verify's path[:, None] moves the accepted
    nodes together (of a sequence with more new tokens than cached ones nothing moves).  weights: moved along if given."""
    import torch
    call, i32, f32 = "llvq_kv_keep", torch.int32, torch.float32
    need = _pool_nbytes(desc)
    try:
        shape, device, (n, pages), heads = keep.shape, keep.get_device(), table.shape, desc.kv_heads
        good = (0 <= device == pool.get_device() == lens.get_device() == table.get_device() and keep.dtype is i32 and
                pool.dtype is torch.uint8 and lens.dtype is i32 and table.dtype is i32 and len(shape) == 3 and shape[0] == n and
                (shape[1] == heads or shape[1] == 1) and lens.shape == (n,) and pool.numel() >= need and keep.is_contiguous() and
                pool.is_contiguous() and lens.is_contiguous() and table.is_contiguous() and
                (counts is None or (counts.get_device() == device and counts.dtype is i32 and counts.shape == (n,) and counts.is_contiguous())) and
                (starts is None or (starts.get_device() == device and starts.dtype is i32 and starts.shape == (n + 1,) and
                                    starts.is_contiguous())) and
                (weights is None or (weights.get_device() == device and weights.dtype is f32 and weights.is_contiguous() and
                                     weights.shape == (desc.pages, heads, desc.page_tokens))))
    except (AttributeError, ValueError):
        good = False
    if good:
        batch = Batch(None if starts is None else starts.data_ptr(), lens.data_ptr(), table.data_ptr(), n, pages, 0)
    else:
        _buffer(keep, call, "keep", i32)
        device = keep.get_device()
        _buffer(pool, call, "pool", torch.uint8, need)
        _one_device(call, device, pool)
        batch = _lists(lens, table, starts, device, call)
        if keep.dim() != 3 or keep.shape[0] != batch.batch or keep.shape[1] not in (1, desc.kv_heads):
            raise ValueError(f"{call}: keep must be [{batch.batch}][{desc.kv_heads} or 1][entries], got {tuple(keep.shape)}")
        shape = keep.shape
        if weights is not None:
            _weights(desc, weights, device, call)
        if counts is not None:
            _vector(counts, call, "counts", i32, (batch.batch,), device)
    err = None if err_count is None else _count(err_count, device, call)
    code = _launch(load_library().llvq_kv_keep, device, stream, desc, pool.data_ptr(), None if weights is None else weights.data_ptr(), batch,
                   keep.data_ptr(), shape[1], shape[2], None if counts is None else counts.data_ptr(), err)
    if code:
        raise LlvqError(code, call)
