"""Block-scaled FP4 quantization (NVFP4 with Four Over Six, RHT16 + SR, 16x16
tiles; MXFP4 with a 32-point Hadamard) for AMD MI355X.

Thin ctypes binding over ``libfp4q.so`` (see ``include/fp4q.h``).  Every
step of the quantization runs in the library's HIP kernels; this module only
allocates torch device buffers, checks dtypes and forwards pointers and the
current stream.  There is no fallback: without the built library, or without
a GPU, the calls raise.

Two layers:
  * ``lib()`` -- the raw C functions (``nvfp4_quantize`` etc.) taking
    integers for device pointers and the stream, returning an int status.
  * tensor helpers with the same names taking/returning torch tensors.
"""
from __future__ import annotations

import ctypes as C
import importlib
import os

FOUR_OVER_SIX = 1 << 0
SR = 1 << 1
RHT16 = 1 << 2
BLOCK2D = 1 << 3
HAD32 = 1 << 4
ROWWISE = 1 << 5
COLWISE = 1 << 6
MSEDEN = 1 << 7
RTN6 = 0

FORMAT_NVFP4 = 0
FORMAT_MXFP4 = 1

STATUS = {0: "FP4_OK", -1: "FP4_E_NULL", -2: "FP4_E_SHAPE", -3: "FP4_E_ALIGN",
          -4: "FP4_E_FLAGS", -5: "FP4_E_WORKSPACE", -6: "FP4_E_HIP"}

ROPE_INTERLEAVED = 1 << 0
ROW_ALPHA = 1 << 8

EXPORTS = ("fp4_workspace_bytes", "fp4_tensor_amax", "nvfp4_quantize", "nvfp4_quantize_noalloc",
           "nvfp4_quantize_rows",
           "nvfp4_requantize_t", "mxfp4_quantize", "mxfp4_gemm", "fp4_dequantize",
           "fp4_kv_write", "fp4_kv_read", "fp4_kv_attention_workspace_bytes", "fp4_kv_attention",
           "qk_norm_rope", "qk_norm_rope_workspace_bytes", "qk_norm_rope_backward",
           "fp4_linear_workspace_bytes", "fp4_linear", "expert_route", "expert_route_backward",
           "fp4_experts_workspace_bytes", "fp4_experts", "residual_norm",
           "residual_norm_workspace_bytes", "residual_norm_backward",
           "fp4_status_str", "fp4_abi_version")


class _CCache(C.Structure):
    """fp4_kv_cache of include/fp4q.h."""
    _fields_ = [(n, C.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales", "k_amax",
                                          "v_amax")] + [
        ("pages", C.c_int64)] + [(n, C.c_int32) for n in ("page_size", "heads", "head_dim",
                                                          "format")] + [("flags", C.c_uint32)]


class _CQueries(C.Structure):
    """fp4_kv_queries of include/fp4q.h."""
    _fields_ = [("q", C.c_void_p), ("q_stride", C.c_int64), ("tokens", C.c_int64),
                ("seqs", C.c_int64), ("cu_q", C.c_void_p), ("max_q", C.c_int64),
                ("kv_lens", C.c_void_p), ("page_table", C.c_void_p), ("table_width", C.c_int64),
                ("q_heads", C.c_int32), ("window", C.c_int32), ("scale", C.c_float),
                ("softcap", C.c_float)]


class _CRope(C.Structure):
    """fp4_qk_rope of include/fp4q.h."""
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("q_stride", C.c_int64),
                ("k_stride", C.c_int64), ("tokens", C.c_int64), ("q_weight", C.c_void_p),
                ("k_weight", C.c_void_p), ("positions", C.c_void_p), ("table", C.c_void_p),
                ("table_rows", C.c_int64), ("q_heads", C.c_int32), ("k_heads", C.c_int32),
                ("head_dim", C.c_int32), ("rot_dim", C.c_int32), ("eps", C.c_float),
                ("flags", C.c_uint32)]


class _CWeights(C.Structure):
    """fp4_weights of include/fp4q.h."""
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("alpha", C.c_void_p),
                ("experts", C.c_int64), ("rows", C.c_int64), ("cols", C.c_int64),
                ("format", C.c_int32), ("flags", C.c_uint32)]


class _CRouting(C.Structure):
    """fp4_routing of include/fp4q.h."""
    _fields_ = [("logits", C.c_void_p), ("stride", C.c_int64), ("tokens", C.c_int64),
                ("bias", C.c_void_p)] + [(n, C.c_int32) for n in (
                    "experts", "top_k", "groups", "top_groups", "group_top", "sigmoid",
                    "renormalize", "logits_bf16")] + [("scale", C.c_float)]


class _CResidual(C.Structure):
    """fp4_residual of include/fp4q.h."""
    _fields_ = [("x", C.c_void_p), ("block", C.c_void_p), ("x_stride", C.c_int64),
                ("block_stride", C.c_int64), ("tokens", C.c_int64), ("block_weight", C.c_void_p),
                ("weight", C.c_void_p), ("gate", C.c_void_p), ("token_gate", C.c_int32),
                ("dim", C.c_int32), ("scale", C.c_float), ("eps", C.c_float)]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4q.so")
_lib = None


class Fp4Error(RuntimeError):
    def __init__(self, fn, status):
        super().__init__("%s failed: %s (%d): %s" % (
            fn, STATUS.get(status, "?"), status, lib().fp4_status_str(status).decode()))
        self.status = status


def lib():
    """Load libfp4q.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libfp4q.so is not built: run __graft_entry__.build() "
                               "(python -m block_scaled_fp4_reduce_amd.build)")
        L = C.CDLL(LIB_PATH)
        vp, i64, u32, u64, sz = C.c_void_p, C.c_int64, C.c_uint32, C.c_uint64, C.c_size_t
        L.fp4_workspace_bytes.restype = sz
        L.fp4_workspace_bytes.argtypes = [i64, i64, u32]
        L.fp4_tensor_amax.restype = C.c_int
        L.fp4_tensor_amax.argtypes = [vp, i64, i64, u32, u64, vp, vp, sz, vp]
        L.nvfp4_quantize.restype = C.c_int
        L.nvfp4_quantize.argtypes = [vp, i64, i64, u32, u64, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.nvfp4_quantize_noalloc.restype = C.c_int
        L.nvfp4_quantize_noalloc.argtypes = [vp, i64, i64, u32, u64, vp, vp, vp, vp, vp, vp, vp, vp]
        L.nvfp4_quantize_rows.restype = C.c_int
        L.nvfp4_quantize_rows.argtypes = [vp, i64, i64, u32, u64, vp, vp, vp, vp, vp]
        L.nvfp4_requantize_t.restype = C.c_int
        L.nvfp4_requantize_t.argtypes = [vp, vp, vp, i64, i64, u32, u64, vp, vp, vp, vp, vp, vp, sz,
                                         vp]
        L.mxfp4_quantize.restype = C.c_int
        L.mxfp4_quantize.argtypes = [vp, i64, i64, u32, vp, vp, vp, vp, vp]
        L.mxfp4_gemm.restype = C.c_int
        L.mxfp4_gemm.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp]
        L.fp4_dequantize.restype = C.c_int
        L.fp4_dequantize.argtypes = [C.c_int, vp, vp, vp, i64, i64, u32, vp, vp]
        cache, queries, rope = C.POINTER(_CCache), C.POINTER(_CQueries), C.POINTER(_CRope)
        L.fp4_kv_write.restype = C.c_int
        L.fp4_kv_write.argtypes = [cache, vp, i64, vp, i64, vp, i64, vp]
        L.fp4_kv_read.restype = C.c_int
        L.fp4_kv_read.argtypes = [cache, vp, i64, vp, i64, vp, i64, vp]
        L.fp4_kv_attention_workspace_bytes.restype = sz
        L.fp4_kv_attention_workspace_bytes.argtypes = [cache, queries]
        L.fp4_kv_attention.restype = C.c_int
        L.fp4_kv_attention.argtypes = [cache, queries, vp, i64, vp, vp, sz, vp]
        L.qk_norm_rope.restype = C.c_int
        L.qk_norm_rope.argtypes = [rope, vp, i64, vp, i64, vp]
        L.qk_norm_rope_workspace_bytes.restype = sz
        L.qk_norm_rope_workspace_bytes.argtypes = [C.c_int]
        L.qk_norm_rope_backward.restype = C.c_int
        L.qk_norm_rope_backward.argtypes = [rope, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp,
                                            sz, vp]
        weights, routing, residual = (C.POINTER(t) for t in (_CWeights, _CRouting, _CResidual))
        L.fp4_linear_workspace_bytes.restype = sz
        L.fp4_linear_workspace_bytes.argtypes = [weights, i64]
        L.fp4_linear.restype = C.c_int
        L.fp4_linear.argtypes = [weights, vp, i64, i64, vp, i64, C.c_int, vp, sz, vp]
        L.expert_route.restype = C.c_int
        L.expert_route.argtypes = [routing, vp, vp, vp]
        L.expert_route_backward.restype = C.c_int
        L.expert_route_backward.argtypes = [routing, vp, vp, vp, i64, vp]
        L.fp4_experts_workspace_bytes.restype = sz
        L.fp4_experts_workspace_bytes.argtypes = [weights, weights, i64, i64]
        L.fp4_experts.restype = C.c_int
        L.fp4_experts.argtypes = [weights, weights, vp, i64, i64, vp, vp, i64, vp, i64, vp, sz, vp]
        L.residual_norm.restype = C.c_int
        L.residual_norm.argtypes = [residual, vp, i64, vp, i64, vp]
        L.residual_norm_workspace_bytes.restype = sz
        L.residual_norm_workspace_bytes.argtypes = [i64, C.c_int]
        L.residual_norm_backward.restype = C.c_int
        L.residual_norm_backward.argtypes = [residual] + [vp, i64] * 4 + [vp, vp, vp, vp, sz, vp]
        L.fp4_status_str.restype = C.c_char_p
        L.fp4_status_str.argtypes = [C.c_int]
        L.fp4_abi_version.restype = C.c_int
        L.fp4_abi_version.argtypes = []
        _lib = L
    return _lib


# ------------------------------------------------------------------ helpers
def _torch():
    import torch
    return torch


def _check(fn, rc):
    if rc != 0:
        raise Fp4Error(fn, rc)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _as_bits(x):
    torch = _torch()
    if x.dtype == torch.bfloat16:
        x = x.view(torch.int16)
    if x.dtype not in (torch.int16, torch.uint16):
        raise TypeError("expected a bfloat16 (or 16-bit bit-pattern) tensor, got %s" % x.dtype)
    if x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("expected a contiguous 2-D tensor on the GPU")
    return x


def fp4_workspace_bytes(rows, cols, flags=0):
    return int(lib().fp4_workspace_bytes(rows, cols, flags))


def _workspace(rows, cols, flags, device, ws=None):
    torch = _torch()
    need = fp4_workspace_bytes(rows, cols, flags)
    if ws is None:
        ws = torch.empty(max(need, 4), dtype=torch.uint8, device=device)
    return ws


# ------------------------------------------------------------------ tensor API
def fp4_tensor_amax(x, flags=0, seed=0, out=None, ws=None, stream=None):
    """Largest magnitude of x (after RHT16 when asked); a 1-element float tensor."""
    torch = _torch()
    xb = _as_bits(x)
    rows, cols = xb.shape
    out = torch.empty(1, dtype=torch.float32, device=x.device) if out is None else out
    ws = _workspace(rows, cols, flags, x.device, ws)
    _check("fp4_tensor_amax", lib().fp4_tensor_amax(
        xb.data_ptr(), rows, cols, flags, seed & (2**64 - 1), out.data_ptr(), ws.data_ptr(),
        ws.numel(), _stream(stream)))
    return out


def nvfp4_quantize(x, flags=0, seed=0, amax=None, want_choice=False, ws=None, stream=None,
                   out=None):
    """NVFP4 quantization.  Returns a dict with ``codes`` [rows][cols/2] uint8,
    ``scales`` (E4M3 bytes), ``alpha`` (1 float), optional ``choice`` and, for
    BLOCK2D|COLWISE, ``codes_t``/``scales_t``.  ``out`` may supply these
    buffers (same keys) to avoid allocation."""
    torch = _torch()
    xb = _as_bits(x)
    rows, cols = xb.shape
    dev = x.device
    two_d = bool(flags & BLOCK2D)
    want_t = two_d and bool(flags & COLWISE)
    srows = rows // 16 if two_d else rows
    o = dict(out or {})
    u8 = torch.uint8
    if "codes" not in o:
        o["codes"] = torch.empty((rows, cols // 2), dtype=u8, device=dev)
    if "scales" not in o:
        o["scales"] = torch.empty((srows, cols // 16), dtype=u8, device=dev)
    if "alpha" not in o:
        o["alpha"] = torch.empty(1, dtype=torch.float32, device=dev)
    if want_choice and "choice" not in o:
        o["choice"] = torch.empty((srows, cols // 16), dtype=u8, device=dev)
    if want_t:
        o.setdefault("codes_t", torch.empty((cols, rows // 2), dtype=u8, device=dev))
        o.setdefault("scales_t", torch.empty((cols // 16, rows // 16), dtype=u8, device=dev))
    if amax is None:
        ws = _workspace(rows, cols, flags, dev, ws)
    _check("nvfp4_quantize", lib().nvfp4_quantize(
        xb.data_ptr(), rows, cols, flags, seed & (2**64 - 1), _ptr(amax), o["alpha"].data_ptr(),
        o["codes"].data_ptr(), o["scales"].data_ptr(), _ptr(o.get("choice")),
        _ptr(o.get("codes_t")), _ptr(o.get("scales_t")), _ptr(ws),
        0 if ws is None else ws.numel(), _stream(stream)))
    return o


def nvfp4_quantize_noalloc(x, flags=0, seed=0, amax=None, out=None, stream=None):
    """nvfp4_quantize without a workspace: the library keeps the amax pass's
    partial maxima in its own fixed device array.  ``out`` must hold every
    output buffer (``codes``, ``scales``, ``alpha``, optional ``choice``,
    ``codes_t``/``scales_t`` for BLOCK2D|COLWISE): this call allocates
    nothing.  Calls overlapping on one device race (see include/fp4q.h)."""
    xb = _as_bits(x)
    rows, cols = xb.shape
    o = out
    _check("nvfp4_quantize_noalloc", lib().nvfp4_quantize_noalloc(
        xb.data_ptr(), rows, cols, flags, seed & (2**64 - 1), _ptr(amax), o["alpha"].data_ptr(),
        o["codes"].data_ptr(), o["scales"].data_ptr(), _ptr(o.get("choice")),
        _ptr(o.get("codes_t")), _ptr(o.get("scales_t")), _stream(stream)))
    return o


def nvfp4_quantize_rows(x, flags=0, seed=0, want_choice=False, stream=None, out=None):
    """NVFP4 with one FP32 scale per row, in one read of x.  Returns a dict
    with ``codes`` [rows][cols/2], ``scales`` [rows][cols/16], ``alpha``
    [rows] (float32) and, when asked, ``choice``."""
    torch = _torch()
    xb = _as_bits(x)
    rows, cols = xb.shape
    dev = x.device
    o = dict(out or {})
    u8 = torch.uint8
    o.setdefault("codes", torch.empty((rows, cols // 2), dtype=u8, device=dev))
    o.setdefault("scales", torch.empty((rows, cols // 16), dtype=u8, device=dev))
    o.setdefault("alpha", torch.empty(max(rows, 1), dtype=torch.float32, device=dev))
    if want_choice:
        o.setdefault("choice", torch.empty((rows, cols // 16), dtype=u8, device=dev))
    _check("nvfp4_quantize_rows", lib().nvfp4_quantize_rows(
        xb.data_ptr(), rows, cols, flags, seed & (2**64 - 1), o["alpha"].data_ptr(),
        o["codes"].data_ptr(), o["scales"].data_ptr(), _ptr(o.get("choice")), _stream(stream)))
    return o


def nvfp4_requantize_t(codes, scales, alpha, flags=0, seed=0, amax=None, want_choice=False,
                       ws=None, stream=None, out=None):
    """NVFP4 of dequantize(X)^T for a 1D NVFP4 tensor X given as ``codes``
    [rows][cols/2], ``scales`` [rows][cols/16] and ``alpha`` (1 float).
    Returns a dict with ``codes`` [cols][rows/2], ``scales`` [cols][rows/16],
    ``alpha`` and, when asked, ``choice``; ``out`` may supply these buffers.
    ``amax`` (1 float) skips the amax pass."""
    torch = _torch()
    for t in (codes, scales, alpha):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("expected contiguous GPU tensors")
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or alpha.dtype != torch.float32:
        raise TypeError("expected uint8 codes/scales and a float32 alpha")
    rows, cols = codes.shape[0], codes.shape[1] * 2
    if tuple(scales.shape) != (rows, cols // 16):
        raise ValueError("scales must be [rows][cols/16]")
    dev = codes.device
    o = dict(out or {})
    u8 = torch.uint8
    o.setdefault("codes", torch.empty((cols, rows // 2), dtype=u8, device=dev))
    o.setdefault("scales", torch.empty((cols, rows // 16), dtype=u8, device=dev))
    o.setdefault("alpha", torch.empty(1, dtype=torch.float32, device=dev))
    if want_choice:
        o.setdefault("choice", torch.empty((cols, rows // 16), dtype=u8, device=dev))
    if amax is None:
        ws = _workspace(rows, cols, flags, dev, ws)
    _check("nvfp4_requantize_t", lib().nvfp4_requantize_t(
        codes.data_ptr(), scales.data_ptr(), alpha.data_ptr(), rows, cols, flags,
        seed & (2**64 - 1), _ptr(amax), o["alpha"].data_ptr(), o["codes"].data_ptr(),
        o["scales"].data_ptr(), _ptr(o.get("choice")), _ptr(ws),
        0 if ws is None else ws.numel(), _stream(stream)))
    return o


def mxfp4_quantize(x, flags=HAD32 | ROWWISE | COLWISE, stream=None, out=None):
    """MXFP4 quantization; returns ``codes_r``/``scales_r`` and/or
    ``codes_c``/``scales_c`` (column-wise = row-wise of the transpose)."""
    torch = _torch()
    xb = _as_bits(x)
    rows, cols = xb.shape
    dev = x.device
    o = dict(out or {})
    u8 = torch.uint8
    if flags & ROWWISE:
        o.setdefault("codes_r", torch.empty((rows, cols // 2), dtype=u8, device=dev))
        o.setdefault("scales_r", torch.empty((rows, cols // 32), dtype=u8, device=dev))
    if flags & COLWISE:
        o.setdefault("codes_c", torch.empty((cols, rows // 2), dtype=u8, device=dev))
        o.setdefault("scales_c", torch.empty((cols, rows // 32), dtype=u8, device=dev))
    _check("mxfp4_quantize", lib().mxfp4_quantize(
        xb.data_ptr(), rows, cols, flags, _ptr(o.get("codes_r")), _ptr(o.get("scales_r")),
        _ptr(o.get("codes_c")), _ptr(o.get("scales_c")), _stream(stream)))
    return o


def mxfp4_gemm(a_codes, a_scales, bt_codes, bt_scales, out=None, stream=None):
    """C = A B (fp32 [M][N]) from row-wise MXFP4 A (codes [M][K/2], scales
    [M][K/32]) and B^T in the same layout (codes [N][K/2], scales [N][K/32])."""
    torch = _torch()
    M, N, K = a_codes.shape[0], bt_codes.shape[0], a_codes.shape[1] * 2
    if bt_codes.shape[1] * 2 != K:
        raise ValueError("A and B^T disagree on K")
    for t in (a_codes, a_scales, bt_codes, bt_scales):
        if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("expected contiguous uint8 GPU tensors")
    out = torch.empty((M, N), dtype=torch.float32, device=a_codes.device) if out is None else out
    _check("mxfp4_gemm", lib().mxfp4_gemm(
        a_codes.data_ptr(), a_scales.data_ptr(), bt_codes.data_ptr(), bt_scales.data_ptr(), M, N, K,
        out.data_ptr(), _stream(stream)))
    return out


def fp4_dequantize(fmt, codes, scales, alpha, rows, cols, flags=0, out=None, stream=None):
    """Decode to fp32 [rows][cols]."""
    torch = _torch()
    out = torch.empty((rows, cols), dtype=torch.float32, device=codes.device) if out is None else out
    _check("fp4_dequantize", lib().fp4_dequantize(
        fmt, codes.data_ptr(), scales.data_ptr(), _ptr(alpha), rows, cols, flags,
        out.data_ptr(), _stream(stream)))
    return out


# ------------------------------------------------------------------ FP4 key/value cache
_native = None


def _binding():
    """The compiled binding of these calls (built beside libfp4q.so)."""
    global _native
    if _native is None:
        lib()                                # a missing build is reported there
        _torch()                             # the binding links to torch's libraries
        _native = importlib.import_module(__name__ + "._calls")
    return _native


def _ints(x, dtype, shape, what):
    if x.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, x.dtype))
    if not x.is_cuda or not x.is_contiguous() or tuple(x.shape) != tuple(shape):
        raise ValueError("%s must be a contiguous GPU tensor %s, got %s" % (
            what, tuple(shape), tuple(x.shape)))
    return x.data_ptr()


class _Address(int):
    """The address of a handle's struct, with the device of its buffers and what
    among them may require a gradient."""

    def __new__(cls, struct, device_index, alpha=None):
        at = super().__new__(cls, C.addressof(struct))
        at.device_index = device_index
        at.alpha = alpha
        return at


class KvCache:
    """A paged FP4 cache of keys and values: the buffers of ``fp4_kv_cache``
    (include/fp4q.h) and what their bytes mean.  ``alloc`` makes the buffers;
    the constructor takes a program's own.  The fields are fixed, since the
    calls use the addresses taken here: other buffers or maxima need another
    handle, or are copied into these tensors."""

    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "k_amax", "v_amax", "fmt", "flags",
                 "pages", "heads", "page_size", "head_dim", "_c", "_at")

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_amax=None, v_amax=None,
                 fmt=FORMAT_NVFP4, flags=0):
        torch = _torch()
        pages, heads, page_size, half = k_codes.shape
        dim, group = half * 2, 16 if fmt == FORMAT_NVFP4 else 32
        for t, shape, what in ((k_codes, (page_size, half), "k_codes"),
                               (k_scales, (page_size, dim // group), "k_scales"),
                               (v_codes, (half, page_size), "v_codes"),
                               (v_scales, (dim // group, page_size), "v_scales")):
            _ints(t, torch.uint8, (pages, heads) + shape, what)
        if fmt == FORMAT_NVFP4:
            for t, what in ((k_amax, "k_amax"), (v_amax, "v_amax")):
                if t is None:
                    raise ValueError("NVFP4 needs %s [heads]" % what)
                _ints(t, torch.float32, (heads,), what)
        for t in (k_scales, v_codes, v_scales, k_amax, v_amax):
            if t is not None and t.device != k_codes.device:
                raise ValueError("the cache's tensors are on different devices: %s and %s" % (
                    k_codes.device, t.device))
        c = _CCache(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                    v_scales.data_ptr(), _ptr(k_amax), _ptr(v_amax), pages, page_size, heads, dim,
                    fmt, flags)
        for name, value in zip(self.__slots__, (k_codes, k_scales, v_codes, v_scales, k_amax, v_amax,
                                                fmt, flags, pages, heads, page_size, dim, c,
                                                _Address(c, k_codes.device.index))):
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        raise AttributeError("the fields of a cache handle are fixed: %s" % name)

    def __delattr__(self, name):
        self.__setattr__(name, None)

    def __copy__(self):
        return self

    @classmethod
    def alloc(cls, pages, page_size, heads, head_dim, fmt=FORMAT_NVFP4, flags=0, k_amax=None,
              v_amax=None, device="cuda"):
        """A cache of `pages` pages.  NVFP4 takes the heads' largest magnitudes
        from calibration (``k_amax``, ``v_amax`` [heads] float32)."""
        torch = _torch()
        group = 16 if fmt == FORMAT_NVFP4 else 32
        new = lambda *shape: torch.empty((pages, heads) + shape, dtype=torch.uint8, device=device)
        return cls(new(page_size, head_dim // 2), new(page_size, head_dim // group),
                   new(head_dim // 2, page_size), new(head_dim // group, page_size), k_amax, v_amax,
                   fmt, flags)


def fp4_kv_write(cache, k, v, slots, stream=None):
    """Quantize keys and values [tokens][heads][head_dim] (bf16) into ``cache``
    at ``slots`` [tokens] (int64; slot s is token s % page_size of page
    s / page_size).  Slots outside the cache are skipped.  What is stored are
    bytes, through which no gradient goes."""
    _binding().kv_write(cache._at, k, v, slots, stream)


def fp4_kv_read(cache, slots, out=None, stream=None):
    """The keys and values at ``slots`` [tokens] as bf16 (k, v), each
    [tokens][heads][head_dim]; ``out`` may supply them."""
    return _binding().kv_read(cache._at, slots, out, stream)


def fp4_kv_attention_workspace_bytes(cache, q, page_table, kv_lens, cu_q=None, max_q=0, scale=None,
                                     softcap=0.0, window=0):
    """Bytes of workspace of ``fp4_kv_attention`` on these arguments."""
    return _binding().kv_attention_ws(cache._at, q, page_table, kv_lens, cu_q, max_q, scale,
                                      softcap, window)


def fp4_kv_attention(cache, q, page_table, kv_lens, cu_q=None, max_q=0, scale=None, softcap=0.0,
                     window=0, want_lse=False, out=None, lse=None, ws=None, stream=None):
    """Causal attention of new tokens over the paged cache.

    q [tokens][q_heads][head_dim] bf16 holds the new tokens of all sequences
    one after another: sequence b's are cu_q[b] .. cu_q[b + 1] - 1 (int32;
    None: one token each; tokens outside get zeros), the last of its kv_lens[b] cached ones (int32, the
    new ones written before).  page_table [seqs][width] (int32) names each
    sequence's pages.  max_q is the largest number of new tokens where the
    program knows it (0: not known).  Scores beyond `softcap` c > 0 level off,
    c tanh(s / c).  Returns out (bf16, like q), or (out, lse) with lse
    [tokens][q_heads] float32.  There is no backward: queries that require a
    gradient are refused in grad mode."""
    return _binding().kv_attention(cache._at, q, page_table, kv_lens, cu_q, max_q, scale, softcap,
                                   window, want_lse, out, lse, ws, stream)


# ------------------------------------------------------------------ norm + rotation
def rope_table(positions, rot_dim, base=10000.0, device="cuda"):
    """Cosines and sines [positions][rot_dim/2][2] (float32) of the angles
    p * base^(-2i/rot_dim), computed in 64 bits."""
    torch = _torch()
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * \
        base ** (-i / rot_dim)
    return torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()


def qk_norm_rope(q, k, q_weight, k_weight, positions, table, eps=1e-6, interleaved=False, out=None,
                 stream=None):
    """RMS norm of each head of q and k ([tokens][heads][head_dim] bf16) with
    its weight ([head_dim] bf16; None: no norm), then the rotation of the
    first 2 * table.shape[1] values by the angles of ``positions`` [tokens]
    (int64) in ``table`` (``rope_table``).  Returns (q, k); ``out`` may supply
    them and may be (q, k) themselves.  Where q, k or a weight requires a
    gradient (and grad mode is on) the results carry it through torch's
    autograd, by ``qk_norm_rope_backward``; ``out`` is refused then.  A capture
    of such a backward needs what torch asks of any: no graph of the same
    leaves from outside the capture is alive."""
    return _binding().norm_rope(q, k, q_weight, k_weight, positions, table, eps, interleaved, out,
                                stream)


_norm_rope_function = None


def _rows(g):
    """g [tokens][heads][head_dim] laid out as the calls take it."""
    tokens, heads, dim = g.shape
    fits = (g.stride()[1:] == (dim, 1) and g.stride(0) >= heads * dim and g.stride(0) % 8 == 0 and
            g.data_ptr() % 16 == 0)
    return g if fits else g.clone(memory_format=_torch().contiguous_format)


def _norm_rope_autograd(*args):
    """qk_norm_rope(q, k, q_weight, k_weight, positions, table, eps, interleaved,
    stream) as a node of torch's autograd graph."""
    global _norm_rope_function
    if _norm_rope_function is None:
        torch = _torch()

        class NormRope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, q_weight, k_weight, positions, table, eps, interleaved, stream):
                ctx.save_for_backward(q, k, q_weight, k_weight, positions, table)
                ctx.how = eps, interleaved
                return qk_norm_rope(q, k, q_weight, k_weight, positions, table, eps, interleaved,
                                    stream=stream)

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dq_out, dk_out):
                x = ctx.saved_tensors
                grads = qk_norm_rope_backward(_rows(dq_out), _rows(dk_out), *x, *ctx.how)
                return tuple(None if g is None or not need else g.to(torch.bfloat16)
                             for g, need in zip(grads, ctx.needs_input_grad)) + (None,) * 5

        _norm_rope_function = NormRope
    return _norm_rope_function.apply(*args)


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, positions, table, eps=1e-6,
                          interleaved=False, out=None, ws=None, stream=None):
    """Gradients of ``qk_norm_rope`` on the same arguments: (dq, dk, dq_weight,
    dk_weight), dq and dk bf16 (``out`` may supply them), the weights' float32
    [head_dim] (None without a weight)."""
    return _binding().norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, positions, table,
                                         eps, interleaved, out, ws, stream)


# ------------------------------------------------------------------ FP4 weights
class Fp4Weights:
    """FP4 weights of a matrix, or of one for every expert: the buffers of
    ``fp4_weights`` (include/fp4q.h), as ``nvfp4_quantize``,
    ``nvfp4_quantize_rows`` or ``mxfp4_quantize`` (without HAD32) make them.

    codes [rows][cols/2] or [experts][rows][cols/2]; scales [..][rows][cols/G]
    or, NVFP4 of 16x16 tiles, [..][rows/16][cols/16]; NVFP4's alpha is one
    float32 a matrix ([1] or [experts]) or one a row ([..][rows]).  The fields
    are fixed, since the calls use the addresses taken here."""

    __slots__ = ("codes", "scales", "alpha", "fmt", "flags", "experts", "rows", "cols", "_c", "_at")

    def __init__(self, codes, scales, alpha=None, fmt=FORMAT_NVFP4):
        torch = _torch()
        if codes.dim() not in (2, 3):
            raise ValueError("codes must be [rows][cols/2] or [experts][rows][cols/2], got %s" % (
                tuple(codes.shape),))
        lead, (rows, half) = tuple(codes.shape[:-2]), codes.shape[-2:]
        cols, group = half * 2, 16 if fmt == FORMAT_NVFP4 else 32
        _ints(codes, torch.uint8, lead + (rows, half), "codes")
        flags = 0
        if fmt == FORMAT_NVFP4:
            by_tile = lead + (rows // 16, cols // 16)
            if tuple(scales.shape) == by_tile != lead + (rows, cols // 16) and rows % 16 == 0:
                flags |= BLOCK2D
        _ints(scales, torch.uint8, by_tile if flags else lead + (rows, cols // group), "scales")
        if fmt == FORMAT_NVFP4:
            if alpha is None:
                raise ValueError("NVFP4 needs alpha")
            by_row = lead + (rows,)
            one = lead or (1,)
            if tuple(alpha.shape) == by_row != one:
                flags |= ROW_ALPHA
            _ints(alpha, torch.float32, by_row if flags & ROW_ALPHA else one, "alpha")
        elif alpha is not None:
            raise ValueError("MXFP4 has no alpha")
        for t in (scales, alpha):
            if t is not None and t.device != codes.device:
                raise ValueError("the weights' tensors are on different devices: %s and %s" % (
                    codes.device, t.device))
        experts = lead[0] if lead else 1
        c = _CWeights(codes.data_ptr(), scales.data_ptr(), _ptr(alpha), experts, rows, cols, fmt,
                      flags)
        for name, value in zip(self.__slots__, (codes, scales, alpha, fmt, flags, experts, rows, cols,
                                                c, _Address(c, codes.device.index, alpha))):
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        raise AttributeError("the fields of a weights handle are fixed: %s" % name)

    def __delattr__(self, name):
        self.__setattr__(name, None)

    def __copy__(self):
        return self


def fp4_linear(w, x, dtype=None, out=None, ws=None, stream=None):
    """x [tokens][cols] (bf16) times the transpose of FP4 weights ``w``
    [rows][cols]: [tokens][rows] in bf16, or float32 with ``dtype``.  The
    products are exact and summed in fp32.  There is no backward: an x or an
    alpha that requires a gradient is refused in grad mode."""
    torch = _torch()
    if dtype not in (None, torch.bfloat16, torch.float32):
        raise TypeError("dtype must be bfloat16 or float32, got %s" % (dtype,))
    return _binding().linear(w._at, x, dtype is torch.float32, out, ws, stream)


# ------------------------------------------------------------------ experts
def expert_route(logits, top_k, scores="softmax", bias=None, groups=1, top_groups=1, group_top=1,
                 renormalize=True, scale=1.0, out=None, stream=None):
    """The ``top_k`` experts of each token from ``logits`` [tokens][experts]
    (float32 or bf16): (weights [tokens][top_k] float32, experts int32).

    With s the softmax or sigmoid of the logits, candidates are in the order of
    the logits or, with ``bias`` [experts] (float32), of s + bias; of several
    ``groups`` only the ``top_groups`` largest stay, by their largest candidate
    or the sum of their two largest scores (``group_top`` 2).  Weights are
    ``scale`` s, over the sum of the chosen s with ``renormalize``.  An expert
    whose logit is -inf is never chosen; places left get expert -1 and weight
    0.  Where logits require a gradient the weights carry it through torch's
    autograd, by ``expert_route_backward``; ``out`` is refused then."""
    return _binding().route(logits, top_k, scores, bias, groups, top_groups, group_top, renormalize,
                            scale, out, stream)


_expert_route_function = None


def _expert_route_autograd(*args):
    """expert_route(logits, top_k, scores, bias, groups, top_groups, group_top,
    renormalize, scale, stream) as a node of torch's autograd graph."""
    global _expert_route_function
    if _expert_route_function is None:
        torch = _torch()

        class ExpertRoute(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, top_k, scores, bias, groups, top_groups, group_top, renormalize,
                        scale, stream):
                w, e = expert_route(logits, top_k, scores, bias, groups, top_groups, group_top,
                                    renormalize, scale, stream=stream)
                ctx.save_for_backward(logits, e)
                ctx.how = scores, renormalize, scale
                ctx.mark_non_differentiable(e)
                return w, e

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dweights, _):
                logits, e = ctx.saved_tensors
                return (expert_route_backward(dweights.contiguous(), logits, e, *ctx.how),) + \
                    (None,) * 9

        _expert_route_function = ExpertRoute
    return _expert_route_function.apply(*args)


def expert_route_backward(dweights, logits, experts, scores="softmax", renormalize=True, scale=1.0,
                          out=None, stream=None):
    """The gradient of the logits (in their type) from that of
    ``expert_route``'s weights and the experts that it chose."""
    return _binding().route_backward(dweights, logits, experts, scores, renormalize, scale, out,
                                     stream)


def fp4_experts_workspace_bytes(gate_up, down, tokens, top_k):
    """Bytes of workspace of ``fp4_experts`` for these weights and sizes."""
    return _binding().experts_ws(gate_up._at, down._at, tokens, top_k)


def fp4_experts(gate_up, down, x, weights, experts, out=None, ws=None, stream=None):
    """The routed experts of each token, out[t] = sum_j weights[t][j]
    D_e (silu(G_e x[t]) * (U_e x[t])) with e = experts[t][j].

    ``gate_up`` holds the experts' G and U [experts][2F][cols] (the first F
    rows are G's), ``down`` their D [experts][cols][F]; x [tokens][cols] bf16,
    weights [tokens][top_k] float32, experts [tokens][top_k] int32 (numbers
    outside the experts are skipped), as ``expert_route`` returns them.  There
    is no backward: tensors that require a gradient are refused in grad mode."""
    return _binding().experts(gate_up._at, down._at, x, weights, experts, out, ws, stream)


# ------------------------------------------------------------------ norms around a block
def residual_norm(x, block, weight, block_weight=None, gate=None, scale=1.0, eps=1e-6, out=None,
                  stream=None):
    """The end of one block and the start of the next: y = ``scale`` x + gate *
    norm(block) and z = norm(y), as (y, z), all [tokens][dim] bf16.

    norm(block) is block's RMS norm times ``block_weight`` [dim], or block
    itself without it; norm(y) is y's times ``weight`` [dim].  ``gate`` is one
    number for every channel ([dim]) or for every token ([tokens][1]), or None;
    all bf16.  ``out`` may supply (y, z) and may be (x, block) themselves.
    Where an input requires a gradient (and grad mode is on) the results carry
    it through torch's autograd, by ``residual_norm_backward``; ``out`` is
    refused then."""
    return _binding().residual(x, block, weight, block_weight, gate, scale, eps, out, stream)


_residual_norm_function = None


def _flat_rows(g):
    """g [tokens][dim] laid out as the calls take it."""
    fits = (g.stride(1) == 1 and g.stride(0) >= g.shape[1] and g.stride(0) % 8 == 0 and
            g.data_ptr() % 16 == 0)
    return g if fits else g.clone(memory_format=_torch().contiguous_format)


def _residual_norm_autograd(*args):
    """residual_norm(x, block, weight, block_weight, gate, scale, eps, stream) as
    a node of torch's autograd graph."""
    global _residual_norm_function
    if _residual_norm_function is None:
        torch = _torch()

        class ResidualNorm(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, block, weight, block_weight, gate, scale, eps, stream):
                ctx.save_for_backward(x, block, weight, block_weight, gate)
                ctx.how = scale, eps
                return residual_norm(x, block, weight, block_weight, gate, scale, eps, stream=stream)

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dy, dz):
                dx, db, dbw, dw, dg = residual_norm_backward(
                    _flat_rows(dy), _flat_rows(dz), *ctx.saved_tensors, *ctx.how)
                return tuple(None if g is None or not need else g.to(torch.bfloat16)
                             for g, need in zip((dx, db, dw, dbw, dg), ctx.needs_input_grad)) + \
                    (None,) * 3

        _residual_norm_function = ResidualNorm
    return _residual_norm_function.apply(*args)


def residual_norm_backward(dy, dz, x, block, weight, block_weight=None, gate=None, scale=1.0,
                           eps=1e-6, out=None, ws=None, stream=None):
    """Gradients of ``residual_norm`` on the same arguments: (dx, dblock,
    dblock_weight, dweight, dgate), dx and dblock bf16 (``out`` may supply
    them), the others float32 (None without that input)."""
    return _binding().residual_backward(dy, dz, x, block, weight, block_weight, gate, scale, eps, out,
                                        ws, stream)
