"""B200-native compressed KV cache: TurboQuant-style 3-bit + QJL keys/values
and attention computed directly over the packed cache.

This package is a thin ctypes binding over ``libtq.so`` (C ABI declared in
``include/tq.h``). Every function here only marshals arguments — tensor
pointers, sizes, the current CUDA stream — and calls the library of the same
name (the calls of a serving step through ``_tq_torch``, a C++ extension, the
others through ctypes); all arithmetic runs in the library's CUDA kernels (or, for
``tq_make_codebook``, its host C++ code). There is no Python or CPU fallback:
if the library is missing, importing the binding raises.

PyTorch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtq.so")

TQ_OK, TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED, TQ_ERR_CUDA, TQ_ERR_WORKSPACE = range(5)
TQ_F32, TQ_BF16 = 0, 1
TQ_DEV_BAD_CODEBOOK, TQ_DEV_BAD_POSITION, TQ_DEV_TIMEOUT = 0x1, 0x2, 0x4
TQ_DEV_BAD_BLOCK, TQ_DEV_BAD_LENGTH, TQ_DEV_NONFINITE = 0x8, 0x10, 0x20
TQ_E4M3, TQ_INT8 = 0, 1

_STATUS = {1: "TQ_ERR_INVALID_ARG", 2: "TQ_ERR_UNSUPPORTED", 3: "TQ_ERR_CUDA", 4: "TQ_ERR_WORKSPACE"}


class TQError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


class Layout(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("key_bits", ctypes.c_int32), ("value_bits", ctypes.c_int32)]


class _Planes(ctypes.Structure):
    _fields_ = [("idx", ctypes.c_void_p), ("sign", ctypes.c_void_p), ("norm", ctypes.c_void_p),
                ("rnorm", ctypes.c_void_p)]


class _Cache8(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("heads", ctypes.c_int32), ("block", ctypes.c_int32), ("code", ctypes.c_int32),
                ("n_blocks", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I32, _I64, _F32, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t

_SIGNATURES = {
    "tq_idx_row_bytes": (_I64, [_I32, _I32]),
    "tq_sign_words": (_I64, [_I32]),
    "tq_packed_bytes": (_I64, [ctypes.POINTER(Layout), _I64, _I32]),
    "tq_make_codebook": (ctypes.c_int, [_I32, _I32, _I32, _P, _I64, _P, _P, _P]),
    "tq_quantize_kv": (ctypes.c_int, [ctypes.POINTER(Layout), _I32, _P, ctypes.c_int, _I64, _I64, _P, _F32,
                                      _P, _I64, _I64, _P, _P, _P, ctypes.POINTER(_Planes), _P, _P]),
    "tq_decode_attention": (ctypes.c_int, [ctypes.POINTER(Layout), _P, ctypes.c_int, _I32, _I32, _I32, _I32, _I64,
                                           _I64, _P, _F32, ctypes.POINTER(_Planes), ctypes.POINTER(_Planes),
                                           _P, _P, _I64, _P, _P, _P, _F32, _P, ctypes.c_int, _P, _P, _SZ, _P, _P]),
    "tq_append_kv": (ctypes.c_int, [ctypes.POINTER(Layout), _I32, _P, ctypes.c_int, _I64, _I64, _P, _F32, _P, _P, _P, _P,
                                    ctypes.POINTER(_Planes), _I64, _I64, _P, _P]),
    "tq_decode_workspace_bytes": (_SZ, [ctypes.POINTER(Layout), _I32, _I32, _I32, _I32, _I64]),
    "tq_decode_attention_noalloc": (ctypes.c_int, [ctypes.POINTER(Layout), _P, ctypes.c_int, _I32, _I32, _I32, _I32,
                                                   _I64, _I64, _P, _F32, ctypes.POINTER(_Planes),
                                                   ctypes.POINTER(_Planes), _P, _P, _I64, _P, _P, _P, _F32, _P,
                                                   ctypes.c_int, _P, _P, _P]),
    "tq_dequantize": (ctypes.c_int, [ctypes.POINTER(Layout), _I32, _I64, ctypes.POINTER(_Planes), _P, _I64, _I64,
                                     _P, _P, _P, ctypes.c_int, _I64, _P]),
    "tq_dequantize_sign_mean": (ctypes.c_int, [ctypes.POINTER(Layout), _I32, _I64, ctypes.POINTER(_Planes), _P, _I64,
                                               _I64, _P, _F32, _P, ctypes.c_int, _I64, _P]),
    "tq_residual_mean": (ctypes.c_int, [_P, _I64, _P, _P, _I32, ctypes.POINTER(ctypes.c_double)]),
    "tq_search_topk": (ctypes.c_int, [ctypes.POINTER(Layout), _P, ctypes.c_int, _I32, ctypes.POINTER(_Planes), _I64,
                                      _P, _P, _P, _I32, _P, _P, _P, _SZ, _P]),
    "tq_search_merge_topk": (ctypes.c_int, [_I32, _I32, _P, _P, _I64, _P, _P, _I64, _P, _P, _P]),
    "tq_search_workspace_bytes": (_SZ, [ctypes.POINTER(Layout), _I32, _I64, _I32]),
    "tq_qk_norm_rope": (ctypes.c_int, [_I32, _I32, _I64, _I32, _I32, ctypes.c_int, _P, _I64, _I64, _P, _I64, _I64, _P,
                                       _I64, _I64, _P, _I64, _I64, _P, _P, _F32, _P, _F32, _P, _P]),
    "tq_cache8_bytes": (_I64, [_I32, _I32, _I32, _I64]),
    "tq_cache8_write": (ctypes.c_int, [ctypes.POINTER(_Cache8), ctypes.c_int, _P, _I64, _I64, _P, _I64, _I64, _I64, _I32,
                                       _P, _P, _P, _I64, _P, _P]),
    "tq_cache8_read": (ctypes.c_int, [ctypes.POINTER(_Cache8), ctypes.c_int, _P, _I64, _I64, _P, _I64, _I64, _I64, _I32,
                                      _P, _P, _P, _I64, _P, _P]),
    "tq_cache8_attention": (ctypes.c_int, [ctypes.POINTER(_Cache8), _P, ctypes.c_int, _I64, _I64, _I64, _I32, _I32, _I32,
                                           _P, _P, _I64, _I32, _I32, _F32, _P, ctypes.c_int, _I64, _I64, _I64, _P, _P,
                                           _SZ, _P, _P]),
    "tq_cache8_attention_workspace_bytes": (_SZ, [ctypes.POINTER(_Cache8), _I32, _I32, _I32]),
    "tq_fit_rotation": (ctypes.c_int, [_I32, _P, _I64, _P, _P]),
    "tq_rotate_normalize": (ctypes.c_int, [_I32, _P, _I64, _P, _P, ctypes.POINTER(_I64)]),
    "tq_last_error_string": (ctypes.c_char_p, []),
    "tq_version": (ctypes.c_char_p, []),
    "tq_kernel_launches": (ctypes.c_uint64, []),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libtq.so is not built ({LIB_PATH}); run `python kv_cache_vector_rope_b200/build.py` "
                          "(the CUDA library is the only implementation; there is no fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


class _NoBinding:
    """Stands where _tq_torch.so is missing or made for another torch: the calls that go through it say so, the others run."""

    def __init__(self, cause: ImportError):
        self._cause = cause

    def __getattr__(self, name):
        raise ImportError(f"{name} needs _tq_torch.so, which is not built or does not load; run "
                          "`python kv_cache_vector_rope_b200/build.py`") from self._cause


try:
    from . import _tq_torch as _bind            # checks and marshalling of the short calls (binding/tq_torch.cpp)
except ImportError as e:
    _bind = _NoBinding(e)


def exported_symbols() -> list[str]:
    return list(_SIGNATURES)


def _check(status: int) -> None:
    if status != TQ_OK:
        raise TQError(status, _lib.tq_last_error_string().decode())


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr()
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return int(t)


def _dev(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TQ_F32
    if t.dtype == torch.bfloat16:
        return TQ_BF16
    raise ValueError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _stream(stream) -> int | None:
    if stream is None:                          # the raw handle: a Stream object costs 3 us a call
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def layout(d: int, key_bits: int = 3, value_bits: int = 3) -> Layout:
    return Layout(d, key_bits, value_bits)


@dataclasses.dataclass
class Planes:
    """Packed planes of n vectors (torch tensors on one device)."""
    idx: torch.Tensor            # uint8 [n, d*bits/8]
    norm: torch.Tensor           # float32 [n]
    sign: torch.Tensor | None = None    # int32 [n, ceil(d/32)] (uint32 bit patterns)
    rnorm: torch.Tensor | None = None   # float32 [n]

    def c(self) -> _Planes:
        return _Planes(_ptr(self.idx), _ptr(self.sign), _ptr(self.norm), _ptr(self.rnorm))

    def rows(self, start: int, stop: int) -> "Planes":
        return Planes(self.idx[start:stop], self.norm[start:stop],
                      None if self.sign is None else self.sign[start:stop],
                      None if self.rnorm is None else self.rnorm[start:stop])

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.idx, self.norm, self.sign, self.rnorm)
                   if t is not None)


def tq_idx_row_bytes(d: int, bits: int) -> int:
    return int(_lib.tq_idx_row_bytes(d, bits))


def tq_sign_words(d: int) -> int:
    return int(_lib.tq_sign_words(d))


def tq_packed_bytes(lay: Layout, n_vectors: int, is_key: bool) -> int:
    return int(_lib.tq_packed_bytes(ctypes.byref(lay), n_vectors, int(is_key)))


def alloc_planes(n: int, d: int, bits: int, is_key: bool, device="cuda") -> Planes:
    """Allocates the planes of n vectors (allocation is PyTorch's)."""
    return Planes(idx=torch.empty((n, tq_idx_row_bytes(d, bits)), dtype=torch.uint8, device=device),
                  norm=torch.empty((n,), dtype=torch.float32, device=device),
                  sign=torch.empty((n, tq_sign_words(d)), dtype=torch.int32, device=device) if is_key else None,
                  rnorm=torch.empty((n,), dtype=torch.float32, device=device) if is_key else None)


def tq_make_codebook(d: int, bits: int, mode: int = 0, samples=None):
    """Lloyd-Max codebook (host). Returns (centroids, boundaries, mse) as float32 arrays and a float."""
    n = 1 << bits
    c = np.zeros(n, dtype=np.float32)
    t = np.zeros(max(n - 1, 1), dtype=np.float32)
    mse = ctypes.c_double(0.0)
    smp = None
    ns = 0
    if samples is not None:
        smp = np.ascontiguousarray(np.asarray(samples, dtype=np.float32).ravel())
        ns = smp.size
    _check(_lib.tq_make_codebook(d, bits, mode, _ptr(smp), ns, c.ctypes.data, t.ctypes.data, ctypes.byref(mse)))
    return c, t[:n - 1], float(mse.value)


def tq_quantize_kv(lay: Layout, is_key: bool, x: torch.Tensor, out: Planes, Pi: torch.Tensor,
                   centroids: torch.Tensor, boundaries: torch.Tensor, S: torch.Tensor | None = None,
                   positions: torch.Tensor | None = None, rope_base: float = 0.0,
                   vectors_per_pi: int = 1, pi_stride: int = 0, d_status: torch.Tensor | None = None,
                   stream=None) -> None:
    """Quantises the rows of x ([n, d], unit stride along d) into `out`."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be [n, d] with unit stride along d")
    _check(_lib.tq_quantize_kv(ctypes.byref(lay), int(is_key), _dev(x, "x"), _dtype_code(x), x.shape[0],
                               x.stride(0), _ptr(positions), float(rope_base), _dev(Pi, "Pi"), vectors_per_pi,
                               pi_stride, _ptr(S), _dev(centroids, "centroids"), _dev(boundaries, "boundaries"),
                               ctypes.byref(out.c()), _ptr(d_status), _stream(stream)))


def tq_append_kv(lay: Layout, is_key: bool, x: torch.Tensor, cache: Planes, ctx_stride: int, slot: int,
                 Pi: torch.Tensor, centroids: torch.Tensor, boundaries: torch.Tensor, S: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, rope_base: float = 0.0, d_status: torch.Tensor | None = None,
                 stream=None) -> None:
    """Quantises row s of x ([n_streams, d]) into cache row s * ctx_stride + slot."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be [n_streams, d] with unit stride along d")
    _check(_lib.tq_append_kv(ctypes.byref(lay), int(is_key), _dev(x, "x"), _dtype_code(x), x.shape[0], x.stride(0),
                             _ptr(positions), float(rope_base), _dev(Pi, "Pi"), _ptr(S), _dev(centroids, "centroids"),
                             _dev(boundaries, "boundaries"), ctypes.byref(cache.c()), ctx_stride, slot,
                             _ptr(d_status), _stream(stream)))


def tq_decode_workspace_bytes(lay: Layout, batch: int, hq: int, hkv: int, nq: int, n_ctx: int) -> int:
    return int(_lib.tq_decode_workspace_bytes(ctypes.byref(lay), batch, hq, hkv, nq, n_ctx))


def decode_workspace(lay: Layout, batch: int, hq: int, hkv: int, nq: int, n_ctx: int, device="cuda") -> torch.Tensor:
    n = tq_decode_workspace_bytes(lay, batch, hq, hkv, nq, n_ctx)
    return torch.empty((max(n, 256) + 255) // 256 * 256, dtype=torch.uint8, device=device)


def tq_decode_attention(lay: Layout, q: torch.Tensor, k: Planes, v: Planes, hkv: int, n_ctx: int,
                        PiK: torch.Tensor, PiV: torch.Tensor, S: torch.Tensor, cK: torch.Tensor, cV: torch.Tensor,
                        out: torch.Tensor, workspace: torch.Tensor, scale: float | None = None,
                        q_positions: torch.Tensor | None = None, rope_base: float = 0.0, pi_stride: int = 0,
                        ctx_stride: int = 0, scores_out: torch.Tensor | None = None,
                        d_status: torch.Tensor | None = None, stream=None) -> None:
    """Attention of q ([batch, hq, nq, d], contiguous) over packed K/V planes of [batch, hkv, ctx] rows."""
    if q.dim() != 4 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [batch, hq, nq, d] tensor")
    if not out.is_contiguous():
        raise ValueError("out must be contiguous [batch, hq, nq, d]")
    batch, hq, nq, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check(_lib.tq_decode_attention(
        ctypes.byref(lay), _dev(q, "q"), _dtype_code(q), batch, hq, hkv, nq, n_ctx, ctx_stride,
        _ptr(q_positions), float(rope_base), ctypes.byref(k.c()), ctypes.byref(v.c()),
        _dev(PiK, "PiK"), _dev(PiV, "PiV"), pi_stride, _dev(S, "S"), _dev(cK, "cK"), _dev(cV, "cV"),
        float(scale), _dev(out, "out"), _dtype_code(out), _ptr(scores_out), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _ptr(d_status), _stream(stream)))


def tq_decode_attention_noalloc(lay: Layout, q: torch.Tensor, k: Planes, v: Planes, hkv: int, n_ctx: int,
                                PiK: torch.Tensor, PiV: torch.Tensor, S: torch.Tensor, cK: torch.Tensor,
                                cV: torch.Tensor, out: torch.Tensor, scale: float | None = None,
                                q_positions: torch.Tensor | None = None, rope_base: float = 0.0, pi_stride: int = 0,
                                ctx_stride: int = 0, scores_out: torch.Tensor | None = None,
                                d_status: torch.Tensor | None = None, stream=None) -> None:
    """tq_decode_attention with the library's fixed device scratch instead of a workspace.

    For callers that cannot allocate device memory at call time. Calls that
    overlap on the GPU share the scratch and must be serialised by the caller."""
    if q.dim() != 4 or not q.is_contiguous() or not out.is_contiguous():
        raise ValueError("q and out must be contiguous [batch, hq, nq, d] tensors")
    batch, hq, nq, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check(_lib.tq_decode_attention_noalloc(
        ctypes.byref(lay), _dev(q, "q"), _dtype_code(q), batch, hq, hkv, nq, n_ctx, ctx_stride,
        _ptr(q_positions), float(rope_base), ctypes.byref(k.c()), ctypes.byref(v.c()),
        _dev(PiK, "PiK"), _dev(PiV, "PiV"), pi_stride, _dev(S, "S"), _dev(cK, "cK"), _dev(cV, "cV"),
        float(scale), _dev(out, "out"), _dtype_code(out), _ptr(scores_out), _ptr(d_status), _stream(stream)))


def tq_dequantize(lay: Layout, is_key: bool, planes: Planes, n_vectors: int, Pi: torch.Tensor,
                  centroids: torch.Tensor, out: torch.Tensor, S: torch.Tensor | None = None,
                  vectors_per_pi: int = 1, pi_stride: int = 0, stream=None) -> None:
    if out.dim() != 2 or out.stride(1) != 1:
        raise ValueError("out must be [n, d] with unit stride along d")
    _check(_lib.tq_dequantize(ctypes.byref(lay), int(is_key), n_vectors, ctypes.byref(planes.c()),
                              _dev(Pi, "Pi"), vectors_per_pi, pi_stride, _ptr(S), _dev(centroids, "centroids"),
                              _dev(out, "out"), _dtype_code(out), out.stride(0), _stream(stream)))


def tq_dequantize_sign_mean(lay: Layout, is_key: bool, planes: Planes, n_vectors: int, Pi: torch.Tensor,
                            centroids: torch.Tensor, e_bar: float, out: torch.Tensor, vectors_per_pi: int = 1,
                            pi_stride: int = 0, stream=None) -> None:
    """x_tilde = Pi^T ||x|| (c[code] + e_bar (2 sign - 1)) for rows 0..n_vectors-1."""
    if out.dim() != 2 or out.stride(1) != 1:
        raise ValueError("out must be [n, d] with unit stride along d")
    _check(_lib.tq_dequantize_sign_mean(ctypes.byref(lay), int(is_key), n_vectors, ctypes.byref(planes.c()),
                                        _dev(Pi, "Pi"), vectors_per_pi, pi_stride, _dev(centroids, "centroids"),
                                        float(e_bar), _dev(out, "out"), _dtype_code(out), out.stride(0),
                                        _stream(stream)))


def tq_qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, q_out: torch.Tensor | None,
                    k_out: torch.Tensor | None, q_weight: torch.Tensor | None = None,
                    k_weight: torch.Tensor | None = None, eps: float = 1e-6, positions: torch.Tensor | None = None,
                    rope_base: float = 10000.0, rot_dim: int | None = None, d_status: torch.Tensor | None = None,
                    stream=None) -> None:
    """Per-head RMS norm and position rotation of q ([tokens, hq, d]) and k ([tokens, hkv, d]) into q_out and k_out.

    The tensors may be strided views (unit stride along d), an output its own input; a side that is None is left out,
    as is the norm of a side without a weight ([d] float32) and the rotation without positions ([tokens] int32)."""
    st = _bind.qk_norm_rope(q, k, q_out, k_out, q_weight, k_weight, eps, positions, rope_base, rot_dim, d_status,
                            None if stream is None else _stream(stream))
    if st:
        _check(st)


_CODE8 = {"e4m3": TQ_E4M3, "int8": TQ_INT8}


@dataclasses.dataclass(slots=True)
class Cache8:
    """A paged 8-bit KV cache (torch tensors on one device): token p of a sequence is row p % block of the page that
    its block table names for p // block; a stored value is code * scale."""
    k: torch.Tensor              # uint8 [n_blocks, heads, block, d]
    v: torch.Tensor
    k_scale: torch.Tensor        # float32 [n_blocks, heads], powers of two
    v_scale: torch.Tensor
    code: str = "e4m3"           # or "int8"

    def c(self) -> _Cache8:
        k, v, ks, vs = self.k, self.v, self.k_scale, self.v_scale
        if k.dim() != 4:
            raise ValueError("codes must be [n_blocks, heads, block, d]")
        n, h, b, d = k.shape
        if (v.shape != k.shape or ks.shape != (n, h) or vs.shape != (n, h) or k.dtype is not torch.uint8
                or v.dtype is not torch.uint8 or ks.dtype is not torch.float32 or vs.dtype is not torch.float32
                or not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous())):
            raise ValueError("a Cache8 has contiguous uint8 [n_blocks, heads, block, d] codes and float32 "
                             "[n_blocks, heads] scales")
        code = _CODE8.get(self.code)
        if code is None:
            raise ValueError(f"unknown code {self.code!r} (e4m3 or int8)")
        return _Cache8(d, h, b, code, n, k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr())

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k, self.v, self.k_scale, self.v_scale))


def tq_cache8_bytes(d: int, heads: int, block: int, n_blocks: int) -> int:
    return int(_lib.tq_cache8_bytes(d, heads, block, n_blocks))


def alloc_cache8(n_blocks: int, heads: int, block: int, d: int, code: str = "e4m3", device="cuda") -> Cache8:
    """Allocates a cache of n_blocks pages (allocation is PyTorch's; it needs no initialisation)."""
    codes = [torch.empty((n_blocks, heads, block, d), dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.empty((n_blocks, heads), dtype=torch.float32, device=device) for _ in range(2)]
    return Cache8(*codes, *scales, code)


def tq_cache8_write(cache: Cache8, k: torch.Tensor, v: torch.Tensor, cu_tokens: torch.Tensor, start: torch.Tensor,
                    block_table: torch.Tensor | None = None, d_status: torch.Tensor | None = None, stream=None) -> None:
    """Quantises rows cu_tokens[b] .. cu_tokens[b+1]-1 of k and v ([tokens, heads, d]) into positions start[b], ...
    of sequence b (cu_tokens int32 [batch+1], start int32 [batch], block_table int32 [batch, blocks])."""
    st = _bind.cache8_rows(True, cache.k, cache.v, cache.k_scale, cache.v_scale, cache.code, k, v, cu_tokens, start,
                           block_table, d_status, None if stream is None else _stream(stream))
    if st:
        _check(st)


def tq_cache8_read(cache: Cache8, k_out: torch.Tensor | None, v_out: torch.Tensor | None, cu_tokens: torch.Tensor,
                   start: torch.Tensor, block_table: torch.Tensor | None = None, d_status: torch.Tensor | None = None,
                   stream=None) -> None:
    """Reads positions start[b], ... of sequence b back into rows cu_tokens[b] .. cu_tokens[b+1]-1 of k_out and v_out."""
    st = _bind.cache8_rows(False, cache.k, cache.v, cache.k_scale, cache.v_scale, cache.code, k_out, v_out, cu_tokens, start,
                           block_table, d_status, None if stream is None else _stream(stream))
    if st:
        _check(st)


def tq_cache8_attention_workspace_bytes(cache: Cache8, batch: int, hq: int, nq: int) -> int:
    return int(_lib.tq_cache8_attention_workspace_bytes(cache.c(), batch, hq, nq))


def cache8_attention_workspace(cache: Cache8, batch: int, hq: int, nq: int) -> torch.Tensor:
    n = tq_cache8_attention_workspace_bytes(cache, batch, hq, nq)
    return torch.empty((max(n, 256) + 255) // 256 * 256, dtype=torch.uint8, device=cache.k.device)


def tq_cache8_attention(cache: Cache8, q: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor,
                        workspace: torch.Tensor, block_table: torch.Tensor | None = None, causal: bool = True,
                        window: int = 0, scale: float | None = None, lse_out: torch.Tensor | None = None,
                        d_status: torch.Tensor | None = None, stream=None) -> None:
    """Attention of q ([batch, hq, nq, d], any strides with unit stride along d) over the first seq_lens[b] tokens of
    each sequence; row i stands at position seq_lens[b] - nq + i. out is as q, lse_out float32 [batch, hq, nq]."""
    st = _bind.cache8_attention(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.code, q, seq_lens, out, workspace,
                                block_table, causal, window, scale, lse_out, d_status,
                                None if stream is None else _stream(stream))
    if st:
        _check(st)


def tq_residual_mean(samples, centroids, boundaries, bits: int) -> float:
    """Mean |u - c[code(u)]| over host samples u (the e_bar of tq_dequantize_sign_mean)."""
    u = np.ascontiguousarray(np.asarray(samples, dtype=np.float32).ravel())
    c = np.ascontiguousarray(np.asarray(centroids, dtype=np.float32))
    t = np.ascontiguousarray(np.asarray(boundaries, dtype=np.float32))
    e = ctypes.c_double(0.0)
    _check(_lib.tq_residual_mean(u.ctypes.data, u.size, c.ctypes.data, t.ctypes.data, bits, ctypes.byref(e)))
    return float(e.value)


def tq_search_workspace_bytes(lay: Layout, n_queries: int, n_db: int, k: int) -> int:
    return int(_lib.tq_search_workspace_bytes(ctypes.byref(lay), n_queries, n_db, k))


def tq_search_topk(lay: Layout, q: torch.Tensor, db: Planes, n_db: int, Pi: torch.Tensor, S: torch.Tensor,
                   centroids: torch.Tensor, k: int, top_idx: torch.Tensor, top_scores: torch.Tensor,
                   workspace: torch.Tensor, stream=None) -> None:
    """k best corpus rows per query ([n_queries, d], contiguous) by estimated inner product."""
    if q.dim() != 2 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [n_queries, d] tensor")
    _check(_lib.tq_search_topk(ctypes.byref(lay), _dev(q, "q"), _dtype_code(q), q.shape[0], ctypes.byref(db.c()),
                               n_db, _dev(Pi, "Pi"), _dev(S, "S"), _dev(centroids, "centroids"), k,
                               _dev(top_idx, "top_idx"), _dev(top_scores, "top_scores"), _dev(workspace, "workspace"),
                               workspace.numel() * workspace.element_size(), _stream(stream)))


def tq_search_merge_topk(idx_a: torch.Tensor, scores_a: torch.Tensor, offset_a: int, idx_b: torch.Tensor,
                         scores_b: torch.Tensor, offset_b: int, idx_out: torch.Tensor, scores_out: torch.Tensor,
                         stream=None) -> None:
    """Merges two [n_queries, k] top-k lists (ids shifted by their shard offsets) into idx_out / scores_out."""
    nq, k = idx_a.shape
    _check(_lib.tq_search_merge_topk(nq, k, _dev(idx_a, "idx_a"), _dev(scores_a, "scores_a"), offset_a,
                                     _dev(idx_b, "idx_b"), _dev(scores_b, "scores_b"), offset_b,
                                     _dev(idx_out, "idx_out"), _dev(scores_out, "scores_out"), _stream(stream)))


def tq_fit_rotation(X, Pi_rand) -> np.ndarray:
    """Per-head rotation Pi_rand V^T from calibration rows X ([n, d], host)."""
    X = np.ascontiguousarray(np.asarray(X, dtype=np.float32))
    P = np.ascontiguousarray(np.asarray(Pi_rand, dtype=np.float32))
    n, d = X.shape
    out = np.zeros((d, d), dtype=np.float32)
    _check(_lib.tq_fit_rotation(d, X.ctypes.data, n, P.ctypes.data, out.ctypes.data))
    return out


def tq_rotate_normalize(X, Pi) -> np.ndarray:
    """Coordinates of Pi x / ||x|| for the non-zero rows of X (host)."""
    X = np.ascontiguousarray(np.asarray(X, dtype=np.float32))
    P = np.ascontiguousarray(np.asarray(Pi, dtype=np.float32))
    n, d = X.shape
    out = np.zeros((n, d), dtype=np.float32)
    m = ctypes.c_int64(0)
    _check(_lib.tq_rotate_normalize(d, X.ctypes.data, n, P.ctypes.data, out.ctypes.data, ctypes.byref(m)))
    return out[:m.value]


def tq_last_error_string() -> str:
    return _lib.tq_last_error_string().decode()


def tq_version() -> str:
    return _lib.tq_version().decode()


def tq_kernel_launches() -> int:
    """Kernels the library has launched (or captured) since it was loaded."""
    return int(_lib.tq_kernel_launches())
