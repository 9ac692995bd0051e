"""ctypes binding to libkq.so -- argument marshalling only.

Every function here has the name of the C entry point it calls (include/kq.h)
and does nothing but turn tensors into pointers, pick the current stream and
raise on a nonzero status.  All arithmetic runs in the CUDA kernels.  If the
library is missing the import fails: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkq.so")

KQ_OK = 0
KQ_ERR_NULL = -1
KQ_ERR_SHAPE = -2
KQ_ERR_UNSUPPORTED = -3
KQ_ERR_ALIGN = -4
KQ_ERR_ARG = -5
KQ_ERR_CUDA = -6
KQ_ERR_TIMEOUT = -7


class KQError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__("%s failed: %d (%s)" % (fn, status, text))
        self.status = status


class _KVCacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class _KVTransformStruct(ctypes.Structure):
    _fields_ = [("Pq", ctypes.c_void_p), ("Pk", ctypes.c_void_p), ("Pv", ctypes.c_void_p),
                ("alpha_k", ctypes.c_float), ("alpha_v", ctypes.c_float), ("rope", ctypes.c_void_p),
                ("rope_positions", ctypes.c_int64), ("rope_dim", ctypes.c_int), ("rope_interleaved", ctypes.c_int)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError("libkq.so not built at %s; run __graft_entry__.build() "
                          "(kronecker_factored_transforms_b200/build.py)" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, I32, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    lib.kq_transform_quant.argtypes = [P, P, P, P, F32, P, P, I64, I32, I32, P]
    lib.kq_transform.argtypes = [P, P, P, P, P, I64, I32, I32, P]
    lib.kq_dequant_inverse.argtypes = [P, P, P, P, P, P, I64, I32, I32, P]
    lib.kq_device_error.argtypes = [P, ctypes.POINTER(ctypes.c_int)]
    lib.kq_selftest_bounded_wait.argtypes = [I64, P]
    lib.kq_w4a4_gemm.argtypes = [P, P, P, P, P, I64, I64, I64, P]
    lib.kq_w4a4_gemm_bf16.argtypes = [P, P, P, P, P, I64, I64, I64, P]
    lib.kq_headwise_transform_quant.argtypes = [P, P, F32, P, P, I64, I32, I32, P]
    lib.kq_transform_quant_two_stage.argtypes = [P, P, P, P, F32, P, P, P, ctypes.c_uint64, I64, I32, I32, P]
    lib.kq_transform_quant_two_stage_static.argtypes = [P, P, P, P, F32, P, P, I64, I32, I32, P]
    lib.kq_headwise_transform_quant_nvfp4.argtypes = [P, P, P, P, P, I64, I32, I32, P]
    lib.kq_kv_append.argtypes = [P, P, P, I64, P, I64, P, I64, P, P, P, I64, I32, P]
    lib.kq_kv_gather.argtypes = [P, P, P, P, I64, P]
    lib.kq_kv_attention.argtypes = [P, P, P, P, I64, P, F32, F32, I32, P, P, P, ctypes.c_uint64, I64, I64, I32, I32, P]
    lib.kq_kv_attention_shared.argtypes = [P, P, P, P, I64, P, I64, P, F32, F32, I32, P, P, P, ctypes.c_uint64, I64,
                                           I64, I32, I32, P]
    lib.kq_kv_attention_workspace_bytes.argtypes = [I64, I64, I32, I32, I32, I32]
    lib.kq_kv_attention_workspace_bytes.restype = ctypes.c_uint64
    for f in (lib.kq_kv_append, lib.kq_kv_gather, lib.kq_kv_attention, lib.kq_kv_attention_shared):
        f.restype = ctypes.c_int
    for f in (lib.kq_transform_quant, lib.kq_transform, lib.kq_dequant_inverse, lib.kq_device_error,
              lib.kq_selftest_bounded_wait, lib.kq_w4a4_gemm, lib.kq_w4a4_gemm_bf16, lib.kq_headwise_transform_quant,
              lib.kq_transform_quant_two_stage, lib.kq_transform_quant_two_stage_static,
              lib.kq_headwise_transform_quant_nvfp4):
        f.restype = ctypes.c_int
    lib.kq_two_stage_workspace_bytes.argtypes = [I64, I32, I32]
    lib.kq_two_stage_workspace_bytes.restype = ctypes.c_uint64
    lib.kq_status_string.argtypes = [I32]
    lib.kq_status_string.restype = ctypes.c_char_p
    lib.kq_kernel_name.argtypes = [I32, I32, I32]
    lib.kq_kernel_name.restype = ctypes.c_char_p
    lib.kq_kernel_for.argtypes = [I64, I32, I32, I32, ctypes.c_float]
    lib.kq_kernel_for.restype = ctypes.c_char_p
    lib.kq_version.argtypes = []
    lib.kq_version.restype = ctypes.c_int
    return lib


lib = _load()

EXPORTED = ("kq_transform_quant", "kq_transform", "kq_dequant_inverse", "kq_device_error",
            "kq_selftest_bounded_wait", "kq_status_string", "kq_kernel_name", "kq_kernel_for", "kq_version", "kq_w4a4_gemm",
            "kq_w4a4_gemm_bf16",
            "kq_headwise_transform_quant", "kq_transform_quant_two_stage", "kq_two_stage_workspace_bytes",
            "kq_transform_quant_two_stage_static", "kq_headwise_transform_quant_nvfp4",
            "kq_kv_append", "kq_kv_gather", "kq_kv_attention", "kq_kv_attention_shared",
            "kq_kv_attention_workspace_bytes")

STATIC_WORKSPACE_BYTES = 64 * 1024 * 1024


def _ptr(t) -> Optional[int]:
    """Device pointer of a tensor (or an int address, or None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _check(fn: str, st: int) -> None:
    if st != KQ_OK:
        raise KQError(fn, st, lib.kq_status_string(st).decode())


def kq_transform_quant(x, P1, P2, cinv, alpha: float, q_out, scale_out, T: int, n1: int, n2: int,
                       stream=None) -> None:
    _check("kq_transform_quant",
           lib.kq_transform_quant(_ptr(x), _ptr(P1), _ptr(P2), _ptr(cinv), float(alpha), _ptr(q_out),
                                  _ptr(scale_out), int(T), int(n1), int(n2), _stream(stream)))


def kq_headwise_transform_quant(x, Ph, alpha: float, q_out, scale_out, T: int, heads: int, head_dim: int,
                                stream=None) -> None:
    _check("kq_headwise_transform_quant",
           lib.kq_headwise_transform_quant(_ptr(x), _ptr(Ph), float(alpha), _ptr(q_out), _ptr(scale_out), int(T),
                                           int(heads), int(head_dim), _stream(stream)))


def kq_two_stage_workspace_bytes(T: int, n1: int, n2: int) -> int:
    return int(lib.kq_two_stage_workspace_bytes(int(T), int(n1), int(n2)))


def kq_transform_quant_two_stage(x, P1, P2, cinv, alpha: float, q_out, scale_out, workspace, workspace_bytes: int,
                                 T: int, n1: int, n2: int, stream=None) -> None:
    _check("kq_transform_quant_two_stage",
           lib.kq_transform_quant_two_stage(_ptr(x), _ptr(P1), _ptr(P2), _ptr(cinv), float(alpha), _ptr(q_out),
                                            _ptr(scale_out), _ptr(workspace), int(workspace_bytes), int(T), int(n1),
                                            int(n2), _stream(stream)))


def kq_transform_quant_two_stage_static(x, P1, P2, cinv, alpha: float, q_out, scale_out, T: int, n1: int, n2: int,
                                        stream=None) -> None:
    _check("kq_transform_quant_two_stage_static",
           lib.kq_transform_quant_two_stage_static(_ptr(x), _ptr(P1), _ptr(P2), _ptr(cinv), float(alpha), _ptr(q_out),
                                                   _ptr(scale_out), int(T), int(n1), int(n2), _stream(stream)))


def kq_headwise_transform_quant_nvfp4(x, Ph, q_out, block_scale_out, scale_out, T: int, heads: int, head_dim: int,
                                      stream=None) -> None:
    _check("kq_headwise_transform_quant_nvfp4",
           lib.kq_headwise_transform_quant_nvfp4(_ptr(x), _ptr(Ph), _ptr(q_out), _ptr(block_scale_out), _ptr(scale_out),
                                                 int(T), int(heads), int(head_dim), _stream(stream)))


def kq_w4a4_gemm(qx, sx, qw, sw, y, M: int, N: int, K: int, stream=None) -> None:
    _check("kq_w4a4_gemm",
           lib.kq_w4a4_gemm(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(y), int(M), int(N), int(K),
                            _stream(stream)))


def kq_w4a4_gemm_bf16(qx, sx, qw, sw, y, M: int, N: int, K: int, stream=None) -> None:
    _check("kq_w4a4_gemm_bf16",
           lib.kq_w4a4_gemm_bf16(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(y), int(M), int(N), int(K),
                                 _stream(stream)))


class _Handle:
    """A C struct the caller fills in once: its address, and the tensors it points into."""

    def __init__(self, struct, tensors, head_dim):
        self._struct = struct
        self.head_dim = head_dim
        self._tensors = [t for t in tensors if t is not None]  # kept alive with the handle
        self.ptr = ctypes.addressof(struct)
        devices = {t.device for t in self._tensors}
        if len(devices) != 1 or next(iter(devices)).type != "cuda":
            raise ValueError("the tensors of a handle lie on one CUDA device, got %s" % sorted(map(str, devices)))
        if not all(t.is_contiguous() for t in self._tensors):
            raise ValueError("the tensors of a handle are contiguous")
        self.device = next(iter(devices)).index


def kv_cache(k_codes, k_scale, v_codes, v_scale) -> _Handle:
    """The kq_kv_cache of four tensors: codes [pages, kv_heads, page_size, head_dim / 2] uint8 and
    scales [pages, kv_heads, page_size] fp32, for keys and for values."""
    import torch
    if k_codes.dim() != 4 or k_codes.shape != v_codes.shape or k_codes.dtype != torch.uint8 \
            or v_codes.dtype != torch.uint8:
        raise ValueError("k_codes and v_codes are uint8 [pages, kv_heads, page_size, head_dim / 2]")
    pages, heads, page, half = k_codes.shape
    for s in (k_scale, v_scale):
        if tuple(s.shape) != (pages, heads, page) or s.dtype != torch.float32:
            raise ValueError("k_scale and v_scale are float32 [pages, kv_heads, page_size]")
    st = _KVCacheStruct(k_codes.data_ptr(), k_scale.data_ptr(), v_codes.data_ptr(), v_scale.data_ptr(), pages, page,
                        heads, 2 * half)
    return _Handle(st, [k_codes, k_scale, v_codes, v_scale], 2 * half)


def kv_transform(Pq, Pk, Pv, alpha_k: float, alpha_v: float, rope=None, interleaved: bool = False) -> _Handle:
    """The kq_kv_transform of bf16 factors [head_dim, head_dim] (as bf16 or 16-bit integer tensors; Pq may be None)
    and a rotary table fp32 [positions, rotated elements] (cosines, then sines) or None."""
    import torch
    for P in (Pq, Pk, Pv):
        if P is not None and (P.shape != Pk.shape or P.dim() != 2 or P.shape[0] != P.shape[1]
                              or P.dtype not in (torch.bfloat16, torch.int16, torch.uint16)):
            raise ValueError("the factors are square matrices of one size, in bf16")
    if rope is not None and (rope.dim() != 2 or rope.dtype != torch.float32):
        raise ValueError("the rotary table is float32 [positions, rotated elements]")
    n, r = (0, 0) if rope is None else rope.shape
    st = _KVTransformStruct(_ptr(Pq), _ptr(Pk), _ptr(Pv), float(alpha_k), float(alpha_v), _ptr(rope), n, r,
                            int(bool(interleaved)))
    return _Handle(st, [Pq, Pk, Pv, rope], Pk.shape[0])


# torch's current device and the raw current stream of a device, the types of the calls' tensors, and those that are the
# same bits (for none, a workspace: any): looked up on the first call.
_current_device = None
_raw_stream = None
_append_kinds = _gather_kinds = _attention_kinds = _shared_kinds = _same_bits = None


def _device_calls():
    global _current_device, _raw_stream, _append_kinds, _gather_kinds, _attention_kinds, _shared_kinds, _same_bits
    import torch
    bf16, int32, int64, fp32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
    _same_bits = {bf16: (torch.int16, torch.uint16), int32: (torch.uint32,), int64: (torch.uint64,), fp32: ()}
    _append_kinds = (bf16, bf16, bf16, int32, int64, bf16)
    _gather_kinds = (int64, bf16, bf16)
    _attention_kinds = (bf16, int32, int32, int32, bf16, fp32, torch.uint8)
    _shared_kinds = (bf16, int32, int32, int32, int32, bf16, fp32, torch.uint8)
    _current_device = torch.cuda.current_device
    # the public way makes a Stream object, which takes as long as the launch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _unusual(fn: str, cache, t, at: int, kind, rows: bool):
    """The address of a tensor that is not of its kind's type, or not dense, where it may be so."""
    if t.get_device() != cache.device:
        raise ValueError("%s: a tensor on %s, the cache on cuda:%d" % (fn, t.device, cache.device))
    if t.dtype is not kind and kind in _same_bits and t.dtype not in _same_bits[kind]:
        raise ValueError("%s: tensor %d is %s, not %s" % (fn, at, t.dtype, kind))
    if not (t.stride(-1) == 1 if rows else t.is_contiguous()):
        raise ValueError("%s: tensor %d is not dense (strides %s)" % (fn, at, t.stride()))
    return t.data_ptr()


def _enter(fn: str, cache, stream, tensors, kinds, rows=0):
    """The stream (a C entry works on the current device: another one is an error here) and the tensors' addresses,
    where these are the numbers that the entry will read there (the first `rows`: rows a stride apart).

    These calls take microseconds on the GPU for small batches, so this is kept short."""
    device = cache.device
    if _current_device() != device:
        raise ValueError("%s: the cache lies on cuda:%d, the current device is cuda:%d" % (fn, device, _current_device()))
    ptrs = []
    for t, kind in zip(tensors, kinds):
        if t is None or t.__class__ is int:
            ptrs.append(t)
        elif t.get_device() == device and t.dtype is kind and t.is_contiguous():  # the usual case
            ptrs.append(t.data_ptr())
        else:
            ptrs.append(_unusual(fn, cache, t, len(ptrs), kind, len(ptrs) < rows))
    if stream is None:
        return _raw_stream(device) or None, ptrs
    return _stream(stream), ptrs


def kq_kv_append(cache, tf, q, q_stride: int, k, k_stride: int, v, v_stride: int, positions, slots, q_out, T: int,
                 q_heads: int, stream=None) -> None:
    if tf.device != cache.device or tf.head_dim != cache.head_dim:
        raise ValueError("kq_kv_append: the transform is of head_dim %d on cuda:%d, the cache of %d on cuda:%d"
                         % (tf.head_dim, tf.device, cache.head_dim, cache.device))
    if _raw_stream is None:
        _device_calls()
    st, (q, k, v, positions, slots, q_out) = _enter(
        "kq_kv_append", cache, stream, (q, k, v, positions, slots, q_out), _append_kinds, 3)
    r = lib.kq_kv_append(cache.ptr, tf.ptr, q, q_stride, k, k_stride, v, v_stride, positions, slots, q_out, T, q_heads, st)
    if r:
        _check("kq_kv_append", r)


def kq_kv_gather(cache, slots, k_out, v_out, T: int, stream=None) -> None:
    if _raw_stream is None:
        _device_calls()
    st, (slots, k_out, v_out) = _enter("kq_kv_gather", cache, stream, (slots, k_out, v_out), _gather_kinds)
    r = lib.kq_kv_gather(cache.ptr, slots, k_out, v_out, T, st)
    if r:
        _check("kq_kv_gather", r)


def kq_kv_attention_workspace_bytes(T: int, B: int, q_heads: int, kv_heads: int, head_dim: int, max_q: int) -> int:
    return int(lib.kq_kv_attention_workspace_bytes(int(T), int(B), int(q_heads), int(kv_heads), int(head_dim),
                                                   int(max_q)))


def kq_kv_attention(cache, q, q_start, page_table, max_pages: int, kv_len, scale: float, softcap: float, window: int,
                    out, lse, workspace, workspace_bytes: int, T: int, B: int, q_heads: int, max_q: int,
                    stream=None) -> None:
    if _raw_stream is None:
        _device_calls()
    st, (q, q_start, page_table, kv_len, out, lse, workspace) = _enter(
        "kq_kv_attention", cache, stream, (q, q_start, page_table, kv_len, out, lse, workspace), _attention_kinds)
    r = lib.kq_kv_attention(cache.ptr, q, q_start, page_table, max_pages, kv_len, scale, softcap, window, out, lse,
                            workspace, workspace_bytes, T, B, q_heads, max_q, st)
    if r:
        _check("kq_kv_attention", r)


def kq_kv_attention_shared(cache, q, q_start, prefix_pages, prefix_len: int, page_table, max_pages: int, kv_len,
                           scale: float, softcap: float, window: int, out, lse, workspace, workspace_bytes: int,
                           T: int, B: int, q_heads: int, max_q: int, stream=None) -> None:
    if _raw_stream is None:
        _device_calls()
    st, (q, q_start, prefix_pages, page_table, kv_len, out, lse, workspace) = _enter(
        "kq_kv_attention_shared", cache, stream, (q, q_start, prefix_pages, page_table, kv_len, out, lse, workspace),
        _shared_kinds)
    r = lib.kq_kv_attention_shared(cache.ptr, q, q_start, prefix_pages, prefix_len, page_table, max_pages, kv_len, scale,
                                   softcap, window, out, lse, workspace, workspace_bytes, T, B, q_heads, max_q, st)
    if r:
        _check("kq_kv_attention_shared", r)


def kq_transform(x, P1, P2, cinv, y_out, T: int, n1: int, n2: int, stream=None) -> None:
    _check("kq_transform",
           lib.kq_transform(_ptr(x), _ptr(P1), _ptr(P2), _ptr(cinv), _ptr(y_out), int(T), int(n1),
                            int(n2), _stream(stream)))


def kq_dequant_inverse(q, scale, P1inv, P2inv, c, x_hat, T: int, n1: int, n2: int, stream=None) -> None:
    _check("kq_dequant_inverse",
           lib.kq_dequant_inverse(_ptr(q), _ptr(scale), _ptr(P1inv), _ptr(P2inv), _ptr(c), _ptr(x_hat),
                                  int(T), int(n1), int(n2), _stream(stream)))


def kq_device_error(stream=None) -> int:
    code = ctypes.c_int(0)
    _check("kq_device_error", lib.kq_device_error(_stream(stream), ctypes.byref(code)))
    return code.value


def kq_selftest_bounded_wait(limit_us: int, stream=None) -> None:
    _check("kq_selftest_bounded_wait", lib.kq_selftest_bounded_wait(int(limit_us), _stream(stream)))


def kq_status_string(status: int) -> str:
    return lib.kq_status_string(int(status)).decode()


def kq_kernel_name(n1: int, n2: int, has_cinv: bool) -> str:
    return lib.kq_kernel_name(int(n1), int(n2), int(bool(has_cinv))).decode()


def kq_kernel_for(T: int, n1: int, n2: int, has_cinv: bool, alpha: float = 0.9) -> str:
    return lib.kq_kernel_for(int(T), int(n1), int(n2), int(bool(has_cinv)), float(alpha)).decode()


def kq_version() -> int:
    return int(lib.kq_version())
