"""Thin ctypes binding of libqmm.so (include/qmm.h).

Functions carry the C names and only marshal arguments: torch tensors become
device pointers, torch dtypes become ``qmm_dtype`` values, and the current
HIP stream is passed unless one is given.  A negative status raises
:class:`QmmError` with the library's message.  The library is required:
importing this module fails loudly when ``libqmm.so`` has not been built.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmm.so")

QMM_F32, QMM_F16, QMM_BF16 = 0, 1, 2
QMM_LAYOUT_ORT, QMM_LAYOUT_TILED, QMM_LAYOUT_TILED_ZP = 0, 1, 2
QMM_OK, QMM_ERR_INVALID_ARG, QMM_ERR_UNSUPPORTED, QMM_ERR_WORKSPACE, QMM_ERR_HIP = 0, -1, -2, -3, -4

_TORCH_TO_QMM = {torch.float32: QMM_F32, torch.float16: QMM_F16, torch.bfloat16: QMM_BF16}

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first "
        "(python -m block_quantized_weight_matmulnbits_amd.build). There is no CPU fallback.")

lib = ctypes.CDLL(LIB_PATH)

_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_f64 = ctypes.c_double
_SIGS = {
    "qmm_last_error": ([], ctypes.c_char_p),
    "qmm_gemv": ([_vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _i32, _i32,
                  _i32, _vp], _i32),
    "qmm_check_g_idx": ([_vp, _i64, _i64, _i32], _i32),
    "qmm_gemm": ([_vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _i32,
                  _i32, _i32, _vp], _i32),
    "qmm_compint8_workspace_size": ([_i64, _i64, _i32], _sz),
    "qmm_lowp_matmul": ([_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _i32, _i32, _vp],
                        _i32),
    "qmm_lowp_quantize": ([_vp, _i32, _i64, _i64, _i32, _i32, _vp, _vp, _vp], _i32),
    "qmm_gemm_compint8": ([_vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _i64,
                           _i32, _i32, _i32, _vp, _sz, _vp], _i32),
    "qmm_gemm_compint8_noalloc": ([_vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i64, _vp, _vp, _i64,
                                   _i64, _i64, _i32, _i32, _i32, _vp], _i32),
    "qmm_int16_workspace_size": ([_i64, _i64, _i32], _sz),
    "qmm_gemm_int16": ([_vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _i32,
                        _vp, _sz, _vp], _i32),
    "qmm_debug_int16_block_dots": ([_vp, _i32, _vp, _vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _sz,
                                    _vp], _i32),
    "qmm_gemm_fp4": ([_vp, _i32, _vp, _vp, _i32, _f32, _vp, _vp, _i64, _i64, _i64, _vp], _i32),
    "qmm_step_create": ([_vp], _i32),
    "qmm_step_add_gemv": ([_vp, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i64, _vp, _vp, _i64, _i64,
                           _i32, _i32, _i32], _i32),
    "qmm_step_add_gemm": ([_vp, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i64, _vp, _vp, _i64, _i64,
                           _i64, _i32, _i32, _i32], _i32),
    "qmm_step_add_gemm_compint8": ([_vp, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i64, _vp, _vp,
                                    _i64, _i64, _i64, _i32, _i32, _i32, _vp, _sz], _i32),
    "qmm_rope_append": ([_vp] * 6 + [_vp, _i32, _i32, _f64, _vp, _vp], _i32),
    "qmm_paged_attention_workspace_size": ([_vp, _i32, _i32, _i32], _sz),
    "qmm_paged_attention": ([_vp, _vp, _vp, _vp, _vp, _f32, _i32, _i64, _f32, _vp, _sz, _vp], _i32),
    "qmm_pages_workspace_size": ([_vp, _i64], _sz),
    "qmm_pages_free": ([_vp, _vp, _i64, _vp], _i32),
    "qmm_pages_fork": ([_vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp], _i32),
    "qmm_pages_reserve": ([_vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp], _i32),
    "qmm_pages_copy": ([_vp, _vp, _vp, _i64, _vp], _i32),
    "qmm_pages_compact": ([_vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "qmm_step_add_rope_append": ([_vp] * 7 + [_vp, _i32, _i32, _f64, _vp], _i32),
    "qmm_step_add_paged_attention": ([_vp, _vp, _vp, _vp, _vp, _vp, _f32, _i32, _i64, _f32, _vp, _sz],
                                     _i32),
    "qmm_step_add_pages_reserve": ([_vp, _vp, _vp, _vp, _i64, _vp, _vp, _sz], _i32),
    "qmm_step_finalize": ([_vp], _i32),
    "qmm_step_launch": ([_vp, _vp], _i32),
    "qmm_step_size": ([_vp], _i32),
    "qmm_step_destroy": ([_vp], None),
    "qconv_int8": ([_vp, _vp, _vp, _vp, _f32, _f32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                    _i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp], _i32),
    "qmm_repacked_bytes": ([_i64, _i64, _i32, _i32, _i32, _i32], _sz),
    "qmm_repack": ([_vp, _vp, _i32, _vp, _i64, _i64, _i32, _i32, _vp, _sz, _vp], _i32),
    "qmm_unrepack": ([_vp, _i32, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp], _i32),
    "qmm_debug_unpack": ([_vp, _i32, _vp, _i32, _vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp], _i32),
    "qmm_debug_quantize_a": ([_vp, _i32, _i64, _i64, _i32, _vp, _vp, _vp], _i32),
    "qmm_debug_compint8_block_dots": ([_vp, _i32, _vp, _i32, _i32, _vp, _i64, _i64, _i64, _i32, _i32,
                                       _vp, _vp, _sz, _vp], _i32),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

EXPORTED = tuple(_SIGS)


class QmmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[qmm status {status}] {message}")
        self.status = status


def _check(status: int) -> None:
    if status != QMM_OK:
        raise QmmError(status, lib.qmm_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dt(t) -> int:
    return _TORCH_TO_QMM[t.dtype]


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


# The current stream's handle without a Stream object around it, where torch
# has the call (the object costs a microsecond of every small operator).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_at(gpu, stream):
    """``stream``, or the current one of GPU number ``gpu``."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(gpu)
    return _stream(stream)


def _elsewhere(gpu, **tensors):
    """The error for the first of ``tensors`` that is not on the GPU of the
    handle they came with (whose number is -1 on the host).  Callers compare
    the numbers in one expression: that is a third of a microsecond a call."""
    name, t = next((n, t) for n, t in tensors.items() if t is not None and (gpu < 0 or t.get_device() != gpu))
    if gpu < 0:
        return ValueError(f"the cache and {name} must be on a GPU: the kernels read device memory")
    return ValueError(f"{name} is on {t.device}, the cache on GPU {gpu}: pass tensors of one GPU")


def qmm_last_error() -> str:
    return lib.qmm_last_error().decode()


class Repacked:
    """A device buffer written by :func:`qmm_repack`: pass it as ``B`` (with
    ``scales=None`` and ``zero_points=None``) to qmm_gemv / qmm_gemm /
    qmm_gemm_compint8.  The tiled buffer itself carries no geometry (the
    kernels derive its regions from K, N, block_size, bits and the scale
    dtype), so the geometry it was repacked with is kept here and every call
    that takes it must pass the same K, N, block_size and bits."""

    def __init__(self, buf, s_dtype, has_zero_points, K, N, block_size, bits):
        self.buf = buf
        self.s_dtype = s_dtype
        self.has_zero_points = bool(has_zero_points)
        self.layout = QMM_LAYOUT_TILED_ZP if has_zero_points else QMM_LAYOUT_TILED
        self.K, self.N, self.block_size, self.bits = int(K), int(N), int(block_size), int(bits)
        self.nbytes = buf.numel() * buf.element_size()

    def check(self, K, N, block_size, bits):
        """Raise ValueError unless (K, N, block_size, bits) are the repack's."""
        got = (int(K), int(N), int(block_size), int(bits))
        want = (self.K, self.N, self.block_size, self.bits)
        if got != want:
            raise ValueError(f"repacked buffer geometry mismatch: it was repacked for (K, N, "
                             f"block_size, bits) = {want}, the call passes {got}. The tiled "
                             "regions are located from these values: pass the repack's.")
        need = qmm_repacked_bytes(K, N, block_size, bits, self.s_dtype, self.has_zero_points)
        if self.nbytes < need:
            raise ValueError(f"repacked buffer holds {self.nbytes} bytes, the geometry needs "
                             f"{need}")


def _weights(B, scales, K, N, block_size, bits):
    """(B pointer, layout, scales pointer, scales dtype) for either layout."""
    if isinstance(B, Repacked):
        if scales is not None:
            raise ValueError("a repacked buffer carries its scales: pass scales=None")
        B.check(K, N, block_size, bits)
        return B.buf.data_ptr(), B.layout, None, B.s_dtype
    return B.data_ptr(), QMM_LAYOUT_ORT, _ptr(scales), _dt(scales)


def _g(g_idx):
    """(pointer, length) of optional int32 group indices."""
    return (None, 0) if g_idx is None else (g_idx.data_ptr(), g_idx.numel())


def qmm_gemv(A, B, scales, zero_points, bias, Y, K, N, block_size, bits, accuracy_level=0,
             stream=None, g_idx=None):
    b, layout, s, sdt = _weights(B, scales, K, N, block_size, bits)
    gp, gn = _g(g_idx)
    _check(lib.qmm_gemv(_ptr(A), _dt(A), b, layout, s, sdt, _ptr(zero_points), gp, gn,
                        _ptr(bias), _ptr(Y), K, N, block_size, bits, accuracy_level,
                        _stream(stream)))


def qmm_check_g_idx(g_idx, K, block_size):
    """Host-side range / shape check of group indices (a CPU int32 tensor)."""
    g = g_idx.contiguous()
    _check(lib.qmm_check_g_idx(g.data_ptr(), g.numel(), K, block_size))


def qmm_gemm(A, B, scales, zero_points, bias, Y, M, K, N, block_size, bits, accuracy_level=0,
             stream=None, g_idx=None):
    b, layout, s, sdt = _weights(B, scales, K, N, block_size, bits)
    gp, gn = _g(g_idx)
    _check(lib.qmm_gemm(_ptr(A), _dt(A), b, layout, s, sdt, _ptr(zero_points), gp, gn,
                        _ptr(bias), _ptr(Y), M, K, N, block_size, bits, accuracy_level,
                        _stream(stream)))


def qmm_repacked_bytes(K, N, block_size, bits, s_dtype, has_zero_points) -> int:
    sdt = s_dtype if isinstance(s_dtype, int) else _TORCH_TO_QMM[s_dtype]
    return int(lib.qmm_repacked_bytes(K, N, block_size, bits, sdt, int(bool(has_zero_points))))


def qmm_repack(B, scales, zero_points, K, N, block_size, bits, out=None, stream=None):
    """Repack (B, scales, zero_points) into ``out`` (allocated when None) and
    return it as a :class:`Repacked`."""
    nbytes = qmm_repacked_bytes(K, N, block_size, bits, scales.dtype, zero_points is not None)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=B.device)
    _check(lib.qmm_repack(_ptr(B), _ptr(scales), _dt(scales), _ptr(zero_points), K, N, block_size,
                          bits, _ptr(out), out.numel() * out.element_size(), _stream(stream)))
    return Repacked(out, _dt(scales), zero_points is not None, K, N, block_size, bits)


def qmm_unrepack(tiled, K, N, block_size, bits, B, scales, zero_points, stream=None):
    if isinstance(tiled, Repacked):
        tiled.check(K, N, block_size, bits)
    buf = tiled.buf if isinstance(tiled, Repacked) else tiled
    _check(lib.qmm_unrepack(_ptr(buf), int(zero_points is not None), K, N, block_size, bits,
                            _dt(scales), _ptr(B), _ptr(scales), _ptr(zero_points),
                            _stream(stream)))


def qmm_compint8_workspace_size(M, K, block_size) -> int:
    return int(lib.qmm_compint8_workspace_size(M, K, block_size))


def qmm_gemm_compint8(A, B, scales, zero_points, bias, Y, M, K, N, block_size, bits, workspace,
                      accuracy_level=4, stream=None, g_idx=None):
    b, layout, s, sdt = _weights(B, scales, K, N, block_size, bits)
    gp, gn = _g(g_idx)
    _check(lib.qmm_gemm_compint8(_ptr(A), _dt(A), b, layout, s, sdt, _ptr(zero_points), gp, gn,
                                 _ptr(bias), _ptr(Y), M, K, N, block_size, bits, accuracy_level,
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream)))


QMM_NOALLOC_SCRATCH_BYTES = 4 * 1024 * 1024


def qmm_gemm_compint8_noalloc(A, B, scales, zero_points, bias, Y, M, K, N, block_size, bits,
                              accuracy_level=4, stream=None, g_idx=None):
    b, layout, s, sdt = _weights(B, scales, K, N, block_size, bits)
    gp, gn = _g(g_idx)
    _check(lib.qmm_gemm_compint8_noalloc(_ptr(A), _dt(A), b, layout, s, sdt, _ptr(zero_points),
                                         gp, gn, _ptr(bias), _ptr(Y), M, K, N, block_size, bits,
                                         accuracy_level, _stream(stream)))


def qmm_int16_workspace_size(M, K, block_size) -> int:
    return int(lib.qmm_int16_workspace_size(M, K, block_size))


def qmm_gemm_int16(A, B, scales, zero_points, bias, Y, M, K, N, block_size, bits, workspace,
                   stream=None):
    """int16 activations (operator layout); ``B`` is the operator's tensor."""
    _check(lib.qmm_gemm_int16(_ptr(A), _dt(A), _ptr(B), QMM_LAYOUT_ORT, _ptr(scales), _dt(scales),
                              _ptr(zero_points), _ptr(bias), _ptr(Y), M, K, N, block_size, bits,
                              _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream(stream)))


def qmm_debug_int16_block_dots(A, B, zero_points, M, K, N, block_size, bits, dots, workspace,
                               stream=None):
    _check(lib.qmm_debug_int16_block_dots(_ptr(A), _dt(A), _ptr(B), _ptr(zero_points), M, K, N,
                                          block_size, bits, _ptr(dots), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(),
                                          _stream(stream)))


QMM_MXFP4, QMM_NVFP4 = 0, 1
FP4_FORMAT = {"mxfp4": QMM_MXFP4, "nvfp4": QMM_NVFP4}


def qmm_gemm_fp4(A, W, scales, fmt, global_scale, bias, Y, M, K, N, stream=None):
    """Block-scaled FP4 weights; ``fmt`` is "mxfp4" / "nvfp4" or the enum."""
    f = FP4_FORMAT.get(fmt, fmt)
    _check(lib.qmm_gemm_fp4(_ptr(A), _dt(A), _ptr(W), _ptr(scales), f, float(global_scale),
                            _ptr(bias), _ptr(Y), M, K, N, _stream(stream)))


class Step:
    """A recorded sequence of calls replayed as one HIP graph (qmm_step_* in
    include/qmm.h).  add_gemv / add_gemm / add_gemm_compint8 /
    add_rope_append / add_paged_attention / add_pages_reserve take the arguments of the functions of the same name (without a stream);
    finalize() validates and captures; launch(stream) replays.  The tensors
    passed are kept referenced for the step's life, since the graph holds
    their device addresses."""

    def __init__(self):
        h = ctypes.c_void_p()
        _check(lib.qmm_step_create(ctypes.byref(h)))
        self._h = h
        self._keep = []

    def _add(self, fn, tensors, *args):
        self._keep.extend(t for t in tensors if t is not None)
        _check(fn(self._h, *args))

    def add_gemv(self, A, B, scales, zero_points, bias, Y, K, N, block_size, bits,
                 accuracy_level=0, g_idx=None):
        b, layout, s, sdt = _weights(B, scales, K, N, block_size, bits)
        gp, gn = _g(g_idx)
        self._add(lib.qmm_step_add_gemv, (A, B, scales, zero_points, bias, Y, g_idx), _ptr(A),
                  _dt(A), b, layout, s, sdt, _ptr(zero_points), gp, gn, _ptr(bias), _ptr(Y), K, N,
                  block_size, bits, accuracy_level)

    def add_gemm(self, A, B, scales, zero_points, bias, Y, M, K, N, block_size, bits,
                 accuracy_level=0, g_idx=None):
        b, layout, s, sdt = _weights(B, scales, K, N, block_size, bits)
        gp, gn = _g(g_idx)
        self._add(lib.qmm_step_add_gemm, (A, B, scales, zero_points, bias, Y, g_idx), _ptr(A),
                  _dt(A), b, layout, s, sdt, _ptr(zero_points), gp, gn, _ptr(bias), _ptr(Y), M, K,
                  N, block_size, bits, accuracy_level)

    def add_gemm_compint8(self, A, B, scales, zero_points, bias, Y, M, K, N, block_size, bits,
                          workspace, accuracy_level=4, g_idx=None):
        b, layout, s, sdt = _weights(B, scales, K, N, block_size, bits)
        gp, gn = _g(g_idx)
        self._add(lib.qmm_step_add_gemm_compint8,
                  (A, B, scales, zero_points, bias, Y, g_idx, workspace), _ptr(A), _dt(A), b,
                  layout, s, sdt, _ptr(zero_points), gp, gn, _ptr(bias), _ptr(Y), M, K, N,
                  block_size, bits, accuracy_level, _ptr(workspace),
                  workspace.numel() * workspace.element_size())

    def add_rope_append(self, q, k, v, out, kv, batch, inv_freq, interleaved=False, factor=1.0,
                        positions=None):
        args = _rope_args(q, k, v, out, kv, batch, inv_freq, interleaved, factor, positions)
        self._add(lib.qmm_step_add_rope_append, (q, k, v, out, kv, batch, inv_freq, positions),
                  *args)

    def add_paged_attention(self, q, kv, batch, out, workspace, scale=None, causal=True, window=0,
                            softcap=0.0, lse=None):
        args = _attention_args(q, kv, batch, out, workspace, scale, causal, window, softcap, lse)
        self._add(lib.qmm_step_add_paged_attention, (q, kv, batch, out, workspace, lse), *args)

    def add_pages_reserve(self, pool, seqs, grow, status, workspace):
        n = _lists(pool, "seqs", seqs, "grow", grow, status, workspace)
        self._add(lib.qmm_step_add_pages_reserve, (pool, seqs, grow, status, workspace), pool._ref,
                  _ptr(seqs), _ptr(grow), n, _ptr(status), _ptr(workspace), workspace.nbytes)

    def finalize(self):
        _check(lib.qmm_step_finalize(self._h))
        return self

    def launch(self, stream=None):
        _check(lib.qmm_step_launch(self._h, _stream(stream)))

    def __len__(self):
        return int(lib.qmm_step_size(self._h))

    def close(self):
        if self._h:
            lib.qmm_step_destroy(self._h)
            self._h = None
            self._keep = []

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def qconv_int8(X, W, bias, w_scale, in_scale, out_scale, in_zp, out_zp, clamp_min, clamp_max,
               stride, pad, Y, stream=None):
    Nb, H, Wd, C = X.shape
    Co, KH, KW, _ = W.shape
    _check(lib.qconv_int8(_ptr(X), _ptr(W), _ptr(bias), _ptr(w_scale), in_scale, out_scale,
                          in_zp, out_zp, clamp_min, clamp_max, Nb, H, Wd, C, Co, KH, KW,
                          stride[0], stride[1], pad[0], pad[1], _ptr(Y), _stream(stream)))


def qmm_debug_unpack(B, scales, zero_points, K, N, block_size, bits, codes=None, zps=None, w=None,
                     stream=None):
    _check(lib.qmm_debug_unpack(_ptr(B), QMM_LAYOUT_ORT, _ptr(scales), _dt(scales),
                                _ptr(zero_points), K, N, block_size, bits, _ptr(codes), _ptr(zps),
                                _ptr(w), _stream(stream)))


def qmm_debug_quantize_a(A, M, K, block_size, qa, sa, stream=None):
    _check(lib.qmm_debug_quantize_a(_ptr(A), _dt(A), M, K, block_size, _ptr(qa), _ptr(sa),
                                    _stream(stream)))


def qmm_debug_compint8_block_dots(A, B, zero_points, M, K, N, block_size, bits, dots, workspace,
                                  stream=None):
    if isinstance(B, Repacked):
        B.check(K, N, block_size, bits)
        b, layout, sdt = B.buf.data_ptr(), B.layout, B.s_dtype
    else:
        b, layout, sdt = _ptr(B), QMM_LAYOUT_ORT, QMM_F32
    _check(lib.qmm_debug_compint8_block_dots(_ptr(A), _dt(A), b, layout, sdt, _ptr(zero_points),
                                             M, K, N, block_size, bits, _ptr(dots),
                                             _ptr(workspace),
                                             workspace.numel() * workspace.element_size(),
                                             _stream(stream)))


LOWP_FORMATS = {"e4m3": 0, "e5m2": 1, "e2m3": 2, "e3m2": 3, "e2m1": 4}
LOWP_LAYOUTS = {"tensor": 0, "mx": 1, "nvfp4": 2}


def qmm_lowp_matmul(lhs, rhs, lhs_scales, rhs_scales, bias, out, m, n, k, layout, lhs_format,
                    rhs_format, stream=None):
    """out[m, n] (f32) = decoded, scaled lhs [m, k] times rhs [n, k]^T (+ bias);
    layout "tensor" / "mx" / "nvfp4", formats "e4m3" / "e5m2" / "e2m3" /
    "e3m2" / "e2m1" (or their qmm_lowp_* integers)."""
    lay = LOWP_LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    lf = LOWP_FORMATS[lhs_format] if isinstance(lhs_format, str) else int(lhs_format)
    rf = LOWP_FORMATS[rhs_format] if isinstance(rhs_format, str) else int(rhs_format)
    _check(lib.qmm_lowp_matmul(_ptr(lhs), _ptr(rhs), _ptr(lhs_scales), _ptr(rhs_scales),
                               _ptr(bias), _ptr(out), m, n, k, lay, lf, rf, _stream(stream)))


def qmm_lowp_quantize(x, codes, scales, rows, cols, fmt, layout, stream=None):
    """codes [rows, cols] uint8 and scales (one f32 per tensor, else
    [rows, ceil(cols / bs)] bytes) of x [rows, cols] (f32 / f16 / bf16)."""
    lay = LOWP_LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    f = LOWP_FORMATS[fmt] if isinstance(fmt, str) else int(fmt)
    _check(lib.qmm_lowp_quantize(_ptr(x), _dt(x), rows, cols, f, lay, _ptr(codes), _ptr(scales),
                                 _stream(stream)))


_INT32 = torch.int32

# struct qmm_heads, as bytes: data, token_stride, head_stride, heads.
_pack_heads = struct.Struct("@Pqqi4x").pack


class _PagedKV(ctypes.Structure):
    _fields_ = ([("k_pages", _vp), ("v_pages", _vp)]
                + [(f"{t}_{d}_stride", _i64) for t in "kv" for d in ("page", "head", "token")]
                + [("pages", _i64)]
                + [(n, _i32) for n in ("dtype", "kv_heads", "page_size", "head_dim")])


class _PagedBatch(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("starts", "lens", "table")]
                + [(n, _i64) for n in ("table_stride", "seqs", "tokens", "width", "max_new",
                                       "max_len")])


class _PagePool(ctypes.Structure):
    _fields_ = ([("data", _vp)]
                + [(n, _i64) for n in ("planes", "pages", "page_bytes", "plane_stride",
                                       "page_stride")]
                + [(n, _vp) for n in ("refs", "table", "lens")]
                + [(n, _i64) for n in ("table_stride", "slots", "width")]
                + [("page_size", _i32)])


def _int32(name, t, shape=None):
    if t.dtype is not _INT32 or not t.is_contiguous() or (shape and t.shape != shape):
        raise ValueError(f"{name} must be a dense int32 tensor"
                         f"{f' of shape {list(shape)}' if shape else ''}, got {t.dtype} "
                         f"{list(t.shape)}")


def _rows(name, t):
    if t.dtype != torch.int32 or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be an int32 tensor [rows, width] with dense rows, got "
                         f"{t.dtype} {list(t.shape)}")


class PagedKV:
    """The pages of one layer's keys and values, each [pages, kv_heads,
    page_size, head_dim] with any strides as long as head_dim is dense (a
    cache laid out token by token is passed as a transposed view)."""

    def __init__(self, k_pages, v_pages):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype:
            raise ValueError(f"k_pages and v_pages must share one shape [pages, kv_heads, page_size, "
                             f"head_dim] and dtype, got {list(k_pages.shape)} {k_pages.dtype} and "
                             f"{list(v_pages.shape)} {v_pages.dtype}")
        if k_pages.dtype not in _TORCH_TO_QMM:
            raise ValueError(f"pages of {k_pages.dtype} are not supported: use float32, float16 or "
                             "bfloat16")
        if k_pages.device != v_pages.device:
            raise ValueError("k_pages and v_pages must be on one device")
        pages, self.kv_heads, self.page_size, self.head_dim = k_pages.shape
        if self.head_dim > 1 and (k_pages.stride(3) != 1 or v_pages.stride(3) != 1):
            raise ValueError("head_dim must be the dense dimension of k_pages and v_pages")
        self.k_pages, self.v_pages, self.dtype = k_pages, v_pages, k_pages.dtype
        self.gpu = k_pages.get_device()
        self._c = _PagedKV(_ptr(k_pages), _ptr(v_pages), *k_pages.stride()[:3],
                           *v_pages.stride()[:3], pages, _dt(k_pages), self.kv_heads,
                           self.page_size, self.head_dim)
        self._ref = ctypes.byref(self._c)


class PagedBatch:
    """Sequences over a paged cache: ``starts`` [seqs + 1] and ``lens`` [seqs]
    (the new tokens included), ``table`` [seqs, width] of page numbers, int32 on
    the device; ``tokens`` rows in all, at most ``max_new`` of one sequence, and
    at most ``max_len`` keys.  The bounds stay; the arrays may change in place."""

    def __init__(self, starts, lens, table, tokens, max_new, max_len):
        _rows("table", table)
        seqs = table.shape[0]
        _int32("starts", starts, (seqs + 1,))
        _int32("lens", lens, (seqs,))
        if not starts.device == lens.device == table.device:
            raise ValueError("starts, lens and table must be on one device")
        self.starts, self.lens, self.table, self.tokens = starts, lens, table, int(tokens)
        self.gpu = table.get_device()
        self._c = _PagedBatch(_ptr(starts), _ptr(lens), _ptr(table), table.stride(0), seqs,
                              self.tokens, table.shape[1], int(max_new), int(max_len))
        self._ref = ctypes.byref(self._c)


class PagePool:
    """The pages of a whole cache, ``data`` [planes, pages, ...] (each page
    dense), with ``refs`` [pages], ``table`` [slots, width] and ``lens`` [slots]
    (int32) for the calls that keep them; qmm_pages_copy needs the data alone."""

    def __init__(self, data, refs=None, table=None, lens=None, page_size=0):
        if data.dim() < 2 or (data.numel() and not data[0, 0].is_contiguous()):
            raise ValueError(f"data must be [planes, pages, ...] with dense pages, got "
                             f"{list(data.shape)} with strides {list(data.stride())}")
        size, slots, width, stride = data.element_size(), 0, 0, 0
        if refs is not None:
            _int32("refs", refs, (data.shape[1],))
            _rows("table", table)
            slots, width = table.shape
            stride = table.stride(0)
            _int32("lens", lens, (slots,))
            if not data.device == refs.device == table.device == lens.device:
                raise ValueError("data, refs, table and lens must be on one device")
        elems = 1
        for n in data.shape[2:]:
            elems *= n
        self.data, self.refs, self.table, self.lens = data, refs, table, lens
        self.page_size, self.gpu = int(page_size), data.get_device()
        self._c = _PagePool(_ptr(data), data.shape[0], data.shape[1], elems * size,
                            data.stride(0) * size, data.stride(1) * size, _ptr(refs), _ptr(table),
                            _ptr(lens), stride, slots, width, self.page_size)
        self._ref = ctypes.byref(self._c)


def _heads(name, t, shape, dtype):
    """The struct of rows of ``shape`` [tokens, heads, head_dim], with the checks
    that need the tensor's own."""
    strides = t.stride()
    if t.shape != shape or t.dtype is not dtype or (strides[2] != 1 and shape[2] > 1):
        raise ValueError(f"{name} must be {dtype} {list(shape)} with dense rows of head_dim, got "
                         f"{t.dtype} {list(t.shape)} with strides {list(strides)}")
    return _pack_heads(t.data_ptr(), strides[0], strides[1], shape[1])


def _rope_args(q, k, v, out, kv, batch, inv_freq, interleaved, factor, positions):
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be a dense float64 vector, got {inv_freq.dtype} "
                         f"{list(inv_freq.shape)}")
    if positions is not None:
        _int32("positions", positions, (batch.tokens,))
    dtype, gpu = kv.dtype, kv.gpu
    own, new = (batch.tokens, q.shape[1], kv.head_dim), (batch.tokens, kv.kv_heads, kv.head_dim)
    rows = (_heads("q", q, own, dtype), _heads("k", k, new, dtype), _heads("v", v, new, dtype),
            _heads("out", out, own, dtype))
    if (not 0 <= gpu == q.get_device() == k.get_device() == v.get_device() == out.get_device() == batch.gpu
            == inv_freq.get_device() or positions is not None and positions.get_device() != gpu):
        raise _elsewhere(gpu, q=q, k=k, v=v, out=out, batch=batch.table, inv_freq=inv_freq, positions=positions)
    return (*rows, kv._ref, batch._ref, inv_freq.data_ptr(), inv_freq.shape[0], interleaved,
            factor, None if positions is None else positions.data_ptr())


def qmm_rope_append(q, k, v, out, kv, batch, inv_freq, interleaved=False, factor=1.0,
                    positions=None, stream=None):
    """Turn q [tokens, heads, head_dim] into ``out`` and append the turned k and
    v [tokens, kv_heads, head_dim] to the cache ``kv``; ``inv_freq`` [half] is
    float64, ``positions`` [tokens] int32 or None (a token's key number)."""
    _check(lib.qmm_rope_append(*_rope_args(q, k, v, out, kv, batch, inv_freq, interleaved, factor,
                                           positions), _stream_at(kv.gpu, stream)))


def qmm_paged_attention_workspace_size(batch, q_heads, kv_heads, head_dim) -> int:
    """Bytes of the workspace; calls on one stream may share it."""
    return int(lib.qmm_paged_attention_workspace_size(batch._ref, q_heads, kv_heads, head_dim))


def _attention_args(q, kv, batch, out, workspace, scale, causal, window, softcap, lse):
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous()
                            or lse.shape != q.shape[:2]):
        raise ValueError(f"lse must be a dense float32 tensor {list(q.shape[:2])}, got {lse.dtype} "
                         f"{list(lse.shape)}")
    if scale is None:
        scale = kv.head_dim ** -0.5
    own, gpu = (batch.tokens, q.shape[1], kv.head_dim), kv.gpu
    q_rows, out_rows = _heads("q", q, own, kv.dtype), _heads("out", out, own, kv.dtype)
    if (not 0 <= gpu == q.get_device() == out.get_device() == batch.gpu == workspace.get_device()
            or lse is not None and lse.get_device() != gpu):
        raise _elsewhere(gpu, q=q, batch=batch.table, out=out, workspace=workspace, lse=lse)
    return (q_rows, kv._ref, batch._ref, out_rows, None if lse is None else lse.data_ptr(), scale,
            causal, window, softcap, workspace.data_ptr(), workspace.nbytes)


def qmm_paged_attention(q, kv, batch, out, workspace, scale=None, causal=True, window=0,
                        softcap=0.0, lse=None, stream=None):
    """Attention of q [tokens, heads, head_dim] over the cache, into ``out`` and,
    where given, ``lse`` [tokens, heads] float32; ``scale`` defaults to
    head_dim ** -0.5."""
    _check(lib.qmm_paged_attention(*_attention_args(q, kv, batch, out, workspace, scale, causal,
                                                    window, softcap, lse),
                                   _stream_at(kv.gpu, stream)))


def qmm_pages_workspace_size(pool, count=0) -> int:
    """Bytes of workspace for lists of ``count`` entries (0: a compaction)."""
    return int(lib.qmm_pages_workspace_size(pool._ref, count))


def _lists(pool, a_name, a, b_name=None, b=None, status=None, workspace=None):
    """Checks int32 lists of one length, the pair of status words and the
    workspace, all on the pool's GPU; the length."""
    _int32(a_name, a)
    n, gpu = a.numel(), pool.gpu
    if b is not None:
        _int32(b_name, b)
        if b.numel() != n:
            raise ValueError(f"{a_name} and {b_name} must have one length, got {n} and {b.numel()}")
    if status is not None:
        _int32("status", status, (2,))
    if (not 0 <= gpu == a.get_device() or b is not None and b.get_device() != gpu
            or status is not None and not gpu == status.get_device() == workspace.get_device()):
        raise _elsewhere(gpu, **{a_name: a, b_name or "": b}, status=status, workspace=workspace)
    return n


def qmm_pages_free(pool, seqs, stream=None):
    n = _lists(pool, "seqs", seqs)
    _check(lib.qmm_pages_free(pool._ref, seqs.data_ptr(), n, _stream_at(pool.gpu, stream)))


def qmm_pages_fork(pool, parents, children, status, workspace, stream=None):
    """``status`` [2] int32, zeroed by the caller, tells on the device whether
    the list was served (qmm_pages_status)."""
    n = _lists(pool, "parents", parents, "children", children, status, workspace)
    _check(lib.qmm_pages_fork(pool._ref, parents.data_ptr(), children.data_ptr(), n,
                              status.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                              _stream_at(pool.gpu, stream)))


def qmm_pages_reserve(pool, seqs, grow, status, workspace, stream=None):
    n = _lists(pool, "seqs", seqs, "grow", grow, status, workspace)
    _check(lib.qmm_pages_reserve(pool._ref, seqs.data_ptr(), grow.data_ptr(), n, status.data_ptr(),
                                 workspace.data_ptr(), workspace.nbytes, _stream_at(pool.gpu, stream)))


def qmm_pages_copy(pool, src, dst, stream=None):
    n = _lists(pool, "src", src, "dst", dst)
    _check(lib.qmm_pages_copy(pool._ref, src.data_ptr(), dst.data_ptr(), n, _stream_at(pool.gpu, stream)))


def qmm_pages_compact(pool, refs_out, table_out, live, workspace, stream=None):
    """``refs_out`` and ``table_out`` take the new counts and table, ``live`` [1]
    the number of used pages, now the first ones."""
    if pool.refs is not None:   # without tables the call itself refuses the pool
        _int32("refs_out", refs_out, pool.refs.shape)
        _int32("table_out", table_out, pool.table.shape)
        _int32("live", live)
    if (not 0 <= pool.gpu == refs_out.get_device() == table_out.get_device() == live.get_device()
            == workspace.get_device()):
        raise _elsewhere(pool.gpu, refs_out=refs_out, table_out=table_out, live=live, workspace=workspace)
    _check(lib.qmm_pages_compact(pool._ref, refs_out.data_ptr(), table_out.data_ptr(),
                                 live.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                                 _stream_at(pool.gpu, stream)))
