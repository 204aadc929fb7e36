"""Python binding of libmkp (run-time polymerized dense GEMM for MI355X).

Argument marshalling only: every step of the GEMM (plan lookup, the
polymerizer, every kernel) runs inside libmkp.so.  PyTorch is used only to
hand over device pointers and the current HIP stream.  If the library has not
been built this module raises on import: there is no fallback path.

Names follow the C-ABI in include/mkp.h: mkp_gemm(M,N,K,A,lda,B,ldb,C,ldc,
stream) and mkp_gemm_batched(...).
"""
from __future__ import annotations

import ctypes
import functools
import json
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmkp.so")

MKP_OK = 0
MKP_ERR_INVALID_ARG = -1
MKP_ERR_UNSUPPORTED = -2
MKP_ERR_OOM = -3
MKP_ERR_HIP = -4
MKP_ERR_BUFFER = -5
MKP_PLAN_EXHAUSTIVE = 1
MKP_PLAN_B_NK = 8
MKP_B_KN = 0
MKP_B_NK = 1
MKP_ACT_NONE = 0
MKP_ACT_RELU = 1
MKP_ACT_GELU = 2
MKP_ACT_GELU_TANH = 3
MKP_ACT_SILU = 4
MKP_BF16 = 0
MKP_F32 = 1
ACTIVATIONS = {None: MKP_ACT_NONE, "none": MKP_ACT_NONE, "relu": MKP_ACT_RELU, "gelu": MKP_ACT_GELU,
               "gelu_tanh": MKP_ACT_GELU_TANH, "silu": MKP_ACT_SILU}


class MkpError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"mkp error {code}: {msg}")
        self.code = code


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python dynamic_shape_gemm_amd/build.py`")

# One HIP runtime per process.  The PyTorch wheel carries its own copy of the
# HIP and HSA runtimes under the same soname as the system's; whichever is
# loaded first is the one libmkp binds to.  If libmkp came first, torch would
# load a second runtime beside it and libmkp's would find no device.  So
# torch, when installed, is loaded before the library.
try:
    import torch  # noqa: F401
except ImportError:
    pass

_lib = ctypes.CDLL(LIB_PATH)
_i64, _p, _int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
_lib.mkp_gemm.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
_lib.mkp_gemm.restype = _int
_lib.mkp_gemm_batched.argtypes = [_i64, _i64, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _p]
_lib.mkp_gemm_batched.restype = _int
_lib.mkp_gemm_batched_noalloc.argtypes = [_i64, _i64, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _p]
_lib.mkp_gemm_batched_noalloc.restype = _int
_lib.mkp_noalloc_scratch_bytes.argtypes = []
_lib.mkp_noalloc_scratch_bytes.restype = ctypes.c_size_t
_lib.mkp_gemm_bt.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p]
_lib.mkp_gemm_bt.restype = _int
_lib.mkp_gemm_batched_bt.argtypes = [_i64, _i64, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _p]
_lib.mkp_gemm_batched_bt.restype = _int
_lib.mkp_gemm_ex.argtypes = [_i64, _i64, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _int, _p, _i64, _i64,
                             ctypes.c_float, ctypes.c_float, _p, _int, _p]
_lib.mkp_gemm_ex.restype = _int
_lib.mkp_conv2d.argtypes = [_i64] * 13 + [_p, _p, _p, _p, _int, _p]
_lib.mkp_conv2d.restype = _int
_grp_args = [_i64, _i64, _i64, _p, _i64, _p, _p, _p, _p, _p, _p]
_lib.mkp_gemm_grouped.argtypes = _grp_args
_lib.mkp_gemm_grouped.restype = _int
_lib.mkp_gemm_grouped_bt.argtypes = _grp_args
_lib.mkp_gemm_grouped_bt.restype = _int
_f32 = ctypes.c_float
_xent_args = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _f32, _f32, _f32, _f32]
_lib.mkp_linear_xent.argtypes = _xent_args + [_p, _p, _p, _i64, _p]
_lib.mkp_linear_xent.restype = _int
_grad_args = [_p, _p, _p, _i64, _p, _i64, _p, _int, _p, _i64, _p]
_lib.mkp_linear_xent_backward.argtypes = _xent_args + _grad_args
_lib.mkp_linear_xent_backward.restype = _int
_distill_args = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _f32, _f32, _f32]
_lib.mkp_linear_distill.argtypes = _distill_args + [_p, _p, _p, _i64, _p]
_lib.mkp_linear_distill.restype = _int
_lib.mkp_linear_distill_backward.argtypes = _distill_args + _grad_args
_lib.mkp_linear_distill_backward.restype = _int
_lib.mkp_linear_loss_workspace.argtypes = [_i64, _i64, _i64, _i64, _p, _i64, _int, _p]
_lib.mkp_linear_loss_workspace.restype = _int
_lib.mkp_plan_describe_grouped.argtypes = [_i64, _i64, _i64, _p, _int, ctypes.c_char_p, ctypes.c_size_t]
_lib.mkp_plan_describe_grouped.restype = _int
_lib.mkp_plan_describe.argtypes = [_i64, _i64, _i64, _i64, _int, ctypes.c_char_p, ctypes.c_size_t]
_lib.mkp_plan_describe.restype = _int
_lib.mkp_plan_with_table.argtypes = [ctypes.c_char_p, _int, _i64, _i64, _i64, _i64, ctypes.c_char_p, ctypes.c_size_t]
_lib.mkp_plan_with_table.restype = _int
_lib.mkp_load_calibration.argtypes = [ctypes.c_char_p]
_lib.mkp_load_calibration.restype = _int
_lib.mkp_calibrate.argtypes = [ctypes.c_char_p, _int]
_lib.mkp_calibrate.restype = _int
_lib.mkp_set_option.argtypes = [ctypes.c_char_p, ctypes.c_char_p]
_lib.mkp_set_option.restype = _int
_lib.mkp_kernel_count.argtypes = []
_lib.mkp_kernel_count.restype = _int
_lib.mkp_kernel_name.argtypes = [_int]
_lib.mkp_kernel_name.restype = ctypes.c_char_p
_lib.mkp_cache_clear.argtypes = []
_lib.mkp_cache_clear.restype = None
_lib.mkp_stats.argtypes = [ctypes.c_char_p, ctypes.c_size_t]
_lib.mkp_stats.restype = _int
_lib.mkp_trace_dump.argtypes = [ctypes.c_char_p, ctypes.c_size_t]
_lib.mkp_trace_dump.restype = _int
_lib.mkp_last_error.argtypes = []
_lib.mkp_last_error.restype = ctypes.c_char_p

# The GEMM and loss entry points through the CPython marshalling module built beside
# the library (a ctypes call spends ~1.5 us converting 10-14 arguments, as
# long as the smallest GEMMs take on the GPU); ctypes where it is absent.
try:
    from . import _mkpfast as _fast
except ImportError:
    _fast = None
_f_gemm = _fast.gemm if _fast else _lib.mkp_gemm
_f_gemm_bt = _fast.gemm_bt if _fast else _lib.mkp_gemm_bt
_f_gemm_batched = _fast.gemm_batched if _fast else _lib.mkp_gemm_batched
_f_gemm_batched_bt = _fast.gemm_batched_bt if _fast else _lib.mkp_gemm_batched_bt
_f_linear_xent = _fast.linear_xent if _fast else _lib.mkp_linear_xent
_f_linear_xent_backward = _fast.linear_xent_backward if _fast else _lib.mkp_linear_xent_backward
_f_linear_distill = _fast.linear_distill if _fast else _lib.mkp_linear_distill
_f_linear_distill_backward = _fast.linear_distill_backward if _fast else _lib.mkp_linear_distill_backward

EXPORTED = ["mkp_gemm", "mkp_gemm_batched", "mkp_gemm_batched_noalloc", "mkp_noalloc_scratch_bytes", "mkp_gemm_bt", "mkp_gemm_batched_bt", "mkp_gemm_ex", "mkp_conv2d", "mkp_gemm_grouped",
            "mkp_gemm_grouped_bt", "mkp_linear_xent", "mkp_linear_xent_backward", "mkp_linear_distill",
            "mkp_linear_distill_backward", "mkp_linear_loss_workspace", "mkp_plan_describe", "mkp_plan_describe_grouped", "mkp_plan_with_table",
            "mkp_load_calibration",
            "mkp_calibrate", "mkp_set_option", "mkp_kernel_count", "mkp_kernel_name", "mkp_cache_clear",
            "mkp_stats", "mkp_trace_dump", "mkp_last_error"]


def last_error() -> str:
    return (_lib.mkp_last_error() or b"").decode()


def _check(rc: int) -> int:
    if rc != MKP_OK:
        raise MkpError(rc, last_error())
    return rc


def _addr(x) -> int:
    """Device address of a torch tensor, or an int address as given."""
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def mkp_gemm(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> int:
    """C[MxN] := A[MxK] . B[KxN] (bf16 in, fp32 out), enqueued on `stream`
    (default: torch's current stream).  Raises MkpError on a bad argument."""
    return _check(_f_gemm(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc, _stream(stream)))


def mkp_gemm_batched(batch, M, N, K, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, stream=None) -> int:
    return _check(_f_gemm_batched(batch, M, N, K, _addr(A), lda, strideA, _addr(B), ldb, strideB, _addr(C),
                                  ldc, strideC, _stream(stream)))


def mkp_gemm_batched_noalloc(batch, M, N, K, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, stream=None) -> int:
    """mkp_gemm_batched without any device allocation: its scratch is the
    library's fixed per-GPU array (calls that overlap on one GPU race)."""
    return _check(_lib.mkp_gemm_batched_noalloc(batch, M, N, K, _addr(A), lda, strideA, _addr(B), ldb, strideB,
                                                _addr(C), ldc, strideC, _stream(stream)))


def mkp_noalloc_scratch_bytes() -> int:
    return int(_lib.mkp_noalloc_scratch_bytes())


def mkp_gemm_raw(M, N, K, A, lda, B, ldb, C, ldc, stream) -> int:
    """As mkp_gemm but returns the status code instead of raising."""
    return _f_gemm(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc, stream or 0)


def mkp_gemm_batched_raw(batch, M, N, K, A, lda, sA, B, ldb, sB, C, ldc, sC, stream) -> int:
    return _f_gemm_batched(batch, M, N, K, _addr(A), lda, sA, _addr(B), ldb, sB, _addr(C), ldc, sC, stream or 0)


def mkp_gemm_bt(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> int:
    """C[MxN] := A[MxK] . B^T with B given as N x K (ldb >= K)."""
    return _check(_f_gemm_bt(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc, _stream(stream)))


def mkp_gemm_batched_bt(batch, M, N, K, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, stream=None) -> int:
    return _check(_f_gemm_batched_bt(batch, M, N, K, _addr(A), lda, strideA, _addr(B), ldb, strideB,
                                     _addr(C), ldc, strideC, _stream(stream)))


def mkp_gemm_bt_raw(M, N, K, A, lda, B, ldb, C, ldc, stream) -> int:
    return _f_gemm_bt(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc, stream or 0)


def mkp_gemm_batched_bt_raw(batch, M, N, K, A, lda, sA, B, ldb, sB, C, ldc, sC, stream) -> int:
    return _f_gemm_batched_bt(batch, M, N, K, _addr(A), lda, sA, _addr(B), ldb, sB, _addr(C), ldc, sC,
                              stream or 0)


def mkp_gemm_ex(batch, M, N, K, A, lda, strideA, B, ldb, strideB, b_layout, C, ldc, strideC,
                alpha=1.0, beta=0.0, bias=None, act=MKP_ACT_NONE, stream=None) -> int:
    """C_b := act(alpha * A_b . op(B_b) + beta * C_b + bias) with op(B) = B
    (b_layout MKP_B_KN) or B^T (MKP_B_NK); act an MKP_ACT_* code or name."""
    return _check(mkp_gemm_ex_raw(batch, M, N, K, A, lda, strideA, B, ldb, strideB, b_layout, C, ldc, strideC,
                                  alpha, beta, bias, act, _stream(stream)))


def mkp_gemm_ex_raw(batch, M, N, K, A, lda, strideA, B, ldb, strideB, b_layout, C, ldc, strideC,
                    alpha, beta, bias, act, stream) -> int:
    if not isinstance(act, int):
        act = ACTIVATIONS[act]
    return _lib.mkp_gemm_ex(batch, M, N, K, _addr(A), lda, strideA, _addr(B), ldb, strideB, b_layout, _addr(C), ldc,
                            strideC, alpha, beta, _addr(bias), act, stream or 0)


def mkp_conv2d_raw(N, H, W, C, K, R, S, stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, x, w, y, bias=None,
                   act=MKP_ACT_NONE, stream=0) -> int:
    if not isinstance(act, int):
        act = ACTIVATIONS[act]
    return _lib.mkp_conv2d(N, H, W, C, K, R, S, stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, _addr(x), _addr(w),
                           _addr(y), _addr(bias), act, stream or 0)


def mkp_conv2d(N, H, W, C, K, R, S, stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, x, w, y, bias=None,
               act=MKP_ACT_NONE, stream=None) -> int:
    """y (N,P,Q,K) fp32 := act(conv2d(x (N,H,W,C) bf16, w (K,R,S,C) bf16) + bias)."""
    return _check(mkp_conv2d_raw(N, H, W, C, K, R, S, stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, x, w, y,
                                 bias, act, _stream(stream)))


def conv_out_size(H, R, stride, pad, dil):
    return (H + 2 * pad - dil * (R - 1) - 1) // stride + 1


def _i64_array(values):
    return (ctypes.c_int64 * max(len(values), 1))(*[int(v) for v in values])


def _ptr_array(values):
    return (ctypes.c_void_p * max(len(values), 1))(*[_addr(v) for v in values])


def _grouped_call(fn, M, K, A, lda, N, B, ldb, C, ldc, stream):
    g = len(N)
    if not (len(B) == len(ldb) == len(C) == len(ldc) == g):
        raise ValueError("N, B, ldb, C and ldc must have one entry per group")
    return fn(g, M, K, _addr(A), lda, ctypes.cast(_i64_array(N), _p), ctypes.cast(_ptr_array(B), _p),
              ctypes.cast(_i64_array(ldb), _p), ctypes.cast(_ptr_array(C), _p), ctypes.cast(_i64_array(ldc), _p),
              stream)


def mkp_gemm_grouped(M, K, A, lda, N, B, ldb, C, ldc, stream=None) -> int:
    """C[g][M x N[g]] := A[M x K] . B[g] (B[g] K x N[g]) for every group, in
    one launch.  N, B, ldb, C, ldc are sequences with one entry per group."""
    return _check(_grouped_call(_lib.mkp_gemm_grouped, M, K, A, lda, N, B, ldb, C, ldc, _stream(stream)))


def mkp_gemm_grouped_bt(M, K, A, lda, N, B, ldb, C, ldc, stream=None) -> int:
    """As mkp_gemm_grouped with each B[g] given as N[g] x K (ldb[g] >= K)."""
    return _check(_grouped_call(_lib.mkp_gemm_grouped_bt, M, K, A, lda, N, B, ldb, C, ldc, _stream(stream)))


def mkp_gemm_grouped_raw(M, K, A, lda, N, B, ldb, C, ldc, stream, bt=False) -> int:
    fn = _lib.mkp_gemm_grouped_bt if bt else _lib.mkp_gemm_grouped
    return _grouped_call(fn, M, K, A, lda, N, B, ldb, C, ldc, stream or 0)


def mkp_plan_describe_grouped(M, K, N, bt=False) -> dict:
    return json.loads(_text_call(_lib.mkp_plan_describe_grouped, len(N), M, K,
                                 ctypes.cast(_i64_array(N), _p), MKP_PLAN_B_NK if bt else 0))


def mkp_linear_xent_raw(M, V, K, X, ldx, W, ldw, bias, labels, scale, softcap, smoothing, z_loss, loss, lse,
                        workspace, workspace_bytes, stream) -> int:
    return _f_linear_xent(M, V, K, _addr(X), ldx, _addr(W), ldw, _addr(bias), _addr(labels), scale, softcap,
                          smoothing, z_loss, _addr(loss), _addr(lse), _addr(workspace), workspace_bytes,
                          stream or 0)


def mkp_linear_xent(M, V, K, X, ldx, W, ldw, bias, labels, scale, softcap, smoothing, z_loss, loss, lse,
                    workspace, workspace_bytes, stream=None) -> int:
    """loss[m], lse[m] := cross entropy of labels[m] (int64) with the logits
    scale X . W^T + bias (X M x K, W V x K, bf16), which are not stored."""
    return _check(mkp_linear_xent_raw(M, V, K, X, ldx, W, ldw, bias, labels, scale, softcap, smoothing, z_loss, loss,
                                      lse, workspace, workspace_bytes, _stream(stream)))


def mkp_linear_xent_backward_raw(M, V, K, X, ldx, W, ldw, bias, labels, scale, softcap, smoothing, z_loss, lse, dloss,
                                 dX, lddx, dW, lddw, dbias, grad_type, workspace, workspace_bytes, stream) -> int:
    return _f_linear_xent_backward(M, V, K, _addr(X), ldx, _addr(W), ldw, _addr(bias), _addr(labels), scale,
                                   softcap, smoothing, z_loss, _addr(lse), _addr(dloss), _addr(dX), lddx,
                                   _addr(dW), lddw, _addr(dbias), grad_type, _addr(workspace), workspace_bytes,
                                   stream or 0)


def mkp_linear_xent_backward(M, V, K, X, ldx, W, ldw, bias, labels, scale, softcap, smoothing, z_loss, lse, dloss,
                             dX, lddx, dW, lddw, dbias, grad_type, workspace, workspace_bytes, stream=None) -> int:
    """dX, dW, dbias (each may be None) := the gradients of
    sum_m dloss[m] loss[m]; lse as mkp_linear_xent wrote it."""
    return _check(mkp_linear_xent_backward_raw(M, V, K, X, ldx, W, ldw, bias, labels, scale, softcap, smoothing, z_loss,
                                               lse, dloss, dX, lddx, dW, lddw, dbias, grad_type, workspace,
                                               workspace_bytes, _stream(stream)))


def mkp_linear_distill_raw(M, V, K, X, ldx, W, ldw, bias, k, ids, ldids, teacher, ldt, teacher_lse, temperature, scale,
                           softcap, loss, lse, workspace, workspace_bytes, stream) -> int:
    return _f_linear_distill(M, V, K, _addr(X), ldx, _addr(W), ldw, _addr(bias), k, _addr(ids), ldids,
                             _addr(teacher), ldt, _addr(teacher_lse), temperature, scale, softcap, _addr(loss),
                             _addr(lse), _addr(workspace), workspace_bytes, stream or 0)


def mkp_linear_distill(M, V, K, X, ldx, W, ldw, bias, k, ids, ldids, teacher, ldt, teacher_lse, temperature, scale,
                       softcap, loss, lse, workspace, workspace_bytes, stream=None) -> int:
    """loss[m] := T^2 KL(teacher || softmax((scale X . W^T + bias) / T)), the
    teacher known by k logits (fp32) at vocabulary entries ids (int64) a row."""
    return _check(mkp_linear_distill_raw(M, V, K, X, ldx, W, ldw, bias, k, ids, ldids, teacher, ldt, teacher_lse,
                                         temperature, scale, softcap, loss, lse, workspace, workspace_bytes,
                                         _stream(stream)))


def mkp_linear_distill_backward_raw(M, V, K, X, ldx, W, ldw, bias, k, ids, ldids, teacher, ldt, teacher_lse,
                                    temperature, scale, softcap, lse, dloss, dX, lddx, dW, lddw, dbias, grad_type,
                                    workspace, workspace_bytes, stream) -> int:
    return _f_linear_distill_backward(M, V, K, _addr(X), ldx, _addr(W), ldw, _addr(bias), k, _addr(ids), ldids,
                                      _addr(teacher), ldt, _addr(teacher_lse), temperature, scale, softcap,
                                      _addr(lse), _addr(dloss), _addr(dX), lddx, _addr(dW), lddw, _addr(dbias),
                                      grad_type, _addr(workspace), workspace_bytes, stream or 0)


def mkp_linear_distill_backward(M, V, K, X, ldx, W, ldw, bias, k, ids, ldids, teacher, ldt, teacher_lse, temperature,
                                scale, softcap, lse, dloss, dX, lddx, dW, lddw, dbias, grad_type, workspace,
                                workspace_bytes, stream=None) -> int:
    """The gradients of sum_m dloss[m] loss[m] of mkp_linear_distill."""
    return _check(mkp_linear_distill_backward_raw(M, V, K, X, ldx, W, ldw, bias, k, ids, ldids, teacher, ldt,
                                                  teacher_lse, temperature, scale, softcap, lse, dloss, dX, lddx, dW,
                                                  lddw, dbias, grad_type, workspace, workspace_bytes,
                                                  _stream(stream)))


def mkp_linear_loss_workspace(M, V, K, k, W, ldw, backward) -> int:
    """Bytes of workspace the vocabulary losses need (k = 0: cross entropy)."""
    n = ctypes.c_int64(0)
    _check(_lib.mkp_linear_loss_workspace(M, V, K, k, _addr(W), ldw, 1 if backward else 0, ctypes.byref(n)))
    return n.value


def _text_call(fn, *args, size=1 << 16):
    buf = ctypes.create_string_buffer(size)
    _check(fn(*args, buf, size))
    return buf.value.decode()


def mkp_plan_describe(batch, M, N, K, align_flags=7, bt=False) -> dict:
    return json.loads(_text_call(_lib.mkp_plan_describe, batch, M, N, K,
                                 align_flags | (MKP_PLAN_B_NK if bt else 0)))


def mkp_plan_with_table(table_text: str, batch, M, N, K, exhaustive=False, bt=False) -> dict:
    flags = (MKP_PLAN_EXHAUSTIVE if exhaustive else 0) | (MKP_PLAN_B_NK if bt else 0)
    return json.loads(_text_call(_lib.mkp_plan_with_table, table_text.encode(), flags, batch, M, N, K))


def mkp_load_calibration(path=None) -> int:
    return _check(_lib.mkp_load_calibration(path.encode() if path else None))


def mkp_calibrate(path: str, max_points: int = 0) -> int:
    return _check(_lib.mkp_calibrate(path.encode(), max_points))


def mkp_set_option(key: str, value) -> int:
    return _check(_lib.mkp_set_option(key.encode(), str(value).encode()))


def mkp_kernel_names() -> list:
    return [_lib.mkp_kernel_name(i).decode() for i in range(_lib.mkp_kernel_count())]


def mkp_cache_clear() -> None:
    _lib.mkp_cache_clear()


def mkp_stats() -> dict:
    return json.loads(_text_call(_lib.mkp_stats))


def mkp_trace_dump() -> list:
    return json.loads(_text_call(_lib.mkp_trace_dump, size=1 << 24))


def gemm(a, b, out=None, stream=None):
    """torch convenience: a (M,K) bf16, b (K,N) bf16 on the GPU, any strides
    with unit column stride; returns (or fills) out (M,N) fp32."""
    import torch
    if a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16:
        raise TypeError("a and b must be bfloat16")
    if a.stride(1) != 1 or b.stride(1) != 1:
        raise ValueError("rows must be contiguous (unit column stride)")
    M, K = a.shape
    K2, N = b.shape
    if K2 != K:
        raise ValueError("inner dimensions differ")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=a.device)
    if out.stride(1) != 1:
        raise ValueError("out rows must be contiguous")
    mkp_gemm(M, N, K, a, max(a.stride(0), 1), b, max(b.stride(0), 1), out, max(out.stride(0), 1), stream)
    return out


def gemm_batched(a, b, out=None, stream=None):
    """torch convenience: a (batch,M,K), b (batch,K,N) bf16 -> out (batch,M,N) fp32."""
    import torch
    batch, M, K = a.shape
    N = b.shape[2]
    if out is None:
        out = torch.empty((batch, M, N), dtype=torch.float32, device=a.device)
    mkp_gemm_batched(batch, M, N, K, a, max(a.stride(1), 1), a.stride(0), b, max(b.stride(1), 1), b.stride(0),
                     out, max(out.stride(1), 1), out.stride(0), stream)
    return out


def gemm_bt(a, w, out=None, stream=None):
    """torch convenience: a (M,K) bf16 and w (N,K) bf16 (a linear layer's
    weight) on the GPU, unit column strides; returns (or fills) out = a . w^T
    (M,N) fp32."""
    import torch
    if a.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise TypeError("a and w must be bfloat16")
    if a.stride(1) != 1 or w.stride(1) != 1:
        raise ValueError("rows must be contiguous (unit column stride)")
    M, K = a.shape
    N, K2 = w.shape
    if K2 != K:
        raise ValueError("inner dimensions differ")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=a.device)
    if out.stride(1) != 1:
        raise ValueError("out rows must be contiguous")
    mkp_gemm_bt(M, N, K, a, max(a.stride(0), 1), w, max(w.stride(0), 1), out, max(out.stride(0), 1), stream)
    return out


def gemm_grouped(a, ws, outs=None, stream=None, bt=False):
    """torch convenience: one A (M,K) bf16 against several weights in one
    launch.  ws: list of (K,N_g) bf16 tensors, or (N_g,K) with bt=True.
    Returns (or fills) the list of (M,N_g) fp32 outputs."""
    import torch
    if a.dtype != torch.bfloat16 or any(w.dtype != torch.bfloat16 for w in ws):
        raise TypeError("a and the weights must be bfloat16")
    if a.stride(1) != 1 or any(w.stride(1) != 1 for w in ws):
        raise ValueError("rows must be contiguous (unit column stride)")
    M, K = a.shape
    Ns = [w.shape[0] if bt else w.shape[1] for w in ws]
    if any((w.shape[1] if bt else w.shape[0]) != K for w in ws):
        raise ValueError("inner dimensions differ")
    if outs is None:
        outs = [torch.empty((M, n), dtype=torch.float32, device=a.device) for n in Ns]
    if any(o.stride(1) != 1 for o in outs):
        raise ValueError("out rows must be contiguous")
    fn = mkp_gemm_grouped_bt if bt else mkp_gemm_grouped
    fn(M, K, a, max(a.stride(0), 1), Ns, ws, [max(w.stride(0), 1) for w in ws], outs,
       [max(o.stride(0), 1) for o in outs], stream)
    return outs


def linear(a, w, bias=None, act=None, out=None, beta=0.0, stream=None):
    """torch convenience for a linear layer: out = act(a . w^T + bias (+ beta
    * out)), a (M,K) bf16, w (N,K) bf16 (the layer's weight), bias (N,) fp32
    or None, act None/"relu"/"gelu"/"gelu_tanh"/"silu"; all in one launch
    sequence of the library (the epilogue runs inside the GEMM)."""
    import torch
    if a.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise TypeError("a and w must be bfloat16")
    if bias is not None and (bias.dtype != torch.float32 or bias.stride(0) != 1):
        raise TypeError("bias must be a contiguous float32 vector")
    if a.stride(1) != 1 or w.stride(1) != 1:
        raise ValueError("rows must be contiguous (unit column stride)")
    M, K = a.shape
    N, K2 = w.shape
    if K2 != K or (bias is not None and bias.shape[0] != N):
        raise ValueError("shapes differ")
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs out")
        out = torch.empty((M, N), dtype=torch.float32, device=a.device)
    if out.stride(1) != 1:
        raise ValueError("out rows must be contiguous")
    mkp_gemm_ex(1, M, N, K, a, max(a.stride(0), 1), 0, w, max(w.stride(0), 1), 0, MKP_B_NK, out,
                max(out.stride(0), 1), 0, 1.0, beta, bias, act, stream)
    return out


def conv2d(x, w, bias=None, act=None, stride=1, padding=0, dilation=1, out=None, stream=None):
    """torch convenience: x (N,H,W,C) bf16 NHWC, w (K,R,S,C) bf16, contiguous;
    returns (or fills) y (N,P,Q,K) fp32 = act(conv2d(x, w) + bias)."""
    import torch
    sh, sw = (stride, stride) if isinstance(stride, int) else stride
    ph, pw = (padding, padding) if isinstance(padding, int) else padding
    dh, dw = (dilation, dilation) if isinstance(dilation, int) else dilation
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise TypeError("x and w must be bfloat16")
    if not x.is_contiguous() or not w.is_contiguous():
        raise ValueError("x and w must be contiguous (NHWC and KRSC)")
    N, H, W, C = x.shape
    K, R, S, C2 = w.shape
    if C2 != C:
        raise ValueError("channel counts differ")
    P, Q = conv_out_size(H, R, sh, ph, dh), conv_out_size(W, S, sw, pw, dw)
    if out is None:
        out = torch.empty((N, P, Q, K), dtype=torch.float32, device=x.device)
    mkp_conv2d(N, H, W, C, K, R, S, sh, sw, ph, pw, dh, dw, x, w, out, bias, act, stream)
    return out


def _loss_inputs(x, w, bias, rows):
    """Checks shared by the vocabulary losses; (M, V, K, ldx, ldw).  rows:
    name -> (tensor or None, dtype, shape)."""
    import torch
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise TypeError("x and w must be bfloat16")
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be (M, K) and w (V, K)")
    M, K = x.shape
    V = w.shape[0]
    if (x.stride(1) != 1 and K > 1) or (w.stride(1) != 1 and K > 1):
        raise ValueError("rows must be contiguous (unit column stride)")
    every = dict(rows, bias=(bias, torch.float32, (V,)), w=(w, w.dtype, tuple(w.shape)), x=(x, x.dtype, tuple(x.shape)))
    every = {name: e for name, e in every.items() if e[0] is not None}
    for name, (t, dtype, shape) in every.items():
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {str(dtype).split('.')[-1]}")
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}")
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must be contiguous along its last axis")
    for name, (t, _, _) in every.items():
        if t.device != x.device or t.device.type != "cuda":
            raise ValueError(f"{name} must be on x's GPU")
    return M, V, K, (x.stride(0) if M > 1 else K), (w.stride(0) if V > 1 else K)


class _LossStream:
    """The stream a vocabulary loss runs on, made current (with its device)
    while the call's outputs and workspace are taken from torch's allocator,
    so that they belong to it.  On another stream than the current one the
    inputs are marked as used there: their memory is not handed out again
    before the call is done with it."""

    def __init__(self, device, stream, *inputs):
        import torch
        current = torch.cuda.current_stream(device)
        if stream is None:
            self.stream = current
        elif isinstance(stream, int):
            self.stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                           else torch.cuda.default_stream(device))
        else:
            self.stream = stream
        if self.stream.device != device:
            raise ValueError("the stream is on another device than x")
        self.handle = self.stream.cuda_stream
        if self.handle != current.cuda_stream:
            for t in inputs:
                if t is not None:
                    t.record_stream(self.stream)
        here = torch.cuda.current_device() == device.index
        self.ctx = None if stream is None and here else torch.cuda.stream(self.stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        return False


# (the size goes by the extents and the weight's alignment alone)
_loss_workspace_bytes = functools.lru_cache(maxsize=1024)(mkp_linear_loss_workspace)


def _loss_workspace(M, V, K, k, w, ldw, backward):
    import torch
    n = _loss_workspace_bytes(M, V, K, k, w.data_ptr() & 15, ldw, backward)
    return torch.empty(n, dtype=torch.uint8, device=w.device), n


def _loss_grads(x, w, bias, need_dx, need_dw, need_dbias, grad_dtype):
    import torch
    if grad_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("grad_dtype must be bfloat16 or float32")
    if need_dbias is None:
        need_dbias = bias is not None
    dx = torch.empty(x.shape, dtype=grad_dtype, device=x.device) if need_dx else None
    dw = torch.empty(w.shape, dtype=grad_dtype, device=x.device) if need_dw else None
    dbias = torch.empty(w.shape[0], dtype=torch.float32, device=x.device) if need_dbias else None
    return dx, dw, dbias, MKP_F32 if grad_dtype == torch.float32 else MKP_BF16


def linear_xent(x, w, labels, bias=None, scale=1.0, softcap=0.0, smoothing=0.0, z_loss=0.0, stream=None):
    """Cross entropy of each row's label with the logits of a linear layer,
    which are not stored: x (M,K) bf16, w (V,K) bf16, labels (M,) int64, bias
    (V,) fp32 or None.  Returns (loss, lse), fp32 (M,); rows whose label is not
    in [0, V) get 0.  The mean over the others is loss.sum() / their number.
    Neither has a grad_fn: gradients come from linear_xent_backward."""
    import torch
    M, V, K, ldx, ldw = _loss_inputs(x, w, bias, {"labels": (labels, torch.int64, (x.shape[0],))})
    with _LossStream(x.device, stream, x, w, labels, bias) as st:
        loss = torch.empty((2, M), dtype=torch.float32, device=x.device)
        loss, lse = loss[0], loss[1]
        ws, n = _loss_workspace(M, V, K, 0, w, ldw, False)
        mkp_linear_xent(M, V, K, x, ldx, w, ldw, bias, labels, scale, softcap, smoothing, z_loss, loss, lse, ws, n, st)
    return loss, lse


def linear_xent_backward(x, w, labels, lse, dloss, bias=None, scale=1.0, softcap=0.0, smoothing=0.0, z_loss=0.0,
                         need_dx=True, need_dw=True, need_dbias=None, grad_dtype=None, stream=None):
    """Gradients of (dloss * loss).sum() for linear_xent's loss: (dx, dw,
    dbias), dx and dw in grad_dtype (bfloat16, the default, or float32), dbias
    fp32 (by default made when there is a bias); None for those not needed.
    lse is linear_xent's; dloss (M,) fp32."""
    import torch
    M = x.shape[0]
    M, V, K, ldx, ldw = _loss_inputs(x, w, bias, {"labels": (labels, torch.int64, (M,)),
                                                  "lse": (lse, torch.float32, (M,))})
    with _LossStream(x.device, stream, x, w, labels, bias, lse, dloss) as st:
        dloss = dloss.contiguous()   # a broadcast scalar has no stride
        _loss_inputs(x, w, None, {"dloss": (dloss, torch.float32, (M,))})
        dx, dw, dbias, gt = _loss_grads(x, w, bias, need_dx, need_dw, need_dbias, grad_dtype or torch.bfloat16)
        ws, n = _loss_workspace(M, V, K, 0, w, ldw, True)
        mkp_linear_xent_backward(M, V, K, x, ldx, w, ldw, bias, labels, scale, softcap, smoothing, z_loss, lse, dloss,
                                 dx, K, dw, K, dbias, gt, ws, n, st)
    return dx, dw, dbias


def _distill_inputs(x, w, bias, ids, teacher, teacher_lse, **rows):
    import torch
    M = x.shape[0]
    k = ids.shape[1] if ids.dim() == 2 else 0
    rows = {name: (t, torch.float32, (M,)) for name, t in rows.items()}
    rows.update(ids=(ids, torch.int64, (M, k)), teacher=(teacher, torch.float32, (M, k)),
                teacher_lse=(teacher_lse, torch.float32, (M,)))
    if k < 1:
        raise ValueError("ids must be (M, k) with k >= 1")
    sizes = _loss_inputs(x, w, bias, rows)
    return sizes + (k, ids.stride(0) if M > 1 else k, teacher.stride(0) if M > 1 else k)


def linear_distill(x, w, ids, teacher, bias=None, temperature=1.0, scale=1.0, softcap=0.0, teacher_lse=None,
                   stream=None):
    """T^2 times the Kullback-Leibler divergence of a linear layer's softmax
    (at temperature T) from a teacher known by its k top logits: x (M,K) bf16,
    w (V,K) bf16, ids (M,k) int64 (entries outside [0, V) are left out),
    teacher (M,k) fp32, teacher_lse (M,) fp32 or None (then the teacher's
    probabilities are normalised over the k).  Returns (loss, lse), fp32 (M,),
    without a grad_fn: gradients come from linear_distill_backward."""
    import torch
    M, V, K, ldx, ldw, k, ldi, ldt = _distill_inputs(x, w, bias, ids, teacher, teacher_lse)
    with _LossStream(x.device, stream, x, w, ids, teacher, bias, teacher_lse) as st:
        loss = torch.empty((2, M), dtype=torch.float32, device=x.device)
        loss, lse = loss[0], loss[1]
        ws, n = _loss_workspace(M, V, K, k, w, ldw, False)
        mkp_linear_distill(M, V, K, x, ldx, w, ldw, bias, k, ids, ldi, teacher, ldt, teacher_lse, temperature, scale,
                           softcap, loss, lse, ws, n, st)
    return loss, lse


def linear_distill_backward(x, w, ids, teacher, lse, dloss, bias=None, temperature=1.0, scale=1.0, softcap=0.0,
                            teacher_lse=None, need_dx=True, need_dw=True, need_dbias=None, grad_dtype=None,
                            stream=None):
    """Gradients of (dloss * loss).sum() for linear_distill's loss, as
    linear_xent_backward gives them."""
    import torch
    M, V, K, ldx, ldw, k, ldi, ldt = _distill_inputs(x, w, bias, ids, teacher, teacher_lse, lse=lse)
    with _LossStream(x.device, stream, x, w, ids, teacher, bias, teacher_lse, lse, dloss) as st:
        dloss = dloss.contiguous()   # a broadcast scalar has no stride
        _loss_inputs(x, w, None, {"dloss": (dloss, torch.float32, (M,))})
        dx, dw, dbias, gt = _loss_grads(x, w, bias, need_dx, need_dw, need_dbias, grad_dtype or torch.bfloat16)
        ws, n = _loss_workspace(M, V, K, k, w, ldw, True)
        mkp_linear_distill_backward(M, V, K, x, ldx, w, ldw, bias, k, ids, ldi, teacher, ldt, teacher_lse, temperature,
                                    scale, softcap, lse, dloss, dx, K, dw, K, dbias, gt, ws, n, st)
    return dx, dw, dbias
