"""Python binding of libqa -- quantized linear layers on AMD MI355X (gfx950).

A thin ctypes layer over the C ABI of ``include/qa.h``: every function has the
name of the C entry point it calls, takes torch tensors that live on the GPU,
allocates the outputs it returns, passes raw device pointers and the current
HIP stream, and raises ``QAError`` on a non-zero status.  All arithmetic runs
in the HIP kernels of ``libqa.so``; there is no fallback path.  If the library
is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqa.so")

QA_F32, QA_F16, QA_BF16 = 0, 1, 2
QA_SCALE_PER_ROW, QA_SCALE_PER_GROUP, QA_SCALE_PER_TENSOR = 0, 1, 2
QA_SMOOTH_DIVIDE, QA_SMOOTH_MULTIPLY = 0, 1
QA_SCORE_SOFTMAX, QA_SCORE_SIGMOID = 0, 1
QA_ACT_NONE, QA_ACT_RELU, QA_ACT_GELU, QA_ACT_GELU_TANH, QA_ACT_SILU = 0, 1, 2, 3, 4

EXPORTS = (
    "qa_status_string", "qa_last_error",
    "qa_outlier_cols_workspace", "qa_outlier_cols", "qa_outlier_topk",
    "qa_quantize_rowwise_int8",
    "qa_qlinear_int8_mixed_workspace", "qa_qlinear_int8_mixed", "qa_qlinear_int8_mixed_offsets",
    "qa_qlinear_int8_mixed_noalloc",
    "qa_qlinear_int8_topk_workspace", "qa_qlinear_int8_topk",
    "qa_quantize_rowwise_int8_asym", "qa_int8_row_sums", "qa_qlinear_int8_asym_workspace", "qa_qlinear_int8_asym",
    "qa_col_absmax_workspace", "qa_col_absmax", "qa_smooth_factors", "qa_quantize_smooth_int8",
    "qa_qlinear_int8_smooth_workspace", "qa_qlinear_int8_smooth",
    "qa_hadamard_quant_int4", "qa_kron_sizes", "qa_kron_quant_int4", "qa_qlinear_kron_w4a4_workspace",
    "qa_qlinear_kron_w4a4",
    "qa_qlinear_w4a4_workspace", "qa_qlinear_w4a4",
    "qa_hadamard_quant_int8", "qa_qlinear_w4a8_workspace", "qa_qlinear_w4a8",
    "qa_hadamard_quant_int4_asym", "qa_w4_column_terms", "qa_qlinear_w4a4_asym_workspace", "qa_qlinear_w4a4_asym",
    "qa_gemm_i8_i32", "qa_gemm_w4a4_group_acc", "qa_gemm_w4a8_group_acc",
    "qa_rmsnorm_int8", "qa_route_experts_workspace", "qa_route_experts", "qa_experts_int8_workspace",
    "qa_experts_int8", "qa_qlinear_int8_lora_workspace", "qa_qlinear_int8_lora",
    "qa_kv_write", "qa_kv_read", "qa_attn_decode_workspace", "qa_attn_decode", "qa_qlinear_int8_act",
    "qa_probe_stream_read",
)

_DTYPE_CODE = {torch.float32: QA_F32, torch.float16: QA_F16, torch.bfloat16: QA_BF16}


class QAError(RuntimeError):
    def __init__(self, fn, status, detail):
        super().__init__("%s failed: %s (%s)" % (fn, status, detail))
        self.status = status
        self.detail = detail


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libqa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libqa.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        S = ctypes.c_int
        sig = {
            "qa_status_string": (ctypes.c_char_p, [S]),
            "qa_last_error": (ctypes.c_char_p, []),
            "qa_outlier_cols_workspace": (SZ, [I64]),
            "qa_outlier_cols": (S, [P, I64, I64, F, P, P, P, P, P, SZ, P]),
            "qa_outlier_topk": (S, [P, I64, I64, I64, P, P, P, P, P, SZ, P]),
            "qa_qlinear_int8_topk_workspace": (SZ, [I64, I64]),
            "qa_qlinear_int8_topk": (S, [P, I64, I64, I64, P, P, P, I64, P, S, P, SZ, P]),
            "qa_quantize_rowwise_int8": (S, [P, I64, I64, P, I32, I32, P, P, P, P, P]),
            "qa_qlinear_int8_mixed_workspace": (SZ, [I64, I64]),
            "qa_qlinear_int8_mixed": (S, [P, I64, I64, P, P, P, I64, F, P, S, P, SZ, P]),
            "qa_qlinear_int8_mixed_offsets": (S, [I64, I64, P]),
            "qa_qlinear_int8_mixed_noalloc": (S, [P, I64, I64, P, P, P, I64, F, P, S, P]),
            "qa_quantize_rowwise_int8_asym": (S, [P, I64, I64, I32, I32, P, P, P, P, P]),
            "qa_int8_row_sums": (S, [P, I64, I64, P, P]),
            "qa_qlinear_int8_asym_workspace": (SZ, [I64, I64]),
            "qa_qlinear_int8_asym": (S, [P, I64, I64, P, P, P, P, I64, P, S, P, SZ, P]),
            "qa_col_absmax_workspace": (SZ, [I64]),
            "qa_col_absmax": (S, [P, I64, I64, P, S, P, SZ, P]),
            "qa_smooth_factors": (S, [P, P, I64, F, P, P]),
            "qa_quantize_smooth_int8": (S, [P, I64, I64, P, S, S, P, P, P]),
            "qa_qlinear_int8_smooth_workspace": (SZ, [I64, I64]),
            "qa_qlinear_int8_smooth": (S, [P, I64, I64, P, S, P, P, I64, P, S, P, SZ, P]),
            "qa_hadamard_quant_int4": (S, [P, I64, I64, I32, S, I32, I32, P, P, P]),
            "qa_kron_sizes": (S, [I64, P, P, P]),
            "qa_kron_quant_int4": (S, [P, I64, I64, I64, I64, P, P, S, I32, I32, I32, P, P, P]),
            "qa_qlinear_kron_w4a4_workspace": (SZ, [I64, I64]),
            "qa_qlinear_kron_w4a4": (S, [P, I64, I64, I64, I64, P, P, P, P, I64, I32, P, S, P, SZ, P]),
            "qa_qlinear_w4a4_workspace": (SZ, [I64, I64]),
            "qa_qlinear_w4a4": (S, [P, I64, I64, P, P, I64, I32, P, S, P, SZ, P]),
            "qa_gemm_i8_i32": (S, [P, P, I64, I64, I64, P, P]),
            "qa_gemm_w4a4_group_acc": (S, [P, P, I64, I64, I64, I32, P, P]),
            "qa_hadamard_quant_int8": (S, [P, I64, I64, I32, I32, I32, P, P, P]),
            "qa_qlinear_w4a8_workspace": (SZ, [I64, I64]),
            "qa_qlinear_w4a8": (S, [P, I64, I64, P, P, I64, I32, P, S, P, SZ, P]),
            "qa_gemm_w4a8_group_acc": (S, [P, P, I64, I64, I64, I32, P, P]),
            "qa_hadamard_quant_int4_asym": (S, [P, I64, I64, I32, P, P, P, P]),
            "qa_w4_column_terms": (S, [P, P, I64, I64, I32, P, P]),
            "qa_qlinear_w4a4_asym_workspace": (SZ, [I64, I64]),
            "qa_qlinear_w4a4_asym": (S, [P, I64, I64, P, P, P, I64, I32, P, S, P, SZ, P]),
            "qa_rmsnorm_int8": (S, [P, I64, P, I64, P, S, I64, I64, F, P, P, P, I64, P, P]),
            "qa_route_experts_workspace": (SZ, [I64, I64, I32]),
            "qa_route_experts": (S, [P, S, I64, I64, I64, P, S, I32, I32, I32, I32, I32, F, P, P, P, P, P, SZ, P]),
            "qa_experts_int8_workspace": (SZ, [I64, I64, I32, I64, I64]),
            "qa_experts_int8": (S, [P, P, I64, I64, P, P, P, I64, I32, P, P, I64, P, P, P, S, P, SZ, P]),
            "qa_qlinear_int8_lora_workspace": (SZ, [I64, I64, I32]),
            "qa_qlinear_int8_lora": (S, [P, P, P, S, I64, I64, P, P, I64, P, P, P, I32, I64, P, P, I64, P, S, P, SZ,
                                         P]),
            "qa_kv_write": (S, [P, I64, P, I64, S, I64, P, I32, I64, I32, I32, I32, P, P, P, P, P]),
            "qa_kv_read": (S, [P, I64, I32, I64, I32, I32, I32, P, P, P, P, P, P, S, P]),
            "qa_attn_decode_workspace": (SZ, [I64, I32, I32, I32, I64, I32]),
            "qa_attn_decode": (S, [P, I64, S, I64, I32, I32, I64, I32, I32, I32, P, P, P, P, P, I64, I64, P, I64, I32, F,
                                   P, S, P, P, SZ, P]),
            "qa_qlinear_int8_act": (S, [P, P, I64, I64, P, P, I64, P, S, P, I64, P, I64, S, P]),
            "qa_probe_stream_read": (S, [P, SZ, I32, I32, I32, P, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().qa_status_string(int(s)).decode()


def last_error() -> str:
    return lib().qa_last_error().decode()


def _check(fn: str, s: int):
    if s != 0:
        raise QAError(fn, status_string(s), last_error())


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, name, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _empty(stream, *args, **kw):
    """torch.empty on the stream the library call runs on: the caching
    allocator then keeps the block for that stream, so memory a call still
    uses is not handed to work on another stream after it is released."""
    if stream is None:
        return torch.empty(*args, **kw)
    with torch.cuda.stream(stream):
        return torch.empty(*args, **kw)


def _workspace(stream, nbytes, device, ws):
    if ws is not None:
        return ws
    return _empty(stream, max(int(nbytes), 1), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- entry points
def qa_outlier_cols_workspace(K: int) -> int:
    return int(lib().qa_outlier_cols_workspace(K))


def qa_outlier_cols(X, threshold=6.0, scratch=None, stream=None):
    """-> (mask u8 [K], idx i32 [K] (first `count` valid), count i32 [1], colmax f32 [K])."""
    _dev(X, "X", torch.float16)
    M, K = X.shape
    dev = X.device
    mask = _empty(stream, K, dtype=torch.uint8, device=dev)
    idx = _empty(stream, K, dtype=torch.int32, device=dev)
    count = _empty(stream, 1, dtype=torch.int32, device=dev)
    colmax = _empty(stream, K, dtype=torch.float32, device=dev)
    nb = qa_outlier_cols_workspace(K)
    scratch = _workspace(stream, nb, dev, scratch)
    _check("qa_outlier_cols", lib().qa_outlier_cols(_p(X), M, K, float(threshold), _p(mask), _p(idx), _p(count),
                                                     _p(colmax), _p(scratch), scratch.numel(), _stream(stream)))
    return mask, idx, count, colmax


def qa_outlier_topk(X, k: int, scratch=None, stream=None):
    """The k columns of largest max |x| (ties: lower column first)
    -> (mask u8 [K], idx i32 [K] (first `count` valid), count i32 [1], colmax f32 [K])."""
    _dev(X, "X", torch.float16)
    M, K = X.shape
    dev = X.device
    mask = _empty(stream, K, dtype=torch.uint8, device=dev)
    idx = _empty(stream, K, dtype=torch.int32, device=dev)
    count = _empty(stream, 1, dtype=torch.int32, device=dev)
    colmax = _empty(stream, K, dtype=torch.float32, device=dev)
    scratch = _workspace(stream, qa_outlier_cols_workspace(K), dev, scratch)
    _check("qa_outlier_topk", lib().qa_outlier_topk(_p(X), M, K, int(k), _p(mask), _p(idx), _p(count), _p(colmax),
                                                     _p(scratch), scratch.numel(), _stream(stream)))
    return mask, idx, count, colmax


def topk_count(share: float, K: int) -> int:
    """Number of decomposed columns for a share of the K dimensions: ceil(share * K)."""
    import math
    return min(K, max(0, math.ceil(share * K)))


def qa_quantize_rowwise_int8(X, mask=None, q_min=-127, q_max=127, s_in=None, z_in=None, stream=None):
    """-> (Xq i8 [rows x K], s f32 [rows] or None in static mode)."""
    _dev(X, "X", torch.float16)
    rows, K = X.shape
    Xq = _empty(stream, (rows, K), dtype=torch.int8, device=X.device)
    s_out = None if s_in is not None else _empty(stream, rows, dtype=torch.float32, device=X.device)
    _check("qa_quantize_rowwise_int8",
           lib().qa_quantize_rowwise_int8(_p(X), rows, K, _p(mask), int(q_min), int(q_max), _p(s_in), _p(z_in),
                                          _p(Xq), _p(s_out), _stream(stream)))
    return Xq, s_out


def qa_qlinear_int8_mixed_workspace(M: int, K: int) -> int:
    return int(lib().qa_qlinear_int8_mixed_workspace(M, K))


def qa_qlinear_int8_mixed(X, Wq, s_w, W16=None, threshold=6.0, out_dtype=torch.float16, out=None,
                          workspace=None, stream=None):
    """LLM.int8() mixed-precision linear -> out [M x N] of out_dtype."""
    _dev(X, "X", torch.float16)
    _dev(Wq, "Wq", torch.int8)
    _dev(s_w, "s_w", torch.float32)
    if W16 is not None:
        _dev(W16, "W16", torch.float16)
    M, K = X.shape
    N = Wq.shape[0]
    if out is None:
        out = _empty(stream, (M, N), dtype=out_dtype, device=X.device)
    workspace = _workspace(stream, qa_qlinear_int8_mixed_workspace(M, K), X.device, workspace)
    _check("qa_qlinear_int8_mixed",
           lib().qa_qlinear_int8_mixed(_p(X), M, K, _p(Wq), _p(s_w), _p(W16), N, float(threshold), _p(out),
                                       _DTYPE_CODE[out.dtype], _p(workspace), workspace.numel(), _stream(stream)))
    return out


NOALLOC_SCRATCH_BYTES = 40 << 20


def qa_qlinear_int8_mixed_noalloc(X, Wq, s_w, out, W16=None, threshold=6.0, stream=None):
    """LLM.int8() mixed-precision linear into the caller's `out` [M x N] (fp32,
    fp16 or bf16) with the library's static per-GPU scratch: nothing is
    allocated, here or in the library.  Calls that overlap on one GPU race."""
    _dev(X, "X", torch.float16)
    _dev(Wq, "Wq", torch.int8)
    _dev(s_w, "s_w", torch.float32)
    _dev(out, "out")
    if W16 is not None:
        _dev(W16, "W16", torch.float16)
    M, K = X.shape
    N = Wq.shape[0]
    if tuple(out.shape) != (M, N):
        raise ValueError("out must be [%d x %d]" % (M, N))
    _check("qa_qlinear_int8_mixed_noalloc",
           lib().qa_qlinear_int8_mixed_noalloc(_p(X), M, K, _p(Wq), _p(s_w), _p(W16), N, float(threshold), _p(out),
                                               _DTYPE_CODE[out.dtype], _stream(stream)))
    return out


def qa_qlinear_int8_mixed_offsets(M: int, K: int):
    """Byte offsets of (idx, count, s_x, Xq) in the workspace of an LLM.int8()
    call with M tokens and K in-features."""
    off = (ctypes.c_size_t * 4)()
    _check("qa_qlinear_int8_mixed_offsets", lib().qa_qlinear_int8_mixed_offsets(int(M), int(K), off))
    return tuple(int(v) for v in off)


def qa_quantize_rowwise_int8_asym(X, q_min=-128, q_max=127, stream=None):
    """Per-row min-max zero-point codes -> (q i8 [rows x K], s f32 [rows], z i32 [rows], rowsum i32 [rows])."""
    _dev(X, "X", torch.float16)
    rows, K = X.shape
    d = X.device
    q = _empty(stream, (rows, K), dtype=torch.int8, device=d)
    s = _empty(stream, rows, dtype=torch.float32, device=d)
    z = _empty(stream, rows, dtype=torch.int32, device=d)
    rs = _empty(stream, rows, dtype=torch.int32, device=d)
    _check("qa_quantize_rowwise_int8_asym",
           lib().qa_quantize_rowwise_int8_asym(_p(X), rows, K, int(q_min), int(q_max), _p(q), _p(s), _p(z), _p(rs),
                                               _stream(stream)))
    return q, s, z, rs


def qa_int8_row_sums(A, stream=None):
    """Row sums of an int8 matrix -> i32 [rows]."""
    _dev(A, "A", torch.int8)
    rows, K = A.shape
    sums = _empty(stream, rows, dtype=torch.int32, device=A.device)
    _check("qa_int8_row_sums", lib().qa_int8_row_sums(_p(A), rows, K, _p(sums), _stream(stream)))
    return sums


def qa_qlinear_int8_asym_workspace(M: int, K: int) -> int:
    return int(lib().qa_qlinear_int8_asym_workspace(M, K))


def qa_qlinear_int8_asym(X, Wq, s_w, w_rowsum, z_w=None, out_dtype=torch.float16, out=None, workspace=None,
                         stream=None):
    """W8A8 linear with per-token zero-point activations -> out [M x N] of out_dtype."""
    _dev(X, "X", torch.float16)
    _dev(Wq, "Wq", torch.int8)
    _dev(s_w, "s_w", torch.float32)
    _dev(w_rowsum, "w_rowsum", torch.int32)
    if z_w is not None:
        _dev(z_w, "z_w", torch.int32)
    M, K = X.shape
    N = Wq.shape[0]
    if out is None:
        out = _empty(stream, (M, N), dtype=out_dtype, device=X.device)
    workspace = _workspace(stream, qa_qlinear_int8_asym_workspace(M, K), X.device, workspace)
    _check("qa_qlinear_int8_asym",
           lib().qa_qlinear_int8_asym(_p(X), M, K, _p(Wq), _p(s_w), _p(z_w), _p(w_rowsum), N, _p(out),
                                      _DTYPE_CODE[out.dtype], _p(workspace), workspace.numel(), _stream(stream)))
    return out


def qa_col_absmax_workspace(K: int) -> int:
    return int(lib().qa_col_absmax_workspace(K))


def qa_col_absmax(A, colmax=None, accumulate=False, scratch=None, stream=None):
    """Column absolute maxima of A fp16 [rows x K] -> colmax f32 [K] (maxed into
    the given colmax when accumulate)."""
    _dev(A, "A", torch.float16)
    rows, K = A.shape
    if colmax is None:
        if accumulate:
            raise ValueError("accumulate needs the running colmax")
        colmax = _empty(stream, K, dtype=torch.float32, device=A.device)
    _dev(colmax, "colmax", torch.float32)
    scratch = _workspace(stream, qa_col_absmax_workspace(K), A.device, scratch)
    _check("qa_col_absmax", lib().qa_col_absmax(_p(A), rows, K, _p(colmax), int(bool(accumulate)), _p(scratch),
                                                 scratch.numel(), _stream(stream)))
    return colmax


def qa_smooth_factors(act_absmax, w_absmax, alpha=0.5, stream=None):
    """SmoothQuant migration factors -> s f32 [K]."""
    _dev(act_absmax, "act_absmax", torch.float32)
    _dev(w_absmax, "w_absmax", torch.float32)
    K = act_absmax.numel()
    if w_absmax.numel() != K:
        raise ValueError("act_absmax and w_absmax differ in length")
    s = _empty(stream, K, dtype=torch.float32, device=act_absmax.device)
    _check("qa_smooth_factors", lib().qa_smooth_factors(_p(act_absmax), _p(w_absmax), K, float(alpha), _p(s),
                                                         _stream(stream)))
    return s


def qa_quantize_smooth_int8(A, s, multiply=False, per_tensor=False, stream=None):
    """Smoothing (A / s, or A * s for a weight) + int8 absmax codes -> (q i8 [rows x K], s_out f32 [rows])."""
    _dev(A, "A", torch.float16)
    _dev(s, "s", torch.float32)
    rows, K = A.shape
    q = _empty(stream, (rows, K), dtype=torch.int8, device=A.device)
    s_out = _empty(stream, rows, dtype=torch.float32, device=A.device)
    _check("qa_quantize_smooth_int8",
           lib().qa_quantize_smooth_int8(_p(A), rows, K, _p(s), QA_SMOOTH_MULTIPLY if multiply else QA_SMOOTH_DIVIDE,
                                         QA_SCALE_PER_TENSOR if per_tensor else QA_SCALE_PER_ROW, _p(q), _p(s_out),
                                         _stream(stream)))
    return q, s_out


def qa_qlinear_int8_smooth_workspace(M: int, K: int) -> int:
    return int(lib().qa_qlinear_int8_smooth_workspace(M, K))


def qa_qlinear_int8_smooth(X, s, Wq, s_w, per_tensor=False, out_dtype=torch.float16, out=None, workspace=None,
                           stream=None):
    """SmoothQuant W8A8 linear -> out [M x N] of out_dtype."""
    _dev(X, "X", torch.float16)
    _dev(s, "s", torch.float32)
    _dev(Wq, "Wq", torch.int8)
    _dev(s_w, "s_w", torch.float32)
    M, K = X.shape
    N = Wq.shape[0]
    if out is None:
        out = _empty(stream, (M, N), dtype=out_dtype, device=X.device)
    workspace = _workspace(stream, qa_qlinear_int8_smooth_workspace(M, K), X.device, workspace)
    _check("qa_qlinear_int8_smooth",
           lib().qa_qlinear_int8_smooth(_p(X), M, K, _p(s), QA_SCALE_PER_TENSOR if per_tensor else QA_SCALE_PER_ROW,
                                        _p(Wq), _p(s_w), N, _p(out), _DTYPE_CODE[out.dtype], _p(workspace),
                                        workspace.numel(), _stream(stream)))
    return out


def qa_qlinear_int8_topk_workspace(M: int, K: int) -> int:
    return int(lib().qa_qlinear_int8_topk_workspace(M, K))


def qa_qlinear_int8_topk(X, Wq, s_w, k: int, W16=None, out_dtype=torch.float16, out=None, workspace=None,
                         stream=None):
    """LLM.int8() linear with the top-k columns decomposed -> out [M x N] of out_dtype."""
    _dev(X, "X", torch.float16)
    _dev(Wq, "Wq", torch.int8)
    _dev(s_w, "s_w", torch.float32)
    if W16 is not None:
        _dev(W16, "W16", torch.float16)
    M, K = X.shape
    N = Wq.shape[0]
    if out is None:
        out = _empty(stream, (M, N), dtype=out_dtype, device=X.device)
    workspace = _workspace(stream, qa_qlinear_int8_topk_workspace(M, K), X.device, workspace)
    _check("qa_qlinear_int8_topk",
           lib().qa_qlinear_int8_topk(_p(X), M, K, int(k), _p(Wq), _p(s_w), _p(W16), N, _p(out),
                                      _DTYPE_CODE[out.dtype], _p(workspace), workspace.numel(), _stream(stream)))
    return out


def qa_hadamard_quant_int4(X, G: int, per_group: bool, q_min=-7, q_max=7, stream=None):
    """-> (packed u32 as int32 [rows x K/8], s f32 [rows x (K/G if per_group else 1)])."""
    _dev(X, "X", torch.float16)
    rows, K = X.shape
    packed = _empty(stream, (rows, K // 8), dtype=torch.int32, device=X.device)
    s = _empty(stream, (rows, K // G if per_group else 1), dtype=torch.float32, device=X.device)
    _check("qa_hadamard_quant_int4",
           lib().qa_hadamard_quant_int4(_p(X), rows, K, int(G), QA_SCALE_PER_GROUP if per_group else QA_SCALE_PER_ROW,
                                        int(q_min), int(q_max), _p(packed), _p(s), _stream(stream)))
    return packed, s


def qa_kron_sizes(n: int):
    """-> (n1, n2, has_kernel): n1 n2 = n, n1 <= n2, n1 + n2 smallest; has_kernel
    tells whether the Kronecker entry points take that pair."""
    n1, n2, hk = ctypes.c_int64(0), ctypes.c_int64(0), ctypes.c_int32(0)
    _check("qa_kron_sizes", lib().qa_kron_sizes(int(n), ctypes.byref(n1), ctypes.byref(n2), ctypes.byref(hk)))
    return n1.value, n2.value, bool(hk.value)


def qa_kron_quant_int4(X, P1, P2, G=None, q_min=-7, q_max=7, stream=None):
    """Kronecker transform P1^T X~ P2 of each row + int4 codes -> (packed u32 as int32 [rows x K/8],
    s f32 [rows x (K/G if G else 1)])."""
    _dev(X, "X", torch.float16)
    _dev(P1, "P1", torch.float32)
    _dev(P2, "P2", torch.float32)
    rows, K = X.shape
    n1, n2 = P1.shape[0], P2.shape[0]
    packed = _empty(stream, (rows, K // 8), dtype=torch.int32, device=X.device)
    s = _empty(stream, (rows, K // G if G else 1), dtype=torch.float32, device=X.device)
    _check("qa_kron_quant_int4",
           lib().qa_kron_quant_int4(_p(X), rows, K, n1, n2, _p(P1), _p(P2),
                                    QA_SCALE_PER_GROUP if G else QA_SCALE_PER_ROW, int(G or 0), int(q_min), int(q_max),
                                    _p(packed), _p(s), _stream(stream)))
    return packed, s


def qa_qlinear_kron_w4a4_workspace(M: int, K: int) -> int:
    return int(lib().qa_qlinear_kron_w4a4_workspace(M, K))


def qa_qlinear_kron_w4a4(X, P1, P2, Wp, s_w, G=128, out_dtype=torch.float32, out=None, workspace=None, stream=None):
    """W4A4 linear with the Kronecker transform of X -> out [M x N]."""
    _dev(X, "X", torch.float16)
    _dev(P1, "P1", torch.float32)
    _dev(P2, "P2", torch.float32)
    _dev(Wp, "Wp", torch.int32)
    _dev(s_w, "s_w", torch.float32)
    M, K = X.shape
    N = Wp.shape[0]
    if out is None:
        out = _empty(stream, (M, N), dtype=out_dtype, device=X.device)
    workspace = _workspace(stream, qa_qlinear_kron_w4a4_workspace(M, K), X.device, workspace)
    _check("qa_qlinear_kron_w4a4",
           lib().qa_qlinear_kron_w4a4(_p(X), M, K, P1.shape[0], P2.shape[0], _p(P1), _p(P2), _p(Wp), _p(s_w), N,
                                      int(G), _p(out), _DTYPE_CODE[out.dtype], _p(workspace), workspace.numel(),
                                      _stream(stream)))
    return out


def qa_qlinear_w4a4_workspace(M: int, K: int) -> int:
    return int(lib().qa_qlinear_w4a4_workspace(M, K))


def qa_qlinear_w4a4(X, Wp, s_w, G=128, out_dtype=torch.float32, out=None, workspace=None, stream=None):
    """W4A4 group-Hadamard linear -> out [M x N]."""
    _dev(X, "X", torch.float16)
    _dev(Wp, "Wp", torch.int32)
    _dev(s_w, "s_w", torch.float32)
    M, K = X.shape
    N = Wp.shape[0]
    if out is None:
        out = _empty(stream, (M, N), dtype=out_dtype, device=X.device)
    workspace = _workspace(stream, qa_qlinear_w4a4_workspace(M, K), X.device, workspace)
    _check("qa_qlinear_w4a4",
           lib().qa_qlinear_w4a4(_p(X), M, K, _p(Wp), _p(s_w), N, int(G), _p(out), _DTYPE_CODE[out.dtype],
                                 _p(workspace), workspace.numel(), _stream(stream)))
    return out


def qa_hadamard_quant_int8(X, G: int, q_min=-127, q_max=127, stream=None):
    """Hadamard rotation + per-row int8 codes -> (q i8 [rows x K], s f32 [rows])."""
    _dev(X, "X", torch.float16)
    rows, K = X.shape
    q = _empty(stream, (rows, K), dtype=torch.int8, device=X.device)
    s = _empty(stream, rows, dtype=torch.float32, device=X.device)
    _check("qa_hadamard_quant_int8",
           lib().qa_hadamard_quant_int8(_p(X), rows, K, int(G), int(q_min), int(q_max), _p(q), _p(s),
                                        _stream(stream)))
    return q, s


def qa_qlinear_w4a8_workspace(M: int, K: int) -> int:
    return int(lib().qa_qlinear_w4a8_workspace(M, K))


def qa_qlinear_w4a8(X, Wp, s_w, G=128, out_dtype=torch.float32, out=None, workspace=None, stream=None):
    """W4A8 group-Hadamard linear (int8 activations, offline int4 weight) -> out [M x N]."""
    _dev(X, "X", torch.float16)
    _dev(Wp, "Wp", torch.int32)
    _dev(s_w, "s_w", torch.float32)
    M, K = X.shape
    N = Wp.shape[0]
    if out is None:
        out = _empty(stream, (M, N), dtype=out_dtype, device=X.device)
    workspace = _workspace(stream, qa_qlinear_w4a8_workspace(M, K), X.device, workspace)
    _check("qa_qlinear_w4a8",
           lib().qa_qlinear_w4a8(_p(X), M, K, _p(Wp), _p(s_w), N, int(G), _p(out), _DTYPE_CODE[out.dtype],
                                 _p(workspace), workspace.numel(), _stream(stream)))
    return out


def qa_hadamard_quant_int4_asym(X, G: int, stream=None):
    """Hadamard rotation + zero-point int4 codes per row -> (packed u32 as int32 [rows x K/8] holding q - 8,
    s f32 [rows], z i32 [rows])."""
    _dev(X, "X", torch.float16)
    rows, K = X.shape
    packed = _empty(stream, (rows, K // 8), dtype=torch.int32, device=X.device)
    s = _empty(stream, rows, dtype=torch.float32, device=X.device)
    z = _empty(stream, rows, dtype=torch.int32, device=X.device)
    _check("qa_hadamard_quant_int4_asym",
           lib().qa_hadamard_quant_int4_asym(_p(X), rows, K, int(G), _p(packed), _p(s), _p(z), _stream(stream)))
    return packed, s, z


def qa_w4_column_terms(Wp, s_w, K: int, G: int, stream=None):
    """c[n] = sum_g s_w[n][g] * sum_{k in g} qw[n][k] of a per-group int4 weight -> f32 [N]."""
    _dev(Wp, "Wp", torch.int32)
    _dev(s_w, "s_w", torch.float32)
    N = Wp.shape[0]
    c = _empty(stream, N, dtype=torch.float32, device=Wp.device)
    _check("qa_w4_column_terms", lib().qa_w4_column_terms(_p(Wp), _p(s_w), N, int(K), int(G), _p(c), _stream(stream)))
    return c


def qa_qlinear_w4a4_asym_workspace(M: int, K: int) -> int:
    return int(lib().qa_qlinear_w4a4_asym_workspace(M, K))


def qa_qlinear_w4a4_asym(X, Wp, s_w, c_w, G=128, out_dtype=torch.float32, out=None, workspace=None, stream=None):
    """W4A4 group-Hadamard linear with zero-point int4 activations -> out [M x N]."""
    _dev(X, "X", torch.float16)
    _dev(Wp, "Wp", torch.int32)
    _dev(s_w, "s_w", torch.float32)
    _dev(c_w, "c_w", torch.float32)
    M, K = X.shape
    N = Wp.shape[0]
    if out is None:
        out = _empty(stream, (M, N), dtype=out_dtype, device=X.device)
    workspace = _workspace(stream, qa_qlinear_w4a4_asym_workspace(M, K), X.device, workspace)
    _check("qa_qlinear_w4a4_asym",
           lib().qa_qlinear_w4a4_asym(_p(X), M, K, _p(Wp), _p(s_w), _p(c_w), N, int(G), _p(out),
                                      _DTYPE_CODE[out.dtype], _p(workspace), workspace.numel(), _stream(stream)))
    return out


def qa_gemm_i8_i32(A, B, stream=None):
    _dev(A, "A", torch.int8)
    _dev(B, "B", torch.int8)
    M, K = A.shape
    N = B.shape[0]
    C = _empty(stream, (M, N), dtype=torch.int32, device=A.device)
    _check("qa_gemm_i8_i32", lib().qa_gemm_i8_i32(_p(A), _p(B), M, K, N, _p(C), _stream(stream)))
    return C


def qa_gemm_w4a4_group_acc(Xp, Wp, K: int, G: int, stream=None):
    _dev(Xp, "Xp", torch.int32)
    _dev(Wp, "Wp", torch.int32)
    M, N = Xp.shape[0], Wp.shape[0]
    acc = _empty(stream, (M, N, K // G), dtype=torch.int32, device=Xp.device)
    _check("qa_gemm_w4a4_group_acc",
           lib().qa_gemm_w4a4_group_acc(_p(Xp), _p(Wp), M, K, N, int(G), _p(acc), _stream(stream)))
    return acc


def qa_gemm_w4a8_group_acc(Xq, Wp, G: int, stream=None):
    _dev(Xq, "Xq", torch.int8)
    _dev(Wp, "Wp", torch.int32)
    M, K = Xq.shape
    N = Wp.shape[0]
    acc = _empty(stream, (M, N, K // G), dtype=torch.int32, device=Xq.device)
    _check("qa_gemm_w4a8_group_acc",
           lib().qa_gemm_w4a8_group_acc(_p(Xq), _p(Wp), M, K, N, int(G), _p(acc), _stream(stream)))
    return acc


def _rows(t, name, dtype):
    """A [rows x columns] tensor whose rows are contiguous -> its row stride."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("%s must be a matrix with contiguous rows" % name)
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _shape(t, name, shape):
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))


def _a(t):
    """Device address of a tensor (None: NULL), as a plain number: a call with twenty of them is host time."""
    return None if t is None else t.data_ptr()


def _s(stream):
    """The given stream's handle, or that of the current device's current stream (without the stream object that
    torch.cuda.current_stream() builds, 3 us of the host's time)."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) if stream is None else stream.cuda_stream


def _like(stream, X, dtype):
    """A contiguous tensor of X's shape (empty_like is the cheapest allocation on the host)."""
    if stream is None and X.is_contiguous():
        return torch.empty_like(X, dtype=dtype)
    return _empty(stream, X.shape, dtype=dtype, device=X.device)


def qa_rmsnorm_int8(X, g, residual=None, eps=1e-6, want_y=False, total=None, stream=None):
    """Residual addition + RMS norm + int8 codes per row.

    X [rows x K] fp32 / fp16 / bf16 (rows may be strided), g [K] and residual
    of the same type -> (Xq i8 [rows x K], s f32 [rows], total or None, y or
    None): total = X + residual (with a residual; into the given `total`,
    which may be X or residual itself), y the norm in X's type if wanted."""
    if X.dtype not in _DTYPE_CODE:
        raise TypeError("X must be fp32, fp16 or bf16, got %s" % X.dtype)
    ldx = _rows(X, "X", X.dtype)
    rows, K = X.shape
    _dev(g, "g", X.dtype)
    _shape(g, "g", (K,))
    ldr = lds = K
    if residual is not None:
        ldr = _rows(residual, "residual", X.dtype)
        _shape(residual, "residual", (rows, K))
        if total is None:
            total = _like(stream, X, X.dtype)
    if total is not None:
        lds = _rows(total, "total", X.dtype)
        _shape(total, "total", (rows, K))
    Xq = _like(stream, X, torch.int8)
    s = _empty(stream, rows, dtype=torch.float32, device=X.device)
    y = _like(stream, X, X.dtype) if want_y else None
    _check("qa_rmsnorm_int8",
           lib().qa_rmsnorm_int8(_a(X), ldx, _a(residual), ldr, _a(g), _DTYPE_CODE[X.dtype], rows, K, float(eps),
                                 _a(Xq), _a(s), _a(total), lds, _a(y), _s(stream)))
    return Xq, s, total, y


def qa_route_experts_workspace(T: int, E: int, k: int) -> int:
    return int(lib().qa_route_experts_workspace(T, E, k))


def qa_route_experts(logits, k: int, bias=None, score=QA_SCORE_SOFTMAX, groups=1, top_groups=1, group_top=1,
                     renorm=True, scale=1.0, workspace=None, stream=None):
    """The k experts of each token -> (ids i32 [T x k], weights f32 [T x k], order i32 [T k], offsets i32 [E + 1]):
    the chosen experts in descending order of score + bias, their weights, and the pairs t k + j by expert.  ids,
    order and offsets are views of one allocation: clone() one that is to be kept or saved without the others."""
    if logits.dtype not in _DTYPE_CODE:
        raise TypeError("logits must be fp32, fp16 or bf16, got %s" % logits.dtype)
    ld = _rows(logits, "logits", logits.dtype)
    T, E = logits.shape
    k = int(k)
    if bias is not None:
        _dev(bias, "bias", torch.float32)
        _shape(bias, "bias", (E,))
    d = logits.device
    n = max(k, 0)
    p, need = T * n, qa_route_experts_workspace(T, E, k)
    w = _empty(stream, (T, n), dtype=torch.float32, device=d)
    # ids, order and offsets are views of one allocation (host time), with the workspace behind them when it is small
    own = workspace is None and need <= 1 << 16
    ints = _empty(stream, 2 * p + E + 1 + (need // 4 if own else 0), dtype=torch.int32, device=d)
    ids, order = ints.as_strided((T, n), (n, 1), 0), ints.as_strided((p,), (1,), p)
    offsets = ints.as_strided((E + 1,), (1,), 2 * p)
    if own:
        ws, ws_bytes = ints.data_ptr() + 4 * (2 * p + E + 1), need
    else:
        workspace = _workspace(stream, need, d, workspace)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel()
    _check("qa_route_experts",
           lib().qa_route_experts(_a(logits), _DTYPE_CODE[logits.dtype], T, E, ld, _a(bias), int(score), int(groups),
                                  int(top_groups), int(group_top), k, int(bool(renorm)), float(scale), _a(ids), _a(w),
                                  _a(order), _a(offsets), ws, ws_bytes, _s(stream)))
    return ids, w, order, offsets


def qa_experts_int8_workspace(T: int, K: int, k: int, E: int, F: int) -> int:
    return int(lib().qa_experts_int8_workspace(T, K, k, E, F))


def qa_experts_int8(Xq, s_x, weights, order, offsets, W13, s13, W2, s2, out_dtype=torch.float16, out=None,
                    workspace=None, stream=None):
    """Gated feed-forward of the routed experts on int8 codes -> out [T x K] of out_dtype.

    Xq i8 [T x K], s_x f32 [T]; weights f32 [T x k], order, offsets from
    qa_route_experts; W13 i8 [E x 2F x K] (gate rows, then up rows), s13 f32
    [E x 2F]; W2 i8 [E x K x F], s2 f32 [E x K].  A part of the experts, e0 ..
    e0 + E - 1: their weights and offsets[e0 : e0 + E + 1]; out is their share of
    the sum."""
    _dev(Xq, "Xq", torch.int8)
    _dev(s_x, "s_x", torch.float32)
    _dev(weights, "weights", torch.float32)
    _dev(order, "order", torch.int32)
    _dev(offsets, "offsets", torch.int32)
    _dev(W13, "W13", torch.int8)
    _dev(s13, "s13", torch.float32)
    _dev(W2, "W2", torch.int8)
    _dev(s2, "s2", torch.float32)
    T, K = Xq.shape
    E, F = W13.shape[0], W2.shape[2]
    k = weights.shape[1]
    _shape(s_x, "s_x", (T,))
    _shape(weights, "weights", (T, k))
    _shape(order, "order", (T * k,))
    _shape(offsets, "offsets", (E + 1,))
    _shape(W13, "W13", (E, 2 * F, K))
    _shape(s13, "s13", (E, 2 * F))
    _shape(W2, "W2", (E, K, F))
    _shape(s2, "s2", (E, K))
    if out is None:
        out = _empty(stream, (T, K), dtype=out_dtype, device=Xq.device)
    _dev(out, "out")
    _shape(out, "out", (T, K))
    workspace = _workspace(stream, qa_experts_int8_workspace(T, K, k, E, F), Xq.device, workspace)
    _check("qa_experts_int8",
           lib().qa_experts_int8(_a(Xq), _a(s_x), T, K, _a(weights), _a(order), _a(offsets), E, k, _a(W13), _a(s13), F,
                                 _a(W2), _a(s2), _a(out), _DTYPE_CODE[out.dtype], _a(workspace), workspace.numel(),
                                 _s(stream)))
    return out


def qa_qlinear_int8_lora_workspace(M: int, K: int, r: int) -> int:
    return int(lib().qa_qlinear_int8_lora_workspace(M, K, r))


def qa_qlinear_int8_lora(Xq, s_x, X, Wq, s_w, A, B, alpha, seg, which, out_dtype=torch.float16, out=None,
                         workspace=None, stream=None):
    """int8 linear with each request's low-rank adapter -> out [M x N] of out_dtype.

    Xq i8 [M x K], s_x f32 [M], X fp16 / bf16 [M x K]; Wq i8 [N x K], s_w f32
    [N]; A [L x r x K], B [L x N x r] of X's type, alpha f32 [L]; seg i32
    [R + 1] token starts of the requests, which i32 [R] their adapters (-1:
    none)."""
    _dev(Xq, "Xq", torch.int8)
    _dev(s_x, "s_x", torch.float32)
    if X.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("X must be fp16 or bf16, got %s" % X.dtype)
    _dev(X, "X", X.dtype)
    _dev(Wq, "Wq", torch.int8)
    _dev(s_w, "s_w", torch.float32)
    _dev(A, "A", X.dtype)
    _dev(B, "B", X.dtype)
    _dev(alpha, "alpha", torch.float32)
    _dev(seg, "seg", torch.int32)
    _dev(which, "which", torch.int32)
    M, K = Xq.shape
    N = Wq.shape[0]
    L, r = A.shape[0], A.shape[1]
    R = which.numel()
    _shape(s_x, "s_x", (M,))
    _shape(X, "X", (M, K))
    _shape(Wq, "Wq", (N, K))
    _shape(s_w, "s_w", (N,))
    _shape(A, "A", (L, r, K))
    _shape(B, "B", (L, N, r))
    _shape(alpha, "alpha", (L,))
    _shape(seg, "seg", (R + 1,))
    if out is None:
        out = _empty(stream, (M, N), dtype=out_dtype, device=Xq.device)
    _dev(out, "out")
    _shape(out, "out", (M, N))
    workspace = _workspace(stream, qa_qlinear_int8_lora_workspace(M, K, r), Xq.device, workspace)
    _check("qa_qlinear_int8_lora",
           lib().qa_qlinear_int8_lora(_a(Xq), _a(s_x), _a(X), _DTYPE_CODE[X.dtype], M, K, _a(Wq), _a(s_w), N, _a(A),
                                      _a(B), _a(alpha), r, L, _a(seg), _a(which), R, _a(out), _DTYPE_CODE[out.dtype],
                                      _a(workspace), workspace.numel(), _s(stream)))
    return out


# The calls of a decoding step are host time: what follows looks at all operands in one expression, and where that
# fails at each by itself, for the error that says which.
def _on(t, name, d):
    """An operand on another device than the first one."""
    if t is not None and t.get_device() != d:
        raise ValueError("%s must be on the same device as the other tensors, got %s" % (name, t.device))


def _cache(cache):
    """The four tensors of a cache -> (bits, pages, heads, page, D, device index): see qa_kv_write."""
    kc, ks, vc, vs = cache
    shape, dt, d, f32 = kc.shape, kc.dtype, kc.get_device(), torch.float32
    if not (len(shape) == 4 and d >= 0 and ks.get_device() == d and vc.get_device() == d and vs.get_device() == d and
            vc.dtype == dt and ks.dtype == f32 and vs.dtype == f32 and vc.shape == shape and ks.shape == shape[:3] and
            vs.shape == shape[:3] and kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and
            vs.is_contiguous()):
        _dev(kc, "k_codes", dt)
        if len(shape) != 4:
            raise ValueError("k_codes must be [pages x heads x page x D (or D / 8 words)], got %s" % list(shape))
        _dev(ks, "k_scales", f32)
        _dev(vc, "v_codes", dt)
        _dev(vs, "v_scales", f32)
        _shape(vc, "v_codes", shape)
        _shape(ks, "k_scales", shape[:3])
        _shape(vs, "v_scales", shape[:3])
        for t, name in ((ks, "k_scales"), (vc, "v_codes"), (vs, "v_scales")):
            _on(t, name, d)
    if dt == torch.int8:
        return 8, shape[0], shape[1], shape[2], shape[3], d
    if dt != torch.int32:
        raise TypeError("cache codes must be int8 (8 bits) or int32 (4 bits, packed), got %s" % dt)
    return 4, shape[0], shape[1], shape[2], 8 * shape[3], d


def _tokens(t, name, heads, D, d):
    """A [tokens x heads x D] tensor whose tokens are contiguous, on device d -> its token stride."""
    shape, stride = t.shape, t.stride()
    if not (len(shape) == 3 and shape[1] == heads and shape[2] == D and t.dtype in _DTYPE_CODE and
            t.get_device() == d and (not shape[0] or (stride[2] == 1 and (heads == 1 or stride[1] == D)))):
        if not t.is_cuda:
            raise TypeError("%s must be a CUDA (HIP) tensor" % name)
        if t.dtype not in _DTYPE_CODE:
            raise TypeError("%s must be fp32, fp16 or bf16, got %s" % (name, t.dtype))
        if len(shape) != 3 or shape[1] != heads or shape[2] != D:
            raise ValueError("%s must be [tokens x %d x %d], got %s" % (name, heads, D, list(shape)))
        _on(t, name, d)
        raise ValueError("%s must have contiguous heads of contiguous values" % name)
    return stride[0] if shape[0] > 1 else heads * D


def _sd(stream, d):
    """The given stream's handle, or that of device d's current stream."""
    return torch._C._cuda_getCurrentRawStream(d) if stream is None else stream.cuda_stream


def qa_kv_write(K, V, slots, cache, stream=None):
    """Keys and values of new tokens into a paged cache of int8 or int4 codes, one scale per token and head.

    K, V [T x heads x D] fp32 / fp16 / bf16 (tokens may be strided: columns of a projection's output); slots i64 [T]
    the tokens' places, page index * page + place in the page (-1: not written); cache = (k_codes, k_scales, v_codes,
    v_scales): codes int8 [pages x heads x page x D], or int32 [pages x heads x page x D / 8] for 4 bits, scales f32
    [pages x heads x page]."""
    bits, pages, heads, page, D, d = _cache(cache)
    if d != torch._C._cuda_getDevice():
        with torch.cuda.device(d):
            return qa_kv_write(K, V, slots, cache, stream)
    ldk, ldv = _tokens(K, "K", heads, D, d), _tokens(V, "V", heads, D, d)
    T = K.shape[0]
    if not (V.dtype == K.dtype and V.shape[0] == T and slots.dtype == torch.int64 and slots.shape == (T,) and
            slots.get_device() == d and slots.is_contiguous()):
        if V.dtype != K.dtype:
            raise TypeError("V must be %s, got %s" % (K.dtype, V.dtype))
        _shape(V, "V", K.shape)
        _dev(slots, "slots", torch.int64)
        _shape(slots, "slots", (T,))
        _on(slots, "slots", d)
    kc, ks, vc, vs = cache
    r = lib().qa_kv_write(K.data_ptr(), ldk, V.data_ptr(), ldv, _DTYPE_CODE[K.dtype], T, slots.data_ptr(), bits, pages,
                          heads, page, D, kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), _sd(stream, d))
    if r:
        _check("qa_kv_write", r)


def qa_kv_read(slots, cache, out_dtype=torch.float16, stream=None):
    """The keys and values at places of a cache (see qa_kv_write) -> (K, V) [T x heads x D] of out_dtype; zeros for a
    slot outside it."""
    bits, pages, heads, page, D, d = _cache(cache)
    if d != torch._C._cuda_getDevice():
        with torch.cuda.device(d):
            return qa_kv_read(slots, cache, out_dtype, stream)
    if not (slots.dtype == torch.int64 and slots.dim() == 1 and slots.get_device() == d and slots.is_contiguous()):
        _dev(slots, "slots", torch.int64)
        if slots.dim() != 1:
            raise ValueError("slots must be [T], got %s" % list(slots.shape))
        _on(slots, "slots", d)
    if out_dtype not in _DTYPE_CODE:
        raise TypeError("out_dtype must be fp32, fp16 or bf16, got %s" % out_dtype)
    T = slots.shape[0]
    K = _empty(stream, (T, heads, D), dtype=out_dtype, device=slots.device)
    V = torch.empty_like(K) if stream is None else _empty(stream, (T, heads, D), dtype=out_dtype, device=slots.device)
    kc, ks, vc, vs = cache
    r = lib().qa_kv_read(slots.data_ptr(), T, bits, pages, heads, page, D, kc.data_ptr(), ks.data_ptr(), vc.data_ptr(),
                         vs.data_ptr(), K.data_ptr(), V.data_ptr(), _DTYPE_CODE[out_dtype], _sd(stream, d))
    if r:
        _check("qa_kv_read", r)
    return K, V


def qa_attn_decode_workspace(B: int, H: int, heads: int, D: int, max_len: int, window: int = 0) -> int:
    return int(lib().qa_attn_decode_workspace(B, H, heads, D, max_len, window))


def qa_attn_decode(q, cache, table, lengths, scale=None, window=0, max_len=None, out_dtype=None, want_lse=False,
                   out=None, workspace=None, stream=None):
    """Attention of one new token per sequence over a paged cache (see qa_kv_write) -> out [B x H x D], or (out, lse
    f32 [B x H]) if wanted.

    q [B x H x D] fp32 / fp16 / bf16 (rows may be strided), H a multiple of the cache's heads; table i32 [B x width]
    the pages of each sequence (rows may be strided), lengths i32 [B] its tokens; scale: 1 / sqrt(D) if not given;
    window: the last tokens that are seen (0: all); max_len: an upper bound of the lengths (the table's places if not
    given), by which the work is split over the card -- lengths past it count as it; out_dtype: q's if not given."""
    bits, pages, heads, page, D, d = _cache(cache)
    if d != torch._C._cuda_getDevice():
        with torch.cuda.device(d):
            return qa_attn_decode(q, cache, table, lengths, scale, window, max_len, out_dtype, want_lse, out, workspace,
                                  stream)
    if q.dim() != 3:
        raise ValueError("q must be [B x H x D], got %s" % list(q.shape))
    B, H, _ = q.shape
    ldq = _tokens(q, "q", H, D, d)
    ldt = _rows(table, "table", torch.int32)
    width = table.shape[1]
    if not (lengths.dtype == torch.int32 and lengths.shape == (B,) and lengths.is_contiguous() and
            lengths.get_device() == d and table.shape[0] == B and table.get_device() == d):
        _dev(lengths, "lengths", torch.int32)
        _shape(lengths, "lengths", (B,))
        _shape(table, "table", (B, width))
        _on(lengths, "lengths", d)
        _on(table, "table", d)
    max_len = width * page if max_len is None else int(max_len)
    if out is None:
        dt = out_dtype or q.dtype
        out = torch.empty_like(q, dtype=dt) if stream is None and q.is_contiguous() else \
            _empty(stream, (B, H, D), dtype=dt, device=q.device)
    else:
        _dev(out, "out")
        _shape(out, "out", (B, H, D))
        _on(out, "out", d)
    if out.dtype not in _DTYPE_CODE or (out_dtype is not None and out.dtype != out_dtype):
        raise TypeError("out must be fp32, fp16 or bf16 (out_dtype), got %s" % out.dtype)
    lse = _empty(stream, (B, H), dtype=torch.float32, device=q.device) if want_lse else None
    L = lib()
    if workspace is None:
        ws, need = None, L.qa_attn_decode_workspace(B, H, heads, D, max_len, window)
        if need:
            workspace = _empty(stream, need, dtype=torch.uint8, device=q.device)
            ws = workspace.data_ptr()
    else:
        _dev(workspace, "workspace")
        _on(workspace, "workspace", d)
        ws, need = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    kc, ks, vc, vs = cache
    r = L.qa_attn_decode(q.data_ptr(), ldq, _DTYPE_CODE[q.dtype], B, H, bits, pages, heads, page, D, kc.data_ptr(),
                         ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), table.data_ptr(), ldt, width, lengths.data_ptr(),
                         max_len, window, D ** -0.5 if scale is None else scale, out.data_ptr(), _DTYPE_CODE[out.dtype],
                         _a(lse), ws, need, _sd(stream, d))
    if r:
        _check("qa_attn_decode", r)
    return (out, lse) if want_lse else out


def qa_qlinear_int8_act(Xq, s_x, Wq, s_w, bias=None, act=QA_ACT_NONE, residual=None, out_dtype=torch.float16, out=None,
                        stream=None):
    """int8 linear on codes with bias, activation and residual: act(X W^T + bias) + residual -> out [M x N].

    Xq i8 [M x K], s_x f32 [M]; Wq i8 [N x K], s_w f32 [N]; bias f32 [N]; act one of QA_ACT_*; residual [M x N] of the
    output's type (rows may be strided); out: the given tensor (rows may be strided, it may be the residual itself) or
    a new one of out_dtype (of the residual's type if there is one)."""
    d = Xq.get_device()
    if d >= 0 and d != torch._C._cuda_getDevice():
        with torch.cuda.device(d):
            return qa_qlinear_int8_act(Xq, s_x, Wq, s_w, bias, act, residual, out_dtype, out, stream)
    i8, f32, shape, wshape = torch.int8, torch.float32, Xq.shape, Wq.shape
    if not (d >= 0 and len(shape) == 2 and len(wshape) == 2 and Xq.dtype == i8 and Wq.dtype == i8 and s_x.dtype == f32 and
            s_w.dtype == f32 and wshape[1] == shape[1] and s_x.shape == shape[:1] and s_w.shape == wshape[:1] and
            s_x.get_device() == d and Wq.get_device() == d and s_w.get_device() == d and Xq.is_contiguous() and
            Wq.is_contiguous() and s_x.is_contiguous() and s_w.is_contiguous()):
        _dev(Xq, "Xq", i8)
        _dev(s_x, "s_x", f32)
        _dev(Wq, "Wq", i8)
        _dev(s_w, "s_w", f32)
        if len(shape) != 2:
            raise ValueError("Xq must be [M x K], got %s" % list(shape))
        _shape(s_x, "s_x", shape[:1])
        _shape(Wq, "Wq", (wshape[0], shape[1]))
        _shape(s_w, "s_w", wshape[:1])
        for t, name in ((s_x, "s_x"), (Wq, "Wq"), (s_w, "s_w")):
            _on(t, name, d)
    M, K = shape
    N = wshape[0]
    if bias is not None:
        _dev(bias, "bias", f32)
        _shape(bias, "bias", (N,))
        _on(bias, "bias", d)
    ldo = ldr = N
    if out is None:
        out = _empty(stream, (M, N), dtype=out_dtype if residual is None else residual.dtype, device=Xq.device)
    else:
        ldo = _rows(out, "out", out.dtype)
        _shape(out, "out", (M, N))
        _on(out, "out", d)
    if out.dtype not in _DTYPE_CODE:
        raise TypeError("out must be fp32, fp16 or bf16, got %s" % out.dtype)
    if residual is not None:
        ldr = _rows(residual, "residual", out.dtype)
        _shape(residual, "residual", (M, N))
        _on(residual, "residual", d)
    r = lib().qa_qlinear_int8_act(Xq.data_ptr(), s_x.data_ptr(), M, K, Wq.data_ptr(), s_w.data_ptr(), N, _a(bias), act,
                                  _a(residual), ldr, out.data_ptr(), ldo, _DTYPE_CODE[out.dtype], _sd(stream, d))
    if r:
        _check("qa_qlinear_int8_act", r)
    return out


def qa_probe_stream_read(src, nbytes: int, wgs: int, lane_bytes: int = 16, unroll: int = 4, sink=None, stream=None):
    """Measurement helper: read src[0 .. nbytes) once (the single-launch HBM read floor)."""
    _dev(src, "src", None)
    if sink is None:
        sink = _empty(stream, (int(wgs) * 512,), dtype=torch.int32, device=src.device)
    _check("qa_probe_stream_read",
           lib().qa_probe_stream_read(_p(src), int(nbytes), int(wgs), int(lane_bytes), int(unroll), _p(sink),
                                      _stream(stream)))
    return sink

