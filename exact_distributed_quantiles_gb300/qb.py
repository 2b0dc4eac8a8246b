"""Thin ctypes binding of ``libqb.so`` with the C entry points' names.

Argument marshalling only: tensors become device pointers, the stream defaults
to torch's current stream, and a non-zero status raises ``QBError``.  Every
step of the computation runs in the library's CUDA kernels; there is no CPU
fallback.  Importing this module raises if ``libqb.so`` has not been built
(``python -m exact_distributed_quantiles_gb300.build``).
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqb.so")

QB_OK, QB_EINVAL, QB_EUNSUPPORTED, QB_ECUDA, QB_EOVERFLOW, QB_EDEVICE = 0, -1, -2, -3, -4, -5
QB_F32, QB_BF16 = 0, 1

EXPORTS = ("qb_status_string", "qb_version", "qb_rank", "qb_sigmoid", "qb_sigmoid_scalar",
           "qb_zero_i32",
           "qb_route_hist_hi", "qb_route_hist_hi_next", "qb_select_hi", "qb_keys_hist_lo",
           "qb_route_hist_lo",
           "qb_finalize", "k3_route_hist", "k3_route_hist_next", "k3_finalize", "lei_inject",
           "qb_device_status",
           "lei_inject_noalloc", "qb_router_gemm", "qb_router_gemm_hist_hi",
           "qb_router_gemm_hist_hi_next", "qb_rank_average",
           "qb_maxvio", "lei_rho", "lei_apply",
           "lei_apply_overlap", "qb_selftest_wait_timeout",
           "qb_balance_loss", "qb_balance_workspace", "qb_balance_grad",
           "qb_expert_order", "qb_order_workspace",
           "qb_fp8_scale_pitch", "qb_fp8_cols_width", "qb_fp8_quantize_rows",
           "qb_fp8_quantize_cols", "qb_fp8_quantize_blocks", "qb_fp8_expert_gemm",
           "qb_fp8_expert_wgrad")

SCORES = {"sigmoid": 0, "softmax": 1}  # QB_SCORE_SIGMOID, QB_SCORE_SOFTMAX


class QBError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed with status {status}: {status_string(status)}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libqb.so not built at {LIB_PATH}; run "
                          "`python -m exact_distributed_quantiles_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    sigs = {
        "qb_status_string": (ctypes.c_char_p, [I]),
        "qb_version": (ctypes.c_char_p, []),
        "qb_rank": (I64, [I64, I, I]),
        "qb_sigmoid": (I, [P, P, I64, P]),
        "qb_sigmoid_scalar": (I, [P, P, I64, P]),
        "qb_zero_i32": (I, [P, I64, P]),
        "qb_route_hist_hi": (I, [P, I, P, I64, I, I, P, P, P, P, P]),
        "qb_route_hist_hi_next": (I, [P, I, P, I64, I, I, P, P, P, P, P]),
        "qb_select_hi": (I, [P, I, I64, P, P, P]),
        "qb_keys_hist_lo": (I, [P, I64, I, P, P, P]),
        "qb_route_hist_lo": (I, [P, I, P, I64, I, I, P, P, P]),
        "qb_finalize": (I, [P, P, P, P, I, P, P, I, P]),
        "k3_route_hist": (I, [P, I, P, I64, I, I, P, I, P, P, P]),
        "k3_route_hist_next": (I, [P, I, P, I64, I, I, P, I, P, P, P]),
        "k3_finalize": (I, [P, I, I, I64, P, P, I, P]),
        "lei_inject": (I, [P, P, I64, I, I, F, I64, P, P]),
        "qb_device_status": (I, [ctypes.POINTER(ctypes.c_int)]),
        "lei_inject_noalloc": (I, [P, P, I64, I, I, F, I64, P]),
        "qb_router_gemm": (I, [P, P, I64, I, I, P, P]),
        "qb_router_gemm_hist_hi": (I, [P, P, I64, I, I, I, P, P, P, P, P, P, P]),
        "qb_router_gemm_hist_hi_next": (I, [P, P, I64, I, I, I, P, P, P, P, P, P, P]),
        "qb_rank_average": (I, [P, I, I, P, P]),
        "qb_maxvio": (I, [P, I64, I, I, I64, P, P, P]),
        "lei_rho": (I, [P, I64, I, I, F, I64, P, P]),
        "lei_apply": (I, [P, I64, I, I64, P, P]),
        "lei_apply_overlap": (I, [P, I64, I, I64, P, P]),
        "qb_selftest_wait_timeout": (I, [I64, P]),
        "qb_balance_loss": (I, [P, I, P, P, I64, I, I, I64, I, F, P, P, P, P, P, I64, P]),
        "qb_balance_workspace": (I64, [I64, I, I64]),
        "qb_balance_grad": (I, [P, I, P, P, P, P, I64, I, I, I64, I, F, P, I, P]),
        "qb_expert_order": (I, [P, I64, I, I, P, P, P, P, P, I64, P]),
        "qb_order_workspace": (I64, [I64, I, I]),
        "qb_fp8_scale_pitch": (I64, [I64]),
        "qb_fp8_cols_width": (I64, [I64, I]),
        "qb_fp8_quantize_rows": (I, [P, I, I64, I64, P, I64, I, P, P, P]),
        "qb_fp8_quantize_cols": (I, [P, I, I64, I64, P, P, I, I64, I, I64, P, P, P]),
        "qb_fp8_quantize_blocks": (I, [P, I, I, I, I, P, P, P, P, P]),
        "qb_fp8_expert_gemm": (I, [P, P, P, P, P, I, I64, I, I, P, I, P]),
        "qb_fp8_expert_wgrad": (I, [P, P, P, P, P, I, I64, I, I, P, I, I, P]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.qb_status_string(int(status)).decode()


def version() -> str:
    return lib.qb_version().decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(fn: str, st: int):
    if st != QB_OK:
        raise QBError(fn, st)


def _dtype(t) -> int:
    if t.dtype == torch.float32:
        return QB_F32
    if t.dtype == torch.bfloat16:
        return QB_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def rank(n_pool: int, E: int, k: int) -> int:
    r = int(lib.qb_rank(int(n_pool), int(E), int(k)))
    if r < 0:
        raise QBError("qb_rank", r)
    return r


def qb_sigmoid(x, s, stream=None):
    _check("qb_sigmoid", lib.qb_sigmoid(_ptr(x), _ptr(s), x.numel(), _stream(stream)))


def qb_sigmoid_scalar(x, s, stream=None):
    _check("qb_sigmoid_scalar", lib.qb_sigmoid_scalar(_ptr(x), _ptr(s), x.numel(), _stream(stream)))


def qb_zero_i32(t, stream=None):
    _check("qb_zero_i32", lib.qb_zero_i32(_ptr(t), t.numel(), _stream(stream)))


def qb_route_hist_hi(logits, bias, k, hist_hi, keys_out=None, topk_out=None, alpha_out=None,
                     stream=None):
    N, E = logits.shape
    _check("qb_route_hist_hi",
           lib.qb_route_hist_hi(_ptr(logits), _dtype(logits), _ptr(bias), N, E, int(k),
                                _ptr(hist_hi), _ptr(keys_out), _ptr(topk_out), _ptr(alpha_out),
                                _stream(stream)))


def qb_route_hist_hi_next(logits, bias, k, hist_hi, keys_out=None, topk_out=None,
                          alpha_out=None, stream=None):
    N, E = logits.shape
    _check("qb_route_hist_hi_next",
           lib.qb_route_hist_hi_next(_ptr(logits), _dtype(logits), _ptr(bias), N, E, int(k),
                                     _ptr(hist_hi), _ptr(keys_out), _ptr(topk_out),
                                     _ptr(alpha_out), _stream(stream)))


def qb_select_hi(hist_hi, r, sel, r_lo, stream=None):
    E = hist_hi.shape[0]
    _check("qb_select_hi", lib.qb_select_hi(_ptr(hist_hi), E, int(r), _ptr(sel), _ptr(r_lo),
                                            _stream(stream)))


def qb_keys_hist_lo(keys, sel, hist_lo, stream=None):
    N, E = keys.shape
    _check("qb_keys_hist_lo", lib.qb_keys_hist_lo(_ptr(keys), N, E, _ptr(sel), _ptr(hist_lo),
                                                  _stream(stream)))


def qb_route_hist_lo(logits, bias, k, sel, hist_lo, stream=None):
    N, E = logits.shape
    _check("qb_route_hist_lo",
           lib.qb_route_hist_lo(_ptr(logits), _dtype(logits), _ptr(bias), N, E, int(k), _ptr(sel),
                                _ptr(hist_lo), _stream(stream)))


def qb_finalize(hist_hi, hist_lo, sel, r_lo, bias_out, qkey_out=None, reset=True, stream=None):
    E = hist_lo.shape[0]
    _check("qb_finalize",
           lib.qb_finalize(_ptr(hist_hi), _ptr(hist_lo), _ptr(sel), _ptr(r_lo), E, _ptr(bias_out),
                           _ptr(qkey_out), 1 if reset else 0, _stream(stream)))


def k3_route_hist(logits, bias, k, bounds, hist, alpha_out, stream=None):
    N, E = logits.shape
    nbins = hist.shape[1]
    _check("k3_route_hist",
           lib.k3_route_hist(_ptr(logits), _dtype(logits), _ptr(bias), N, E, int(k), _ptr(bounds),
                             nbins, _ptr(hist), _ptr(alpha_out), _stream(stream)))


def k3_route_hist_next(logits, bias, k, bounds, hist, alpha_out, stream=None):
    N, E = logits.shape
    nbins = hist.shape[1]
    _check("k3_route_hist_next",
           lib.k3_route_hist_next(_ptr(logits), _dtype(logits), _ptr(bias), N, E, int(k),
                                  _ptr(bounds), nbins, _ptr(hist), _ptr(alpha_out),
                                  _stream(stream)))


def k3_finalize(hist, r, bounds, bias_out, reset=True, stream=None):
    E, nbins = hist.shape
    _check("k3_finalize", lib.k3_finalize(_ptr(hist), E, nbins, int(r), _ptr(bounds),
                                          _ptr(bias_out), 1 if reset else 0, _stream(stream)))


def lei_inject(grad, topk_idx, eta, workspace, batch_tokens=0, stream=None):
    N, E = grad.shape
    k = topk_idx.shape[1]
    _check("lei_inject",
           lib.lei_inject(_ptr(grad), _ptr(topk_idx), N, E, int(k), float(eta), int(batch_tokens),
                          _ptr(workspace), _stream(stream)))


def lei_rho(topk_idx, E, eta, workspace, batch_tokens=0, stream=None):
    """First half of lei_inject: eta*rho per local batch into workspace."""
    N, k = topk_idx.shape
    _check("lei_rho", lib.lei_rho(_ptr(topk_idx), N, int(E), int(k), float(eta),
                                  int(batch_tokens), _ptr(workspace), _stream(stream)))


def lei_apply(grad, workspace, batch_tokens=0, stream=None):
    """Second half of lei_inject: grad += workspace[batch(row)]."""
    N, E = grad.shape
    _check("lei_apply", lib.lei_apply(_ptr(grad), N, E, int(batch_tokens), _ptr(workspace),
                                      _stream(stream)))


def lei_apply_overlap(grad, workspace, batch_tokens=0, stream=None):
    """lei_apply launched to run beside the kernel enqueued just before it
    on the stream (it must not touch grad or write workspace)."""
    N, E = grad.shape
    _check("lei_apply_overlap",
           lib.lei_apply_overlap(_ptr(grad), N, E, int(batch_tokens), _ptr(workspace),
                                 _stream(stream)))


def lei_inject_noalloc(grad, topk_idx, eta, batch_tokens=0, stream=None):
    """lei_inject with the library's own fixed scratch instead of a caller
    workspace (for callers that cannot allocate device memory)."""
    N, E = grad.shape
    k = topk_idx.shape[1]
    _check("lei_inject_noalloc",
           lib.lei_inject_noalloc(_ptr(grad), _ptr(topk_idx), N, E, int(k), float(eta),
                                  int(batch_tokens), _stream(stream)))


def qb_router_gemm(hidden, w_t, logits_out, stream=None):
    M, H = hidden.shape
    E = w_t.shape[0]
    _check("qb_router_gemm", lib.qb_router_gemm(_ptr(hidden), _ptr(w_t), M, H, E, _ptr(logits_out),
                                                _stream(stream)))


def qb_router_gemm_hist_hi(hidden, w_t, bias, k, logits_out, hist_hi, keys_out=None,
                           topk_out=None, alpha_out=None, stream=None):
    M, H = hidden.shape
    E = w_t.shape[0]
    _check("qb_router_gemm_hist_hi",
           lib.qb_router_gemm_hist_hi(_ptr(hidden), _ptr(w_t), M, H, E, int(k), _ptr(bias),
                                      _ptr(logits_out), _ptr(hist_hi), _ptr(keys_out),
                                      _ptr(topk_out), _ptr(alpha_out), _stream(stream)))


def qb_router_gemm_hist_hi_next(hidden, w_t, bias, k, logits_out, hist_hi, keys_out=None,
                                topk_out=None, alpha_out=None, stream=None):
    M, H = hidden.shape
    E = w_t.shape[0]
    _check("qb_router_gemm_hist_hi_next",
           lib.qb_router_gemm_hist_hi_next(_ptr(hidden), _ptr(w_t), M, H, E, int(k), _ptr(bias),
                                           _ptr(logits_out), _ptr(hist_hi), _ptr(keys_out),
                                           _ptr(topk_out), _ptr(alpha_out), _stream(stream)))


def qb_rank_average(qkeys, bias_out, stream=None):
    """qkeys: int16/uint16 [P, E] selected keys of P ranks -> centred average bias."""
    P, E = qkeys.shape
    _check("qb_rank_average", lib.qb_rank_average(_ptr(qkeys), P, E, _ptr(bias_out),
                                                  _stream(stream)))


def qb_maxvio(topk, E, loads_out, maxvio_out, batch_tokens=0, stream=None):
    N, k = topk.shape
    _check("qb_maxvio", lib.qb_maxvio(_ptr(topk), N, int(E), k, int(batch_tokens),
                                      _ptr(loads_out), _ptr(maxvio_out), _stream(stream)))


# ------------------------------------------------ balance loss, experts' products

_FP8 = (torch.float8_e4m3fn, torch.uint8)
_U8 = (torch.uint8,)
_BOOL = (torch.bool, torch.uint8)
_I32 = (torch.int32,)
_F32 = (torch.float32,)
_FLOATS = (torch.float32, torch.bfloat16)
_DTYPE = {torch.float32: QB_F32, torch.bfloat16: QB_BF16}


def _need(fn, name, t, dtypes, shape):
    """The address of a contiguous CUDA tensor of one of the types and of the shape; refuses others."""
    if t is None:
        raise TypeError(f"{fn}: {name} is required")
    if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.is_cuda:
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{fn}: {name} must be on the GPU, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{fn}: {name} must be {' or '.join(str(d) for d in dtypes)}, "
                        f"got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{fn}: {name} must be contiguous")


def _optional(fn, name, t, dtypes, shape):
    return None if t is None else _need(fn, name, t, dtypes, shape)


# the current stream's handle without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_int(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _score(score) -> int:
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return SCORES[score]


def _batches(N, batch_tokens) -> int:
    return -(-N // batch_tokens) if batch_tokens else 1


def _scratch(fn, t):
    """(address, bytes) of a workspace."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{fn}: workspace must be a contiguous CUDA tensor")
    return t.data_ptr(), t.nbytes


def _workspace(name, nbytes, device):
    if nbytes < 0:
        raise QBError(name, int(nbytes))
    return torch.zeros(max(16, int(nbytes)), dtype=torch.uint8, device=device)


def balance_workspace(N, E, batch_tokens=0, device="cuda"):
    """A zeroed workspace for qb_balance_loss; reusable call after call."""
    return _workspace("qb_balance_workspace",
                      lib.qb_balance_workspace(int(N), int(E), int(batch_tokens)), device)


def order_workspace(N, E, k, device="cuda"):
    """A workspace for qb_expert_order."""
    return _workspace("qb_order_workspace", lib.qb_order_workspace(int(N), int(E), int(k)), device)


def fp8_scale_pitch(n) -> int:
    """Bytes of one row of scales for n values: one for each 128, in whole 32-bit words."""
    return (n + 511) // 512 * 4


def fp8_cols_width(M, G) -> int:
    """Columns of qb_fp8_quantize_cols' codes for M rows in G groups."""
    return (M + 127 * G) // 128 * 128


def qb_balance_loss(logits, topk_idx, coeff, counts, tokens, prob_sum, loss, workspace,
                    token_mask=None, batch_tokens=0, score="sigmoid", stream=None):
    """Load-balance loss per local batch, with the per-expert counts and share sums."""
    fn = "qb_balance_loss"
    N, E = logits.shape
    k = topk_idx.shape[1]
    nb = _batches(N, batch_tokens)
    _check(fn, lib.qb_balance_loss(
        _need(fn, "logits", logits, _FLOATS, (N, E)), _DTYPE[logits.dtype],
        _need(fn, "topk_idx", topk_idx, _I32, (N, k)),
        _optional(fn, "token_mask", token_mask, _BOOL, (N,)), N, E, k, batch_tokens, _score(score),
        coeff, _need(fn, "counts", counts, _I32, (nb, E)), _need(fn, "tokens", tokens, _I32, (nb,)),
        _need(fn, "prob_sum", prob_sum, _F32, (nb, E)), _need(fn, "loss", loss, _F32, (nb,)),
        *_scratch(fn, workspace), _stream_int(stream)))


def qb_balance_grad(logits, counts, tokens, loss_grad, coeff, k, grad, token_mask=None,
                    batch_tokens=0, score="sigmoid", accumulate=False, stream=None):
    """Gradient of qb_balance_loss with respect to the logits, into grad (or added to it)."""
    fn = "qb_balance_grad"
    N, E = logits.shape
    nb = _batches(N, batch_tokens)
    _check(fn, lib.qb_balance_grad(
        _need(fn, "logits", logits, _FLOATS, (N, E)), _DTYPE[logits.dtype],
        _optional(fn, "token_mask", token_mask, _BOOL, (N,)),
        _need(fn, "counts", counts, _I32, (nb, E)), _need(fn, "tokens", tokens, _I32, (nb,)),
        _need(fn, "loss_grad", loss_grad, _F32, (nb,)), N, E, k, batch_tokens, _score(score), coeff,
        _need(fn, "grad", grad, _F32, (N, E)), 1 if accumulate else 0, _stream_int(stream)))


def qb_expert_order(topk_idx, E, counts, offsets, slot_of, token_of, workspace, stream=None):
    """Per-expert counts and offsets, and the stable order of the top-k entries by expert."""
    fn = "qb_expert_order"
    N, k = topk_idx.shape
    _check(fn, lib.qb_expert_order(
        _need(fn, "topk_idx", topk_idx, _I32, (N, k)), N, E, k,
        _need(fn, "counts", counts, _I32, (E,)), _need(fn, "offsets", offsets, _I32, (E + 1,)),
        _need(fn, "slot_of", slot_of, _I32, (N, k)),
        _need(fn, "token_of", token_of, _I32, (N * k,)), *_scratch(fn, workspace),
        _stream_int(stream)))


def _source(fn, x, row_idx):
    """(address, type, source rows, row stride, row indexes, rows of the result, K); x may have
    strided rows."""
    if x.dtype not in _FLOATS:
        raise TypeError(f"{fn}: x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() != 2 or x.stride(1) != 1 or not x.is_cuda:
        raise ValueError(f"{fn}: x must be [rows, K] on the GPU, each row contiguous")
    T, K = x.shape
    M, index = T, None
    if row_idx is not None:
        M = row_idx.numel()
        index = _need(fn, "row_idx", row_idx, _I32, (M,))
    return x.data_ptr(), _DTYPE[x.dtype], T, x.stride(0) if T > 1 else K, index, M, K


def qb_fp8_quantize_rows(x, q, scale, row_idx=None, stream=None):
    """e4m3 codes of x's rows (of the rows row_idx names), a scale for each 128 columns."""
    fn = "qb_fp8_quantize_rows"
    px, dtype, T, ld, index, M, K = _source(fn, x, row_idx)
    _check(fn, lib.qb_fp8_quantize_rows(
        px, dtype, T, ld, index, M, K, _need(fn, "q", q, _FP8, (M, K)),
        _need(fn, "scale", scale, _U8, (M, fp8_scale_pitch(K))), _stream_int(stream)))


def qb_fp8_quantize_cols(x, q_t, scale_t, offsets=None, row_idx=None, stream=None):
    """Transposed codes of x's rows in groups, a scale for each 128 tokens of a group."""
    fn = "qb_fp8_quantize_cols"
    px, dtype, T, ld, index, M, K = _source(fn, x, row_idx)
    G = 1 if offsets is None else offsets.numel() - 1
    width = q_t.shape[1]
    _check(fn, lib.qb_fp8_quantize_cols(
        px, dtype, T, ld, index, _optional(fn, "offsets", offsets, _I32, (G + 1,)), G, M, K, width,
        _need(fn, "q_t", q_t, _FP8, (K, width)),
        _need(fn, "scale_t", scale_t, _U8, (K, fp8_scale_pitch(width))), _stream_int(stream)))


def qb_fp8_quantize_blocks(w, q, scale, q_t=None, scale_t=None, stream=None):
    """Codes of weights w [G, N, K] in blocks of 128 x 128, and of their transposes."""
    fn = "qb_fp8_quantize_blocks"
    G, N, K = w.shape
    both = q_t is not None or scale_t is not None
    _check(fn, lib.qb_fp8_quantize_blocks(
        _need(fn, "w", w, _FLOATS, (G, N, K)), _DTYPE[w.dtype], G, N, K,
        _need(fn, "q", q, _FP8, (G, N, K)),
        _need(fn, "scale", scale, _U8, (G, -(-N // 128), fp8_scale_pitch(K))),
        _need(fn, "q_t", q_t, _FP8, (G, K, N)) if both else None,
        _need(fn, "scale_t", scale_t, _U8, (G, -(-K // 128), fp8_scale_pitch(N))) if both else None,
        _stream_int(stream)))


def qb_fp8_expert_gemm(a, a_scale, b, b_scale, out, offsets=None, stream=None):
    """out[r] = A[r] . B[g]^T for the rows offsets[g] .. offsets[g+1] - 1 of each expert g."""
    fn = "qb_fp8_expert_gemm"
    M, K = a.shape
    G, N = b.shape[:2]
    one = G == 1 and offsets is None
    _check(fn, lib.qb_fp8_expert_gemm(
        _need(fn, "a", a, _FP8, (M, K)),
        _need(fn, "a_scale", a_scale, _U8, (M, fp8_scale_pitch(K))),
        _need(fn, "b", b, _FP8, (G, N, K)),
        _need(fn, "b_scale", b_scale, _U8, (G, -(-N // 128), fp8_scale_pitch(K))),
        None if one else _need(fn, "offsets", offsets, _I32, (G + 1,)), G, M, N, K,
        _need(fn, "out", out, _FLOATS, (M, N)), _DTYPE[out.dtype], _stream_int(stream)))


def qb_fp8_expert_wgrad(a_t, a_scale, b_t, b_scale, out, offsets=None, accumulate=False,
                        stream=None):
    """out[g] (+)= A B^T over group g's columns, the experts' weight gradients."""
    fn = "qb_fp8_expert_wgrad"
    G, N, K = out.shape
    width = a_t.shape[1]
    one = G == 1 and offsets is None
    _check(fn, lib.qb_fp8_expert_wgrad(
        _need(fn, "a_t", a_t, _FP8, (N, width)),
        _need(fn, "a_scale", a_scale, _U8, (N, fp8_scale_pitch(width))),
        _need(fn, "b_t", b_t, _FP8, (K, width)),
        _need(fn, "b_scale", b_scale, _U8, (K, fp8_scale_pitch(width))),
        None if one else _need(fn, "offsets", offsets, _I32, (G + 1,)), G, width, N, K,
        _need(fn, "out", out, _FLOATS, (G, N, K)), _DTYPE[out.dtype], 1 if accumulate else 0,
        _stream_int(stream)))


def device_status() -> int:
    flags = ctypes.c_int(0)
    st = lib.qb_device_status(ctypes.byref(flags))
    if st == QB_ECUDA:
        raise QBError("qb_device_status", st)
    return int(flags.value)


# ---------------------------------------------------------------- convenience

class EQBState:
    """Device buffers of one router's EQB global batch (caller-owned memory).

    hist_hi / hist_lo: int32 [E,256]; sel / r_lo: int32 [E]."""

    def __init__(self, E: int, device="cuda"):
        self.E = E
        self.hist_hi = torch.zeros(E, 256, dtype=torch.int32, device=device)
        self.hist_lo = torch.zeros(E, 256, dtype=torch.int32, device=device)
        self.sel = torch.empty(E, dtype=torch.int32, device=device)
        self.r_lo = torch.empty(E, dtype=torch.int32, device=device)
        self.qkey = torch.empty(E, dtype=torch.int16, device=device)


def eqb_global_batch(microbatches, bias, k, state: EQBState | None = None, keys=None,
                     bias_out=None, reset=True, stream=None):
    """Hi pass per microbatch, select, lo pass over the stored keys, finalize.

    ``keys`` (uint16 as int16 [N_pool, E]) receives the keys of every
    microbatch in order; allocated when None.  Returns (state, bias_out)."""
    E = bias.shape[0]
    n_pool = sum(int(m.shape[0]) for m in microbatches)
    state = state or EQBState(E, bias.device)
    if keys is None:
        keys = torch.empty(n_pool, E, dtype=torch.int16, device=bias.device)
    if bias_out is None:
        bias_out = torch.empty_like(bias)
    row = 0
    first = True
    for m in microbatches:
        n = int(m.shape[0])
        if n == 0:
            continue  # issues no work
        # every microbatch after the first continues the batch on this stream
        route = qb_route_hist_hi if first else qb_route_hist_hi_next
        route(m, bias, k, state.hist_hi, keys_out=keys[row:row + n], stream=stream)
        first = False
        row += n
    r = rank(n_pool, E, k)
    qb_select_hi(state.hist_hi, r, state.sel, state.r_lo, stream=stream)
    qb_keys_hist_lo(keys, state.sel, state.hist_lo, stream=stream)
    qb_finalize(state.hist_hi, state.hist_lo, state.sel, state.r_lo, bias_out, qkey_out=state.qkey,
                reset=reset, stream=stream)
    return state, bias_out
