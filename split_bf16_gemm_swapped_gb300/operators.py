"""The operators around the decode projection: residual addition + RMS norm to
8-bit codes, quantisation, the product of 8-bit codes, log probabilities.

As in the package's other calls, PyTorch supplies device memory and streams
and every step runs in the library's kernels (``include/splitk.h`` says what
each computes).  A single-token call takes the GPU a few microseconds, so the
binding keeps its own share small: plain comparisons, one allocation an
output, and the current stream's handle without a stream object.
"""
from __future__ import annotations

import torch

from . import SplitKError, load_library

__all__ = ["splitk_rmsnorm_i8", "splitk_quantize_i8", "splitk_gemm_i8", "splitk_logprobs"]

_BF16, _F16, _F32, _I8, _I64 = torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.int64
_CODES = {_BF16: 0, _F32: 1, _F16: 2}          # SPLITK_DTYPE_*
_empty = torch.empty
# the handle of a device's current stream (what torch.cuda.current_stream()
# wraps in an object, at the cost of a small kernel)
_stream_handle = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _type_error(name, t, allowed):
    return TypeError(f"{name} must be {allowed}, not {str(t.dtype)[6:]}")


def _other_device(device, **ts):
    """The error for operands that are not all on one GPU."""
    for name, t in ts.items():
        if t is not None and t.device != device:
            return ValueError(f"{name} must be on {device}, the operands' device")
    return ValueError("operands must be CUDA tensors")


def _given(t, name, shape, dtype, at):
    """Checks an output that the caller brings: a contiguous tensor of this
    shape and type on device `at`."""
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    if t.get_device() != at:
        raise ValueError(f"{name} must be on the operands' device")
    return t


def _rows(t, name):
    """(rows, width, row stride) of a tensor read as rows along its last
    dimension: [M, D] with contiguous rows any distance apart, or a contiguous
    [L, M, D]."""
    shape = t.shape
    if len(shape) == 2:
        rows, width = shape
        if t.is_contiguous():
            return rows, width, width
        step, inner = t.stride()
        if inner == 1 or width == 1:
            return rows, width, (step if rows > 1 else width)
    elif len(shape) == 3 and t.is_contiguous():
        return shape[0] * shape[1], shape[2], shape[2]
    raise ValueError(f"{name} is [M, D] with contiguous rows, or a contiguous [L, M, D]")


def _on_device(fn, at):
    """fn, called with device `at` current."""
    def call(*args):
        with torch.cuda.device(at):
            return fn(*args)
    return call


def _entry(name, at):
    """The library's entry point `name` for operands on device `at`."""
    fn = getattr(load_library(), name)
    return fn if _current_device() == at else _on_device(fn, at)


def splitk_rmsnorm_i8(x, weight, residual=None, eps: float = 1e-6, q=None, scale=None, residual_out=None,
                      stream=None):
    """Residual addition, RMS norm and 8-bit codes with a scale per row:
    y = x + residual, n = y * weight / sqrt(mean(y^2) + eps), codes
    q = round(n / scale) with scale = max|n| / 127.

    x [M, D] (rows any distance apart) or contiguous [L, M, D], bfloat16;
    residual contiguous of x's shape, bfloat16 or float32; weight [D],
    bfloat16 or float32.  Returns (q int8, scale float32 [M] or [L, M],
    residual_out): the sum y in the residual's type, None without a residual.
    residual_out may be the residual itself (updated in place)."""
    M, D, stride = _rows(x, "x")
    shape, at = x.shape, x.get_device()
    if x.dtype is not _BF16:
        raise _type_error("x", x, "bfloat16")
    if weight.dtype is not _BF16 and weight.dtype is not _F32:
        raise _type_error("weight", weight, "bfloat16 or float32")
    if weight.shape != (D,) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous tensor of shape ({D},)")
    if at < 0 or weight.get_device() != at or (residual is not None and residual.get_device() != at):
        raise _other_device(x.device, weight=weight, residual=residual)
    r_type = r_in = r_out = None
    if residual is not None:
        r_type = residual.dtype
        if r_type is not _BF16 and r_type is not _F32:
            raise _type_error("residual", residual, "bfloat16 or float32")
        r_in = _given(residual, "residual", shape, r_type, at).data_ptr()
        residual_out = (_empty(shape, dtype=r_type, device=residual.device) if residual_out is None
                        else _given(residual_out, "residual_out", shape, r_type, at))
        r_out = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    q = _empty(shape, dtype=_I8, device=x.device) if q is None else _given(q, "q", shape, _I8, at)
    scale = (_empty(shape[:-1], dtype=_F32, device=x.device) if scale is None
             else _given(scale, "scale", shape[:-1], _F32, at))
    rc = _entry("splitk_rmsnorm_i8", at)(
        x.data_ptr(), stride, r_in, r_out, _CODES.get(r_type, 0), weight.data_ptr(), _CODES[weight.dtype], eps,
        q.data_ptr(), scale.data_ptr(), M, D,
        _stream_handle(at) if stream is None else stream.cuda_stream)
    if rc != 0:
        raise SplitKError(rc, "splitk_rmsnorm_i8")
    return q, scale, residual_out


def splitk_quantize_i8(x, q=None, scale=None, stream=None):
    """8-bit codes with a scale per row, scale = max|x| / 127: activations
    (a row is a token) or weights (a row is a channel).  x as in
    splitk_rmsnorm_i8; returns (q int8, scale float32)."""
    M, D, stride = _rows(x, "x")
    shape, at = x.shape, x.get_device()
    if x.dtype is not _BF16:
        raise _type_error("x", x, "bfloat16")
    if at < 0:
        raise _other_device(x.device)
    q = _empty(shape, dtype=_I8, device=x.device) if q is None else _given(q, "q", shape, _I8, at)
    scale = (_empty(shape[:-1], dtype=_F32, device=x.device) if scale is None
             else _given(scale, "scale", shape[:-1], _F32, at))
    rc = _entry("splitk_quantize_i8", at)(
        x.data_ptr(), stride, q.data_ptr(), scale.data_ptr(), M, D,
        _stream_handle(at) if stream is None else stream.cuda_stream)
    if rc != 0:
        raise SplitKError(rc, "splitk_quantize_i8")
    return q, scale


def splitk_gemm_i8(a_q, a_scale, b_q, b_scale, c=None, bias=None, out_dtype=None, stream=None):
    """c = (b_q @ a_q^T) * b_scale * a_scale + bias: 8-bit codes with a scale
    per channel (a_scale [L, N] or [N]) and per token (b_scale [L, M] or [M]).

    a_q [L, N, K] or [N, K] and b_q [L, M, K] or [M, K] int8, contiguous, K a
    multiple of 16; bias [L, N] or [N] bfloat16.  Returns c [L, M, N] or
    [M, N]: bfloat16, or float32 where out_dtype or the c given says so."""
    if a_q.dtype is not _I8 or b_q.dtype is not _I8:
        raise TypeError("a_q and b_q must be int8")
    if a_scale.dtype is not _F32 or b_scale.dtype is not _F32:
        raise TypeError("a_scale and b_scale must be float32")
    a_shape, b_shape = a_q.shape, b_q.shape
    if len(a_shape) == 2 and len(b_shape) == 2:
        (N, K), (M, Kb) = a_shape, b_shape
        L, channels, tokens, outputs = 1, (N,), (M,), (M, N)
        fits = K == Kb
    elif len(a_shape) == 3 and len(b_shape) == 3:
        (L, N, K), (Lb, M, Kb) = a_shape, b_shape
        channels, tokens, outputs = (L, N), (L, M), (L, M, N)
        fits = K == Kb and L == Lb
    else:
        raise ValueError("a_q is [L, N, K] or [N, K]; b_q is [L, M, K] or [M, K]")
    if not fits or a_scale.shape != channels or b_scale.shape != tokens:
        raise ValueError(f"shape mismatch: a_q{tuple(a_shape)} a_scale{tuple(a_scale.shape)} "
                         f"b_q{tuple(b_shape)} b_scale{tuple(b_scale.shape)}")
    if not (a_q.is_contiguous() and a_scale.is_contiguous() and b_q.is_contiguous() and b_scale.is_contiguous()):
        raise ValueError("operands must be contiguous")
    at = a_q.get_device()
    if (at < 0 or a_scale.get_device() != at or b_q.get_device() != at or b_scale.get_device() != at or
            (bias is not None and bias.get_device() != at)):
        raise _other_device(a_q.device, a_scale=a_scale, b_q=b_q, b_scale=b_scale, bias=bias)
    if bias is not None and (bias.dtype is not _BF16 or bias.shape != channels or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous bfloat16 tensor of shape {channels}")
    if out_dtype is None:
        out_dtype = _BF16 if c is None else c.dtype
    if out_dtype is not _BF16 and out_dtype is not _F32:
        raise TypeError(f"c must be bfloat16 or float32, not {str(out_dtype)[6:]}")
    c = _empty(outputs, dtype=out_dtype, device=a_q.device) if c is None else _given(c, "c", outputs, out_dtype, at)
    rc = _entry("splitk_gemm_i8", at)(
        a_q.data_ptr(), a_scale.data_ptr(), b_q.data_ptr(), b_scale.data_ptr(),
        None if bias is None else bias.data_ptr(), c.data_ptr(), _CODES[out_dtype], M, N, K, L,
        _stream_handle(at) if stream is None else stream.cuda_stream)
    if rc != 0:
        raise SplitKError(rc, "splitk_gemm_i8")
    return c


def splitk_logprobs(logits, tokens=None, top_k: int = 0, logprob=None, entropy=None, top_ids=None,
                    top_logprobs=None, stream=None):
    """Log probabilities of the given tokens, the entropy of each row and its
    top_k most probable tokens (0..32; equal logits by the lowest index).

    logits [M, V] (rows any distance apart) or contiguous [L, M, V], bfloat16,
    float16 or float32; tokens int64 [M] or [L, M], contiguous.  Returns
    (logprob, entropy, top_ids int64 [..., top_k], top_logprobs), float32 but
    the ids; logprob is None without tokens, the alternatives with top_k = 0."""
    M, V, stride = _rows(logits, "logits")
    kind = logits.dtype
    if kind not in _CODES:
        raise _type_error("logits", logits, "bfloat16, float16 or float32")
    device, at, shape = logits.device, logits.get_device(), logits.shape[:-1]
    if at < 0 or (tokens is not None and tokens.get_device() != at):
        raise _other_device(device, tokens=tokens)
    t_ptr = l_ptr = i_ptr = p_ptr = None
    if tokens is not None:
        if tokens.dtype is not _I64 or tokens.shape != shape or not tokens.is_contiguous():
            raise ValueError(f"tokens must be a contiguous int64 tensor of shape {tuple(shape)}")
        logprob = (_empty(shape, dtype=_F32, device=device) if logprob is None
                   else _given(logprob, "logprob", shape, _F32, at))
        t_ptr, l_ptr = tokens.data_ptr(), logprob.data_ptr()
    elif logprob is not None:
        raise ValueError("logprob needs tokens")
    entropy = (_empty(shape, dtype=_F32, device=device) if entropy is None
               else _given(entropy, "entropy", shape, _F32, at))
    if top_k > 0:
        tops = (*shape, top_k)
        top_ids = (_empty(tops, dtype=_I64, device=device) if top_ids is None
                   else _given(top_ids, "top_ids", tops, _I64, at))
        top_logprobs = (_empty(tops, dtype=_F32, device=device) if top_logprobs is None
                        else _given(top_logprobs, "top_logprobs", tops, _F32, at))
        i_ptr, p_ptr = top_ids.data_ptr(), top_logprobs.data_ptr()
    elif top_ids is not None or top_logprobs is not None:
        raise ValueError("the alternatives' outputs need top_k > 0")
    rc = _entry("splitk_logprobs", at)(
        logits.data_ptr(), _CODES[kind], stride, t_ptr, l_ptr, entropy.data_ptr(), top_k, i_ptr, p_ptr, M, V,
        _stream_handle(at) if stream is None else stream.cuda_stream)
    if rc != 0:
        raise SplitKError(rc, "splitk_logprobs")
    return logprob, entropy, top_ids, top_logprobs
