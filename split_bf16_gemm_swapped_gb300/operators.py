"""The operators around the decode projection: residual addition + RMS norm to
8-bit codes, quantisation, the product of 8-bit codes, log probabilities.

As in the package's other calls, PyTorch supplies device memory and streams
and every step runs in the library's kernels (``include/splitk.h`` says what
each computes).  The binding is compiled (``csrc/operators_binding.cpp``,
``_lib/_operators.so``): a single-token call takes the GPU a few microseconds,
less than its checks would take here.

A call's stream is the device's current one, or the one given as `stream`.
Outputs a call makes belong to that stream, as if it had been current.  As with
PyTorch's own calls, tensors of another stream are the caller's to order
(stream.wait_stream) and to keep until the work is done (tensor.record_stream).
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import threading

from . import SplitKError, _build, load_library

__all__ = ["splitk_rmsnorm_i8", "splitk_quantize_i8", "splitk_gemm_i8", "splitk_logprobs"]


def _load():
    """The compiled binding; raises if it has not been built."""
    load_library()
    path = _build.OPERATORS_LIB
    if not path.exists():
        raise RuntimeError(
            f"{path} is missing: build the binding first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    if _build.operators_built_for() != _build.operators_abi():
        raise RuntimeError(
            f"{path} was built for another PyTorch or Python ({_build.operators_built_for() or 'unknown'}; this is "
            f"{_build.operators_abi()}): build it again (python -c 'import __graft_entry__ as g; g.build()')")
    loader = importlib.machinery.ExtensionFileLoader("_operators", str(path))
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_operators", loader))
    import torch  # noqa: F401  (the binding's types)
    loader.exec_module(module)
    return module


class _Unloaded:
    """Stands for the binding until the first call: the names of this module need
    neither PyTorch nor the built binding."""

    _lock = threading.Lock()

    def __getattr__(self, name):
        global _native
        if name.startswith("__"):
            raise AttributeError(name)
        with self._lock:
            if _native is self:
                _native = _load()
        return getattr(_native, name)


_native = _Unloaded()


def splitk_rmsnorm_i8(x, weight, residual=None, eps: float = 1e-6, q=None, scale=None, residual_out=None,
                      stream=None):
    """Residual addition, RMS norm and 8-bit codes with a scale per row:
    y = x + residual, n = y * weight / sqrt(mean(y^2) + eps), codes
    q = round(n / scale) with scale = max|n| * (1 / 127), in float32.

    x [M, D] (rows any distance apart) or contiguous [L, M, D], bfloat16;
    residual contiguous of x's shape, bfloat16 or float32; weight [D],
    bfloat16 or float32.  Returns (q int8, scale float32 [M] or [L, M],
    residual_out): the sum y in the residual's type, None without a residual.
    residual_out may be the residual itself (updated in place)."""
    out = _native.rmsnorm_i8(x, weight, residual, eps, q, scale, residual_out, stream)
    if type(out) is int:
        raise SplitKError(out, "splitk_rmsnorm_i8")
    return out


def splitk_quantize_i8(x, q=None, scale=None, stream=None):
    """8-bit codes with a scale per row: activations (a row is a token) or weights
    (a row is a channel).  x as in splitk_rmsnorm_i8; returns (q int8, scale
    float32), to the bit what scale = (x.float().abs().amax(-1) / 127) and
    torch.round(x.float() / scale[..., None]) give on the GPU (scale at least
    2**-126)."""
    out = _native.quantize_i8(x, q, scale, stream)
    if type(out) is int:
        raise SplitKError(out, "splitk_quantize_i8")
    return out


def splitk_gemm_i8(a_q, a_scale, b_q, b_scale, c=None, bias=None, out_dtype=None, stream=None):
    """c = (b_q @ a_q^T) * b_scale * a_scale + bias: 8-bit codes with a scale
    per channel (a_scale [L, N] or [N]) and per token (b_scale [L, M] or [M]).

    a_q [L, N, K] or [N, K] and b_q [L, M, K] or [M, K] int8, contiguous, K a
    multiple of 16; bias [L, N] or [N] bfloat16.  Returns c [L, M, N] or
    [M, N]: bfloat16, or float32 where out_dtype or the c given says so."""
    out = _native.gemm_i8(a_q, a_scale, b_q, b_scale, c, bias, out_dtype, stream)
    if type(out) is int:
        raise SplitKError(out, "splitk_gemm_i8")
    return out


def splitk_logprobs(logits, tokens=None, top_k: int = 0, logprob=None, entropy=None, top_ids=None,
                    top_logprobs=None, stream=None):
    """Log probabilities of the given tokens, the entropy of each row and its
    top_k most probable tokens (0..32; equal logits by the lowest index).

    logits [M, V] (rows any distance apart) or contiguous [L, M, V], bfloat16,
    float16 or float32; tokens int64 [M] or [L, M], contiguous.  Returns
    (logprob, entropy, top_ids int64 [..., top_k], top_logprobs), float32 but
    the ids; logprob is None without tokens, the alternatives with top_k = 0."""
    out = _native.logprobs(logits, tokens, top_k, logprob, entropy, top_ids, top_logprobs, stream)
    if type(out) is int:
        raise SplitKError(out, "splitk_logprobs")
    return out
