"""GB300-native split-K BF16 decode GEMM: ``C[M, N] = B[M, K] @ A[N, K]^T``.

A thin ctypes binding over the C ABI in ``include/splitk.h``
(``_lib/libsplitk_sm103a.so``, built in-tree by ``__graft_entry__.build()`` or
``split_bf16_gemm_swapped_gb300._build.build_all()``).  It only marshals
arguments: every step of the GEMM runs in the library's sm_103a kernels, and
there is no CPU or PyTorch fallback -- if the library is missing, importing a
function that needs it raises.

PyTorch supplies device memory and streams.  Tensors:
  a  weights      [L, N, K] (or [N, K]) bfloat16, CUDA, contiguous
  b  activations  [L, M, K] (or [M, K]) bfloat16, CUDA, contiguous
  c  output       [L, M, N] (or [M, N]) bfloat16, CUDA, contiguous
"""
from __future__ import annotations

import ctypes
from pathlib import Path

from . import _build

__all__ = [
    "SplitKError", "Plan", "Fault", "library_path", "load_library",
    "splitk_plan", "splitk_plan_for", "splitk_gemm_bf16", "splitk_gemm_bf16_planned",
    "splitk_gemm_bf16_hostio", "splitk_gemm_bf16_zerocopy", "splitk_gemm_bf16_noalloc",
    "splitk_gemm_bf16_bias",
    "splitk_plan_check_for", "splitk_plan_candidates_for", "splitk_tune",
    "splitk_plan_w4a16", "splitk_plan_w4a16_for", "splitk_gemm_w4a16", "splitk_gemm_w4a16_planned",
    "splitk_plan_w8a16", "splitk_plan_w8a16_for", "splitk_gemm_w8a16", "splitk_gemm_w8a16_planned",
    "splitk_rmsnorm_i8", "splitk_quantize_i8", "splitk_gemm_i8", "splitk_logprobs",
    "splitk_get_fault",
    "splitk_get_status",
    "splitk_set_wait_limit_ns", "splitk_debug_inject", "splitk_release", "splitk_cache_info",
    "splitk_strerror", "splitk_version", "splitk_set_trace", "FLAG_NO_PDL",
    "INJECT_SKIP_PUBLISH", "TRACE_SLOTS", "TRACE_FIELDS",
    "STATUS",
]

FLAG_NO_PDL = 0x1
INJECT_SKIP_PUBLISH = 0x1

STATUS = {
    0: "SPLITK_OK", -1: "SPLITK_ERR_INVALID_SHAPE", -2: "SPLITK_ERR_MISALIGNED",
    -3: "SPLITK_ERR_UNSUPPORTED_SPLIT", -4: "SPLITK_ERR_NO_FIT", -5: "SPLITK_ERR_CUDA",
    -6: "SPLITK_ERR_TIMEOUT", -7: "SPLITK_ERR_NULL", -8: "SPLITK_ERR_CACHE_FULL",
    -9: "SPLITK_ERR_UNSUPPORTED_DEVICE", -10: "SPLITK_ERR_BAD_PLAN",
    -11: "SPLITK_ERR_SCRATCH", -12: "SPLITK_ERR_NOT_MAPPED", -13: "SPLITK_ERR_CAPTURE",
    -14: "SPLITK_ERR_INVALID_ARGUMENT",
}


class SplitKError(RuntimeError):
    def __init__(self, code: int, where: str = ""):
        self.code = int(code)
        self.name = STATUS.get(self.code, str(code))
        msg = f"{self.name}: {splitk_strerror(self.code)}"
        super().__init__(f"{where}: {msg}" if where else msg)


class Plan(ctypes.Structure):
    _fields_ = [
        ("mma_m", ctypes.c_int), ("mma_n", ctypes.c_int), ("stages", ctypes.c_int),
        ("split_k", ctypes.c_int), ("k_tiles_per_cta", ctypes.c_int),
        ("mailbox_dedicated", ctypes.c_int), ("mailbox_quads", ctypes.c_int),
        ("reduce_rounds", ctypes.c_int), ("grid", ctypes.c_uint * 3),
        ("cluster", ctypes.c_uint * 3), ("smem_bytes", ctypes.c_size_t),
        ("ctas_per_sm", ctypes.c_int), ("pdl_trigger", ctypes.c_int),
        ("reduce_scatter", ctypes.c_int), ("b_resident", ctypes.c_int),
        ("a_tmem_tiles", ctypes.c_int), ("tmem_cols", ctypes.c_uint),
        ("mma_issuers", ctypes.c_int), ("b_loader", ctypes.c_int),
        ("l2_prefetch", ctypes.c_int), ("weight_format", ctypes.c_int),
        ("w4_smem_tiles", ctypes.c_int), ("b_stages", ctypes.c_int),
        ("persistent", ctypes.c_int), ("w4_decoders", ctypes.c_int),
    ]

    def as_dict(self) -> dict:
        d = {k: getattr(self, k) for k, _ in self._fields_}
        d["grid"] = list(self.grid)
        d["cluster"] = list(self.cluster)
        return d

    def __repr__(self) -> str:
        return f"Plan({self.as_dict()})"


class Fault(ctypes.Structure):
    _fields_ = [("code", ctypes.c_int), ("role", ctypes.c_int), ("index", ctypes.c_int),
                ("parity", ctypes.c_int), ("block", ctypes.c_int * 3),
                ("cluster_rank", ctypes.c_int)]

    def as_dict(self) -> dict:
        d = {k: getattr(self, k) for k, _ in self._fields_}
        d["block"] = list(self.block)
        return d


_lib = None


def library_path() -> Path:
    return _build.SPLITK_LIB


def load_library():
    """Loads the CUDA library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not path.exists():
        raise RuntimeError(
            f"{path} is missing: build the sm_103a library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(str(path))
    vp, i, u, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
    lib.splitk_plan.argtypes = [i, i, i, i, i, ctypes.POINTER(Plan)]
    lib.splitk_plan.restype = i
    lib.splitk_plan_for.argtypes = [i, i, i, i, i, i, sz, sz, ctypes.POINTER(Plan)]
    lib.splitk_plan_for.restype = i
    lib.splitk_gemm_bf16.argtypes = [vp, vp, vp, i, i, i, i, i, vp]
    lib.splitk_gemm_bf16.restype = i
    lib.splitk_plan_w4a16_for.argtypes = [i, i, i, i, i, i, sz, sz, ctypes.POINTER(Plan)]
    lib.splitk_plan_w4a16_for.restype = i
    lib.splitk_plan_w4a16.argtypes = [i, i, i, i, i, ctypes.POINTER(Plan)]
    lib.splitk_plan_w4a16.restype = i
    lib.splitk_gemm_w4a16.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.splitk_gemm_w4a16.restype = i
    lib.splitk_gemm_w4a16_planned.argtypes = [vp, vp, vp, vp, i, i, i, i, ctypes.POINTER(Plan), u, vp]
    lib.splitk_gemm_w4a16_planned.restype = i
    lib.splitk_plan_w8a16_for.argtypes = [i, i, i, i, i, i, sz, sz, ctypes.POINTER(Plan)]
    lib.splitk_plan_w8a16_for.restype = i
    lib.splitk_plan_w8a16.argtypes = [i, i, i, i, i, ctypes.POINTER(Plan)]
    lib.splitk_plan_w8a16.restype = i
    lib.splitk_gemm_w8a16.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.splitk_gemm_w8a16.restype = i
    lib.splitk_gemm_w8a16_planned.argtypes = [vp, vp, vp, vp, i, i, i, i, ctypes.POINTER(Plan), u, vp]
    lib.splitk_gemm_w8a16_planned.restype = i
    lib.splitk_plan_check_for.argtypes = [ctypes.POINTER(Plan), i, i, i, i, sz, sz]
    lib.splitk_plan_check_for.restype = i
    lib.splitk_plan_candidates_for.argtypes = [i, i, i, i, i, i, sz, sz, ctypes.POINTER(Plan), i]
    lib.splitk_plan_candidates_for.restype = i
    lib.splitk_tune.argtypes = [ctypes.POINTER(vp), i, vp, vp, i, i, i, i, i, i, vp, ctypes.POINTER(Plan),
                                ctypes.POINTER(ctypes.c_float)]
    lib.splitk_tune.restype = i
    lib.splitk_gemm_bf16_bias.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.splitk_gemm_bf16_bias.restype = i
    lib.splitk_gemm_bf16_planned.argtypes = [vp, vp, vp, i, i, i, i, ctypes.POINTER(Plan), u, vp]
    lib.splitk_gemm_bf16_planned.restype = i
    lib.splitk_gemm_bf16_hostio.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.splitk_gemm_bf16_hostio.restype = i
    lib.splitk_gemm_bf16_zerocopy.argtypes = [vp, vp, vp, i, i, i, i, i, vp]
    lib.splitk_gemm_bf16_zerocopy.restype = i
    lib.splitk_gemm_bf16_noalloc.argtypes = [vp, vp, vp, i, i, i, i, i, vp]
    lib.splitk_gemm_bf16_noalloc.restype = i
    ll, f = ctypes.c_longlong, ctypes.c_float
    lib.splitk_rmsnorm_i8.argtypes = [vp, ll, vp, vp, i, vp, i, f, vp, vp, i, i, vp]
    lib.splitk_rmsnorm_i8.restype = i
    lib.splitk_quantize_i8.argtypes = [vp, ll, vp, vp, i, i, vp]
    lib.splitk_quantize_i8.restype = i
    lib.splitk_gemm_i8.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.splitk_gemm_i8.restype = i
    lib.splitk_logprobs.argtypes = [vp, i, ll, vp, vp, vp, i, vp, vp, i, i, vp]
    lib.splitk_logprobs.restype = i
    lib.splitk_get_fault.argtypes = [ctypes.POINTER(Fault)]
    lib.splitk_get_fault.restype = i
    lib.splitk_get_status.argtypes = []
    lib.splitk_get_status.restype = i
    lib.splitk_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.splitk_set_wait_limit_ns.restype = i
    lib.splitk_debug_inject.argtypes = [u]
    lib.splitk_debug_inject.restype = i
    lib.splitk_set_trace.argtypes = [vp, sz]
    lib.splitk_set_trace.restype = i
    lib.splitk_release.argtypes = []
    lib.splitk_release.restype = None
    lib.splitk_cache_info.argtypes = [ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(i)]
    lib.splitk_cache_info.restype = i
    lib.splitk_strerror.argtypes = [i]
    lib.splitk_strerror.restype = ctypes.c_char_p
    lib.splitk_version.argtypes = []
    lib.splitk_version.restype = i
    _lib = lib
    return lib


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise SplitKError(rc, where)


# ---------------------------------------------------------------- planning
def splitk_plan(M: int, N: int, K: int, L: int = 1, split_k: int = 0) -> Plan:
    out = Plan()
    _check(load_library().splitk_plan(M, N, K, L, split_k, ctypes.byref(out)), "splitk_plan")
    return out


def splitk_plan_for(M: int, N: int, K: int, L: int, split_k: int, num_sms: int,
                    smem_per_sm: int, smem_per_block_optin: int) -> Plan:
    out = Plan()
    _check(load_library().splitk_plan_for(M, N, K, L, split_k, num_sms, smem_per_sm,
                                          smem_per_block_optin, ctypes.byref(out)),
           "splitk_plan_for")
    return out


# ---------------------------------------------------------------- GEMM
def _dims(a, b):
    import torch
    if a.dim() not in (2, 3) or b.dim() != a.dim():
        raise ValueError("a is [L, N, K] or [N, K]; b is [L, M, K] or [M, K]")
    if a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16:
        raise TypeError("a and b must be bfloat16")
    if a.dim() == 2:
        (N, K), (M, Kb), L = a.shape, b.shape, 1
        Lb = 1
    else:
        (L, N, K), (Lb, M, Kb) = a.shape, b.shape
    if K != Kb or L != Lb:
        raise ValueError(f"shape mismatch: a{tuple(a.shape)} b{tuple(b.shape)}")
    return int(M), int(N), int(K), int(L)


def _stream_handle(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(int(stream.cuda_stream))


def _out(c, a, M, N, L):
    import torch
    shape = (M, N) if a.dim() == 2 else (L, M, N)
    if c is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=a.device)
    if tuple(c.shape) != shape or c.dtype != torch.bfloat16 or not c.is_contiguous():
        raise ValueError(f"c must be a contiguous bfloat16 tensor of shape {shape}")
    if c.device != a.device:
        raise ValueError(f"c must be on {a.device}, the operands' device")
    return c


def _require_cuda(*ts):
    for t in ts:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("operands must be contiguous CUDA tensors")
    if len({str(t.device) for t in ts}) > 1:
        raise ValueError("operands must be on one device")


def splitk_gemm_bf16(a, b, c=None, split_k: int = 0, stream=None):
    """c = b @ a^T (per batch), written once; returns c."""
    import torch
    M, N, K, L = _dims(a, b)
    _require_cuda(a, b)
    c = _out(c, a, M, N, L)
    _require_cuda(c)
    with torch.cuda.device(a.device):
        rc = load_library().splitk_gemm_bf16(
            a.data_ptr(), b.data_ptr(), c.data_ptr(), M, N, K, L, int(split_k),
            _stream_handle(stream, a.device))
    _check(rc, "splitk_gemm_bf16")
    return c


WEIGHTS_BF16 = 0
WEIGHTS_E2M1_E8M0 = 1
WEIGHTS_E4M3_E8M0 = 2


def splitk_plan_w4a16_for(M: int, N: int, K: int, L: int, split_k: int, num_sms: int,
                          smem_per_sm: int, smem_per_block_optin: int) -> Plan:
    """The A16W4 plan for a described device (no CUDA)."""
    p = Plan()
    _check(load_library().splitk_plan_w4a16_for(M, N, K, L, split_k, num_sms, smem_per_sm,
                                                smem_per_block_optin, ctypes.byref(p)),
           "splitk_plan_w4a16_for")
    return p


def splitk_plan_w4a16(M: int, N: int, K: int, L: int = 1, split_k: int = 0) -> Plan:
    p = Plan()
    _check(load_library().splitk_plan_w4a16(M, N, K, L, split_k, ctypes.byref(p)), "splitk_plan_w4a16")
    return p


def _w4_dims(a_q, a_s, b):
    import torch
    if a_q.dtype != torch.uint8 or a_s.dtype != torch.uint8:
        raise TypeError("A16W4 codes and scales are uint8 tensors")
    if b.dtype != torch.bfloat16:
        raise TypeError("b must be bfloat16")
    if a_q.dim() not in (2, 3) or a_s.dim() != a_q.dim() or b.dim() != a_q.dim():
        raise ValueError("a_q is [L, N, K/2] or [N, K/2], a_s [L, N, K/32] or [N, K/32], b [L, M, K] or [M, K]")
    if a_q.dim() == 2:
        a_q, a_s = a_q.unsqueeze(0), a_s.unsqueeze(0)
    if b.dim() == 2:
        b = b.unsqueeze(0)
    L, N, K2 = a_q.shape
    K = 2 * K2
    if tuple(a_s.shape) != (L, N, K // 32) or b.shape[0] != L or b.shape[2] != K:
        raise ValueError(f"shape mismatch a_q{tuple(a_q.shape)} a_s{tuple(a_s.shape)} b{tuple(b.shape)}")
    for t in (a_q, a_s, b):
        if not t.is_contiguous():
            raise ValueError("operands must be contiguous")
    return int(b.shape[1]), N, K, L


def splitk_gemm_w4a16(a_q, a_s, b, c=None, split_k: int = 0, stream=None):
    """c = b @ dequant(a_q, a_s)^T (4-bit E2M1 codes, E8M0 scales per 32 k)."""
    import torch
    M, N, K, L = _w4_dims(a_q, a_s, b)
    _require_cuda(a_q, a_s, b)
    c = _out(c, b, M, N, L)
    with torch.cuda.device(b.device):
        rc = load_library().splitk_gemm_w4a16(a_q.data_ptr(), a_s.data_ptr(), b.data_ptr(), c.data_ptr(),
                                              M, N, K, L, int(split_k), _stream_handle(stream, b.device))
    _check(rc, "splitk_gemm_w4a16")
    return c


def splitk_gemm_w4a16_planned(a_q, a_s, b, c, plan: Plan, flags: int = 0, stream=None):
    import torch
    M, N, K, L = _w4_dims(a_q, a_s, b)
    _require_cuda(a_q, a_s, b)
    c = _out(c, b, M, N, L)
    with torch.cuda.device(b.device):
        rc = load_library().splitk_gemm_w4a16_planned(a_q.data_ptr(), a_s.data_ptr(), b.data_ptr(),
                                                      c.data_ptr(), M, N, K, L, ctypes.byref(plan),
                                                      int(flags), _stream_handle(stream, b.device))
    _check(rc, "splitk_gemm_w4a16_planned")
    return c


# ---------------------------------------------------------------- A16W8
def splitk_plan_w8a16_for(M: int, N: int, K: int, L: int, split_k: int, num_sms: int,
                          smem_per_sm: int, smem_per_block_optin: int) -> Plan:
    """The A16W8 plan for a described device (no CUDA)."""
    p = Plan()
    _check(load_library().splitk_plan_w8a16_for(M, N, K, L, split_k, num_sms, smem_per_sm,
                                                smem_per_block_optin, ctypes.byref(p)),
           "splitk_plan_w8a16_for")
    return p


def splitk_plan_w8a16(M: int, N: int, K: int, L: int = 1, split_k: int = 0) -> Plan:
    p = Plan()
    _check(load_library().splitk_plan_w8a16(M, N, K, L, split_k, ctypes.byref(p)), "splitk_plan_w8a16")
    return p


def _w8_dims(a_q, a_s, b):
    import torch
    if a_q.dtype != torch.uint8 or a_s.dtype != torch.uint8:
        raise TypeError("A16W8 codes and scales are uint8 tensors")
    if b.dtype != torch.bfloat16:
        raise TypeError("b must be bfloat16")
    if a_q.dim() not in (2, 3) or a_s.dim() != a_q.dim() or b.dim() != a_q.dim():
        raise ValueError("a_q is [L, N, K] or [N, K], a_s [L, N, K/32] or [N, K/32], b [L, M, K] or [M, K]")
    if a_q.dim() == 2:
        a_q, a_s = a_q.unsqueeze(0), a_s.unsqueeze(0)
    if b.dim() == 2:
        b = b.unsqueeze(0)
    L, N, K = a_q.shape
    if tuple(a_s.shape) != (L, N, K // 32) or b.shape[0] != L or b.shape[2] != K:
        raise ValueError(f"shape mismatch a_q{tuple(a_q.shape)} a_s{tuple(a_s.shape)} b{tuple(b.shape)}")
    for t in (a_q, a_s, b):
        if not t.is_contiguous():
            raise ValueError("operands must be contiguous")
    return int(b.shape[1]), N, K, L


def splitk_gemm_w8a16(a_q, a_s, b, c=None, split_k: int = 0, stream=None):
    """c = b @ dequant(a_q, a_s)^T (8-bit E4M3 codes, E8M0 scales per 32 k)."""
    import torch
    M, N, K, L = _w8_dims(a_q, a_s, b)
    _require_cuda(a_q, a_s, b)
    c = _out(c, b, M, N, L)
    with torch.cuda.device(b.device):
        rc = load_library().splitk_gemm_w8a16(a_q.data_ptr(), a_s.data_ptr(), b.data_ptr(), c.data_ptr(),
                                              M, N, K, L, int(split_k), _stream_handle(stream, b.device))
    _check(rc, "splitk_gemm_w8a16")
    return c


def splitk_gemm_w8a16_planned(a_q, a_s, b, c, plan: Plan, flags: int = 0, stream=None):
    import torch
    M, N, K, L = _w8_dims(a_q, a_s, b)
    _require_cuda(a_q, a_s, b)
    c = _out(c, b, M, N, L)
    with torch.cuda.device(b.device):
        rc = load_library().splitk_gemm_w8a16_planned(a_q.data_ptr(), a_s.data_ptr(), b.data_ptr(),
                                                      c.data_ptr(), M, N, K, L, ctypes.byref(plan),
                                                      int(flags), _stream_handle(stream, b.device))
    _check(rc, "splitk_gemm_w8a16_planned")
    return c


def splitk_plan_check_for(plan: Plan, M: int, N: int, K: int, L: int, smem_per_sm: int,
                          smem_per_block_optin: int) -> int:
    """The launch-time plan check for a described device; returns the status."""
    return load_library().splitk_plan_check_for(ctypes.byref(plan), M, N, K, L, smem_per_sm,
                                                smem_per_block_optin)


def splitk_plan_candidates_for(M: int, N: int, K: int, L: int, split_k: int, num_sms: int,
                               smem_per_sm: int, smem_per_block_optin: int) -> list:
    """Every valid tactic for the shape on a described device (the plan's
    own choice first)."""
    lib = load_library()
    n = lib.splitk_plan_candidates_for(M, N, K, L, split_k, num_sms, smem_per_sm,
                                       smem_per_block_optin, None, 0)
    _check(n if n < 0 else 0, "splitk_plan_candidates_for")
    arr = (Plan * max(n, 1))()
    got = lib.splitk_plan_candidates_for(M, N, K, L, split_k, num_sms, smem_per_sm,
                                         smem_per_block_optin, arr, n)
    _check(got if got < 0 else 0, "splitk_plan_candidates_for")
    return [Plan.from_buffer_copy(arr[k]) for k in range(n)]


def splitk_tune(a_list, b, c=None, split_k: int = 0, reps: int = 64, stream=None):
    """The fastest candidate tactic measured on this device, cycling through
    the same-shape weight tensors `a_list`; returns (plan, us_per_call)."""
    import torch
    M, N, K, L = _dims(a_list[0], b)
    for a in a_list:
        if tuple(a.shape) != tuple(a_list[0].shape) or a.dtype != a_list[0].dtype:
            raise ValueError("the weight tensors must have one shape and dtype")
    _require_cuda(*a_list, b)
    c = _out(c, a_list[0], M, N, L)
    ptrs = (ctypes.c_void_p * len(a_list))(*[a.data_ptr() for a in a_list])
    plan = Plan()
    us = ctypes.c_float(0.0)
    with torch.cuda.device(b.device):
        rc = load_library().splitk_tune(ptrs, len(a_list), b.data_ptr(), c.data_ptr(), M, N, K, L,
                                        int(split_k), int(reps), _stream_handle(stream, b.device),
                                        ctypes.byref(plan), ctypes.byref(us))
    _check(rc, "splitk_tune")
    return plan, float(us.value)


def splitk_gemm_bf16_bias(a, b, bias, c=None, split_k: int = 0, stream=None):
    """c = b @ a^T + bias (bias [L, N] or [N] bfloat16, added in FP32 before
    the one rounding); returns c."""
    import torch
    M, N, K, L = _dims(a, b)
    _require_cuda(a, b, bias)
    if bias.dtype != torch.bfloat16 or bias.numel() != L * N:
        raise ValueError("bias must be a bfloat16 tensor of L*N elements")
    c = _out(c, a, M, N, L)
    _require_cuda(c)
    with torch.cuda.device(a.device):
        rc = load_library().splitk_gemm_bf16_bias(
            a.data_ptr(), b.data_ptr(), bias.data_ptr(), c.data_ptr(), M, N, K, L,
            int(split_k), _stream_handle(stream, a.device))
    _check(rc, "splitk_gemm_bf16_bias")
    return c


def splitk_gemm_bf16_noalloc(a, b, c, split_k: int = 0, stream=None):
    """c = b @ a^T through the allocation-free entry point.

    For callers that cannot allocate device memory (see splitk.h): the C
    call allocates nothing, so `c` must be given -- this wrapper does not
    create it either.  Same kernel and results as splitk_gemm_bf16."""
    import torch
    M, N, K, L = _dims(a, b)
    _require_cuda(a, b)
    if c is None:
        raise ValueError("splitk_gemm_bf16_noalloc needs a preallocated output c")
    c = _out(c, a, M, N, L)
    _require_cuda(c)
    with torch.cuda.device(a.device):
        rc = load_library().splitk_gemm_bf16_noalloc(
            a.data_ptr(), b.data_ptr(), c.data_ptr(), M, N, K, L, int(split_k),
            _stream_handle(stream, a.device))
    _check(rc, "splitk_gemm_bf16_noalloc")
    return c


def splitk_gemm_bf16_planned(a, b, c, plan: Plan, flags: int = 0, stream=None):
    import torch
    M, N, K, L = _dims(a, b)
    _require_cuda(a, b)
    c = _out(c, a, M, N, L)
    _require_cuda(c)
    with torch.cuda.device(a.device):
        rc = load_library().splitk_gemm_bf16_planned(
            a.data_ptr(), b.data_ptr(), c.data_ptr(), M, N, K, L, ctypes.byref(plan),
            int(flags), _stream_handle(stream, a.device))
    _check(rc, "splitk_gemm_bf16_planned")
    return c


def splitk_gemm_bf16_hostio(a, b_host, c_host, b_dev, c_dev, split_k: int = 0, stream=None):
    """Copies b_host -> b_dev, runs the GEMM, copies c_dev -> c_host (all async)."""
    import torch
    M, N, K, L = _dims(a, b_dev)
    _require_cuda(a, b_dev, c_dev)
    if b_host.is_cuda or c_host.is_cuda:
        raise ValueError("b_host and c_host must be host tensors")
    if b_host.numel() != b_dev.numel() or c_host.numel() != c_dev.numel() or \
            c_dev.numel() != L * M * N:
        raise ValueError("host and device buffers must match in size")
    with torch.cuda.device(a.device):
        rc = load_library().splitk_gemm_bf16_hostio(
            a.data_ptr(), b_host.data_ptr(), c_host.data_ptr(), b_dev.data_ptr(),
            c_dev.data_ptr(), M, N, K, L, int(split_k), _stream_handle(stream, a.device))
    _check(rc, "splitk_gemm_bf16_hostio")
    return c_host


def splitk_gemm_bf16_zerocopy(a, b_host, c_host, split_k: int = 0, stream=None):
    """c_host = b_host @ a^T with the activations read from, and the output
    written to, pinned host memory by the kernel itself (no copy engines);
    returns c_host.  Synchronize the stream before reading it."""
    import torch
    if b_host.is_cuda or c_host.is_cuda:
        raise ValueError("b_host and c_host must be host tensors")
    _require_cuda(a)
    if a.dtype != torch.bfloat16 or b_host.dtype != torch.bfloat16 or c_host.dtype != torch.bfloat16:
        raise TypeError("a, b_host and c_host must be bfloat16")
    if a.dim() != b_host.dim() or a.dim() not in (2, 3) or not (a.is_contiguous() and b_host.is_contiguous()
                                                                and c_host.is_contiguous()):
        raise ValueError("a and b_host must be contiguous [N, K] and [M, K] (or batched [L, ...])")
    a3 = a if a.dim() == 3 else a.unsqueeze(0)
    b3 = b_host if b_host.dim() == 3 else b_host.unsqueeze(0)
    L, N, K = a3.shape
    if b3.shape[0] != L or b3.shape[2] != K:
        raise ValueError("a and b_host disagree on L or K")
    M = b3.shape[1]
    if c_host.numel() != L * M * N:
        raise ValueError("c_host must hold L * M * N values")
    with torch.cuda.device(a.device):
        rc = load_library().splitk_gemm_bf16_zerocopy(
            a.data_ptr(), b_host.data_ptr(), c_host.data_ptr(), M, N, K, L, int(split_k),
            _stream_handle(stream, a.device))
    _check(rc, "splitk_gemm_bf16_zerocopy")
    return c_host


# ---------------------------------------------------------------- 8-bit codes, log probabilities
DTYPE_BF16, DTYPE_F32, DTYPE_F16 = 0, 1, 2


def _dtype_code(t, name, *allowed):
    """The library's code of t's type, one of `allowed` (torch type names)."""
    kind = str(t.dtype)[6:]
    if kind not in allowed:
        raise TypeError(f"{name} must be {' or '.join(allowed)}, not {kind}")
    return {"bfloat16": DTYPE_BF16, "float32": DTYPE_F32, "float16": DTYPE_F16}[kind]


def _same_device(device, **ts):
    """Every tensor given is a CUDA tensor on `device`."""
    for name, t in ts.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}, the operands' device")
    if device.type != "cuda":
        raise ValueError("operands must be CUDA tensors")


def _given(t, name, shape, dtype, device):
    """t if it is a contiguous tensor of this shape and type, or a new one."""
    import torch
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    _same_device(device, **{name: t})
    return t


def _rows(t, name):
    """(rows, width, row stride) of a tensor read as rows along its last
    dimension: [M, D] with contiguous rows any distance apart, or a contiguous
    [L, M, D]."""
    if t.dim() not in (2, 3) or (t.dim() == 3 and not t.is_contiguous()) or t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} is [M, D] with contiguous rows, or a contiguous [L, M, D]")
    width = t.shape[-1]
    if t.dim() == 3:
        return t.shape[0] * t.shape[1], width, width
    rows = t.shape[0]
    return rows, width, (t.stride(0) if rows > 1 else width)


def _call(fn, device, stream, where, *args):
    """One library call on `device` (made current) and `stream` (the current
    one when None)."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if torch.cuda.current_device() == device.index:
        rc = fn(*args, stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream.cuda_stream)
    _check(rc, where)


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
    import torch
    M, D, stride = _rows(x, "x")
    _dtype_code(x, "x", "bfloat16")
    w_code = _dtype_code(weight, "weight", "bfloat16", "float32")
    if tuple(weight.shape) != (D,) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous tensor of shape ({D},)")
    device, shape = x.device, tuple(x.shape)
    _same_device(device, weight=weight, residual=residual)
    r_code, r_in, r_out = DTYPE_BF16, None, None
    if residual is not None:
        r_code = _dtype_code(residual, "residual", "bfloat16", "float32")
        r_in = _given(residual, "residual", shape, residual.dtype, device).data_ptr()
        residual_out = _given(residual_out, "residual_out", shape, residual.dtype, device)
        r_out = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    q = _given(q, "q", shape, torch.int8, device)
    scale = _given(scale, "scale", shape[:-1], torch.float32, device)
    _call(load_library().splitk_rmsnorm_i8, device, stream, "splitk_rmsnorm_i8",
          x.data_ptr(), stride, r_in, r_out, r_code, weight.data_ptr(), w_code, eps, q.data_ptr(),
          scale.data_ptr(), M, D)
    return q, scale, residual_out


def splitk_quantize_i8(x, q=None, scale=None, stream=None):
    """8-bit codes with a scale per row, scale = max|x| / 127: activations
    (a row is a token) or weights (a row is a channel).  x as in
    splitk_rmsnorm_i8; returns (q int8, scale float32)."""
    import torch
    M, D, stride = _rows(x, "x")
    _dtype_code(x, "x", "bfloat16")
    device, shape = x.device, tuple(x.shape)
    _same_device(device)
    q = _given(q, "q", shape, torch.int8, device)
    scale = _given(scale, "scale", shape[:-1], torch.float32, device)
    _call(load_library().splitk_quantize_i8, device, stream, "splitk_quantize_i8",
          x.data_ptr(), stride, q.data_ptr(), scale.data_ptr(), M, D)
    return q, scale


def splitk_gemm_i8(a_q, a_scale, b_q, b_scale, c=None, bias=None, out_dtype=None, stream=None):
    """c = (b_q @ a_q^T) * b_scale * a_scale + bias: 8-bit codes with a scale
    per channel (a_scale [L, N] or [N]) and per token (b_scale [L, M] or [M]).

    a_q [L, N, K] or [N, K] and b_q [L, M, K] or [M, K] int8, contiguous, K a
    multiple of 16; bias [L, N] or [N] bfloat16.  Returns c [L, M, N] or
    [M, N]: bfloat16, or float32 where out_dtype or the c given says so."""
    import torch
    if a_q.dtype != torch.int8 or b_q.dtype != torch.int8:
        raise TypeError("a_q and b_q must be int8")
    if a_scale.dtype != torch.float32 or b_scale.dtype != torch.float32:
        raise TypeError("a_scale and b_scale must be float32")
    if a_q.dim() not in (2, 3) or b_q.dim() != a_q.dim():
        raise ValueError("a_q is [L, N, K] or [N, K]; b_q is [L, M, K] or [M, K]")
    batch = tuple(a_q.shape[:-2])
    (N, K), (M, Kb) = a_q.shape[-2:], b_q.shape[-2:]
    if K != Kb or tuple(b_q.shape[:-2]) != batch or tuple(a_scale.shape) != (*batch, N) or \
            tuple(b_scale.shape) != (*batch, M):
        raise ValueError(f"shape mismatch: a_q{tuple(a_q.shape)} a_scale{tuple(a_scale.shape)} "
                         f"b_q{tuple(b_q.shape)} b_scale{tuple(b_scale.shape)}")
    if not (a_q.is_contiguous() and a_scale.is_contiguous() and b_q.is_contiguous() and b_scale.is_contiguous()):
        raise ValueError("operands must be contiguous")
    device = a_q.device
    _same_device(device, a_scale=a_scale, b_q=b_q, b_scale=b_scale, bias=bias)
    if bias is not None and (bias.dtype != torch.bfloat16 or tuple(bias.shape) != (*batch, N) or
                             not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous bfloat16 tensor of shape {(*batch, N)}")
    if out_dtype is None:
        out_dtype = torch.bfloat16 if c is None else c.dtype
    c = _given(c, "c", (*batch, M, N), out_dtype, device)
    c_code = _dtype_code(c, "c", "bfloat16", "float32")
    _call(load_library().splitk_gemm_i8, device, stream, "splitk_gemm_i8",
          a_q.data_ptr(), a_scale.data_ptr(), b_q.data_ptr(), b_scale.data_ptr(),
          None if bias is None else bias.data_ptr(), c.data_ptr(), c_code, M, N, K, batch[0] if batch else 1)
    return c


def splitk_logprobs(logits, tokens=None, top_k: int = 0, logprob=None, entropy=None, top_ids=None,
                    top_logprobs=None, stream=None):
    """Log probabilities of the given tokens, the entropy of each row and its
    top_k most probable tokens (0..32; equal logits by the lowest index).

    logits [M, V] (rows any distance apart) or contiguous [L, M, V], bfloat16,
    float16 or float32; tokens int64 [M] or [L, M], contiguous.  Returns
    (logprob, entropy, top_ids int64 [..., top_k], top_logprobs), float32 but
    the ids; logprob is None without tokens, the alternatives with top_k = 0."""
    import torch
    M, V, stride = _rows(logits, "logits")
    code = _dtype_code(logits, "logits", "bfloat16", "float16", "float32")
    device, shape = logits.device, tuple(logits.shape[:-1])
    _same_device(device, tokens=tokens)
    t_ptr = l_ptr = i_ptr = p_ptr = None
    if tokens is not None:
        if tokens.dtype != torch.int64 or tuple(tokens.shape) != shape or not tokens.is_contiguous():
            raise ValueError(f"tokens must be a contiguous int64 tensor of shape {shape}")
        logprob = _given(logprob, "logprob", shape, torch.float32, device)
        t_ptr, l_ptr = tokens.data_ptr(), logprob.data_ptr()
    elif logprob is not None:
        raise ValueError("logprob needs tokens")
    entropy = _given(entropy, "entropy", shape, torch.float32, device)
    if top_k:
        top_ids = _given(top_ids, "top_ids", (*shape, top_k), torch.int64, device)
        top_logprobs = _given(top_logprobs, "top_logprobs", (*shape, top_k), torch.float32, device)
        i_ptr, p_ptr = top_ids.data_ptr(), top_logprobs.data_ptr()
    elif top_ids is not None or top_logprobs is not None:
        raise ValueError("the alternatives' outputs need top_k > 0")
    _call(load_library().splitk_logprobs, device, stream, "splitk_logprobs",
          logits.data_ptr(), code, stride, t_ptr, l_ptr, entropy.data_ptr(), top_k, i_ptr, p_ptr, M, V)
    return logprob, entropy, top_ids, top_logprobs


# ---------------------------------------------------------------- status
def splitk_get_fault() -> dict:
    f = Fault()
    rc = load_library().splitk_get_fault(ctypes.byref(f))
    if rc not in (0, -6):
        raise SplitKError(rc, "splitk_get_fault")
    return f.as_dict()


def splitk_get_status() -> int:
    return int(load_library().splitk_get_status())


def splitk_set_wait_limit_ns(ns: int) -> None:
    _check(load_library().splitk_set_wait_limit_ns(int(ns)), "splitk_set_wait_limit_ns")


def splitk_debug_inject(flags: int) -> None:
    _check(load_library().splitk_debug_inject(int(flags)), "splitk_debug_inject")


def splitk_set_trace(buffer=None) -> None:
    """Trace later launches into `buffer` (a CUDA tensor, 16 uint64 words per
    CTA, see splitk.h); None turns tracing off."""
    if buffer is None:
        _check(load_library().splitk_set_trace(None, 0), "splitk_set_trace")
    else:
        _check(load_library().splitk_set_trace(buffer.data_ptr(),
                                               buffer.numel() * buffer.element_size()),
               "splitk_set_trace")


TRACE_SLOTS = 16
TRACE_FIELDS = ("sm_rank", "start", "synced", "weights_issued", "act_ready", "first_full",
                "last_full", "mma_done", "reduced", "stored", "end", "bar_init", "map_ready",
                "prefetched", "tmem_alloc", "epi_synced")


def splitk_release() -> None:
    load_library().splitk_release()


def splitk_cache_info() -> dict:
    """The memory the library owns on the current CUDA device: device and
    page-locked host bytes of its tensor-map pool, and the maps in it."""
    dev_b, host_b, maps = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_int()
    _check(load_library().splitk_cache_info(ctypes.byref(dev_b), ctypes.byref(host_b), ctypes.byref(maps)),
           "splitk_cache_info")
    return {"device_bytes": dev_b.value, "host_bytes": host_b.value, "maps": maps.value}


def splitk_strerror(code: int) -> str:
    return load_library().splitk_strerror(int(code)).decode()


def splitk_version() -> int:
    return int(load_library().splitk_version())
