"""What the 4-bit operators and the logits' adjustment refuse, without a GPU: the C
ABI checks its arguments before it touches CUDA, and the binding checks its
tensors before the library."""
from __future__ import annotations

import ctypes

import pytest
import torch

import split_bf16_gemm_swapped_gb300 as sk
from split_bf16_gemm_swapped_gb300 import _build

OK, SHAPE, ALIGN, NULL, DEVICE, ARG = 0, -1, -2, -7, -9, -14
P = 0x10000          # an aligned address that is never read: every call here is refused
U8, I8, F16, F32, F64, I32, I64 = (torch.uint8, torch.int8, torch.float16, torch.float32, torch.float64, torch.int32,
                                   torch.int64)


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build_splitk()
    _build.build_operators()


def quantize(x=P, kind=0, stride=64, q=P, s=P, M=2, K=64):
    return sk.load_library().splitk_quantize_mx4(x, kind, stride, q, s, M, K, None)


def test_quantize_refusals():
    for kw in (dict(x=None), dict(q=None), dict(s=None)):
        assert quantize(**kw) == NULL, kw
    for kw in (dict(M=0), dict(K=0), dict(K=48), dict(K=16), dict(stride=63), dict(M=-1), dict(M=(1 << 30) + 1),
               dict(K=(1 << 30) + 32, stride=1 << 31)):
        assert quantize(**kw) == SHAPE, kw
    assert quantize(kind=3) == ARG and quantize(kind=-1) == ARG
    for kw in (dict(x=P + 1), dict(x=P + 2, kind=1), dict(q=P + 8)):
        assert quantize(**kw) == ALIGN, kw


def dequantize(q=P, s=P, out=P, kind=0, M=2, K=64):
    return sk.load_library().splitk_dequantize_mx4(q, s, out, kind, M, K, None)


def test_dequantize_refusals():
    for kw in (dict(q=None), dict(s=None), dict(out=None)):
        assert dequantize(**kw) == NULL, kw
    for kw in (dict(M=0), dict(K=0), dict(K=33), dict(M=(1 << 30) + 1), dict(M=1 << 30, K=1 << 30)):
        assert dequantize(**kw) == SHAPE, kw
    assert dequantize(kind=3) == ARG and dequantize(kind=-1) == ARG
    for kw in (dict(q=P + 8), dict(out=P + 8)):
        assert dequantize(**kw) == ALIGN, kw


def rmsnorm(x=P, stride=64, r=None, r_out=None, r_type=0, w=P, w_type=0, eps=1e-6, q=P, s=P, M=2, D=64):
    return sk.load_library().splitk_rmsnorm_mx4(x, stride, r, r_out, r_type, w, w_type, eps, q, s, M, D, None)


def test_rmsnorm_refusals():
    for kw in (dict(x=None), dict(w=None), dict(q=None), dict(s=None), dict(r=P), dict(r_out=P)):
        assert rmsnorm(**kw) == NULL, kw
    for kw in (dict(M=0), dict(D=0), dict(D=72, stride=72), dict(stride=63), dict(D=(1 << 30) + 32, stride=1 << 31),
               dict(M=(1 << 30) + 1)):
        assert rmsnorm(**kw) == SHAPE, kw
    for kw in (dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(w_type=2),
               dict(r=P, r_out=P, r_type=2), dict(r=P, r_out=P, r_type=-1)):
        assert rmsnorm(**kw) == ARG, kw
    for kw in (dict(x=P + 1), dict(w=P + 1), dict(w=P + 2, w_type=1), dict(q=P + 4), dict(r=P + 1, r_out=P),
               dict(r=P, r_out=P + 2, r_type=1)):
        assert rmsnorm(**kw) == ALIGN, kw


def gemm(a=P, sa=P, b=P, sb=P, bias=None, c=P, c_type=0, M=2, N=64, K=64, L=1):
    return sk.load_library().splitk_gemm_mx4(a, sa, b, sb, bias, c, c_type, M, N, K, L, None)


def test_gemm_refusals():
    for kw in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(c=None)):
        assert gemm(**kw) == NULL, kw
    for kw in (dict(M=0), dict(N=0), dict(K=0), dict(L=0), dict(K=80), dict(K=16), dict(L=65536),
               dict(N=65535 * 128 + 1), dict(K=(1 << 30) + 32), dict(M=-5), dict(M=(1 << 30) + 1),
               dict(M=1 << 30, N=65535 * 128, L=60000)):
        assert gemm(**kw) == SHAPE, kw
    assert gemm(c_type=2) == ARG and gemm(c_type=-1) == ARG
    for kw in (dict(a=P + 8), dict(b=P + 4), dict(bias=P + 1), dict(c=P + 1), dict(c=P + 2, c_type=1)):
        assert gemm(**kw) == ALIGN, kw


def adjust(x=P, kind=0, stride=100, out=P, out_stride=100, M=2, V=100, how=True, **parts):
    h = sk.Adjust(**{k: v for k, v in parts.items() if v is not None})
    return sk.load_library().splitk_adjust_logits(x, kind, stride, ctypes.byref(h) if how else None, out, out_stride, M, V,
                                                  None)


def test_adjust_refusals():
    for kw in (dict(x=None), dict(out=None), dict(how=False), dict(history_length=3), dict(bias_count=1),
               dict(bias_count=1, bias_ids=P), dict(bias_count=1, bias_values=P), dict(repetition=P), dict(lengths=P)):
        assert adjust(**kw) == NULL, kw
    for kw in (dict(M=0), dict(V=0), dict(stride=99), dict(out_stride=99), dict(V=(1 << 22) + 1, stride=1 << 23,
                                                                                  out_stride=1 << 23), dict(M=-1)):
        assert adjust(**kw) == SHAPE, kw
    for kw in (dict(kind=3), dict(kind=-1), dict(history=P, history_length=-1), dict(history=P, history_length=(1 << 30) + 1),
               dict(bias_count=1025, bias_ids=P, bias_values=P), dict(bias_count=-1)):
        assert adjust(**kw) == ARG, kw
    assert adjust(x=P, out=P, stride=100, out_stride=101) == ARG          # in place, rows over other rows
    some = dict(history=P, history_length=4, bias_ids=P, bias_values=P, bias_count=2)
    for kw in (dict(x=P + 1), dict(x=P + 2, kind=1), dict(out=P + 1), dict(allowed=P + 2), dict(some, history=P + 4),
               dict(some, lengths=P + 4), dict(some, prompt_lengths=P + 4), dict(some, repetition=P + 2),
               dict(some, presence=P + 2), dict(some, frequency=P + 1), dict(some, bias_ids=P + 4),
               dict(some, bias_values=P + 2)):
        assert adjust(**kw) == ALIGN, kw


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses here are not memory")
def test_a_machine_without_the_gpu_is_refused():
    assert quantize() == dequantize() == rmsnorm() == gemm() == adjust() == DEVICE
    assert gemm(M=1 << 30, N=1, K=32) == DEVICE


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_the_binding_refuses_other_types():
    for call in (lambda: sk.splitk_quantize_mx4(meta(2, 64, dtype=F64)),
                 lambda: sk.splitk_dequantize_mx4(meta(2, 32, dtype=I8), meta(2, 2, dtype=U8)),
                 lambda: sk.splitk_rmsnorm_mx4(meta(2, 64, dtype=F16), meta(64)),
                 lambda: sk.splitk_rmsnorm_mx4(meta(2, 64), meta(64, dtype=F16)),
                 lambda: sk.splitk_gemm_mx4(meta(64, 32, dtype=I8), meta(64, 2, dtype=U8), meta(2, 32, dtype=U8),
                                            meta(2, 2, dtype=U8)),
                 lambda: sk.splitk_adjust_logits(meta(2, 64, dtype=F64)),
                 lambda: sk.splitk_adjust_logits(None)):
        with pytest.raises(TypeError):
            call()


def test_the_binding_refuses_other_shapes():
    def product(a=(64, 32), sa=(64, 2), b=(2, 32), sb=(2, 2)):
        return sk.splitk_gemm_mx4(*(meta(*s, dtype=U8) for s in (a, sa, b, sb)))

    for match, call in (
            ("multiple of 32", lambda: sk.splitk_quantize_mx4(meta(2, 48))),
            ("x is", lambda: sk.splitk_quantize_mx4(meta(64))),
            ("x is", lambda: sk.splitk_quantize_mx4(meta(64, 32).t())),
            ("scale", lambda: sk.splitk_dequantize_mx4(torch.zeros(2, 32, dtype=U8), torch.zeros(2, 3, dtype=U8))),
            ("weight", lambda: sk.splitk_rmsnorm_mx4(meta(2, 64), meta(63))),
            ("multiple of 32", lambda: sk.splitk_rmsnorm_mx4(meta(2, 63), meta(63))),
            ("shape mismatch", lambda: product(b=(2, 16))),
            ("shape mismatch", lambda: product(sa=(64, 3))),
            ("shape mismatch", lambda: product(sb=(3, 2))),
            ("multiple of 32", lambda: product(a=(64, 24), b=(2, 24))),
            ("a_q is", lambda: product(b=(1, 2, 32)))):
        with pytest.raises(ValueError, match=match):
            call()


def test_the_binding_refuses_parts_that_do_not_belong_together():
    x = torch.zeros(2, 100)
    i64, f32 = dict(dtype=I64), dict(dtype=F32)
    for match, kw in (("need a history", dict(presence=torch.zeros(2, **f32))),
                      ("need a history", dict(lengths=torch.zeros(2, **i64))),
                      ("belong together", dict(bias_ids=torch.zeros(2, 3, **i64))),
                      ("bias_values", dict(bias_ids=torch.zeros(2, 3, **i64), bias_values=torch.zeros(2, 4, **f32))),
                      ("history", dict(history=torch.zeros(3, 4, **i64))),
                      ("history", dict(history=torch.zeros(2, 4, dtype=I32))),
                      ("repetition", dict(history=torch.zeros(2, 4, **i64), repetition=torch.zeros(2, dtype=F64))),
                      ("allowed", dict(allowed=torch.zeros(2, 3, dtype=I32))),
                      ("out", dict(out=torch.zeros(2, 99))),
                      ("out", dict(out=torch.zeros(2, 100, dtype=torch.bfloat16)))):
        with pytest.raises(ValueError, match=match):
            sk.splitk_adjust_logits(x, **kw)


def test_the_binding_refuses_tensors_that_are_not_on_a_gpu():
    cpu = torch.zeros(2, 64, dtype=torch.bfloat16)
    codes, scale = torch.zeros(2, 32, dtype=U8), torch.zeros(2, 2, dtype=U8)
    for call in (lambda: sk.splitk_quantize_mx4(cpu), lambda: sk.splitk_dequantize_mx4(codes, scale),
                 lambda: sk.splitk_rmsnorm_mx4(cpu, torch.zeros(64)),
                 lambda: sk.splitk_gemm_mx4(codes, scale, codes, scale), lambda: sk.splitk_adjust_logits(cpu)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="device"):
        sk.splitk_gemm_mx4(meta(64, 32, dtype=U8), meta(64, 2, dtype=U8), codes, scale)


# ---------------------------------------------------------------- the product's shared memory
LAYOUT = r"""
#include <stdio.h>
#include "splitk_mx4.cuh"
int main() {
  for (int tokens : {16, 32, 64, 128, 256}) {
    for (int stages = 1; stages <= splitk::kMxStages; ++stages) {
      for (int split = 1; split <= 4; ++split) {
        printf("%d %d %d %u %u\n", tokens, stages, split, splitk::mx_ring_bytes(tokens, stages),
               splitk::mx_bars_at(tokens, stages, split));
      }
    }
  }
}
"""


def test_a_shares_sums_end_before_the_barriers(tmp_path):
    """Sums of a tile's shares lie over the ring, and the barriers behind both, whatever
    tile, depth and split are chosen: 128 weight rows of f32 a token."""
    import subprocess
    (tmp_path / "layout.cu").write_text(LAYOUT)
    exe = tmp_path / "layout"
    res = subprocess.run([_build._nvcc(), *_build.ARCH_FLAGS, "-std=c++17", "-I", str(_build.INCLUDE), "-I", str(_build.CSRC),
                          str(tmp_path / "layout.cu"), "-o", str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    rows = [tuple(map(int, line.split())) for line in subprocess.run([exe], capture_output=True, text=True).stdout.splitlines()]
    assert len(rows) == 5 * 4 * 4
    for tokens, stages, split, ring, bars in rows:
        # a stage: two K tiles of 128 bytes of 128 weight rows and half of the tokens
        assert ring >= stages * 2 * 128 * (128 + tokens // 2)
        assert bars >= ring and bars % 8 == 0, (tokens, stages, split)
        if split > 1:
            assert bars >= tokens * 128 * 4, (tokens, stages, split, bars)
