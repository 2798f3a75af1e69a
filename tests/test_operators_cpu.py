"""What the operators around the projection refuse, without a GPU: the C ABI
checks its arguments before it touches CUDA, and the binding checks its
tensors before the library."""
from __future__ import annotations

import ctypes

import pytest
import torch

import split_bf16_gemm_swapped_gb300 as sk
from split_bf16_gemm_swapped_gb300 import _build

OK, SHAPE, ALIGN, NULL, DEVICE, ARG = 0, -1, -2, -7, -9, -14
P = 0x10000          # an aligned address that is never read: every call here is refused


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build_splitk()
    _build.build_operators()


def rmsnorm(x=P, stride=64, r=None, r_out=None, r_type=0, w=P, w_type=0, eps=1e-6, q=P, s=P, M=2, D=64):
    return sk.load_library().splitk_rmsnorm_i8(x, stride, r, r_out, r_type, w, w_type, eps, q, s, M, D, None)


def test_rmsnorm_refusals():
    for kw in (dict(x=None), dict(w=None), dict(q=None), dict(s=None), dict(r=P), dict(r_out=P)):
        assert rmsnorm(**kw) == NULL, kw
    for kw in (dict(M=0), dict(D=0), dict(M=-1), dict(stride=63), dict(D=(1 << 30) + 1, stride=1 << 31),
               dict(M=(1 << 30) + 1)):
        assert rmsnorm(**kw) == SHAPE, kw
    for kw in (dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(w_type=2),
               dict(r=P, r_out=P, r_type=2), dict(r=P, r_out=P, r_type=-1)):
        assert rmsnorm(**kw) == ARG, kw
    for kw in (dict(x=P + 1), dict(w=P + 1), dict(w=P + 2, w_type=1), dict(s=P + 2), dict(r=P + 1, r_out=P),
               dict(r=P, r_out=P + 2, r_type=1)):
        assert rmsnorm(**kw) == ALIGN, kw


def quantize(x=P, stride=64, q=P, s=P, M=2, D=64):
    return sk.load_library().splitk_quantize_i8(x, stride, q, s, M, D, None)


def test_quantize_refusals():
    for kw in (dict(x=None), dict(q=None), dict(s=None)):
        assert quantize(**kw) == NULL, kw
    for kw in (dict(M=0), dict(D=0), dict(stride=10)):
        assert quantize(**kw) == SHAPE, kw
    for kw in (dict(x=P + 1), dict(s=P + 1)):
        assert quantize(**kw) == ALIGN, kw


def gemm(a=P, sa=P, b=P, sb=P, bias=None, c=P, c_type=0, M=2, N=64, K=64, L=1):
    return sk.load_library().splitk_gemm_i8(a, sa, b, sb, bias, c, c_type, M, N, K, L, None)


def test_gemm_refusals():
    for kw in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(c=None)):
        assert gemm(**kw) == NULL, kw
    for kw in (dict(M=0), dict(N=0), dict(K=0), dict(L=0), dict(K=72), dict(K=8), dict(L=65536),
               dict(N=65535 * 128 + 1), dict(K=(1 << 30) + 16), dict(M=-5),
               dict(M=1 << 30, N=65535 * 128, L=60000)):
        assert gemm(**kw) == SHAPE, kw
    assert gemm(c_type=2) == ARG and gemm(c_type=-1) == ARG
    for kw in (dict(a=P + 8), dict(b=P + 4), dict(sa=P + 2), dict(sb=P + 1), dict(bias=P + 1), dict(c=P + 1),
               dict(c=P + 2, c_type=1)):
        assert gemm(**kw) == ALIGN, kw


def logprobs(x=P, kind=0, stride=100, t=P, lp=P, h=P, k=4, ids=P, tops=P, M=2, V=100):
    return sk.load_library().splitk_logprobs(x, kind, stride, t, lp, h, k, ids, tops, M, V, None)


def test_logprobs_refusals():
    for kw in (dict(x=None), dict(h=None), dict(t=None), dict(lp=None), dict(ids=None), dict(tops=None)):
        assert logprobs(**kw) == NULL, kw
    for kw in (dict(M=0), dict(V=0, stride=1), dict(stride=99), dict(V=(1 << 22) + 1, stride=1 << 23)):
        assert logprobs(**kw) == SHAPE, kw
    for kw in (dict(kind=3), dict(kind=-1), dict(k=-1), dict(k=33), dict(V=3)):
        assert logprobs(**kw) == ARG, kw
    for kw in (dict(x=P + 1), dict(x=P + 2, kind=1), dict(t=P + 4), dict(lp=P + 2), dict(h=P + 2), dict(ids=P + 4),
               dict(tops=P + 1)):
        assert logprobs(**kw) == ALIGN, kw


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses here are not memory")
def test_a_machine_without_the_gpu_is_refused():
    assert rmsnorm() == quantize() == gemm() == logprobs() == DEVICE


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_the_binding_refuses_other_types():
    i8, f32, f16 = torch.int8, torch.float32, torch.float16
    with pytest.raises(TypeError):
        sk.splitk_rmsnorm_i8(meta(2, 64, dtype=f16), meta(64))
    with pytest.raises(TypeError):
        sk.splitk_rmsnorm_i8(meta(2, 64), meta(64, dtype=f16))
    with pytest.raises(TypeError):
        sk.splitk_quantize_i8(meta(2, 64, dtype=f32))
    with pytest.raises(TypeError):
        sk.splitk_gemm_i8(meta(64, 64), meta(64, dtype=f32), meta(2, 64, dtype=i8), meta(2, dtype=f32))
    with pytest.raises(TypeError):
        sk.splitk_gemm_i8(meta(64, 64, dtype=i8), meta(64), meta(2, 64, dtype=i8), meta(2, dtype=f32))
    with pytest.raises(TypeError):
        sk.splitk_logprobs(meta(2, 64, dtype=torch.float64))


def test_the_binding_refuses_other_shapes():
    i8, f32 = torch.int8, torch.float32
    with pytest.raises(ValueError, match="weight"):
        sk.splitk_rmsnorm_i8(meta(2, 64), meta(63))
    with pytest.raises(ValueError, match="x is"):
        sk.splitk_rmsnorm_i8(meta(64), meta(64))
    with pytest.raises(ValueError, match="x is"):
        sk.splitk_quantize_i8(meta(64, 2).t())
    with pytest.raises(ValueError, match="shape mismatch"):
        sk.splitk_gemm_i8(meta(64, 64, dtype=i8), meta(64, dtype=f32), meta(2, 32, dtype=i8), meta(2, dtype=f32))
    with pytest.raises(ValueError, match="shape mismatch"):
        sk.splitk_gemm_i8(meta(64, 64, dtype=i8), meta(64, dtype=f32), meta(2, 64, dtype=i8), meta(3, dtype=f32))
    with pytest.raises(ValueError, match="contiguous"):
        sk.splitk_gemm_i8(meta(64, 64, dtype=i8).t(), meta(64, dtype=f32), meta(2, 64, dtype=i8), meta(2, dtype=f32))


def test_the_binding_refuses_tensors_that_are_not_on_a_gpu():
    i8, f32 = torch.int8, torch.float32
    cpu = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sk.splitk_rmsnorm_i8(cpu, torch.zeros(64))
    with pytest.raises(ValueError, match="CUDA"):
        sk.splitk_quantize_i8(cpu)
    with pytest.raises(ValueError, match="CUDA"):
        sk.splitk_gemm_i8(torch.zeros(64, 64, dtype=i8), torch.zeros(64), torch.zeros(2, 64, dtype=i8), torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        sk.splitk_logprobs(cpu)
    with pytest.raises(ValueError, match="device"):
        sk.splitk_rmsnorm_i8(meta(2, 64), torch.zeros(64, dtype=f32))


def test_gemm_refuses_token_counts_past_its_index_arithmetic():
    """Counts of tiles and blocks round M up in 32 bits."""
    for M in ((1 << 30) + 1, (1 << 31) - 255, (1 << 31) - 1):
        for N, K in ((1, 16), (16, 64)):
            assert gemm(M=M, N=N, K=K) == SHAPE, (M, N, K)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses here are not memory")
def test_gemm_takes_token_counts_up_to_two_to_the_30():
    assert gemm(M=1 << 30, N=1, K=16) == DEVICE


UNBUILT = """
import sys
sys.modules["torch"] = None                       # an import of it raises
from pathlib import Path
from split_bf16_gemm_swapped_gb300 import _build
_build.OPERATORS_LIB = Path({missing!r})
import split_bf16_gemm_swapped_gb300 as sk
from split_bf16_gemm_swapped_gb300 import *
assert all(hasattr(sk, name) for name in sk.__all__)
assert splitk_logprobs is sk.splitk_logprobs and splitk_logprobs.__doc__
print("imported")
"""


def test_the_names_need_neither_pytorch_nor_the_binding(tmp_path):
    import subprocess
    import sys
    from pathlib import Path
    code = UNBUILT.format(missing=str(tmp_path / "missing.so"))
    res = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parent.parent, capture_output=True,
                         text=True, timeout=300)
    assert res.returncode == 0 and "imported" in res.stdout, res.stderr[-2000:]


def test_a_call_without_the_binding_raises(tmp_path):
    import subprocess
    import sys
    from pathlib import Path
    code = f"""
from pathlib import Path
from split_bf16_gemm_swapped_gb300 import _build
_build.OPERATORS_LIB = Path({str(tmp_path / "missing.so")!r})
import torch, split_bf16_gemm_swapped_gb300 as sk
for call in (lambda: sk.splitk_quantize_i8(torch.zeros(1, 8)), lambda: sk.splitk_logprobs(torch.zeros(1, 8))):
    try:
        call()
    except RuntimeError as e:
        assert "missing" in str(e), e
        print("raised")
"""
    res = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parent.parent, capture_output=True,
                         text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.count("raised") == 2, res.stderr[-2000:]


def test_the_binding_is_built_again_for_another_pytorch(monkeypatch, tmp_path):
    """It uses PyTorch's C++ types: newer than its sources is not enough."""
    lib, built = tmp_path / "_operators.so", []
    monkeypatch.setattr(_build, "OPERATORS_LIB", lib)
    monkeypatch.setattr(_build, "OPERATORS_STAMP", tmp_path / "_operators.abi", raising=False)

    def compile(cmd, cwd=None):
        from pathlib import Path
        built.append(cmd)
        Path(cmd[cmd.index("-o") + 1]).write_bytes(b"")

    monkeypatch.setattr(_build, "_run", compile)
    for _ in range(2):
        _build.build_operators()
    assert len(built) == 1 and lib.exists()
    version = _build.importlib.metadata.version
    monkeypatch.setattr(_build.importlib.metadata, "version",
                        lambda name: "0.0.1" if name == "torch" else version(name))
    for _ in range(2):
        _build.build_operators()
    assert len(built) == 2
    soabi = _build.sysconfig.get_config_var
    monkeypatch.setattr(_build.sysconfig, "get_config_var",
                        lambda name: "other" if name == "SOABI" else soabi(name))
    for _ in range(2):
        _build.build_operators()
    assert len(built) == 3


def test_a_binding_of_another_pytorch_is_not_loaded(monkeypatch, tmp_path):
    from split_bf16_gemm_swapped_gb300 import operators
    stamp = tmp_path / "_operators.abi"
    monkeypatch.setattr(_build, "OPERATORS_STAMP", stamp, raising=False)
    for text in (None, "torch 0.0.1, other"):
        if text:
            stamp.write_text(text)
        with pytest.raises(RuntimeError, match="another PyTorch"):
            operators._load()
