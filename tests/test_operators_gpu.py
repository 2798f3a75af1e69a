"""The operators around the projection on the GPU, against plain 64-bit
implementations: residual addition + RMS norm to 8-bit codes, quantisation,
the product of 8-bit codes, and log probabilities.

Tolerances are bounds of f32 arithmetic, derived where they are stated; u is
the unit roundoff of f32, 2^-24.  Outputs in bf16 are held to the bit: they are
the f32 result rounded once."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import split_bf16_gemm_swapped_gb300 as sk  # noqa: E402

DEV = torch.device("cuda:0")
U = 2.0 ** -24
BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(shape, g, dtype=F32, scale=1.0):
    return (scale * torch.randn(shape, device=DEV, generator=g)).to(dtype)


# ---------------------------------------------------------------- norm and codes
def check_codes(q, scale, n, rel):
    """Codes and scales of the 64-bit rows n, each of whose values the f32
    computation has to a relative error of `rel`."""
    want = torch.clamp_min(n.abs().amax(-1) / 127, 2.0 ** -126)
    assert ((scale.double() - want).abs() <= rel * want).all()
    # a code is the nearest whole number to a value off by `rel` of at most 127
    off = (q.double() - n / want[..., None]).abs().max().item()
    assert off <= 0.5 + 127 * 2 * rel, off
    assert q.min() >= -127 and q.max() <= 127


def norm_ref(x, r, w, eps):
    y = x.double() if r is None else x.double() + r.double()
    n = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    return y, n


def norm_rel(D):
    """A thread adds at most 32 squares in registers (64 passes' worth for
    rows past 32768), ten more additions join the threads, and the mean, root,
    quotients and products round a dozen times."""
    return (max(32, D / 1024) + 10 + 12) * U


def check_norm(x, r, w, eps=1e-6, **kw):
    keep = None if r is None else r.clone()
    q, scale, out = sk.splitk_rmsnorm_i8(x, w, r, eps=eps, **kw)
    torch.cuda.synchronize()
    y, n = norm_ref(x, keep, w, eps)
    check_codes(q, scale, n, norm_rel(x.shape[-1]))
    if r is not None:
        assert out.dtype == r.dtype
        assert torch.equal(out, (x.float() + keep.float()).to(r.dtype))     # one f32 sum, rounded once
    else:
        assert out is None
    return q, scale, out


WIDTHS = [1, 7, 8, 31, 64, 255, 256, 264, 513, 1000, 1024, 1032, 4096, 4999, 7168, 16384, 32768, 32769, 40000]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("residual", [None, BF16, F32])
@pytest.mark.parametrize("weight", [BF16, F32])
def test_norm_codes(D, residual, weight):
    g = gen(D)
    M = 5
    x = randn((M, D), g, BF16)
    r = None if residual is None else randn((M, D), g, residual, 4.0)
    w = (1 + randn((D,), g, F32, 0.1)).to(weight)
    check_norm(x, r, w)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 33, 500])
@pytest.mark.parametrize("D", [96, 2048, 7168])
def test_norm_row_counts(M, D):
    g = gen(M * D)
    check_norm(randn((M, D), g, BF16), randn((M, D), g, BF16), randn((D,), g, BF16))


@pytest.mark.parametrize("offset,pad", [(0, 8), (0, 3), (1, 0), (8, 8), (3, 5)])
@pytest.mark.parametrize("D", [256, 250, 2000])
def test_norm_rows_cut_from_a_wider_tensor(offset, pad, D):
    g = gen(D + offset)
    x = randn((6, offset + D + pad), g, BF16)[:, offset:offset + D]
    check_norm(x, randn((6, D), g, F32), randn((D,), g, F32))


@pytest.mark.parametrize("D", [64, 1001, 7168, 33000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_residual_in_place(D, dtype):
    g = gen(D)
    x, r, w = randn((7, D), g, BF16), randn((7, D), g, dtype), randn((D,), g, BF16)
    q0, s0, out0 = sk.splitk_rmsnorm_i8(x, w, r)
    same = r.clone()
    q1, s1, out1 = sk.splitk_rmsnorm_i8(x, w, same, residual_out=same)
    torch.cuda.synchronize()
    assert out1.data_ptr() == same.data_ptr()
    assert torch.equal(out0, same) and torch.equal(q0, q1) and torch.equal(s0, s1)


def test_norm_takes_batched_rows_and_given_outputs():
    g = gen(3)
    x, r, w = randn((3, 4, 512), g, BF16), randn((3, 4, 512), g, BF16), randn((512,), g, F32)
    q = torch.empty((3, 4, 512), dtype=torch.int8, device=DEV)
    scale = torch.empty((3, 4), device=DEV)
    out = torch.empty_like(r)
    got = check_norm(x, r, w, q=q, scale=scale, residual_out=out)
    assert got[0] is q and got[1] is scale and got[2] is out


def test_norm_of_rows_without_codes():
    """Zeros code to zeros; NaN and infinity give the scale NaN, in their row
    alone."""
    g = gen(4)
    x = randn((6, 300), g, BF16)
    x[0] = 0
    x[2, 17] = float("nan")
    x[3, 299] = float("inf")
    x[4, 0] = float("-inf")
    w = torch.ones(300, device=DEV)
    q, scale, _ = sk.splitk_rmsnorm_i8(x, w)
    torch.cuda.synchronize()
    assert (q[0] == 0).all() and scale[0].item() == 2.0 ** -126
    assert torch.isnan(scale[[2, 3, 4]]).all() and torch.isfinite(scale[[0, 1, 5]]).all()
    check_codes(q[[1, 5]], scale[[1, 5]], norm_ref(x[[1, 5]], None, w, 1e-6)[1], norm_rel(300))
    w[9] = float("nan")
    _, scale, _ = sk.splitk_rmsnorm_i8(x, w)
    assert torch.isnan(scale).all()


@pytest.mark.parametrize("D", [1, 5, 64, 1000, 4096, 16384, 50001])
@pytest.mark.parametrize("M", [1, 130])
def test_quantise(D, M):
    g = gen(D + M)
    x = randn((M, D), g, BF16, 3.0)
    x[M // 2] *= 1e-30
    q, scale = sk.splitk_quantize_i8(x)
    torch.cuda.synchronize()
    check_codes(q, scale, x.double(), 4 * U)
    # the row's largest value is a full code
    assert (q.abs().amax(-1) == 127).all()


def test_quantise_tiny_rows():
    """Rows under the smallest scale: codes of the floor, finite."""
    x = torch.tensor([[2.0 ** -130, -2.0 ** -127, 0.0, 2.0 ** -133]], device=DEV).to(BF16)
    q, scale = sk.splitk_quantize_i8(x)
    torch.cuda.synchronize()
    assert scale.item() == 2.0 ** -126
    assert q.tolist() == [[0, 0, 0, 0]]               # -2^-127 is half a scale: to even


# ---------------------------------------------------------------- product
def codes(shape, g, full=False):
    lo = -128 if full else -127
    return torch.randint(lo, 128, shape, device=DEV, generator=g, dtype=torch.int32).to(torch.int8)


def check_product(a, sa, b, sb, bias=None, out=None, exact_sum=True):
    c = sk.splitk_gemm_i8(a, sa, b, sb, bias=bias, out_dtype=F32)
    torch.cuda.synchronize()
    assert sk.splitk_get_status() == 0
    total = torch.matmul(b.double(), a.double().transpose(-1, -2))          # whole numbers below 2^53: exact
    v = total * sb.double()[..., :, None] * sa.double()[..., None, :]
    ref = v if bias is None else v + bias.double()[..., None, :]
    # two products and an addition of f32; sums past 2^24 round once for each
    # 16 codes of K (truncated at worst: 2 u) and once for each part of K
    terms = 3 * U * (v.abs() + ref.abs())
    if not exact_sum:
        size = torch.matmul(b.double().abs(), a.double().abs().transpose(-1, -2))
        terms = terms + 2 * U * (a.shape[-1] / 16 + 16) * size * sb.double()[..., :, None] * sa.double()[..., None, :]
    err = (c.double() - ref).abs()
    assert (err <= terms).all(), (err - terms).max().item()
    if out == F32:
        return c
    rounded = sk.splitk_gemm_i8(a, sa, b, sb, bias=bias)
    assert torch.equal(rounded, c.to(BF16))
    return rounded


def product_inputs(L, M, N, K, seed, batched=True):
    g = gen(seed)
    a, b = codes((L, N, K), g, True), codes((L, M, K), g, True)
    sa = 0.001 + 0.01 * torch.rand((L, N), device=DEV, generator=g)
    sb = 0.001 + 0.01 * torch.rand((L, M), device=DEV, generator=g)
    bias = randn((L, N), g, BF16)
    return (a, sa, b, sb, bias) if batched else (a[0], sa[0], b[0], sb[0], bias[0])


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257])
@pytest.mark.parametrize("N,K", [(128, 128), (100, 272), (1000, 1024), (257, 2064)])
def test_product_shapes(M, N, K):
    a, sa, b, sb, bias = product_inputs(1, M, N, K, M + N + K, batched=False)
    # random codes: the sums stay below 2^24 for K <= 2064 (16-sigma: 5476 * sqrt(2064) * 16 = 4.0e6)
    check_product(a, sa, b, sb, bias=bias if M % 2 else None, out=F32 if M % 3 == 0 else BF16)


@pytest.mark.parametrize("K", [16, 32, 48, 64, 80, 112, 144, 240, 496, 528, 1040, 4112])
@pytest.mark.parametrize("M", [1, 20, 70])
def test_product_k_tails(K, M):
    a, sa, b, sb, _ = product_inputs(1, M, 144, K, K + M, batched=False)
    check_product(a, sa, b, sb, out=F32)


@pytest.mark.parametrize("M", [1, 12, 40, 150])
def test_product_batches(M):
    a, sa, b, sb, bias = product_inputs(3, M, 200, 320, M)
    c = check_product(a, sa, b, sb, bias=bias)
    for l in range(3):
        one = sk.splitk_gemm_i8(a[l], sa[l], b[l], sb[l], bias=bias[l])
        assert torch.equal(one, c[l])


@pytest.mark.parametrize("M,N,K", [(1, 7168, 2048), (16, 4096, 7168), (64, 2304, 7168), (128, 1024, 16384),
                                   (300, 2000, 7168)])
def test_product_workload_shapes(M, N, K):
    a, sa, b, sb, bias = product_inputs(1, M, N, K, M, batched=False)
    check_product(a, sa, b, sb, bias=bias)


@pytest.mark.parametrize("M", [1, 30, 100, 300])
def test_product_of_extreme_codes(M):
    """Every code -128: sums past 2^24, where f32 rounds them (these are whole
    multiples of 2^14: exact all the same); and mixed extremes."""
    K = 4096
    a = torch.full((130, K), -128, dtype=torch.int8, device=DEV)
    b = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    one = torch.ones(130, device=DEV), torch.ones(M, device=DEV)
    c = sk.splitk_gemm_i8(a, one[0], b, one[1], out_dtype=F32)
    assert (c == float(K * 128 * 128)).all()
    g = gen(M)
    a = torch.where(torch.rand((130, K), device=DEV, generator=g) < 0.5, 127, 126).to(torch.int8)
    check_product(a, one[0], torch.full_like(b, 127), one[1], out=F32, exact_sum=False)


@pytest.mark.parametrize("M", [1, 8, 33, 129])
def test_product_runs_the_same_twice(M):
    a, sa, b, sb, bias = product_inputs(1, M, 1000, 4096, M, batched=False)
    first = sk.splitk_gemm_i8(a, sa, b, sb, bias=bias)
    for _ in range(3):
        assert torch.equal(sk.splitk_gemm_i8(a, sa, b, sb, bias=bias), first)


def test_product_writes_its_output_and_nothing_else():
    for M, N in ((3, 77), (50, 130), (140, 300)):
        a, sa, b, sb, _ = product_inputs(1, M, N, 256, M, batched=False)
        for dtype in (BF16, F32):
            room = torch.full((M + 2, N), 7.0, dtype=dtype, device=DEV)
            sk.splitk_gemm_i8(a, sa, b, sb, c=room[1:M + 1])
            torch.cuda.synchronize()
            assert (room[0] == 7).all() and (room[M + 1] == 7).all()
            assert torch.equal(room[1:M + 1], sk.splitk_gemm_i8(a, sa, b, sb, out_dtype=dtype))


def test_nan_scales_reach_their_tokens_alone():
    a, sa, b, sb, _ = product_inputs(1, 40, 256, 256, 5, batched=False)
    sb[11] = float("nan")
    c = sk.splitk_gemm_i8(a, sa, b, sb)
    assert torch.isnan(c[11]).all()
    c[11] = 0
    assert torch.isfinite(c).all()


@pytest.mark.parametrize("M,N,K", [(33, 64, 64), (47, 1000, 2048), (100, 500, 256), (300, 200, 4096), (1000, 65, 1024),
                                   (64, 2048, 2048), (700, 17, 16), (2_097_153, 1, 16)])
def test_product_of_few_weights_and_many_tokens(M, N, K):
    a, sa, b, sb, bias = product_inputs(1, M, N, K, M, batched=False)
    check_product(a, sa, b, sb, bias=bias)
    check_product(a, sa, b, sb, out=F32)


@pytest.mark.parametrize("M,N,K", [(33, 500, 7184), (64, 701, 7168), (65, 257, 16384), (129, 1000, 7168), (257, 300, 8208),
                                   (12, 18433, 7168), (20, 18433, 272), (40, 18432, 80), (300, 9001, 144),
                                   (1000, 2100, 1040), (513, 4098, 2064)])
@pytest.mark.parametrize("L", [1, 2])
def test_product_tiles_of_odd_sizes(M, N, K, L):
    a, sa, b, sb, bias = product_inputs(L, M, N, K, M + N, batched=L > 1)
    check_product(a, sa, b, sb, bias=bias if M % 2 else None)


@pytest.mark.parametrize("M,K", [(64, 256), (40, 4096), (300, 2048)])
def test_product_reports_a_wait_that_runs_out(M, K):
    """The pair's second CTA keeps its tiles to itself: the first one's bounded
    wait runs out, the call says so, and the next call is right again."""
    a, sa, b, sb, _ = product_inputs(1, M, 512, K, M, batched=False)
    sk.splitk_set_wait_limit_ns(5_000_000)
    sk.splitk_debug_inject(sk.INJECT_SKIP_PUBLISH)
    try:
        sk.splitk_gemm_i8(a, sa, b, sb)
        torch.cuda.synchronize()
        assert sk.splitk_get_fault()["code"] == -6
    finally:
        sk.splitk_debug_inject(0)
        sk.splitk_set_wait_limit_ns(0)
    assert sk.splitk_get_status() == 0
    check_product(a, sa, b, sb)


# ---------------------------------------------------------------- log probabilities
def logprob_ref(x, t, k):
    x = x.double().cpu()
    empty = torch.isneginf(x).all(-1)
    # distances to the maximum first: 64 bits do not hold the type's lowest
    # value and a logarithm's difference from it
    top = x.amax(-1, keepdim=True)
    order, x = x, x - torch.where(torch.isneginf(top), 0.0, top)
    lse = torch.where(empty, 0.0, torch.logsumexp(x, -1))
    lp = x - lse[:, None]
    p = torch.where(empty[:, None], 0.0, lp.exp())
    h = -torch.special.xlogy(p, p).sum(-1)
    ids = torch.sort(order, dim=-1, descending=True, stable=True).indices[:, :k]
    return lp, h, ids


def check_logprobs(x, t, k):
    M, V = x.shape
    logprob, entropy, ids, tops = sk.splitk_logprobs(x, t, top_k=k)
    torch.cuda.synchronize()
    lp, h, want = logprob_ref(x, t, k)
    # A logit's distance to the maximum rounds twice (relative 2 u), its exp
    # is off by 2^-22 and that much of the distance; at most V / 512 + 24
    # additions follow one another.  The result adds three roundings of its size.
    def bound(v):
        return 2 * U * (torch.nan_to_num(v.abs(), posinf=0.0) + h + V / 512 + 40)
    if t is not None:
        ref = lp.gather(1, t.cpu()[:, None])[:, 0]
        got = logprob.double().cpu()
        same = torch.isneginf(ref) & torch.isneginf(got)
        assert (same | ((got - ref).abs() <= bound(ref))).all()
    assert ((entropy.double().cpu() - h).abs() <= 2 * bound(h) + 2 * U * h).all()
    if k:
        assert torch.equal(ids.cpu(), want)
        ref, got = lp.gather(1, want), tops.double().cpu()
        same = torch.isneginf(ref) & torch.isneginf(got)
        assert (same | ((got - ref).abs() <= 2 * U * (torch.nan_to_num(ref.abs(), posinf=0.0) + h[:, None] +
                                                      V / 512 + 40))).all()
    return logprob, entropy, ids, tops


VOCABS = [1, 2, 5, 255, 256, 257, 300, 511, 1000, 4096, 4097, 8191, 16384, 32768, 50001, 65536, 131072]


@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_logprobs_vocabularies(V, dtype):
    g = gen(V)
    x = randn((4, V), g, dtype, 3.0)
    t = torch.randint(0, V, (4,), device=DEV, generator=g)
    for k in (0, 1, min(20, V), min(32, V)):
        check_logprobs(x, t, k)


@pytest.mark.parametrize("M", [1, 2, 3, 37, 38, 75, 76, 152, 153, 400])
def test_logprobs_row_counts(M):
    g = gen(M)
    check_logprobs(randn((M, 20000), g, BF16, 3.0), torch.randint(0, 20000, (M,), device=DEV, generator=g), 8)


@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 4), (7, 9), (8, 8)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_logprobs_rows_of_a_padded_buffer(offset, pad, dtype):
    """What stands beside a row (larger than all of it) is not read as part of
    it, whatever the alignment of its ends."""
    g = gen(offset)
    for V in (3, 100, 1000, 9001):
        room = torch.full((5, offset + V + pad), 1e4, dtype=dtype, device=DEV)
        room[:, offset:offset + V] = randn((5, V), g, dtype, 2.0)
        x = room[:, offset:offset + V]
        check_logprobs(x, torch.randint(0, V, (5,), device=DEV, generator=g), min(V, 4))


def test_logprobs_equal_logits_go_by_the_lowest_index():
    for V in (40, 5000, 70000):
        x = torch.zeros((3, V), dtype=BF16, device=DEV)
        x[1, V - 1] = -0.0
        x[2, ::7] = 1.0
        check_logprobs(x, torch.zeros(3, dtype=torch.int64, device=DEV), 32)
    # -0 equals 0
    x = torch.full((1, 600), -1.0, device=DEV)
    x[0, 3], x[0, 500] = -0.0, 0.0
    assert check_logprobs(x, None, 2)[2].tolist() == [[3, 500]]


@pytest.mark.parametrize("order", ["rising", "falling", "steps"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logprobs_sorted_rows(order, dtype):
    V = 30000
    v = torch.arange(V, device=DEV, dtype=F32) / 1000
    v = v if order == "rising" else v.flip(0) if order == "falling" else (v * 2).floor()
    check_logprobs(v.to(dtype).repeat(3, 1), torch.tensor([0, 1, V - 1], device=DEV), 32)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("V", [50, 7000, 60001])
def test_logprobs_masked_rows(dtype, V):
    """-inf masks that leave many, few, one and no logits."""
    g = gen(V)
    x = randn((7, V), g, dtype, 3.0)
    x[1, ::2] = float("-inf")
    x[2, 3:] = float("-inf")
    x[3, :V - 1] = float("-inf")
    x[4] = float("-inf")
    x[5, :V // 2] = float("-inf")
    x[6] = float("-inf")
    x[6, V // 3] = -3.0
    t = torch.tensor([0, 0, 1, V - 1, 5, V // 2, V // 3], device=DEV)
    logprob, entropy, ids, tops = check_logprobs(x, t, 10)
    assert logprob[3].item() == 0 and entropy[3].item() == 0
    assert math.isinf(logprob[4].item()) and entropy[4].item() == 0
    assert ids[4].tolist() == list(range(10)) and torch.isneginf(tops[4]).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_logprobs_masks_of_the_lowest_value(dtype):
    low = torch.finfo(dtype).min
    g = gen(9)
    x = randn((4, 9000), g, dtype, 3.0)
    x[0, 10:] = low                      # a few real logits first
    x[1, :8990] = low                    # and last: the maximum rises from the lowest value
    x[2] = low                           # every logit masked: all equal
    check_logprobs(x, torch.tensor([3, 8995, 0, 0], device=DEV), 12)


@pytest.mark.parametrize("M", [1, 160])
@pytest.mark.parametrize("V", [300, 20011, 131072])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logprobs_of_rows_with_few_kept_logits(dtype, V, M):
    """About as many logits as alternatives are kept, anywhere in the row: the
    masked ones of the lowest index follow them."""
    g = gen(V + M)
    for low in (float("-inf"), torch.finfo(dtype).min):
        for keep in (1, 19, 20, 21, 140):
            x = torch.full((M, V), low, dtype=dtype, device=DEV)
            at = torch.rand((M, V), device=DEV, generator=g).argsort(dim=1)[:, :keep]
            x.scatter_(1, at, randn((M, keep), g, dtype, 3.0))
            check_logprobs(x, at[:, 0].contiguous(), 20)


@pytest.mark.parametrize("levels", [2, 3, 40])
@pytest.mark.parametrize("V", [300, 20011, 131072])
def test_logprobs_of_rows_with_few_values(V, levels):
    g = gen(V + levels)
    for kept in (0.0, 0.001, 0.5):
        x = torch.randint(1, levels, (5, V), device=DEV, generator=g).to(BF16)
        x *= torch.rand((5, V), device=DEV, generator=g) < kept
        check_logprobs(x, torch.zeros(5, dtype=torch.int64, device=DEV), 32)


@pytest.mark.parametrize("V", [129, 200, 640, 777, 1024, 1300, 1919, 1920, 3968, 4100])
def test_logprobs_of_short_rows(V):
    """Rows whose lanes have a logit or two, in few CTAs and in many."""
    g = gen(V)
    for M in (3, 250, 700):
        for dtype in (BF16, F32):
            check_logprobs(randn((M, V), g, dtype, 3.0), torch.randint(0, V, (M,), device=DEV, generator=g), 32)


def test_logprobs_of_rows_of_nan_alone():
    for M, V in ((1, 131072), (1, 500), (200, 40000)):
        x = torch.full((M, V), float("nan"), dtype=BF16, device=DEV)
        logprob, entropy, ids, tops = sk.splitk_logprobs(x, torch.zeros(M, dtype=torch.int64, device=DEV), top_k=20)
        assert torch.isnan(logprob).all() and torch.isnan(entropy).all() and torch.isnan(tops).all()
        assert (ids >= 0).all() and (ids < V).all()


def test_logprobs_of_rows_with_nan_and_infinity():
    g = gen(10)
    x = randn((4, 3000), g, F32)
    x[1, 1234] = float("nan")
    x[2, 77] = float("inf")
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    logprob, entropy, ids, tops = sk.splitk_logprobs(x, t, top_k=5)
    assert torch.isnan(logprob[[1, 2]]).all() and torch.isnan(entropy[[1, 2]]).all()
    assert torch.isnan(tops[[1, 2]]).all()
    assert (ids >= 0).all() and (ids < 3000).all()
    for row in (0, 3):
        check_logprobs(x[row:row + 1], t[row:row + 1], 5)
        assert torch.isfinite(logprob[row]) and torch.isfinite(tops[row]).all()


def test_logprobs_of_large_logits_keep_their_differences():
    """A common offset does not cost precision: the distances to the maximum
    are exact."""
    g = gen(11)
    x = torch.randint(-40, 40, (3, 5000), device=DEV, generator=g).float()
    a = sk.splitk_logprobs(x, torch.zeros(3, dtype=torch.int64, device=DEV), top_k=4)
    b = sk.splitk_logprobs(x + 2.0 ** 20, torch.zeros(3, dtype=torch.int64, device=DEV), top_k=4)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


@pytest.mark.parametrize("M,V", [(1, 900), (3, 5000), (40, 40000), (700, 3000), (2, 131072), (200, 70001)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_logprobs_of_rows_that_are_all_but_decided(M, V, dtype):
    """log(1 + s) of a small s keeps s's precision, wherever the largest logit
    stands and however the row is shared out."""
    g = gen(M + V)
    for D in (4.0, 9.0, 15.5):
        for low in (float("-inf"), -1000.0):
            x = torch.full((M, V), low, dtype=dtype, device=DEV)
            at = torch.rand((M, V), device=DEV, generator=g).argsort(dim=1)[:, :4]
            x.scatter_(1, at[:, 1:], 2.0 - D)
            x.scatter_(1, at[:, :1], 2.0)
            logprob, entropy, ids, tops = sk.splitk_logprobs(x, at[:, 0].contiguous(), top_k=1)
            s = 3 * math.exp(-D)
            ref, h = -math.log1p(s), math.log1p(s) + s * D / (1 + s)
            # the exponent D log2 e rounds twice (1.5 2^-24 D as a share of s); the
            # power of two, the sum and the logarithm add a few 2^-24
            share = 2.0 ** -24 * (1.5 * D + 12)
            assert ((logprob.double() - ref).abs() <= share * -ref).all()
            assert ((entropy.double() - h).abs() <= 2 * share * h).all()
            assert (ids == at[:, :1]).all() and torch.equal(tops[:, 0], logprob)


def test_logprobs_token_outside_the_vocabulary():
    x = torch.zeros((4, 100), device=DEV)
    out = sk.splitk_logprobs(x, torch.tensor([-1, 100, 1 << 40, 99], device=DEV))
    assert torch.isnan(out[0][:3]).all() and abs(out[0][3].item() + math.log(100)) < 1e-6
    assert out[2] is None and out[3] is None


def test_logprobs_without_tokens_and_batched():
    g = gen(12)
    x = randn((2, 3, 800), g, BF16)
    t = torch.randint(0, 800, (2, 3), device=DEV, generator=g)
    logprob, entropy, ids, tops = sk.splitk_logprobs(x, t, top_k=3)
    assert logprob.shape == (2, 3) and entropy.shape == (2, 3) and ids.shape == tops.shape == (2, 3, 3)
    none, h, i, p = sk.splitk_logprobs(x.view(6, 800), top_k=3)
    assert none is None and torch.equal(h, entropy.view(6)) and torch.equal(i, ids.view(6, 3))


def test_logprobs_past_32_bit_offsets():
    """Rows whose logits start past 2^32 elements of a buffer."""
    stride = (1 << 31) + 8
    room = torch.empty(2 * stride + 512, dtype=BF16, device=DEV)
    x = torch.as_strided(room, (3, 512), (stride, 1))
    x.copy_(randn((3, 512), gen(13), BF16, 3.0))
    check_logprobs(x, torch.tensor([1, 2, 3], device=DEV), 5)


# ---------------------------------------------------------------- streams, graphs, the chain
def test_operators_run_on_the_stream_they_are_given():
    """Behind a long wait on their own stream, with inputs written there."""
    s = torch.cuda.Stream()
    g = gen(14)
    x, w = randn((8, 1024), g, BF16), randn((1024,), g, F32)
    a = codes((512, 1024), g)
    sa = torch.rand(512, device=DEV, generator=g) * 0.01
    ref_q, ref_s, _ = sk.splitk_rmsnorm_i8(x, w)
    ref = sk.splitk_logprobs(sk.splitk_gemm_i8(a, sa, ref_q, ref_s), top_k=4)
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
    q, sc, _ = sk.splitk_rmsnorm_i8(late, w, stream=s)
    c = sk.splitk_gemm_i8(a, sa, q, sc, stream=s)
    got = sk.splitk_logprobs(c, top_k=4, stream=s)
    s.synchronize()
    for u, v in zip(got[1:], ref[1:]):
        assert torch.equal(u, v)


def test_the_example_runs():
    import subprocess
    import sys
    from pathlib import Path
    root = Path(__file__).resolve().parent.parent
    res = subprocess.run([sys.executable, str(root / "examples" / "quantized_head.py"), "--tokens", "3", "--width", "512",
                          "--vocabulary", "1001", "--steps", "3"], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-2000:]
    assert "3 steps of 3 tokens" in res.stdout


def test_the_chain_in_a_graph():
    g = gen(15)
    M, D, V = 4, 2048, 5000
    x, r, w = randn((M, D), g, BF16), randn((M, D), g, BF16), randn((D,), g, BF16)
    a, sa = sk.splitk_quantize_i8(randn((V, D), g, BF16, 0.05))
    t = torch.randint(0, V, (M,), device=DEV, generator=g)

    def step():
        q, sc, out = sk.splitk_rmsnorm_i8(x, w, r)
        logits = sk.splitk_gemm_i8(a, sa, q, sc)
        return (out, logits, *sk.splitk_logprobs(logits, t, top_k=6))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (1, 2):
        x.copy_(randn((M, D), gen(seed), BF16))
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(outs, step()):
            assert torch.equal(u, v)
    assert sk.splitk_get_status() == 0


def plain_codes(x):
    """Codes and scales by elementary 32-bit operations."""
    x = x.float()
    scale = (x.abs().amax(-1) / 127).clamp_min(2.0 ** -126)
    return torch.round(x / scale[..., None]).to(torch.int8), scale


@pytest.mark.parametrize("M,D", [(2000, 7168), (3000, 1000), (700, 4999), (300, 16384), (40, 33000), (5000, 255), (1, 7168)])
def test_codes_are_the_formulas_to_the_bit(M, D):
    """No tolerance: x is exact in 32 bits, and the scale and the quotient are
    one rounding each.  Rows with outliers, rows whose values are whole
    multiples of a unit (most of them halves between two codes when the largest
    is 254 units), and tiny ones."""
    g = gen(D)
    x = randn((M, D), g, BF16)
    x = torch.where(torch.rand(D, device=DEV, generator=g) < 0.01, x * 30, x)
    steps = torch.randint(-254, 255, (M, D), device=DEV, generator=g).to(BF16)       # below 256: exact in bf16
    steps[:, 0] = torch.randint(128, 255, (M,), device=DEV, generator=g).to(BF16)
    even = steps.clone()
    even[:, 0] = 254
    tiny = randn((M, D), g, BF16, 2.0 ** -120)
    for rows in (x, steps, even, tiny):
        q, scale = sk.splitk_quantize_i8(rows)
        ref_q, ref_s = plain_codes(rows)
        assert torch.equal(scale, ref_s)
        assert torch.equal(q, ref_q), (q != ref_q).sum().item()


def test_every_code_of_every_largest_value():
    """Each bf16 mantissa as a row's largest value, with every bf16 value below
    it whose code is not 0: quotients have no other mantissas."""
    top = (128 + torch.arange(128, device=DEV)).float()                   # 128 .. 255
    values = top.repeat(9) * 2.0 ** -torch.arange(9, device=DEV).repeat_interleave(128).float()
    x = torch.where(values <= top[:, None], values, 0.0)
    x = torch.cat([x, -x], 1)
    for unit in (1.0, 2.0 ** -100, 2.0 ** 100):
        q, scale = sk.splitk_quantize_i8((unit * x).to(BF16))
        ref_q, ref_s = plain_codes(unit * x)
        assert torch.equal(scale, ref_s) and torch.equal(q, ref_q)


@pytest.mark.parametrize("D", [64, 1000, 4999, 7168, 16384, 33000])
def test_codes_of_the_norm_are_those_of_its_rows(D):
    """Features of one magnitude and a weight that carries the row: n is then a
    known f32 (the root of a power of four is exact), and so are its codes."""
    g = gen(D)
    M = 50
    sign = torch.where(torch.rand((M, D), device=DEV, generator=g) < 0.5, -1.0, 1.0)
    w = torch.randint(1, 255, (D,), device=DEV, generator=g).float()
    w[D // 2] = 254
    # mean(y^2) = 4 exactly (sums of 4 below 2^24), and eps is far below its last bit
    q, scale, _ = sk.splitk_rmsnorm_i8((2 * sign).to(BF16), w, eps=1e-12)
    ref_q, ref_s = plain_codes(sign * w)
    assert torch.equal(scale, ref_s) and torch.equal(q, ref_q)


def test_norm_whose_rows_pass_the_range_has_no_codes():
    """n past f32 is an infinity: the scale is NaN, as for one in the row."""
    x = torch.zeros((2, 256), dtype=BF16, device=DEV)
    x[0, 0] = x[1, 0] = 1
    w = torch.full((256,), 3e38, device=DEV)
    w[1:] = 1
    _, scale, _ = sk.splitk_rmsnorm_i8(x, w)
    assert torch.isnan(scale).all()


def check_nan_rows(x):
    """Rows that hold a NaN: no values, but alternatives that are tokens of the
    row, each one once."""
    M, V = x.shape
    for k in (1, 5, 20, 32):
        if k > V:
            continue
        t = torch.zeros(M, dtype=torch.int64, device=DEV)
        logprob, entropy, ids, tops = sk.splitk_logprobs(x, t, top_k=k)
        assert torch.isnan(logprob).all() and torch.isnan(entropy).all() and torch.isnan(tops).all()
        assert (ids >= 0).all() and (ids < V).all()
        assert (ids.sort(dim=1).values.diff(dim=1) > 0).all()


@pytest.mark.parametrize("V", [1, 5, 33, 200, 255, 256, 300, 511, 4000, 8192])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_logprobs_of_short_rows_of_nan_and_few_others(V, dtype):
    """Groups that hold NaN and masked logits, or NaN and what is beside the
    row, at every alignment of a row's ends."""
    nan, inf = float("nan"), float("inf")
    g = gen(V)
    for offset, pad in ((0, 0), (1, 0), (3, 6), (7, 1)):
        for M in (1, 200):
            room = torch.zeros((M, offset + V + pad), dtype=dtype, device=DEV)
            x = room[:, offset:offset + V]
            x.fill_(nan)
            check_nan_rows(x)
            if V == 1:
                continue
            for other in (-inf, -3.0, inf):
                for few in (1, 2, 3, 40):
                    x.fill_(nan)
                    x[:, torch.randperm(V, device=DEV, generator=g)[:min(few, V - 1)]] = other
                    check_nan_rows(x)


@pytest.mark.parametrize("M,V", [(1, 131072), (3, 50001), (300, 50001), (1, 40000), (700, 8000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logprobs_of_long_rows_of_nan_and_masks(M, V, dtype):
    """A masked logit in each group of 256 and NaN beside it, and fewer finite
    logits than alternatives."""
    nan, inf = float("nan"), float("inf")
    for step in (7, 200, 256, 3000):
        for finite in (0, 3):
            x = torch.full((M, V), nan, dtype=dtype, device=DEV)
            x[:, ::step] = -inf
            x[:, V // 3:V // 3 + finite] = 1.0
            check_nan_rows(x)
            x = torch.full((M, V), -inf, dtype=dtype, device=DEV)
            x[:, step // 2::step] = nan
            x[:, V // 3:V // 3 + finite] = 1.0
            check_nan_rows(x)


def stream_of_memory(t):
    """The stream whose memory a tensor lies in."""
    at = t.data_ptr()
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= at < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("no segment holds the tensor")


def made_on(s, **kw):
    """What each operator makes, on stream s."""
    x = torch.ones((4, 512), dtype=BF16, device=DEV)
    w = torch.ones(512, device=DEV)
    a, sa = torch.ones((256, 512), dtype=torch.int8, device=DEV), torch.ones(256, device=DEV)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    for operand in (x, w, a, sa, t):
        operand.record_stream(s)
    q, scale, out = sk.splitk_rmsnorm_i8(x, w, x, **kw)
    c = sk.splitk_gemm_i8(a, sa, q, scale, **kw)
    return (q, scale, out, c, *sk.splitk_quantize_i8(x, **kw), *sk.splitk_logprobs(c, t, top_k=2, **kw))


def test_outputs_are_of_the_memory_of_the_stream_given():
    s = torch.cuda.Stream()
    external = torch.cuda.ExternalStream(s.cuda_stream)
    current = torch.cuda.current_stream()
    for stream in (s, external):
        made = made_on(s, stream=stream)
        assert torch.cuda.current_stream() == current                   # as before
        assert all(stream_of_memory(t) == s.cuda_stream for t in made)
        s.synchronize()
    with torch.cuda.stream(s):
        assert all(stream_of_memory(t) == s.cuda_stream for t in made_on(s))
        default = made_on(current, stream=current)
    assert all(stream_of_memory(t) == current.cuda_stream for t in default)
    torch.cuda.synchronize()


def test_an_output_is_no_block_that_another_stream_still_writes():
    """A block freed on the current stream, whose last kernel there waits, does
    not become the output of a call on a stream given; and an output dropped
    while that stream still writes it does not come back on the current one."""
    g = gen(30)
    s = torch.cuda.Stream()
    a, b = codes((1024, 512), g), codes((300, 512), g)
    sa, sb = torch.rand(1024, device=DEV, generator=g), torch.rand(300, device=DEV, generator=g)
    ref = sk.splitk_gemm_i8(a, sa, b, sb, out_dtype=F32)
    torch.cuda.synchronize()
    victim = torch.empty((300, 1024), device=DEV)
    torch.cuda._sleep(50_000_000)
    victim.fill_(7)
    del victim
    c = sk.splitk_gemm_i8(a, sa, b, sb, out_dtype=F32, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(c, ref)
    at = c.data_ptr()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
    del c
    c = sk.splitk_gemm_i8(a, sa, b, sb, out_dtype=F32, stream=s)
    assert c.data_ptr() == at                            # in the stream's order: its own memory again
    del c
    other = torch.full((300, 1024), 3.0, device=DEV)
    assert other.data_ptr() != at
    torch.cuda.synchronize()
    assert (other == 3).all()


@pytest.mark.parametrize("M", [1, 16, 64, 300])
@pytest.mark.parametrize("K", [2048, 16384, 65536, 262144])
def test_product_of_codes_of_one_sign(M, K):
    """Sums far past 2^24, where additions may truncate: within the bound that
    the header gives, and never above the sum by more than its one rounding to
    nearest where that is what the additions do (half a unit of 2^-23 an
    addition of 16 codes)."""
    g = gen(K + M)
    a = torch.randint(100, 128, (300, K), device=DEV, generator=g, dtype=torch.int32).to(torch.int8)
    b = torch.randint(100, 128, (M, K), device=DEV, generator=g, dtype=torch.int32).to(torch.int8)
    c = sk.splitk_gemm_i8(a, torch.ones(300, device=DEV), b, torch.ones(M, device=DEV), out_dtype=F32).double()
    total = torch.matmul(b.double(), a.double().T)
    off = (c - total) / total
    # (the scales are 1: two products and the output round nothing)
    most = (K / 16 + 16) * 2.0 ** -23
    assert off.abs().max().item() <= most
    assert off.max().item() <= most / 2


FIRST_IN_A_GRAPH = """
import torch, split_bf16_gemm_swapped_gb300 as sk
dev = torch.device("cuda:0")
b = torch.randint(-127, 128, (64, 512), dtype=torch.int32, device=dev).to(torch.int8)
a = torch.randint(-127, 128, (1000, 512), dtype=torch.int32, device=dev).to(torch.int8)
sa, sb = torch.rand(1000, device=dev), torch.rand(64, device=dev)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    c = sk.splitk_gemm_i8(a, sa, b, sb)
    _, h, ids, top = sk.splitk_logprobs(c, top_k=3)
g.replay()
torch.cuda.synchronize()
ref = sk.splitk_gemm_i8(a, sa, b, sb)
_, h2, ids2, top2 = sk.splitk_logprobs(ref, top_k=3)
assert torch.equal(c, ref) and torch.equal(h, h2) and torch.equal(ids, ids2) and torch.equal(top, top2)
assert sk.splitk_get_status() == 0
print("same")
"""


def test_an_operators_first_call_may_be_captured():
    """Preparing its kernels is nothing that a capture forbids."""
    import subprocess
    import sys
    from pathlib import Path
    root = Path(__file__).resolve().parent.parent
    res = subprocess.run([sys.executable, "-c", FIRST_IN_A_GRAPH], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "same" in res.stdout, res.stdout[-2000:] + res.stderr[-2000:]


@pytest.mark.parametrize("M,N,K,runs", [(64, 18432, 1024, 6000), (64, 18432, 1280, 2000), (20, 18432, 1024, 2000),
                                        (20, 18432, 2048, 1000), (128, 14336, 1024, 2000), (128, 7168, 2048, 1000),
                                        (256, 18432, 1024, 1000), (300, 7168, 2048, 500), (1000, 4100, 1040, 300)])
def test_every_run_of_the_tiles_is_exact(M, N, K, runs):
    """A tile's codes are all read before the next tile's copy takes their place,
    and what one CTA of a pair converts is there when the other's MMAs read it:
    in each of many runs (the sums are whole numbers below 2^24)."""
    g = gen(M + N)
    a, b = codes((N, K), g), codes((M, K), g)
    one = torch.ones(N, device=DEV), torch.ones(M, device=DEV)
    ref = torch.matmul(b.double(), a.double().T).float()
    c = torch.empty((M, N), device=DEV)
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(runs):
        c.fill_(0.5)
        sk.splitk_gemm_i8(a, one[0], b, one[1], c=c)
        wrong += (c != ref).any()
    assert wrong.item() == 0
    assert sk.splitk_get_status() == 0


@pytest.mark.parametrize("M", [1, 4, 128])
def test_rows_before_a_wide_down_projection(M):
    D = 53248
    g = gen(M)
    x = randn((M, D), g, BF16)
    q, scale = sk.splitk_quantize_i8(x)
    ref_q, ref_s = plain_codes(x)
    assert torch.equal(scale, ref_s) and torch.equal(q, ref_q)
    check_norm(x, randn((M, D), g, BF16), randn((D,), g, F32))


@pytest.mark.parametrize("N,K", [(32000, 2048), (50257, 1024), (131072, 1040)])
@pytest.mark.parametrize("M", [1, 12, 40, 130])
def test_product_of_a_vocabulary_head(M, N, K):
    a, sa, b, sb, bias = product_inputs(1, M, N, K, M + N, batched=False)
    check_product(a, sa, b, sb, bias=bias if M == 12 else None, out=F32 if M == 40 else BF16)


def test_the_chain_in_threads_on_streams_of_their_own():
    """Each thread runs the chain on its own stream while the others do, with
    tokens enough for either product kernel, and gets what it gets alone."""
    import threading
    D, V, steps = 1024, 4000, 60
    g = gen(40)
    a, sa = sk.splitk_quantize_i8(randn((V, D), g, BF16, 0.05))
    w = randn((D,), g, F32)
    inputs = [(randn((M, D), g, BF16), randn((M, D), g, BF16)) for M in (1, 8, 40, 200)]

    def chain(x, r, **kw):
        q, s, out = sk.splitk_rmsnorm_i8(x, w, r, **kw)
        logits = sk.splitk_gemm_i8(a, sa, q, s, out_dtype=F32, **kw)
        return (q, s, out, logits, *sk.splitk_logprobs(logits, top_k=7, **kw)[1:])

    alone = [[t.clone() for t in chain(x, r)] for x, r in inputs]
    torch.cuda.synchronize()
    wrong, errors = [0] * len(inputs), []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for step in range(steps):
                # the stream given, or the thread's current one
                if step % 2:
                    got = chain(*inputs[i], stream=s)
                else:
                    with torch.cuda.stream(s):
                        got = chain(*inputs[i])
                s.synchronize()
                wrong[i] += not all(torch.equal(u, v) for u, v in zip(got, alone[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:                      # a thread's exception fails the test, not the thread alone
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(inputs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert wrong == [0] * len(inputs)
    torch.cuda.synchronize()
    assert sk.splitk_get_status() == 0


def guarded(shape, dtype, value):
    """A contiguous output inside a buffer full of `value`, and what is around it."""
    n = math.prod(shape)
    room = torch.full((n + 64,), value, dtype=dtype, device=DEV)
    return room[32:32 + n].view(shape), (room[:32], room[32 + n:])


def untouched(guards, value):
    return all(bool((g == value).all()) for g in guards)


@pytest.mark.parametrize("M,D", [(1, 1), (3, 77), (5, 512), (130, 7168), (2, 16392), (3, 40001)])
def test_norm_and_codes_write_their_outputs_and_nothing_else(M, D):
    g = gen(M + D)
    x, r, w = randn((M, D), g, BF16), randn((M, D), g, F32), randn((D,), g, F32)
    (q, gq), (s, gs), (out, go) = guarded((M, D), torch.int8, 99), guarded((M,), F32, 7.0), guarded((M, D), F32, 7.0)
    sk.splitk_rmsnorm_i8(x, w, r, q=q, scale=s, residual_out=out)
    torch.cuda.synchronize()
    assert untouched(gq, 99) and untouched(gs, 7.0) and untouched(go, 7.0)
    ref = sk.splitk_rmsnorm_i8(x, w, r)
    assert torch.equal(q, ref[0]) and torch.equal(s, ref[1]) and torch.equal(out, ref[2])
    sk.splitk_quantize_i8(x, q=q, scale=s)
    torch.cuda.synchronize()
    assert untouched(gq, 99) and untouched(gs, 7.0)


@pytest.mark.parametrize("M,V,k", [(1, 5, 5), (3, 1000, 20), (200, 4100, 32), (2, 131072, 32), (700, 8000, 1)])
def test_logprobs_write_their_outputs_and_nothing_else(M, V, k):
    g = gen(M + V)
    t = torch.randint(0, V, (M,), device=DEV, generator=g)
    for fill in (None, float("nan"), float("-inf")):
        x = randn((M, V), g, BF16, 3.0)
        if fill is not None:
            x[:, V // 2:] = fill
        (lp, g0), (h, g1) = guarded((M,), F32, 7.0), guarded((M,), F32, 7.0)
        (ids, g2), (tops, g3) = guarded((M, k), torch.int64, 7), guarded((M, k), F32, 7.0)
        sk.splitk_logprobs(x, t, top_k=k, logprob=lp, entropy=h, top_ids=ids, top_logprobs=tops)
        torch.cuda.synchronize()
        assert all(untouched(gd, 7) for gd in (g0, g1, g2, g3))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logprobs_of_the_largest_vocabulary(dtype):
    V = 1 << 22
    g = gen(22)
    x = randn((2, V), g, dtype, 3.0)
    x[1, 1000:] = float("-inf")
    check_logprobs(x, torch.tensor([V - 1, 3], device=DEV), 32)
