"""Microscaled 4-bit codes on the GPU against plain 64-bit implementations:
quantisation and back, residual addition + RMS norm to codes, the product of codes.

Codes and values are held to the bit where the formulas are exact; other
tolerances are bounds of f32 arithmetic, derived where they are stated (u is the
unit roundoff of f32, 2^-24)."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import split_bf16_gemm_swapped_gb300 as sk  # noqa: E402

DEV = torch.device("cuda:0")
U = 2.0 ** -24
U8, BF16, F16, F32, F64 = torch.uint8, torch.bfloat16, torch.float16, torch.float32, torch.float64
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(shape, g, dtype=F32, scale=1.0):
    return (scale * torch.randn(shape, device=DEV, generator=g)).to(dtype)


def sync():
    torch.cuda.synchronize()
    assert sk.splitk_get_status() == 0, sk.splitk_get_fault()


# ---------------------------------------------------------------- the format, in 64 bits
def nearest(q):
    """The codes 0..7 of magnitudes q >= 0, ties to the even one, from 5 on 6 or the
    tie's 4."""
    grid = torch.tensor(GRID, dtype=F64, device=q.device)
    middle = (grid[1:] + grid[:-1]) / 2
    code = torch.bucketize(q, middle)                          # middles below q: a middle itself goes down
    tie = (code < 7) & (q == middle[code.clamp_max(6)]) & (code % 2 == 1)
    return code + tie.long()


def power_of_two(e):
    """2^e as f64, from its bits (torch.ldexp and torch.pow may be a bit off)."""
    return ((e.long() + 1023) << 52).view(F64)


def scale_codes(top):
    """Of blocks with the largest magnitude `top` (finite)."""
    exponent = torch.frexp(top).exponent.long() - 1            # floor(log2)
    return torch.where(top == 0, 1, (exponent - 2 + 127).clamp_min(1))


def quantised(v):
    """(codes [.., K] 0..15, scale codes [.., K/32]) of f64 rows, NaN blocks among them."""
    b = v.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    s = scale_codes(torch.where(bad, 0.0, top))
    q = b * power_of_two(127 - s)[..., None]
    code = nearest(torch.where(bad[..., None], 0.0, q.abs())) + 8 * (torch.signbit(b) & ~bad[..., None]).long()
    return code.flatten(-2), torch.where(bad, 255, s)


def unpack(codes):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(U8).contiguous()


def values(codes, scale):
    """f64 values of packed codes."""
    table = torch.tensor(GRID + tuple(-x for x in GRID), dtype=F64, device=codes.device)
    by = power_of_two(scale.long() - 127)
    by = torch.where(scale == 255, float("nan"), by)
    return (table[unpack(codes)].unflatten(-1, (-1, 32)) * by[..., None]).flatten(-2)


def check_quantised(x, codes, scale):
    want, want_scale = quantised(x.double())
    assert torch.equal(scale.long(), want_scale)
    assert torch.equal(unpack(codes), want)


# ---------------------------------------------------------------- quantise
WIDTHS = [32, 64, 96, 224, 256, 480, 1024, 1056, 4096, 7168, 16384, 40000]


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("M", [1, 3, 130])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_quantise(K, M, dtype):
    g = gen(K + M)
    x = randn((M, K), g, dtype, 3.0)
    x[M // 2] *= 1e-4
    codes, scale = sk.splitk_quantize_mx4(x)
    sync()
    assert codes.shape == (M, K // 2) and scale.shape == (M, K // 32) and codes.dtype == scale.dtype == U8
    check_quantised(x, codes, scale)


@pytest.mark.parametrize("offset,pad", [(0, 8), (0, 3), (1, 0), (8, 8), (3, 5)])
@pytest.mark.parametrize("K", [32, 96, 2016, 8192])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_quantise_rows_cut_from_a_wider_tensor(offset, pad, K, dtype):
    x = randn((7, offset + K + pad), gen(K + offset), dtype)[:, offset:offset + K]
    codes, scale = sk.splitk_quantize_mx4(x)
    sync()
    check_quantised(x, codes, scale)


def test_quantise_every_bf16_value():
    """Each beside a largest value of every binade near its own, and alone."""
    bits = torch.arange(1 << 16, device=DEV, dtype=torch.int32)
    v = (bits << 16).view(F32).to(BF16)
    v = v[torch.isfinite(v)]
    blocks = []
    for up in (0, 1, 2, 3, 4, 5):
        top = torch.ldexp(torch.ones_like(v, dtype=F64), torch.frexp(v.double()).exponent.double() - 1 + up)
        top = torch.where(v == 0, 0.0, top.clamp_max(2.0 ** 127)).to(BF16)
        b = torch.zeros(len(v), 32, dtype=BF16, device=DEV)
        b[:, 5], b[:, 30] = v, top * (1.5 if up % 2 else 1.0)
        blocks.append(b)
    x = torch.cat(blocks)
    x = x[torch.isfinite(x).all(1)]
    codes, scale = sk.splitk_quantize_mx4(x)
    sync()
    check_quantised(x, codes, scale)
    assert scale.min() >= 1 and scale.max() <= 252


def test_quantise_halves_between_codes():
    """Every middle of two codes, and the f32 values beside it."""
    grid = torch.tensor(GRID, dtype=F64)
    middle = (grid[1:] + grid[:-1]) / 2
    near = torch.cat([middle.float(), torch.nextafter(middle.float(), torch.tensor(0.0)),
                      torch.nextafter(middle.float(), torch.tensor(9.0)), torch.tensor([7.9999995, 6.0, 6.5, 4.0])])
    for power in (-100, -3, 0, 90):
        x = torch.zeros(len(near), 64, device=DEV)
        x[:, 0], x[:, 31], x[:, 40] = near.to(DEV) * 2.0 ** power, 4.0 * 2.0 ** power, -near.to(DEV) * 2.0 ** power
        codes, scale = sk.splitk_quantize_mx4(x)
        sync()
        check_quantised(x, codes, scale)


def test_quantise_blocks_without_codes():
    """NaN and infinity give the scale NaN in their block alone; zeros and the
    smallest numbers code to multiples of the smallest scale."""
    x = randn((4, 128), gen(1), F32)
    x[0, 40], x[1, 0], x[2, 127] = float("nan"), float("inf"), float("-inf")
    x[3] = 0
    x[3, 64], x[3, 70], x[3, 100] = 2.0 ** -127, -2.0 ** -149, -0.0
    codes, scale = sk.splitk_quantize_mx4(x)
    sync()
    check_quantised(x, codes, scale)
    assert scale[0, 1] == scale[1, 0] == scale[2, 3] == 255 and (scale == 255).sum() == 3
    assert (scale[3] == 1).all() and codes[3, 32] == 1


def test_quantise_takes_batched_rows_and_given_outputs():
    x = randn((3, 4, 512), gen(2), BF16)
    codes, scale = torch.empty((3, 4, 256), dtype=U8, device=DEV), torch.empty((3, 4, 16), dtype=U8, device=DEV)
    got = sk.splitk_quantize_mx4(x, codes, scale)
    sync()
    assert got[0] is codes and got[1] is scale
    check_quantised(x, codes, scale)


# ---------------------------------------------------------------- dequantise
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_dequantise_every_code_and_scale(dtype):
    pairs = torch.arange(256, device=DEV, dtype=torch.int32).to(U8)
    codes = pairs.expand(256, 256).contiguous()                        # 512 values a row
    scale = torch.arange(256, device=DEV, dtype=torch.int32).to(U8)[:, None].expand(256, 16).contiguous()
    out = sk.splitk_dequantize_mx4(codes, scale, out_dtype=dtype)
    sync()
    want = values(codes, scale).to(F32)                                # 64 bits to 32: exact, or infinite past 2^128
    assert out.dtype == dtype
    assert torch.equal(out.nan_to_num(nan=7e7), want.to(dtype).nan_to_num(nan=7e7))
    assert torch.isnan(out[255]).all() and torch.isfinite(out[:141]).all()      # 6 * 2^14 passes f16


@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (5, 4064), (130, 7168), (1000, 64)])
def test_dequantise_gives_back_what_was_coded(M, K):
    x = randn((M, K), gen(M + K), BF16)
    codes, scale = sk.splitk_quantize_mx4(x)
    out = sk.splitk_dequantize_mx4(codes, scale)
    sync()
    assert out.dtype == BF16 and torch.equal(out.double(), values(codes, scale))
    # a value is at most half a step of its code off, or cut off above 6 scales
    by = power_of_two(scale.long() - 127).repeat_interleave(32, -1)
    assert ((out.double() - x.double()).abs() <= by * torch.where(x.double().abs() > 6 * by, 2.0, 1.0)).all()
    again, again_scale = sk.splitk_quantize_mx4(out)
    sync()
    assert torch.equal(sk.splitk_dequantize_mx4(again, again_scale), out)


# ---------------------------------------------------------------- norm
def check_norm(x, r, w, eps=1e-6, **kw):
    keep = None if r is None else r.clone()
    codes, scale, out = sk.splitk_rmsnorm_mx4(x, w, r, eps=eps, **kw)
    sync()
    y = x.float() if r is None else x.float() + keep.float()
    if r is None:
        assert out is None
    else:
        assert out.dtype == r.dtype and torch.equal(out, y.to(r.dtype))
    D = x.shape[-1]
    # The sum: a thread's at most 32 squares are f32, joined in 64 bits; then a
    # root, a quotient and two products round once each (the mean, once more).
    rel = (32 + 1 + 5) * U
    n = y.double() / (y.double().square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    b = n.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    s = scale.long()
    assert ((s == scale_codes(top * (1 - rel))) | (s == scale_codes(top * (1 + rel)))).all()
    q = (b * power_of_two(127 - s)[..., None]).flatten(-2)
    code = unpack(codes)
    low, high = nearest(q.abs() * (1 - rel)), nearest(q.abs() * (1 + rel))
    assert ((code & 7) >= low).all() and ((code & 7) <= high).all()
    assert ((code & 8 > 0) == torch.signbit(n)).all()
    return codes, scale, out


@pytest.mark.parametrize("D", [32, 64, 96, 256, 288, 512, 544, 1024, 4096, 4992, 7168, 8224, 16384, 16416, 32768, 32800, 40000])
@pytest.mark.parametrize("residual", [None, BF16, F32])
@pytest.mark.parametrize("weight", [BF16, F32])
def test_norm(D, residual, weight):
    g = gen(D)
    x = randn((5, D), g, BF16)
    r = None if residual is None else randn((5, D), g, residual, 4.0)
    check_norm(x, r, (1 + randn((D,), g, F32, 0.1)).to(weight))


@pytest.mark.parametrize("M", [1, 2, 3, 4, 33, 500, 2000])
@pytest.mark.parametrize("D", [96, 2048, 7168])
def test_norm_row_counts(M, D):
    g = gen(M * D)
    check_norm(randn((M, D), g, BF16), randn((M, D), g, BF16), randn((D,), g, BF16))


@pytest.mark.parametrize("offset,pad", [(0, 8), (0, 3), (1, 0), (8, 8), (3, 5)])
@pytest.mark.parametrize("D", [64, 256, 2016, 33024])
def test_norm_rows_cut_from_a_wider_tensor(offset, pad, D):
    g = gen(D + offset)
    x = randn((6, offset + D + pad), g, BF16)[:, offset:offset + D]
    check_norm(x, randn((6, D), g, F32), randn((D,), g, F32))


@pytest.mark.parametrize("D", [64, 7168, 33024])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_of_operands_at_odd_places(D, dtype):
    """A residual, its sum and a weight that start at an element of no alignment."""
    g = gen(D)
    flat = lambda n, t: randn((n + 1,), g, t)[1:]                      # noqa: E731
    r, out = flat(3 * D, dtype).view(3, D), flat(3 * D, dtype).view(3, D)
    check_norm(randn((3, D), g, BF16), r, flat(D, F32), residual_out=out)


@pytest.mark.parametrize("D", [64, 1024, 7168, 33024])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_residual_in_place(D, dtype):
    g = gen(D)
    x, r, w = randn((7, D), g, BF16), randn((7, D), g, dtype), randn((D,), g, BF16)
    q0, s0, out0 = sk.splitk_rmsnorm_mx4(x, w, r)
    same = r.clone()
    q1, s1, out1 = sk.splitk_rmsnorm_mx4(x, w, same, residual_out=same)
    sync()
    assert out1 is same and torch.equal(out0, same) and torch.equal(q0, q1) and torch.equal(s0, s1)


def test_norm_of_rows_without_codes():
    """NaN, infinity and squares past the range give the scale NaN, in their row
    alone; zeros code to zeros."""
    x = randn((7, 320), gen(4), BF16)
    x[0] = 0
    x[2, 17], x[3, 319], x[4, 0] = float("nan"), float("inf"), float("-inf")
    x[5] = 3e38
    codes, scale, _ = sk.splitk_rmsnorm_mx4(x, torch.ones(320, device=DEV))
    sync()
    assert (codes[0] == 0).all() and (scale[0] == 1).all()
    assert (scale[[2, 3, 4, 5]] == 255).all() and (codes[[2, 3, 4, 5]] == 0).all() and (scale[[0, 1, 6]] < 255).all()
    w = torch.ones(320, device=DEV)
    w[33] = float("nan")
    _, scale, _ = sk.splitk_rmsnorm_mx4(x[[1, 6]], w)
    sync()
    assert (scale[:, 1] == 255).all() and (scale[:, [0] + list(range(2, 10))] < 255).all()


def test_norm_is_the_elementary_operations_to_the_bit():
    """The formula in 32 bits, in its order, with the mean in 64: of 15 million
    values none may differ but in a row whose mean the f32 sums of a thread moved
    to its neighbour (a few rows in a hundred)."""
    g = gen(9)
    x, r, w = randn((2048, 7168), g, BF16), randn((2048, 7168), g, F32, 4.0), (1 + randn((7168,), g, F32, 0.1)).to(BF16)
    codes, scale, out = sk.splitk_rmsnorm_mx4(x, w, r)
    sync()
    y = x.float() + r
    mean = y.double().square().mean(1, keepdim=True).float()
    n = y * w.float() * (1 / torch.sqrt(mean + 1e-6))
    want, want_scale = quantised(n.double())
    off = ((unpack(codes) != want).any(1) | (scale.long() != want_scale).any(1)).sum().item()
    assert off <= 2, off


@pytest.mark.parametrize("D,residual", [(64, None), (64, BF16), (1024, None), (1024, F32), (7168, None), (7168, BF16)])
def test_norm_of_other_rows_is_the_elementary_operations_to_the_bit(D, residual):
    """As above.  A thread's sums move the mean to a neighbour in up to one row of four
    here; the factor then moves by at most one in 2^23, which takes a value of a row
    over a border of codes once in some 10^7: of 2048 rows less than one, on average."""
    g = gen(D)
    x, w = randn((2048, D), g, BF16), (1 + randn((D,), g, F32, 0.1)).to(BF16)
    r = None if residual is None else randn((2048, D), g, residual, 4.0)
    codes, scale, _ = sk.splitk_rmsnorm_mx4(x, w, r)
    sync()
    y = x.float() if r is None else x.float() + r.float()
    n = y * w.float() * (1 / torch.sqrt(y.double().square().mean(1, keepdim=True).float() + 1e-6))
    want, want_scale = quantised(n.double())
    off = ((unpack(codes) != want).any(1) | (scale.long() != want_scale).any(1)).sum().item()
    assert off <= 2, off


@pytest.mark.parametrize("M", [1, 700])
@pytest.mark.parametrize("D", [64, 512, 544, 1024, 2048, 4992, 7168, 20480])
def test_norm_joins_its_threads_sums_without_a_loss(M, D):
    """Whole numbers whose squares a thread sums exactly (32 of at most 723^2 are below
    2^24), so that the mean is the exact one, rounded once; and weights that bring every
    value of the row to a border between two codes, where another mean shows."""
    g = gen(D)
    grid = torch.tensor(GRID, dtype=F64, device=DEV)
    middle = (grid[1:] + grid[:-1]) / 2
    for _ in range(30):
        y = torch.randint(1, 724, (D,), device=DEV, generator=g) * (2 * torch.randint(0, 2, (D,), device=DEV, generator=g) - 1)
        x = torch.randint(-200, 201, (D,), device=DEV, generator=g).to(BF16)
        r = (y - x.long()).float()
        factor = 1 / torch.sqrt(y.double().square().mean().float() + 1e-6)
        goal = middle[torch.randint(0, 7, (D,), device=DEV, generator=g)]
        goal[::32] = 5.0                                               # every block's scale is 1
        w = (goal / (y.double() * factor.double())).float()
        codes, scale, _ = sk.splitk_rmsnorm_mx4(x.expand(M, D).contiguous(), w, r.expand(M, D).contiguous())
        sync()
        want, want_scale = quantised((y.float() * w * factor).double())
        assert (scale.long() == want_scale).all() and (unpack(codes) == want).all()


# ---------------------------------------------------------------- product
def random_codes(shape, g, low=120, high=134):
    """Codes, and scale codes of a few binades."""
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), device=DEV, generator=g, dtype=torch.int32).to(U8)
    scale = torch.randint(low, high, (*shape[:-1], shape[-1] // 32), device=DEV, generator=g, dtype=torch.int32).to(U8)
    return codes, scale


def check_product(a, sa, b, sb, bias=None, exact=False):
    c = sk.splitk_gemm_mx4(a, sa, b, sb, bias=bias, out_dtype=F32)
    sync()
    K = 2 * a.shape[-1]
    av, bv = values(a, sa), values(b, sb)
    ref = torch.matmul(bv, av.transpose(-1, -2))
    if bias is not None:
        ref = ref + bias.double()[..., None, :]
    if exact:
        assert torch.equal(c.double(), ref)
    else:
        # exact products; a sum of 16 of them or more is added at a time, truncated at
        # worst (2 u of what is summed so far, at most the sum of magnitudes), and once
        # for each part of K; the bias rounds once
        size = torch.matmul(bv.abs(), av.abs().transpose(-1, -2))
        bound = 2 * U * (K / 16 + 16) * size + U * ref.abs()
        err = (c.double() - ref).abs()
        assert (err <= bound).all(), (err - bound).max().item()
    rounded = sk.splitk_gemm_mx4(a, sa, b, sb, bias=bias)
    sync()
    assert torch.equal(rounded, c.to(BF16))
    return c


def product_inputs(L, M, N, K, seed, batched=True, **kw):
    g = gen(seed)
    shape = (lambda *s: s) if batched else (lambda *s: s[1:])
    a, sa = random_codes(shape(L, N, K), g, **kw)
    b, sb = random_codes(shape(L, M, K), g, **kw)
    return a, sa, b, sb


def test_product_of_one_block_by_hand():
    """Row n of the weights holds one code at one place, token m another: each
    output is one product, at its own row, column and scale."""
    g = gen(1)
    for K in (32, 64, 256, 512):
        at = torch.randint(0, K, (128,), device=DEV, generator=g)
        a = torch.zeros(128, K, dtype=torch.long, device=DEV)
        a[torch.arange(128), at] = torch.randint(0, 16, (128,), device=DEV, generator=g)
        b = torch.randint(0, 16, (8, K), device=DEV, generator=g)
        sa = torch.randint(100, 150, (128, K // 32), device=DEV, generator=g).to(U8)
        sb = torch.randint(100, 150, (8, K // 32), device=DEV, generator=g).to(U8)
        check_product(pack(a), sa, pack(b), sb, exact=True)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 256, 257, 600])
@pytest.mark.parametrize("N,K", [(128, 256), (100, 544), (1000, 1024), (257, 4128)])
def test_product_shapes(M, N, K):
    check_product(*product_inputs(1, M, N, K, M * N + K, batched=False))


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 192, 224, 256, 288, 480, 512, 1056, 2080, 4128])
@pytest.mark.parametrize("M", [1, 20, 70, 300])
def test_product_k_tails(K, M):
    check_product(*product_inputs(1, M, 200, K, M + K))


@pytest.mark.parametrize("M", [1, 12, 40, 150, 300])
@pytest.mark.parametrize("K", [512, 992])
def test_product_batches(M, K):
    g = gen(M)
    bias = randn((3, 300), g, BF16, 100.0)
    check_product(*product_inputs(3, M, 300, K, M), bias=bias)


@pytest.mark.parametrize("M,N,K", [(1, 7168, 2048), (16, 4096, 7168), (64, 2304, 7168), (128, 1024, 16384), (1000, 2048, 7168),
                                   (513, 18432, 512), (300, 4000, 2016), (1, 500, 16384), (2048, 4096, 1024)])
def test_product_workload_shapes(M, N, K):
    check_product(*product_inputs(1, M, N, K, M + N + K, batched=False))


@pytest.mark.parametrize("M", [1, 9, 40, 100, 300, 700])
@pytest.mark.parametrize("K", [256, 2016, 16384])
def test_product_of_one_scale_is_exact(M, K):
    """Sums of quarters up to 36 K stay below 2^24 of them."""
    a, sa, b, sb = product_inputs(1, M, 384, K, M + K, low=127, high=128)
    check_product(a, sa, b, sb, exact=4 * 36 * K < 2 ** 24)


@pytest.mark.parametrize("M", [1, 16, 100, 300])
def test_product_of_extreme_scales(M):
    """Scales of every code whose products stay in range, and codes of zero."""
    g = gen(M)
    a, _, b, _ = product_inputs(1, M, 256, 512, M)
    sa = torch.randint(1, 60, (1, 256, 16), device=DEV, generator=g).to(U8)
    sb = torch.randint(190, 240, (1, M, 16), device=DEV, generator=g).to(U8)
    check_product(a, sa, b, sb)
    check_product(torch.zeros_like(a), sa, b, sb, exact=True)


@pytest.mark.parametrize("M", [3, 50, 300])
def test_nan_scales_reach_their_rows_alone(M):
    a, sa, b, sb = product_inputs(1, M, 300, 1024, M, batched=False)
    sa[17, 5], sa[299, 31], sb[1, 30], sb[M - 1, 0] = 255, 255, 255, 255
    c = sk.splitk_gemm_mx4(a, sa, b, sb)
    sync()
    want = torch.zeros(M, 300, dtype=torch.bool, device=DEV)
    want[:, 17] = want[:, 299] = want[1] = want[M - 1] = True
    assert torch.equal(torch.isnan(c), want)


@pytest.mark.parametrize("by", ["quantise", "norm"])
@pytest.mark.parametrize("M", [3, 50, 300])
@pytest.mark.parametrize("K", [32, 1056, 4128])
def test_nan_and_infinite_values_reach_their_rows_alone(M, K, by):
    """What the quantisation and the norm make of them, zeros under a scale that is no
    number, on both sides; the last 64 of K are half full."""
    g = gen(M + K)
    w, x = randn((300, K), g, BF16), randn((M, K), g, BF16)
    w[17, K - 1], w[129, 0], w[299, K // 2] = float("nan"), float("inf"), float("-inf")
    x[0, 0], x[1, K - 1], x[M - 1, 5] = float("inf"), float("nan"), float("-inf")
    a = sk.splitk_quantize_mx4(w)
    b = sk.splitk_quantize_mx4(x) if by == "quantise" else sk.splitk_rmsnorm_mx4(x, torch.ones(K, device=DEV))[:2]
    c = sk.splitk_gemm_mx4(*a, *b, out_dtype=F32)
    sync()
    assert (a[1] == 255).any(1).sum() == 3 and (b[1] == 255).any(1).sum() == 3
    want = torch.zeros(M, 300, dtype=torch.bool, device=DEV)
    want[:, [17, 129, 299]] = True
    want[[0, 1, M - 1]] = True
    assert torch.equal(torch.isnan(c), want) and torch.isfinite(c[~want]).all()


@pytest.mark.parametrize("M", [1, 8, 33, 129, 700])
def test_product_runs_the_same_twice(M):
    ops = product_inputs(1, M, 1000, 4096, M)
    first = sk.splitk_gemm_mx4(*ops, out_dtype=F32)
    for _ in range(20):
        assert torch.equal(sk.splitk_gemm_mx4(*ops, out_dtype=F32), first)
    sync()


@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("K", [1024, 1152, 1056])
def test_product_of_scales_at_odd_places(offset, K):
    """Scale codes need no alignment."""
    a, sa, b, sb = product_inputs(1, 40, 200, K, K, batched=False)
    odd = lambda s: torch.cat([s.new_zeros(offset), s.flatten()])[offset:].view(s.shape)      # noqa: E731
    want = sk.splitk_gemm_mx4(a, sa, b, sb, out_dtype=F32)
    got = sk.splitk_gemm_mx4(a, odd(sa), b, odd(sb), out_dtype=F32)
    sync()
    assert torch.equal(got, want)


def test_product_agrees_with_the_bf16_product_of_4_bit_weights():
    """The same weights in splitk_gemm_w4a16, with the tokens' values in bf16."""
    g = gen(5)
    a, sa = random_codes((512, 1024), g)
    b, sb = random_codes((4, 1024), g)
    wide = sk.splitk_gemm_w4a16(a, sa, sk.splitk_dequantize_mx4(b, sb))
    c = sk.splitk_gemm_mx4(a, sa, b, sb)
    sync()
    size = torch.matmul(values(b, sb).abs(), values(a, sa).abs().T)
    # both round to bf16, and differ before that by the order of their sums
    assert ((c.double() - wide.double()).abs() <= 2.0 ** -8 * (c.double().abs() + wide.double().abs()) +
            4 * U * (1024 / 16 + 16) * size).all()


@pytest.mark.parametrize("M,K", [(4, 256), (64, 4096), (300, 2048)])
def test_product_reports_a_wait_that_runs_out(M, K):
    ops = product_inputs(1, M, 256, K, 1)
    want = sk.splitk_gemm_mx4(*ops)
    sync()
    sk.splitk_set_wait_limit_ns(20_000_000)
    sk.splitk_debug_inject(sk.INJECT_SKIP_PUBLISH)
    try:
        sk.splitk_gemm_mx4(*ops)
        torch.cuda.synchronize()
        assert sk.splitk_get_status() == -6
    finally:
        sk.splitk_debug_inject(0)
        sk.splitk_set_wait_limit_ns(0)
    assert torch.equal(sk.splitk_gemm_mx4(*ops), want)
    sync()
