"""The operators of a decode step in 4 bits together, as a server runs them: norm to
codes, product of codes, adjustment of the logits, log probabilities; their streams,
graphs and threads, the memory of their outputs, and that they write nothing else."""
from __future__ import annotations

import math
import subprocess
import sys
import threading
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import split_bf16_gemm_swapped_gb300 as sk  # noqa: E402

DEV = torch.device("cuda:0")
ROOT = Path(__file__).resolve().parent.parent
U8, BF16, F16, F32 = torch.uint8, torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(shape, g, dtype=BF16, scale=1.0):
    return (scale * torch.randn(shape, device=DEV, generator=g)).to(dtype)


def same(a, b):
    """Bit for bit, but NaN for NaN."""
    if a.is_floating_point():
        return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(nan=0.0), b.nan_to_num(nan=0.0))
    return torch.equal(a, b)


class Step:
    """A decode step's end with weights of its own, and a row's parameters."""

    def __init__(self, M, D, V, seed, H=50, B=6):
        g = gen(seed)
        self.w = randn((D,), g, F32)
        self.head, self.head_scale = sk.splitk_quantize_mx4(randn((V, D), g, BF16, 0.05))
        self.x, self.r = randn((M, D), g), randn((M, D), g, BF16, 4.0)
        self.how = dict(
            history=torch.randint(0, V, (M, H), device=DEV, generator=g),
            lengths=torch.randint(0, H + 1, (M,), device=DEV, generator=g),
            prompt_lengths=torch.randint(0, H // 2, (M,), device=DEV, generator=g),
            repetition=1 + torch.rand(M, device=DEV, generator=g), presence=torch.rand(M, device=DEV, generator=g),
            frequency=torch.rand(M, device=DEV, generator=g),
            bias_ids=torch.randint(0, V, (M, B), device=DEV, generator=g), bias_values=randn((M, B), g, F32, 5.0),
            allowed=torch.randint(-2**31, 2**31, (M, -(-V // 32)), device=DEV, generator=g).to(torch.int32))

    def __call__(self, **kw):
        codes, scale, out = sk.splitk_rmsnorm_mx4(self.x, self.w, self.r, **kw)
        logits = sk.splitk_gemm_mx4(self.head, self.head_scale, codes, scale, out_dtype=F32, **kw)
        adjusted = sk.splitk_adjust_logits(logits, **self.how, **kw)
        _, entropy, ids, top = sk.splitk_logprobs(adjusted, top_k=6, **kw)
        return codes, scale, out, logits, adjusted, entropy, ids, top


def test_the_chain_answers_as_its_formulas_do():
    """The chain's own logits, adjusted by elementary operations, have its most probable
    tokens; and what the codes stand for multiplies to its logits."""
    step = Step(5, 1024, 5000, 1)
    codes, scale, _, logits, adjusted, _, ids, top = step()
    torch.cuda.synchronize()
    a = sk.splitk_dequantize_mx4(step.head, step.head_scale, out_dtype=F32).double()
    b = sk.splitk_dequantize_mx4(codes, scale, out_dtype=F32).double()
    # exact products; 1024 of them added 16 or more at a time, each time off by 2 u at most
    bound = 2 * 2.0 ** -24 * (1024 / 16 + 16) * (b.abs() @ a.abs().T)
    assert ((logits.double() - b @ a.T).abs() <= bound).all()
    want = logits.clone()
    for m in range(5):
        n, p = int(step.how["lengths"][m]), int(step.how["prompt_lengths"][m])
        said = step.how["history"][m, :n]
        count = torch.bincount(said[p:], minlength=5000).float()
        seen = torch.bincount(said, minlength=5000) > 0
        row, rep = want[m], step.how["repetition"][m]
        row = torch.where(seen, torch.where(row > 0, row / rep, row * rep), row)
        row = torch.where(count > 0, row - step.how["frequency"][m] * count - step.how["presence"][m], row)
        for i, v in zip(step.how["bias_ids"][m].tolist(), step.how["bias_values"][m]):
            row[i] += v
        ok = (step.how["allowed"][m].long()[torch.arange(5000, device=DEV) // 32] >> (torch.arange(5000, device=DEV) % 32)) & 1
        want[m] = row.masked_fill(ok == 0, float("-inf"))
    # five roundings of values below 64 (2^-19 apart), two of a bias listed twice
    assert ((want - adjusted).abs().nan_to_num(nan=0.0) <= 8 * 2.0 ** -19).all()
    lp = torch.log_softmax(adjusted.double(), 1)
    assert torch.equal(torch.sort(lp, dim=1, descending=True, stable=True).indices[:, :6], ids)
    assert ((lp.gather(1, ids) - top.double()).abs() <= 1e-5).all()
    assert sk.splitk_get_status() == 0


@pytest.mark.parametrize("M", [1, 40, 300])
def test_the_chain_on_a_stream_given(M):
    """Behind a long wait on its own stream, with inputs written there."""
    s = torch.cuda.Stream()
    step = Step(M, 1024, 3000, M)
    ref = [t.clone() for t in step()]
    x = step.x
    step.x = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        step.x.copy_(x)
    got = step(stream=s)
    s.synchronize()
    assert all(same(u, v) for u, v in zip(got, ref))


def test_quantisation_on_a_stream_given():
    s = torch.cuda.Stream()
    x = randn((64, 2048), gen(2))
    ref = sk.splitk_quantize_mx4(x)
    back = sk.splitk_dequantize_mx4(*ref)
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
    got = sk.splitk_quantize_mx4(late, stream=s)
    out = sk.splitk_dequantize_mx4(*got, stream=s)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]) and torch.equal(out, back)


@pytest.mark.parametrize("M", [1, 4, 40, 200])
def test_the_chain_in_graphs(M):
    """Two captured graphs of one chain, replayed in turn beside calls, with inputs
    changed between; replayed at once on streams of their own."""
    step = Step(M, 2048, 5000, 15 + M)
    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step())
    for seed in (1, 2):
        step.x.copy_(randn(step.x.shape, gen(seed)))
        step.how["lengths"].copy_(torch.randint(0, 51, (M,), device=DEV, generator=gen(seed)))
        for i in (0, 1, 0):
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(same(u, v) for u, v in zip(outs[i], step()))
    ref = [t.clone() for t in step()]
    for o in outs:
        for t in o:
            t.zero_()
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(same(u, v) for o in outs for u, v in zip(o, ref))
    assert sk.splitk_get_status() == 0


FIRST_IN_A_GRAPH = """
import torch, split_bf16_gemm_swapped_gb300 as sk
dev = torch.device("cuda:0")
x = torch.randn(%d, 512, device=dev).to(torch.bfloat16)
a = torch.randint(0, 256, (1000, 256), dtype=torch.int32, device=dev).to(torch.uint8)
sa = torch.randint(120, 130, (1000, 16), dtype=torch.int32, device=dev).to(torch.uint8)
w = torch.ones(512, device=dev)
h = torch.randint(0, 1000, (x.shape[0], 20), device=dev)
f = torch.ones(x.shape[0], device=dev)
def step():
    q, s, _ = sk.splitk_rmsnorm_mx4(x, w)
    c = sk.splitk_gemm_mx4(a, sa, q, s)
    return q, s, c, sk.splitk_adjust_logits(c, history=h, frequency=f), *sk.splitk_quantize_mx4(x), sk.splitk_dequantize_mx4(q, s)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(u, v) for u, v in zip(out, step()))
assert sk.splitk_get_status() == 0
print("same")
"""


@pytest.mark.parametrize("M", [3, 200])
def test_an_operators_first_call_may_be_captured(M):
    res = subprocess.run([sys.executable, "-c", FIRST_IN_A_GRAPH % M], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "same" in res.stdout, res.stdout[-2000:] + res.stderr[-2000:]


def stream_of_memory(t):
    """The stream whose memory a tensor lies in."""
    at = t.data_ptr()
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= at < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("no segment holds the tensor")


def test_outputs_are_of_the_memory_of_the_stream_given():
    s = torch.cuda.Stream()
    step = Step(4, 512, 1000, 3)
    torch.cuda.synchronize()

    def made(**kw):
        codes, scale, *rest = step(**kw)
        return (codes, scale, *rest, *sk.splitk_quantize_mx4(step.x, **kw), sk.splitk_dequantize_mx4(codes, scale, **kw))

    current = torch.cuda.current_stream()
    for stream in (s, torch.cuda.ExternalStream(s.cuda_stream)):
        outs = made(stream=stream)
        assert torch.cuda.current_stream() == current
        assert all(stream_of_memory(t) == s.cuda_stream for t in outs)
        s.synchronize()
    with torch.cuda.stream(s):
        assert all(stream_of_memory(t) == s.cuda_stream for t in made())
        default = made(stream=current)
    assert all(stream_of_memory(t) == current.cuda_stream for t in default)
    torch.cuda.synchronize()


def test_the_chain_in_threads_on_streams_of_their_own():
    """Each thread runs its chain while the others run theirs, and gets what it gets
    alone: products of one and of many tiles, each holding tensor memory."""
    steps = [Step(M, 1024, 4000, 40 + M) for M in (1, 8, 40, 100, 300)]
    alone = [[t.clone() for t in step()] for step in steps]
    torch.cuda.synchronize()
    wrong, errors = [0] * len(steps), []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for turn in range(40):
                if turn % 2:
                    got = steps[i](stream=s)
                else:
                    with torch.cuda.stream(s):
                        got = steps[i]()
                s.synchronize()
                wrong[i] += not all(same(u, v) for u, v in zip(got, alone[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(steps))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert wrong == [0] * len(steps)
    torch.cuda.synchronize()
    assert sk.splitk_get_status() == 0


def test_products_beside_the_other_products():
    """Kernels that hold tensor memory run at once on streams of their own: this one,
    the 8-bit one and the bf16 one."""
    g = gen(50)
    x, a = randn((200, 1024), g), randn((3000, 1024), g, BF16, 0.05)
    a4, a8 = sk.splitk_quantize_mx4(a), sk.splitk_quantize_i8(a)
    x4, x8 = sk.splitk_quantize_mx4(x), sk.splitk_quantize_i8(x)
    few = x[:8].contiguous()
    runs = [lambda **kw: sk.splitk_gemm_mx4(*a4, *x4, **kw), lambda **kw: sk.splitk_gemm_i8(*a8, *x8, **kw),
            lambda **kw: sk.splitk_gemm_bf16(a, few, **kw), lambda **kw: sk.splitk_gemm_mx4(*a4, x4[0][:8], x4[1][:8], **kw)]
    ref = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(30):
        got = [run(stream=s) for run, s in zip(runs, streams)]
        for s in streams:
            s.synchronize()
        assert all(torch.equal(u.view(v.shape), v) for u, v in zip(got, ref))
    assert sk.splitk_get_status() == 0


# ---------------------------------------------------------------- every run, and nothing else written
@pytest.mark.parametrize("M,N,K,runs", [(1, 7168, 2048, 2000), (16, 4096, 7168, 2000), (20, 18432, 1024, 1000), (64, 18432, 1280, 1000),
                                        (128, 14336, 1024, 1000), (128, 7168, 4096, 1000), (256, 18432, 1024, 500),
                                        (300, 7168, 2048, 500), (1000, 4100, 1056, 300), (2048, 18432, 512, 200)])
def test_every_run_of_the_product_is_exact(M, N, K, runs):
    """Each slot of the ring is read before the next copy or the next scales take its
    place, and the accumulator before the next tile's (one scale: the sums are whole
    quarters below 2^24 of them, whatever their order)."""
    g = gen(M + N)
    a = torch.randint(0, 256, (N, K // 2), device=DEV, generator=g, dtype=torch.int32).to(U8)
    b = torch.randint(0, 256, (M, K // 2), device=DEV, generator=g, dtype=torch.int32).to(U8)
    sa, sb = torch.full((N, K // 32), 127, dtype=U8, device=DEV), torch.full((M, K // 32), 127, dtype=U8, device=DEV)
    # scales that change from block to block on both sides and cancel: a mixed-up one shows
    e = torch.arange(K // 32, device=DEV) % 5
    sa, sb = (sa + e.to(U8)).contiguous(), (sb - e.to(U8)).contiguous()
    av, bv = (sk.splitk_dequantize_mx4(q, s, out_dtype=F32) for q, s in ((a, sa), (b, sb)))
    ref = torch.matmul(bv.double(), av.double().T).float()
    c = torch.empty((M, N), device=DEV)
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(runs):
        c.fill_(0.5)
        sk.splitk_gemm_mx4(a, sa, b, sb, c=c)
        wrong += (c != ref).any()
    assert wrong.item() == 0
    assert sk.splitk_get_status() == 0


def guarded(shape, dtype, value, skew=0):
    """A contiguous output inside a buffer full of `value`, and what is around it."""
    n = math.prod(shape)
    room = torch.full((n + 128,), value, dtype=dtype, device=DEV)
    return room[64 + skew:64 + skew + n].view(shape), (room[:64 + skew], room[64 + skew + n:])


def untouched(guards, value):
    return all(bool((g == value).all()) for g in guards)


@pytest.mark.parametrize("M,D", [(1, 32), (3, 96), (5, 512), (130, 7168), (2, 16416), (3, 40000)])
def test_norm_and_codes_write_their_outputs_and_nothing_else(M, D):
    g = gen(M + D)
    x, r, w = randn((M, D), g), randn((M, D), g, F32), randn((D,), g, F32)
    (q, gq), (s, gs), (out, go) = guarded((M, D // 2), U8, 99), guarded((M, D // 32), U8, 7), guarded((M, D), F32, 7.0)
    sk.splitk_rmsnorm_mx4(x, w, r, codes=q, scale=s, residual_out=out)
    torch.cuda.synchronize()
    assert untouched(gq, 99) and untouched(gs, 7) and untouched(go, 7.0)
    ref = sk.splitk_rmsnorm_mx4(x, w, r)
    assert torch.equal(q, ref[0]) and torch.equal(s, ref[1]) and torch.equal(out, ref[2])
    sk.splitk_quantize_mx4(x, codes=q, scale=s)
    back, gb = guarded((M, D), BF16, 7.0)
    sk.splitk_dequantize_mx4(q, s, out=back)
    torch.cuda.synchronize()
    assert untouched(gq, 99) and untouched(gs, 7) and untouched(gb, 7.0)
    ref = sk.splitk_quantize_mx4(x)
    assert torch.equal(q, ref[0]) and torch.equal(s, ref[1]) and torch.equal(back, sk.splitk_dequantize_mx4(q, s))


@pytest.mark.parametrize("M,N,K", [(1, 100, 64), (7, 1000, 544), (30, 257, 1024), (64, 4100, 512), (100, 130, 4096), (129, 301, 256),
                                   (300, 2049, 480), (1000, 515, 256)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("skew", [0, 1])
def test_product_writes_its_output_and_nothing_else(M, N, K, dtype, skew):
    g = gen(M + N)
    a, sa = sk.splitk_quantize_mx4(randn((N, K), g))
    b, sb = sk.splitk_quantize_mx4(randn((M, K), g))
    c, gc = guarded((M, N), dtype, 7.0, skew)
    sk.splitk_gemm_mx4(a, sa, b, sb, c=c)
    torch.cuda.synchronize()
    assert untouched(gc, 7.0)
    assert torch.equal(c, sk.splitk_gemm_mx4(a, sa, b, sb, out_dtype=dtype))
    assert sk.splitk_get_status() == 0


@pytest.mark.parametrize("M,V", [(1, 5), (3, 1000), (7, 4099), (2, 131072), (300, 8001)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("skew", [0, 3])
def test_adjustment_writes_its_output_and_nothing_else(M, V, dtype, skew):
    g = gen(M + V)
    x = randn((M, V), g, dtype)
    how = dict(history=torch.randint(-2, V + 2, (M, 40), device=DEV, generator=g), frequency=torch.rand(M, device=DEV, generator=g),
               bias_ids=torch.randint(-2, V + 2, (M, 5), device=DEV, generator=g), bias_values=randn((M, 5), g, F32),
               allowed=torch.randint(-2**31, 2**31, (M, -(-V // 32)), device=DEV, generator=g).to(torch.int32))
    out, go = guarded((M, V), dtype, 7.0, skew)
    sk.splitk_adjust_logits(x, **how, out=out)
    torch.cuda.synchronize()
    assert untouched(go, 7.0)
    assert same(out, sk.splitk_adjust_logits(x, **how))


# ---------------------------------------------------------------- sizes of whole models
@pytest.mark.parametrize("N,K", [(32000, 2048), (50257, 1024), (131072, 1056)])
@pytest.mark.parametrize("M", [1, 12, 40, 130])
def test_product_of_a_vocabulary_head(M, N, K):
    g = gen(M + N)
    a, sa = sk.splitk_quantize_mx4(randn((N, K), g))
    b, sb = sk.splitk_quantize_mx4(randn((M, K), g))
    c = sk.splitk_gemm_mx4(a, sa, b, sb, out_dtype=F32)
    av, bv = (sk.splitk_dequantize_mx4(q, s, out_dtype=F32).double() for q, s in ((a, sa), (b, sb)))
    # exact products; at least 16 of them are added at a time, each time off by 2 u at most
    bound = 2 * 2.0 ** -24 * (K / 16 + 16) * (bv.abs() @ av.abs().T)
    assert ((c.double() - bv @ av.T).abs() <= bound).all()
    assert sk.splitk_get_status() == 0


@pytest.mark.parametrize("M,N,K", [(16, 20480, 4096), (40, 19600, 8192), (100, 20000, 4128), (300, 10300, 8192), (520, 7000, 4096),
                                   (1, 300, (1 << 20) + 32), (200, 500, 1 << 18)])
def test_product_of_a_round_of_tiles_and_a_few_and_of_long_rows(M, N, K):
    """A few tiles more than there are pairs of SMs run on several pairs each, after the
    others or alone; rows of many K tiles."""
    g = gen(M + K)
    a, sa = sk.splitk_quantize_mx4(randn((N, K), g))
    b, sb = sk.splitk_quantize_mx4(randn((M, K), g))
    bias = randn((N,), g)
    c = sk.splitk_gemm_mx4(a, sa, b, sb, bias=bias, out_dtype=F32)
    av, bv = (sk.splitk_dequantize_mx4(q, s, out_dtype=F32).double() for q, s in ((a, sa), (b, sb)))
    ref = bv @ av.T + bias.double()
    # exact products; at least 16 of them are added at a time, each time off by 2 u at most
    bound = 2 * 2.0 ** -24 * (K / 16 + 16) * (bv.abs() @ av.abs().T) + 2.0 ** -24 * ref.abs()
    assert ((c.double() - ref).abs() <= bound).all()
    assert sk.splitk_get_status() == 0


@pytest.mark.parametrize("M", [1, 4, 128])
def test_rows_before_a_wide_down_projection(M):
    """Widths of 53248: norm to codes, then the product with K as long."""
    D, N = 53248, 512
    g = gen(M)
    x, r, w = randn((M, D), g), randn((M, D), g), randn((D,), g, F32)
    codes, scale, out = sk.splitk_rmsnorm_mx4(x, w, r)
    y = x.float() + r.float()
    assert torch.equal(out, y.to(BF16))
    n = (y.double() / (y.double().square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double())
    values = sk.splitk_dequantize_mx4(codes, scale, out_dtype=F32).double()
    # half a step of 2 scales, a quarter of the block's largest magnitude at most (or cut
    # off: 6 of below 8 scales, a quarter again)
    top = n.unflatten(-1, (-1, 32)).abs().amax(-1).repeat_interleave(32, -1)
    assert ((values - n).abs() <= top / 4 * (1 + 1e-5)).all()
    a, sa = sk.splitk_quantize_mx4(randn((N, D), g))
    c = sk.splitk_gemm_mx4(a, sa, codes, scale, out_dtype=F32)
    av = sk.splitk_dequantize_mx4(a, sa, out_dtype=F32).double()
    bound = 2 * 2.0 ** -24 * (D / 16 + 16) * (values.abs() @ av.abs().T)
    assert ((c.double() - values @ av.T).abs() <= bound).all()
    assert sk.splitk_get_status() == 0


def test_product_offsets_past_32_bits():
    """More than 2^31 outputs, and more than 2^31 bytes of codes."""
    g = gen(60)
    K = 256
    a, sa = sk.splitk_quantize_mx4(randn((150_000, K), g))
    b, sb = sk.splitk_quantize_mx4(randn((15_000, K), g))
    c = sk.splitk_gemm_mx4(a, sa, b, sb)
    bv = sk.splitk_dequantize_mx4(b, sb, out_dtype=F32)
    for n in (0, 77_777, 149_999):
        av = sk.splitk_dequantize_mx4(a[n:n + 1].contiguous(), sa[n:n + 1].contiguous(), out_dtype=F32)
        ref = (bv.double() @ av.double().T)[:, 0]
        bound = 2 * 2.0 ** -24 * 32 * (bv.abs().double() @ av.abs().double().T)[:, 0] + ref.abs() * 2.0 ** -8
        assert ((c[:, n].double() - ref).abs() <= bound).all()
    del c
    wide, wide_s = a.repeat(120, 1), sa.repeat(120, 1)                 # 18 million rows are refused: in batches
    one = sk.splitk_gemm_mx4(a, sa, b[:3].contiguous(), sb[:3].contiguous())
    c = sk.splitk_gemm_mx4(wide.view(120, 150_000, -1), wide_s.view(120, 150_000, -1),
                           b[:3].repeat(120, 1, 1), sb[:3].repeat(120, 1, 1))
    assert torch.equal(c, one.expand(120, -1, -1))
    assert sk.splitk_get_status() == 0


# ---------------------------------------------------------------- the example
@pytest.mark.parametrize("tokens", [3, 70])
def test_the_example_runs(tokens):
    res = subprocess.run([sys.executable, str(ROOT / "examples" / "quantized_head.py"), "--format", "mx4", "--tokens", str(tokens),
                          "--width", "512", "--vocabulary", "1001", "--steps", "3"], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-2000:]
    assert f"3 steps of {tokens} tokens" in res.stdout
