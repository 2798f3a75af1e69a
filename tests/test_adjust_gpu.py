"""splitk_adjust_logits on the GPU against the elementary 32-bit operations of its
formula, to the bit, with each row's tokens counted on the host."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import split_bf16_gemm_swapped_gb300 as sk  # noqa: E402

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def sync():
    torch.cuda.synchronize()
    assert sk.splitk_get_status() == 0, sk.splitk_get_fault()


def bits(allowed):
    """[M, V] truth values as words of 32."""
    M, V = allowed.shape
    words = -(-V // 32)
    padded = torch.zeros(M, 32 * words, dtype=torch.long, device=DEV)
    padded[:, :V] = allowed
    return (padded.view(M, words, 32) << torch.arange(32, device=DEV)).sum(-1).to(torch.int32)


def reference(x, history=None, lengths=None, prompt_lengths=None, repetition=None, presence=None, frequency=None,
              bias_ids=None, bias_values=None, allowed=None, **_):
    M, V = x.shape
    y = x.float().clone()
    for m in range(M):
        row = y[m]
        if history is not None:
            H = history.shape[1]
            n = H if lengths is None else max(0, min(int(lengths[m]), H))
            p = 0 if prompt_lengths is None else int(prompt_lengths[m])
            tokens = history[m, :n]
            inside = (tokens >= 0) & (tokens < V)
            said = torch.zeros(V, dtype=torch.bool, device=DEV)
            said[tokens[inside]] = True
            new = tokens[inside & (torch.arange(n, device=DEV) >= p)]
            count = torch.bincount(new, minlength=V).float()
            if repetition is not None:
                row = torch.where(said, torch.where(row > 0, row / repetition[m], row * repetition[m]), row)
            if frequency is not None:
                row = torch.where(count > 0, row - frequency[m] * count, row)
            if presence is not None:
                row = torch.where(count > 0, row - presence[m], row)
        if bias_ids is not None:
            sums = {}
            for i, v in zip(bias_ids[m].tolist(), bias_values[m]):
                if 0 <= i < V:
                    sums[i] = v if i not in sums else sums[i] + v      # in 32 bits, in order
            for i, v in sums.items():
                row = row.clone()
                row[i] = row[i] + v
        if allowed is not None:
            ok = (allowed[m].long()[torch.arange(V, device=DEV) // 32] >> (torch.arange(V, device=DEV) % 32)) & 1
            row = row.masked_fill(ok == 0, float("-inf"))
        y[m] = row
    return y.to(x.dtype)


def same(a, b):
    """Equal, NaN for NaN (and 0 for -0)."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(nan=0.0), b.nan_to_num(nan=0.0))


def logits(M, V, g, dtype, pad=0, offset=0):
    return (2.5 * torch.randn(M, offset + V + pad, device=DEV, generator=g)).to(dtype)[:, offset:offset + V]


def parts(M, V, g, H=0, B=0, allow=None):
    """A row's history has few tokens often, some that no vocabulary has, and any length."""
    how = {}
    rand = lambda *s: torch.rand(*s, device=DEV, generator=g)          # noqa: E731
    if H:
        how["history"] = (V * rand(M, H) ** 3).long().clamp_(0, V - 1)
        how["history"][rand(M, H) < 0.05] = -1
        how["history"][rand(M, H) < 0.05] = V + 3
        how["lengths"] = (rand(M) * (H + 1)).long()
        how["prompt_lengths"] = (how["lengths"] * rand(M)).long()
        how["repetition"], how["presence"], how["frequency"] = 1 + 0.3 * rand(M), rand(M), 0.5 * rand(M)
    if B:
        how["bias_ids"] = torch.randint(-1, V, (M, B), device=DEV, generator=g)
        how["bias_values"] = 5 * torch.randn(M, B, device=DEV, generator=g)
    if allow is not None:
        how["allowed"] = bits(rand(M, V) < allow)
    return how


def check(x, **how):
    keep = x.clone()
    want = reference(x, **how)
    out = sk.splitk_adjust_logits(x, **how)
    sync()
    assert out.dtype == x.dtype and out.shape == x.shape
    assert same(out, want)
    if how.get("out") is None:
        assert same(x, keep)
    return out


VOCABS = [1, 5, 8, 31, 32, 33, 255, 256, 1000, 2047, 2048, 2049, 4096, 4104, 9001, 32000, 50257]


@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_vocabularies(V, dtype):
    g = gen(V)
    check(logits(3, V, g, dtype), **parts(3, V, g, H=70, B=9, allow=0.7))


@pytest.mark.parametrize("M", [1, 2, 37, 300])
@pytest.mark.parametrize("H,B,allow", [(0, 0, None), (40, 0, None), (0, 12, None), (0, 0, 0.5), (33, 5, 0.001)])
def test_parts(M, H, B, allow):
    g = gen(M + H)
    check(logits(M, 3000, g, BF16), **parts(M, 3000, g, H, B, allow))


@pytest.mark.parametrize("leave", ["lengths", "prompt_lengths", "repetition", "presence", "frequency"])
def test_each_part_may_be_left_out(leave):
    g = gen(7)
    how = parts(5, 999, g, H=200)
    del how[leave]
    check(logits(5, 999, g, F32), **how)


@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 4), (7, 9), (8, 8)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("V", [1000, 2049])
def test_rows_of_a_padded_buffer(offset, pad, dtype, V):
    g = gen(offset + pad)
    how = parts(4, V, g, H=100, B=3, allow=0.8)
    x = logits(4, V, g, dtype, pad, offset)
    want = check(x, **how)
    # into rows of such a buffer, whose other elements stay as they are
    buffer = torch.full((4, offset + V + pad), 3.0, device=DEV, dtype=dtype)
    out = buffer[:, offset:offset + V]
    assert sk.splitk_adjust_logits(x, out=out, **how) is out
    sync()
    assert same(out, want) and (buffer[:, :offset] == 3).all() and (buffer[:, offset + V:] == 3).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("V,pad", [(4096, 0), (5001, 7)])
def test_in_place(dtype, V, pad):
    g = gen(V)
    x, how = logits(6, V, g, dtype, pad), parts(6, V, g, H=300, B=20, allow=0.9)
    want = reference(x, **how)
    assert sk.splitk_adjust_logits(x, out=x, **how) is x
    sync()
    assert same(x, want)


def test_batched_rows():
    g = gen(3)
    x, how = logits(12, 500, g, BF16), parts(12, 500, g, H=30, B=4, allow=0.5)
    want = reference(x, **how)
    out = sk.splitk_adjust_logits(x.view(3, 4, 500), **{k: v.view(3, 4, *v.shape[1:]) for k, v in how.items()})
    sync()
    assert out.shape == (3, 4, 500) and same(out.view(12, 500), want)


def test_rows_that_allow_nothing_and_lengths_at_their_ends():
    g = gen(4)
    how = parts(6, 700, g, H=50, B=2, allow=0.5)
    how["allowed"][2] = 0
    how["allowed"][3] = -1
    how["lengths"] = torch.tensor([0, 1, 50, 51, -3, 49], device=DEV)
    how["prompt_lengths"] = torch.tensor([0, 1, 50, 0, 5, 60], device=DEV)
    out = check(logits(6, 700, g, F32), **how)
    assert torch.isneginf(out[2]).all() and torch.isfinite(out[3]).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_masked_infinite_and_nan_logits(dtype):
    """Logits that are -inf, of the type's lowest value, +inf or NaN, counted or
    not, allowed or not."""
    g = gen(5)
    x = logits(4, 300, g, dtype)
    x[:, 0:40] = float("-inf")
    x[:, 40:80] = torch.finfo(dtype).min
    x[:, 80:90] = float("nan")
    x[:, 90:100] = float("inf")
    x[:, 100:110] = 0.0
    x[:, 110:120] = -0.0
    how = parts(4, 300, g, H=400, B=60, allow=0.8)
    how["bias_values"][:, 5] = float("-inf")
    check(x, **how)


def test_a_token_biased_twice_has_the_sum_in_order():
    """Sums whose order shows: 1e8 + 3 - 1e8 is 0 or 3 in 32 bits."""
    x = torch.zeros(2, 100, device=DEV)
    ids = torch.tensor([[7, 9, 7, 7, -1, 100, 9], [7, 7, 7, 9, 9, 200, -5]], device=DEV)
    v = torch.tensor([[1e8, 2.0, 3.0, -1e8, 5.0, 6.0, 0.5], [1e8, -1e8, 3.0, 0.25, 0.5, 1.0, 1.0]], device=DEV)
    out = check(x, bias_ids=ids, bias_values=v)
    assert out[0, 7] == 0 and out[1, 7] == 3 and out[0, 9] == 2.5 and out[1, 9] == 0.75


@pytest.mark.parametrize("H", [1, 2, 255, 256, 257, 5000, 40000])
def test_history_lengths(H):
    g = gen(H)
    check(logits(3, 20000, g, BF16), **parts(3, 20000, g, H))


def test_a_token_said_often():
    """One token fills a long history: its count is exact, with and without a prompt."""
    H = 100_000
    x = torch.ones(2, 64, device=DEV)
    history = torch.full((2, H), 5, device=DEV)
    prompt = torch.tensor([0, H - 1], device=DEV)
    check(x, history=history, prompt_lengths=prompt, frequency=torch.ones(2, device=DEV), presence=torch.ones(2, device=DEV),
          repetition=torch.full((2,), 2.0, device=DEV))


@pytest.mark.parametrize("B", [1, 2, 255, 256, 257, 1024])
def test_bias_counts(B):
    g = gen(B)
    check(logits(3, 500, g, F32), **parts(3, 500, g, B=B))


def repeated(how, M, V, B, g):
    """bias_ids of one token, of tokens that are there twice (beside each other and half
    the list apart), of some and a padding of zeros, and of different ones."""
    rows = {"one": torch.full((B,), min(5, V - 1)), "twice": torch.arange(B) // 2, "apart": torch.arange(B) % (B // 2),
            "padded": torch.cat([torch.arange(1, 21), torch.zeros(B - 20, dtype=torch.long)]), "different": torch.arange(B)}
    return (rows[how] % V).to(DEV).expand(M, B).contiguous()


@pytest.mark.parametrize("how", ["one", "twice", "apart", "padded"])
@pytest.mark.parametrize("dtype,M,V", [(F32, 2, 700), (BF16, 3, 9001), (F16, 2, 40000)])
@pytest.mark.parametrize("B", [300, 1023, 1024])
def test_biases_of_the_same_tokens(how, dtype, M, V, B):
    """The sum in the list's order, whatever of it one token takes."""
    g = gen(B)
    values = torch.randn(M, B, device=DEV, generator=g) * torch.where(torch.rand(M, B, device=DEV, generator=g) < 0.2, 1e4, 1.0)
    check(logits(M, V, g, dtype), bias_ids=repeated(how, M, V, B, g), bias_values=values, **parts(M, V, g, H=40, allow=0.9))


@pytest.mark.parametrize("how", ["one", "twice", "apart", "padded"])
@pytest.mark.parametrize("M,V", [(1, 131072), (64, 32000)])
def test_biases_of_the_same_tokens_take_no_longer(how, M, V):
    """A list is gone over once for each of its tokens, by as many threads: 1024 steps, a
    few microseconds, beside a list of different tokens (a pass for each entry of one
    token took a thousand times as long)."""
    g, B = gen(1), 1024
    x, v = logits(M, V, g, BF16), torch.randn(M, B, device=DEV, generator=g)
    out = torch.empty_like(x)

    def time(ids):
        best = float("inf")
        for _ in range(5):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(4):
                sk.splitk_adjust_logits(x, bias_ids=ids, bias_values=v, out=out)
            end.record()
            torch.cuda.synchronize()
            best = min(best, start.elapsed_time(end) / 4)
        return best

    other, same_tokens = time(repeated("different", M, V, B, g)), time(repeated(how, M, V, B, g))
    assert same_tokens <= 10 * other + 0.02, (same_tokens, other)


def test_more_biases_than_it_takes_are_refused():
    with pytest.raises(sk.SplitKError, match="INVALID_ARGUMENT"):
        sk.splitk_adjust_logits(torch.zeros(1, 50, device=DEV), bias_ids=torch.zeros(1, 1025, dtype=torch.long, device=DEV),
                                bias_values=torch.zeros(1, 1025, device=DEV))


def test_an_empty_history_and_no_biases():
    x = logits(3, 100, gen(1), BF16)
    out = sk.splitk_adjust_logits(x, history=torch.zeros(3, 0, dtype=torch.long, device=DEV),
                                  lengths=torch.zeros(3, dtype=torch.long, device=DEV), presence=torch.ones(3, device=DEV),
                                  bias_ids=torch.zeros(3, 0, dtype=torch.long, device=DEV),
                                  bias_values=torch.zeros(3, 0, device=DEV))
    sync()
    assert torch.equal(out, x)


@pytest.mark.parametrize("M,V", [(1, 131072), (65, 50001), (200, 131072), (3, 200000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_workload_sizes(M, V, dtype):
    g = gen(M + V)
    x, how = logits(M, V, g, dtype), parts(M, V, g, H=600, B=8, allow=0.9)
    few = torch.unique(torch.cat([torch.randint(0, M, (6,), device=DEV, generator=g), torch.tensor([0, M - 1], device=DEV)]))
    out = sk.splitk_adjust_logits(x, **how)
    sync()
    assert same(out[few], reference(x[few], **{k: v[few] for k, v in how.items()}))
    # the others by a check that needs no loop: what is banned, and what nothing touches
    allowed = (how["allowed"].long()[:, :, None] >> torch.arange(32, device=DEV) & 1).flatten(1)[:, :V] > 0
    assert torch.isneginf(out[~allowed]).all()
    inside = how["history"].clamp(0, V - 1)
    touched = torch.zeros(M, V, dtype=torch.bool, device=DEV).scatter_(1, inside, True)
    touched.scatter_(1, how["bias_ids"].clamp_min(0), True)
    free = allowed & ~touched
    assert torch.equal(out[free], x[free])


@pytest.mark.parametrize("V", [50003, 50048])
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("H", [0, 300, 600])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_large_batches(dtype, H, pad, V):
    """Batches of more than 2048 vectors an SM, which the longest spans take: every type,
    short and long histories, and logits whose rows lie otherwise between 16-byte
    boundaries than the outputs'."""
    each = 16 // dtype.itemsize
    M = 2048 * torch.cuda.get_device_properties(0).multi_processor_count // (V // each) + 2
    g = gen(V + H + pad)
    x, how = logits(M, V, g, dtype, pad), parts(M, V, g, H=H, B=8, allow=0.9)
    few = torch.tensor([0, 1, M // 2, M - 2, M - 1], device=DEV)
    out = sk.splitk_adjust_logits(x, **how)
    sync()
    assert same(out[few], reference(x[few], **{k: v[few] for k, v in how.items()}))
    allowed = (how["allowed"].long()[:, :, None] >> torch.arange(32, device=DEV) & 1).flatten(1)[:, :V] > 0
    assert torch.isneginf(out[~allowed]).all()
    touched = torch.zeros(M, V, dtype=torch.bool, device=DEV).scatter_(1, how["bias_ids"].clamp_min(0), True)
    if H:
        touched.scatter_(1, how["history"].clamp(0, V - 1), True)
    free = allowed & ~touched
    assert torch.equal(out[free], x[free])


def test_past_32_bit_offsets():
    """Logits of more than 2^31 elements: the last rows as the first."""
    M, V = 17000, 131072
    x = torch.zeros(M, V, dtype=BF16, device=DEV)
    g = gen(8)
    rows = [0, 1, M - 2, M - 1]
    for m in rows:
        x[m] = torch.randn(V, device=DEV, generator=g).to(BF16)
    history = torch.randint(0, V, (M, 16), device=DEV, generator=g)
    how = dict(history=history, repetition=torch.full((M,), 1.5, device=DEV), presence=torch.full((M,), 0.5, device=DEV))
    sk.splitk_adjust_logits(x, out=x, **how)
    sync()
    g = gen(8)
    for m in rows:
        y = torch.randn(1, V, device=DEV, generator=g).to(BF16)
        assert same(x[m:m + 1], reference(y, **{k: v[m:m + 1] for k, v in how.items()}))
