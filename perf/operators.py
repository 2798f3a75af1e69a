"""The operators around the decode projection, as they are measured: residual
addition + RMS norm to 8-bit codes, quantisation to 8-bit codes, the matrix
product of 8-bit codes, and log probabilities of a vocabulary's logits.

`run` computes each in its plain form (elementary torch operations in 32 bits,
rounded once at the end), or, with `own`, through the package's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
DTYPES = {"bf16": BF16, "f16": F16, "f32": F32}
EPS = 1e-6
TINY = 2.0 ** -126          # the smallest scale of a row of codes


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token between two projections of the single-token decode
        {"name": "norm one token", "op": "norm", "M": 1, "D": 7168, "residual": "bf16", "weight": "bf16", "pad": 0},
        # a prefill chunk of the same model width
        {"name": "norm prefill", "op": "norm", "M": 2048, "D": 7168, "residual": "bf16", "weight": "bf16", "pad": 0},
        # an odd width with a 32-bit residual stream, rows cut out of a wider tensor
        {"name": "norm odd f32 stream", "op": "norm", "M": 333, "D": 4999, "residual": "f32", "weight": "f32", "pad": 9},
        # activations that follow no norm (before the down projection), a decode batch
        {"name": "quantise activations", "op": "quantise", "M": 128, "D": 16384, "pad": 0},
        # a projection's weights laid out in codes, a scale for each channel
        {"name": "quantise weights", "op": "quantise", "M": 18432, "D": 7168, "pad": 0},
        # the single-token decode projection
        {"name": "product one token", "op": "product", "L": 1, "M": 1, "N": 7168, "K": 2048, "bias": False, "out": "bf16"},
        # the small-batch decode projection
        {"name": "product small batch", "op": "product", "L": 1, "M": 16, "N": 4096, "K": 7168, "bias": True, "out": "bf16"},
        # the wide projection of a decode batch
        {"name": "product wide", "op": "product", "L": 1, "M": 64, "N": 18432, "K": 7168, "bias": False, "out": "bf16"},
        # a prefill chunk of odd length through a long-K projection
        {"name": "product prefill", "op": "product", "L": 1, "M": 1000, "N": 7168, "K": 16384, "bias": False, "out": "f32"},
        # the answer to one token: sampled id, entropy, 20 alternatives
        {"name": "logprobs one token", "op": "logprobs", "M": 1, "V": 131072, "k": 20, "type": "bf16", "masked": "none", "pad": 0},
        # a batch under a grammar: odd vocabulary, 32-bit logits in a padded buffer, most tokens masked
        {"name": "logprobs masked batch", "op": "logprobs", "M": 65, "V": 50001, "k": 5, "type": "f32", "masked": "most", "pad": 15},
        # a prompt's log probabilities
        {"name": "logprobs prompt", "op": "logprobs", "M": 1024, "V": 131072, "k": 20, "type": "bf16", "masked": "none", "pad": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quantise", "product", "product", "logprobs", "logprobs"])
    if op in ("norm", "quantise"):
        D = _log(rng, 64, 16384)
        D = D if rng.random() < 0.4 else -(-D // 16) * 16          # any width, or a whole number of 16s
        case = {"op": op, "M": _log(rng, 1, min(4096, 18432 * 7168 // D)), "D": D, "pad": rng.choice([0, 0, 16, 3])}
        if op == "norm":
            case.update(residual=rng.choice(["none", "bf16", "f32"]), weight=rng.choice(["bf16", "f32"]))
        return case
    if op == "product":
        K = 16 * _log(rng, 4, 1024)
        N = _log(rng, 64, 18432)
        L = rng.choice([1, 1, 1, 2])
        most = 1000 * 7168 * 16384 // (L * N * K)
        return {"op": op, "L": L, "M": _log(rng, 1, max(1, min(1000, most))), "N": N, "K": K,
                "bias": rng.random() < 0.3, "out": rng.choice(["bf16", "bf16", "f32"])}
    V = _log(rng, 1000, 200000)
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    return {"op": op, "M": _log(rng, 1, min(1024, 1024 * 131072 // V // (2 if kind == "f32" else 1))), "V": V,
            "k": rng.choice([0, 1, 5, 20, 32]), "type": kind, "masked": rng.choice(["none", "some", "most"]),
            "pad": rng.choice([0, 0, 8, 1])}


def work(case):
    if case["op"] == "norm":
        M, D = case["M"], case["D"]
        r = {"none": 0, "bf16": 2, "f32": 4}[case["residual"]]
        # x and the residual in; the residual, codes and scales out
        return {"bytes": M * D * (2 + 2 * r + 1) + 4 * M + D * (2 if case["weight"] == "bf16" else 4),
                "flops": 8 * M * D}
    if case["op"] == "quantise":
        M, D = case["M"], case["D"]
        return {"bytes": M * D * 3 + 4 * M, "flops": 4 * M * D}
    if case["op"] == "product":
        L, M, N, K = case["L"], case["M"], case["N"], case["K"]
        out = 2 if case["out"] == "bf16" else 4
        return {"bytes": L * (N * K + M * K + 4 * (N + M) + M * N * out + (2 * N if case["bias"] else 0)),
                "flops": 2 * L * M * N * K}
    M, V, k = case["M"], case["V"], case["k"]
    size = 4 if case["type"] == "f32" else 2
    return {"bytes": M * V * size + 8 * M + M * (8 + 12 * k), "flops": 6 * M * V}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(rows, width, pad, g):
    """[rows, width] bf16, one feature in a hundred 30 times as large as the
    others (the outlier channels of real activations), cut out of a buffer
    that is `pad` wider."""
    x = torch.randn(rows, width + pad, device="cuda", dtype=F32, generator=g)
    loud = torch.rand(width + pad, device="cuda", generator=g) < 0.01
    return torch.where(loud, x * 30, x).to(BF16)[:, :width]


def _codes(shape, g):
    """8-bit codes as rows scaled to their largest value hold them."""
    return (torch.randn(shape, device="cuda", dtype=F32, generator=g) * 32).round_().clamp_(-127, 127).to(torch.int8)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] in ("norm", "quantise"):
        M, D = case["M"], case["D"]
        s["x"] = _activations(M, D, case["pad"], g)
        s["values"] = torch.empty(M, D, device="cuda", dtype=BF16)
        if case["op"] == "norm":
            s["r"] = None
            if case["residual"] != "none":
                s["r"] = (4 * torch.randn(M, D, device="cuda", dtype=F32, generator=g)).to(DTYPES[case["residual"]])
            s["w"] = (1 + 0.1 * torch.randn(D, device="cuda", dtype=F32, generator=g)).to(DTYPES[case["weight"]])
    elif case["op"] == "product":
        L, M, N, K = case["L"], case["M"], case["N"], case["K"]
        s["a"] = _codes((L, N, K), g)
        s["b"] = _codes((L, M, K), g)
        s["a_scale"] = 0.0002 + 0.0004 * torch.rand(L, N, device="cuda", generator=g)
        s["b_scale"] = 0.01 + 0.05 * torch.rand(L, M, device="cuda", generator=g)
        s["bias_values"] = torch.randn(L, N, device="cuda", dtype=F32, generator=g).to(BF16) if case["bias"] else None
    else:
        M, V = case["M"], case["V"]
        x = 2.5 * torch.randn(M, V + case["pad"], device="cuda", dtype=F32, generator=g)
        hot = torch.randint(0, V, (M, 8), device="cuda", generator=g)
        x.scatter_add_(1, hot, 10 * torch.rand(M, 8, device="cuda", generator=g))       # a few likely tokens
        if case["masked"] != "none":
            # "some": a tenth of the tokens banned; "most": a handful allowed, and every seventh row allows none
            allowed = torch.rand(M, V + case["pad"], device="cuda", generator=g)
            allowed = allowed < (0.9 if case["masked"] == "some" else 20.0 / V)
            if case["masked"] == "most":
                allowed[3::7] = False
            x.masked_fill_(~allowed, float("-inf"))
        s["x"] = x.to(DTYPES[case["type"]])[:, :V]
        s["t"] = torch.where(torch.rand(M, device="cuda", generator=g) < 0.8, hot[:, 0],
                             torch.randint(0, V, (M,), device="cuda", generator=g))
    return s


# ---------------------------------------------------------------- plain forms
def _row_codes(n):
    scale = (n.abs().amax(dim=1) / 127).clamp_min(TINY)
    return torch.round(n / scale[:, None]), scale


def _plain_norm(s):
    y = s["x"].float()
    if s["r"] is not None:
        y = y + s["r"].float()
    n = y * torch.rsqrt(y.square().mean(dim=1, keepdim=True) + EPS) * s["w"].float()
    q, scale = _row_codes(n)
    return {"values": (q * scale[:, None]).to(BF16), "scale": scale,
            "residual": None if s["r"] is None else y.to(s["r"].dtype)}


def _plain_quantise(s):
    q, scale = _row_codes(s["x"].float())
    return {"values": (q * scale[:, None]).to(BF16), "scale": scale}


def _plain_product(s):
    c = torch.matmul(s["b"].float(), s["a"].float().transpose(1, 2))
    c = c * s["b_scale"][:, :, None] * s["a_scale"][:, None, :]
    if s["bias_values"] is not None:
        c = c + s["bias_values"].float()[:, None, :]
    return c.to(DTYPES[s["out"]])


def _plain_logprobs(s):
    x, t, V, k = s["x"].float(), s["t"], s["V"], s["k"]
    top = x.amax(dim=1, keepdim=True)
    d = x - torch.where(top == float("-inf"), 0.0, top)            # an empty row stays at -inf
    e = torch.exp(d)
    total = e.sum(dim=1)
    norm = torch.log(torch.where(total == 0, 1.0, total))          # an empty row: 0
    mean = torch.where(e == 0, 0.0, e * d).sum(dim=1) / torch.where(total == 0, 1.0, total)
    out = {"logprob": d.gather(1, t[:, None])[:, 0] - norm, "entropy": norm - mean}
    if k:
        # one whole number for value and place, so that equal values go by the lowest index
        bits = (x + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() << 32
        key = key | torch.arange(V - 1, -1, -1, device=x.device)
        ids = V - 1 - (torch.topk(key, k, dim=1).values & 0xFFFFFFFF)
        out["top_ids"] = ids
        out["top_logprobs"] = d.gather(1, ids) - norm[:, None]
    return out


def run(state):
    s = state
    if not own:
        plain = {"norm": _plain_norm, "quantise": _plain_quantise, "product": _plain_product,
                 "logprobs": _plain_logprobs}
        return plain[s["op"]](s)
    import split_bf16_gemm_swapped_gb300 as sk
    if s["op"] == "norm":
        q, scale, residual = sk.splitk_rmsnorm_i8(s["x"], s["w"], s["r"], eps=EPS)
        torch.mul(q, scale[:, None], out=s["values"])              # the codes as the values they stand for
        return {"values": s["values"], "scale": scale, "residual": residual}
    if s["op"] == "quantise":
        q, scale = sk.splitk_quantize_i8(s["x"])
        torch.mul(q, scale[:, None], out=s["values"])
        return {"values": s["values"], "scale": scale}
    if s["op"] == "product":
        return sk.splitk_gemm_i8(s["a"], s["a_scale"], s["b"], s["b_scale"], bias=s["bias_values"],
                                 out_dtype=DTYPES[s["out"]])
    logprob, entropy, ids, tops = sk.splitk_logprobs(s["x"], s["t"], top_k=s["k"])
    out = {"logprob": logprob, "entropy": entropy}
    if s["k"]:
        out["top_ids"], out["top_logprobs"] = ids, tops
    return out


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "quantise"):
        v = s["x"].double()
        if case["op"] == "norm":
            v = v if s["r"] is None else v + s["r"].double()
            residual = None if s["r"] is None else v
            v = v / (v.pow(2).sum(1, keepdim=True) / case["D"] + EPS).sqrt() * s["w"].double()
        scale = torch.maximum(v.abs().max(1).values / 127, torch.tensor(TINY, dtype=torch.float64, device="cuda"))
        out = {"values": torch.round(v / scale[:, None]) * scale[:, None], "scale": scale}
        if case["op"] == "norm":
            out["residual"] = residual
        return out
    if case["op"] == "product":
        a, b = s["a"].double() * s["a_scale"].double()[..., None], s["b"].double() * s["b_scale"].double()[..., None]
        c = torch.einsum("lmk,lnk->lmn", b, a)
        return c if s["bias_values"] is None else c + s["bias_values"].double()[:, None]
    rows = [[], [], [], []]
    for at in range(0, case["M"], 128):                            # some rows at a time: 64 bits of a prompt's logits
        x, t = s["x"][at:at + 128].double(), s["t"][at:at + 128]
        empty = torch.isneginf(x).all(1)
        lse = torch.where(empty, 0.0, torch.logsumexp(x, 1))
        lp = x - lse[:, None]
        rows[0].append(lp[torch.arange(len(t), device="cuda"), t])
        rows[1].append(-torch.special.xlogy(lp.exp(), lp.exp()).sum(1))
        if case["k"]:
            _, order = torch.sort(x, dim=1, descending=True, stable=True)
            ids = order[:, :case["k"]]
            rows[2].append(ids)
            rows[3].append(torch.gather(lp, 1, ids))
    rows = [torch.cat(r) if r else None for r in rows]
    out = {"logprob": rows[0], "entropy": rows[1]}
    if case["k"]:
        out.update(top_ids=rows[2], top_logprobs=rows[3])
    return out
