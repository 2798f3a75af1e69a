"""The operators of a decode step in 4 bits, as they are measured: quantisation to
microscaled 4-bit floats (E2M1 codes, an E8M0 scale for 32 of them) and back,
residual addition + RMS norm to such codes, the matrix product of two operands
held so, and the adjustment of a vocabulary's logits (penalties for repeated
tokens, biases, grammar masks) before log probabilities are taken.

`run` computes each in its plain form (elementary torch operations in 32 bits,
rounded once at the end), or, with `own`, through the package's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
DTYPES = {"bf16": BF16, "f16": F16, "f32": F32}
EPS = 1e-6
BLOCK = 32                  # codes that share a scale


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # activations that follow no norm (before the down projection), a decode batch
        {"name": "quantise activations", "op": "quantise", "M": 128, "D": 16384, "type": "bf16", "pad": 0},
        # a projection's weights laid out in codes
        {"name": "quantise weights", "op": "quantise", "M": 18432, "D": 7168, "type": "bf16", "pad": 0},
        # one token between two projections of the single-token decode
        {"name": "norm one token", "op": "norm", "M": 1, "D": 7168, "residual": "bf16", "weight": "bf16", "pad": 0},
        # a prefill chunk of the same model width, a 32-bit residual stream
        {"name": "norm prefill", "op": "norm", "M": 2048, "D": 7168, "residual": "f32", "weight": "bf16", "pad": 0},
        # the single-token decode projection
        {"name": "product one token", "op": "product", "L": 1, "M": 1, "N": 7168, "K": 2048, "bias": False, "out": "bf16"},
        # the small-batch decode projection
        {"name": "product small batch", "op": "product", "L": 1, "M": 16, "N": 4096, "K": 7168, "bias": True, "out": "bf16"},
        # the wide projection of a decode batch
        {"name": "product wide", "op": "product", "L": 1, "M": 64, "N": 18432, "K": 7168, "bias": False, "out": "bf16"},
        # a prefill chunk of odd length through a long-K projection
        {"name": "product odd chunk", "op": "product", "L": 1, "M": 1000, "N": 7168, "K": 16384, "bias": False, "out": "f32"},
        # a prefill chunk through the wide projection
        {"name": "product prefill", "op": "product", "L": 1, "M": 2048, "N": 18432, "K": 7168, "bias": False, "out": "bf16"},
        # one conversation: its history, some biased tokens
        {"name": "adjust one row", "op": "adjust", "M": 1, "V": 131072, "H": 1500, "B": 20, "type": "bf16",
         "masked": "none", "pad": 0},
        # a batch under a grammar: odd vocabulary, 32-bit logits in a padded buffer, most tokens masked
        {"name": "adjust grammar batch", "op": "adjust", "M": 65, "V": 50001, "H": 300, "B": 0, "type": "f32",
         "masked": "most", "pad": 15},
        # a large batch of long conversations, biases and some banned tokens
        {"name": "adjust large batch", "op": "adjust", "M": 256, "V": 131072, "H": 4096, "B": 64, "type": "bf16",
         "masked": "some", "pad": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantise", "norm", "product", "product", "adjust", "adjust"])
    if op in ("quantise", "norm"):
        D = BLOCK * _log(rng, 2, 512)
        case = {"op": op, "M": _log(rng, 1, min(4096, 18432 * 7168 // D)), "D": D, "pad": rng.choice([0, 0, 16, 3])}
        if op == "norm":
            case.update(residual=rng.choice(["none", "bf16", "f32"]), weight=rng.choice(["bf16", "f32"]))
        else:
            case.update(type=rng.choice(["bf16", "bf16", "f16", "f32"]))
        return case
    if op == "product":
        K = BLOCK * _log(rng, 2, 512)
        N = _log(rng, 64, 18432)
        L = rng.choice([1, 1, 1, 2])
        most = 2048 * 18432 * 7168 // (L * N * K)
        return {"op": op, "L": L, "M": _log(rng, 1, max(1, min(2048, most))), "N": N, "K": K,
                "bias": rng.random() < 0.3, "out": rng.choice(["bf16", "bf16", "f32"])}
    V = _log(rng, 1000, 200000)
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    return {"op": op, "M": _log(rng, 1, min(256, 256 * 131072 // V // (2 if kind == "f32" else 1))), "V": V,
            "H": rng.choice([0, _log(rng, 1, 4096), _log(rng, 1, 4096)]), "B": rng.choice([0, 0, _log(rng, 1, 300)]),
            "type": kind, "masked": rng.choice(["none", "some", "most"]), "pad": rng.choice([0, 0, 8, 1])}


def work(case):
    size = {"none": 0, "bf16": 2, "f16": 2, "f32": 4}
    if case["op"] in ("quantise", "norm"):
        M, D = case["M"], case["D"]
        held = M * D // 2 + M * D // BLOCK
        if case["op"] == "quantise":
            return {"bytes": M * D * size[case["type"]] + held, "flops": 4 * M * D}
        # x and the residual in; the residual, codes and scales out
        return {"bytes": M * D * (2 + 2 * size[case["residual"]]) + held + D * size[case["weight"]], "flops": 8 * M * D}
    if case["op"] == "product":
        L, M, N, K = case["L"], case["M"], case["N"], case["K"]
        return {"bytes": L * ((N + M) * (K // 2 + K // BLOCK) + M * N * size[case["out"]] + (2 * N if case["bias"] else 0)),
                "flops": 2 * L * M * N * K}
    M, V = case["M"], case["V"]
    mask = 0 if case["masked"] == "none" else 4 * -(-V // 32)
    return {"bytes": M * (2 * V * size[case["type"]] + 8 * case["H"] + 12 * case["B"] + mask + 28), "flops": 6 * M * V}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(rows, width, pad, g):
    """[rows, width] f32, one feature in a hundred 30 times as large as the
    others (the outlier channels of real activations), cut out of a buffer
    that is `pad` wider."""
    x = torch.randn(rows, width + pad, device="cuda", dtype=F32, generator=g)
    loud = torch.rand(width + pad, device="cuda", generator=g) < 0.01
    return torch.where(loud, x * 30, x)


def _packed(x):
    """Rows in codes, low nibble first, and the codes of their scales."""
    q, scale = _row_codes(x)
    a = q.abs()
    # 0, 0.5, 1, 1.5, 2, 3, 4, 6 are the codes 0..7
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, 2 + a, 4 + a / 2)).to(torch.uint8)
    code = torch.where(q < 0, code + 8, code)
    return code[..., 0::2] | (code[..., 1::2] << 4), (scale.view(torch.int32) >> 23).to(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] in ("quantise", "norm"):
        M, D = case["M"], case["D"]
        kind = DTYPES[case["type"]] if case["op"] == "quantise" else BF16
        s["x"] = _activations(M, D, case["pad"], g).to(kind)[:, :D]
        if case["op"] == "norm":
            s["r"] = None
            if case["residual"] != "none":
                s["r"] = (4 * torch.randn(M, D, device="cuda", dtype=F32, generator=g)).to(DTYPES[case["residual"]])
            s["w"] = (1 + 0.1 * torch.randn(D, device="cuda", dtype=F32, generator=g)).to(DTYPES[case["weight"]])
    elif case["op"] == "product":
        L, M, N, K = case["L"], case["M"], case["N"], case["K"]
        s["a"], s["a_scale"] = _packed(0.02 * torch.randn(L, N, K, device="cuda", dtype=F32, generator=g))
        s["b"], s["b_scale"] = _packed(_activations(L * M, K, 0, g).view(L, M, K))
        s["bias_values"] = torch.randn(L, N, device="cuda", dtype=F32, generator=g).to(BF16) if case["bias"] else None
    else:
        M, V, H, B = case["M"], case["V"], case["H"], case["B"]
        x = 2.5 * torch.randn(M, V + case["pad"], device="cuda", dtype=F32, generator=g)
        s["x"] = x.to(DTYPES[case["type"]])[:, :V]
        rand = lambda *shape: torch.rand(*shape, device="cuda", generator=g)            # noqa: E731
        s["history"] = None
        if H:
            # a few tokens are most of a text: those near the start of the vocabulary
            s["history"] = (V * rand(M, H) ** 4).long().clamp_(0, V - 1)
            s["lengths"] = (H * (0.5 + 0.5 * rand(M))).long()
            s["lengths"][2::5] = 0                                                      # some have said nothing yet
            s["prompts"] = (s["lengths"] * rand(M)).long()
            s["repetition"] = 1 + 0.3 * rand(M)
            s["presence"] = rand(M)
            s["frequency"] = 0.5 * rand(M)
        s["bias_ids"] = None
        if B:
            s["bias_ids"] = torch.randint(0, V, (M, B), device="cuda", generator=g)
            s["bias_ids"][:, B // 2 + 1:][rand(M, B - B // 2 - 1) < 0.3] = -1           # lists of unequal length
            s["bias_values"] = 5 * torch.randn(M, B, device="cuda", dtype=F32, generator=g)
        s["allowed"] = None
        if case["masked"] != "none":
            # "some": a tenth of the tokens banned; "most": a handful allowed, and every seventh row allows none
            words = -(-V // 32)
            allowed = rand(M, 32 * words) < (0.9 if case["masked"] == "some" else 20.0 / V)
            if case["masked"] == "most":
                allowed[3::7] = False
            bits = torch.arange(32, device="cuda")
            packed = torch.empty(M, words, dtype=torch.int32, device="cuda")
            for m in range(M):
                packed[m] = (allowed[m].view(words, 32).long() << bits).sum(1).to(torch.int32)
            s["allowed"] = packed
    return s


# ---------------------------------------------------------------- plain forms
def _row_codes(n):
    """The values of f32 rows' codes, a multiple of their block's scale each, and
    the scales: 2^(floor(log2(max)) - 2), from 2^-126 on."""
    blocks = n.unflatten(-1, (-1, BLOCK))
    top = blocks.abs().amax(-1)
    exponent = torch.where(top == 0, -126, torch.frexp(top).exponent - 3).clamp_min(-126)
    scale = ((exponent + 127) << 23).view(F32)
    q = blocks / scale[..., None]
    a = q.abs().clamp_max(6)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign(torch.round(a / step) * step, q)
    return q.flatten(-2), scale


def _values(q, scale):
    return (q.unflatten(-1, (-1, BLOCK)) * scale[..., None]).flatten(-2)


_TABLE = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _unpacked(codes, scale, dtype=F32):
    table = torch.tensor(_TABLE, device=codes.device, dtype=dtype)
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    power = (scale.int() << 23).view(F32) if dtype == F32 else ((scale.long() + 896) << 52).view(F64)
    return _values(table[q.int()], power)


def _plain_quantise(s):
    q, scale = _row_codes(s["x"].float())
    return {"values": _values(q, scale).to(BF16), "scale": scale.to(BF16)}


def _plain_norm(s):
    y = s["x"].float()
    if s["r"] is not None:
        y = y + s["r"].float()
    # the mean in 64 bits: a value beside the border of two codes goes by its last bits
    mean = y.double().square().mean(dim=1, keepdim=True).float()
    q, scale = _row_codes(y * s["w"].float() * (1 / torch.sqrt(mean + EPS)))
    return {"values": _values(q, scale).to(BF16), "scale": scale.to(BF16),
            "residual": None if s["r"] is None else y.to(s["r"].dtype)}


def _plain_product(s):
    a, b = _unpacked(s["a"], s["a_scale"]), _unpacked(s["b"], s["b_scale"])
    c = torch.matmul(b, a.transpose(1, 2))
    if s["bias_values"] is not None:
        c = c + s["bias_values"].float()[:, None, :]
    return c.to(DTYPES[s["out"]])


def _plain_adjust(s):
    x, M, V = s["x"].float(), s["M"], s["V"]
    if s["history"] is not None:
        at = torch.arange(s["H"], device=x.device)
        said = torch.zeros(M, V, device=x.device).scatter_add_(1, s["history"], (at < s["lengths"][:, None]).float()) > 0
        new = (at < s["lengths"][:, None]) & (at >= s["prompts"][:, None])
        count = torch.zeros(M, V, device=x.device).scatter_add_(1, s["history"], new.float())
        r = s["repetition"][:, None]
        x = torch.where(said, torch.where(x > 0, x / r, x * r), x)
        x = x - s["frequency"][:, None] * count
        x = x - s["presence"][:, None] * (count > 0)
    if s["bias_ids"] is not None:
        kept = s["bias_ids"] >= 0
        bias = torch.zeros(M, V, device=x.device, dtype=F64)
        bias.scatter_add_(1, s["bias_ids"].clamp_min(0), torch.where(kept, s["bias_values"], 0.0).double())
        x = x + bias.float()
    if s["allowed"] is not None:
        bits = s["allowed"][:, :, None] >> torch.arange(32, device=x.device, dtype=torch.int32) & 1
        x = x.masked_fill(bits.flatten(1)[:, :V] == 0, float("-inf"))
    return x.to(s["x"].dtype)


def run(state):
    s = state
    if not own:
        plain = {"quantise": _plain_quantise, "norm": _plain_norm, "product": _plain_product, "adjust": _plain_adjust}
        return plain[s["op"]](s)
    import split_bf16_gemm_swapped_gb300 as sk
    if s["op"] in ("quantise", "norm"):
        out = {}
        if s["op"] == "quantise":
            codes, scale = sk.splitk_quantize_mx4(s["x"])
        else:
            codes, scale, out["residual"] = sk.splitk_rmsnorm_mx4(s["x"], s["w"], s["r"], eps=EPS)
        # codes and scales as the values they stand for, which bf16 holds
        out["values"] = sk.splitk_dequantize_mx4(codes, scale)
        out["scale"] = (scale.to(torch.int16) << 7).view(BF16)
        return out
    if s["op"] == "product":
        return sk.splitk_gemm_mx4(s["a"], s["a_scale"], s["b"], s["b_scale"], bias=s["bias_values"],
                                  out_dtype=DTYPES[s["out"]])
    args = {}
    if s["history"] is not None:
        args.update(history=s["history"], lengths=s["lengths"], prompt_lengths=s["prompts"], repetition=s["repetition"],
                    presence=s["presence"], frequency=s["frequency"])
    if s["bias_ids"] is not None:
        args.update(bias_ids=s["bias_ids"], bias_values=s["bias_values"])
    return sk.splitk_adjust_logits(s["x"], allowed=s["allowed"], **args)


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("quantise", "norm"):
        out = {"values": [], "scale": []}
        if case["op"] == "norm":
            out["residual"] = None if s["r"] is None else s["x"].double() + s["r"].double()
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64, device="cuda")
        for at in range(0, case["M"], 1024):                        # some rows at a time
            v = s["x"][at:at + 1024].double()
            if case["op"] == "norm":
                v = v if s["r"] is None else v + s["r"][at:at + 1024].double()
                v = v / (v.pow(2).sum(1, keepdim=True) / case["D"] + EPS).sqrt() * s["w"].double()
            b = v.reshape(len(v), -1, BLOCK)
            top = b.abs().max(2).values.clamp_min(2.0 ** -124)
            floor = torch.floor(torch.log2(top))
            power = ((floor.long() + 1023) << 52).view(F64)
            # (a power of two's logarithm may be a bit off)
            scale = torch.where(power > top, power / 2, torch.where(2 * power <= top, 2 * power, power)) / 4
            q = (b / scale[..., None]).abs()
            # between two neighbours of the grid: the nearer one, the middle to the even code
            hi = torch.searchsorted(grid, q.contiguous()).clamp_max(7)
            lo = (hi - 1).clamp_min(0)
            down, up = q - grid[lo], grid[hi] - q
            pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
            out["values"].append((torch.sign(b) * grid[pick] * scale[..., None]).flatten(1))
            out["scale"].append(scale)
        out["values"], out["scale"] = torch.cat(out["values"]), torch.cat(out["scale"])
        return out
    if case["op"] == "product":
        a, b = (_unpacked(s[n], s[n + "_scale"], F64) for n in ("a", "b"))
        c = torch.einsum("lmk,lnk->lmn", b, a)
        return c if s["bias_values"] is None else c + s["bias_values"].double()[:, None]
    rows = []
    for m in range(case["M"]):
        x = s["x"][m].double()
        if s["history"] is not None:
            n, p = int(s["lengths"][m]), int(s["prompts"][m])
            said = torch.bincount(s["history"][m, :n], minlength=case["V"]) > 0
            count = torch.bincount(s["history"][m, p:n], minlength=case["V"])
            r, f, q = (s[k][m].double() for k in ("repetition", "frequency", "presence"))
            x = torch.where(said & (x > 0), x / r, torch.where(said, x * r, x)) - f * count - torch.where(count > 0, q, 0.0)
        if s["bias_ids"] is not None:
            kept = s["bias_ids"][m] >= 0
            x = x.index_add(0, s["bias_ids"][m][kept], s["bias_values"][m][kept].double())
        if s["allowed"] is not None:
            v = torch.arange(case["V"], device="cuda")
            x = torch.where((s["allowed"][m].long()[v // 32] >> (v % 32)) % 2 == 1, x, -math.inf)
        rows.append(x)
    return torch.stack(rows)
