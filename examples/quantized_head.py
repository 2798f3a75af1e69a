"""The end of a decode step with 8-bit weights and activations: the last
projection's output joins the residual stream and is normed to codes, the
vocabulary head multiplies them with its codes, and the logits become the next
token of each sequence, its log probability and its alternatives.

    python examples/quantized_head.py [--tokens 4] [--width 7168] [--vocabulary 32000] [--steps 20]

Random weights; the same step in bf16 (``splitk_gemm_bf16``) runs beside it for
comparison.
"""
from __future__ import annotations

import argparse
import sys
from pathlib import Path

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))

import torch  # noqa: E402

import split_bf16_gemm_swapped_gb300 as sk  # noqa: E402


class QuantizedHead:
    """The final norm and the vocabulary projection, weights held as 8-bit
    codes with a scale for each vocabulary entry."""

    def __init__(self, norm: torch.Tensor, head: torch.Tensor, eps: float = 1e-6):
        self.norm, self.eps = norm, eps
        self.codes, self.scales = sk.splitk_quantize_i8(head)       # a row is a channel: laid out once

    def logits(self, x: torch.Tensor, residual: torch.Tensor) -> torch.Tensor:
        """[M, V] f32 logits of the activations x; `residual` takes their sum."""
        q, scale, _ = sk.splitk_rmsnorm_i8(x, self.norm, residual, eps=self.eps, residual_out=residual)
        return sk.splitk_gemm_i8(self.codes, self.scales, q, scale, out_dtype=torch.float32)

    def step(self, x: torch.Tensor, residual: torch.Tensor, alternatives: int):
        """The most probable token of each row, its log probability, the
        distribution's entropy, and the alternatives with theirs."""
        logits = self.logits(x, residual)
        _, entropy, ids, logprobs = sk.splitk_logprobs(logits, top_k=alternatives)
        return ids[:, 0], logprobs[:, 0], entropy, ids, logprobs


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4)
    ap.add_argument("--width", type=int, default=7168)
    ap.add_argument("--vocabulary", type=int, default=32000)
    ap.add_argument("--alternatives", type=int, default=5)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()

    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(0)
    head = (0.05 * torch.randn(a.vocabulary, a.width, device=dev, generator=g)).bfloat16()
    norm = (1 + 0.1 * torch.randn(a.width, device=dev, generator=g)).bfloat16()
    x = torch.randn(a.tokens, a.width, device=dev, generator=g).bfloat16()
    residual = (4 * torch.randn(a.tokens, a.width, device=dev, generator=g)).bfloat16()

    # the same step with bf16 weights and activations
    y = x.float() + residual.float()
    n = (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * norm.float()).bfloat16()
    wide = sk.splitk_gemm_bf16(head, n)
    _, wide_entropy, wide_ids, wide_logprobs = sk.splitk_logprobs(wide, top_k=a.alternatives)

    quantized = QuantizedHead(norm, head)
    kept = residual.clone()
    token, logprob, entropy, ids, logprobs = quantized.step(x, kept, a.alternatives)
    # the bf16 step's first choice, as the quantized logits see it
    at, _, _, _ = sk.splitk_logprobs(quantized.logits(x, residual.clone()), wide_ids[:, 0].contiguous())
    for m in range(min(a.tokens, 4)):
        print(f"row {m}: token {token[m].item()} at {logprob[m].item():.3f} (entropy {entropy[m].item():.3f}), "
              f"alternatives {ids[m].tolist()}")
        print(f"        bf16: {wide_ids[m, 0].item()} at {wide_logprobs[m, 0].item():.3f} "
              f"(entropy {wide_entropy[m].item():.3f}), here at {at[m].item():.3f}")

    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        quantized.step(x, residual, a.alternatives)
    end.record()
    torch.cuda.synchronize()
    if sk.splitk_get_status() != 0:
        raise SystemExit(f"a kernel reported a timeout: {sk.splitk_get_fault()}")
    print(f"{a.steps} steps of {a.tokens} tokens: {start.elapsed_time(end) / a.steps * 1e3:.1f} us a step")


if __name__ == "__main__":
    main()
