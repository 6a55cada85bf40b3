"""A gated feed-forward block trained in bf16, then quantised to 4 bits and served.

    python examples/ffn_train_then_4bit.py [--tokens M] [--width K] [--hidden N] [--steps S] [--format nv|mx]

Training: y = (silu(x Wg) * (x Wu)) Wd against a fixed random block, with the
library's forward and backward products and plain SGD on FP32 master weights.
Serving: the three weights are quantised once (each [out, in], as a linear
layer stores them), and a prompt and single tokens run through gemm_fp4_linear,
which quantises the activations on the way.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_matrix_multiply_gb300 as gemm  # noqa: E402


class GatedFFN:
    """bf16 weights Wg, Wu [K,N] and Wd [N,K] with FP32 masters."""

    def __init__(self, K: int, N: int, gen: torch.Generator):
        def w(rows, cols):
            return torch.randn(rows, cols, device="cuda", generator=gen) * rows ** -0.5
        self.K, self.N = K, N
        self.master = [w(K, N), w(K, N), w(N, K)]
        self.weights = [m.bfloat16() for m in self.master]

    def forward(self, x: torch.Tensor, save: bool):
        M, (Wg, Wu, Wd) = x.shape[0], self.weights
        z = torch.empty(M, self.N, dtype=torch.bfloat16, device="cuda")
        y = torch.empty(M, self.K, dtype=torch.bfloat16, device="cuda")
        G, U = (torch.empty(M, self.N, device="cuda") for _ in range(2)) if save else (None, None)
        gemm.gemm_gated("bf16", "silu", x, Wg, Wu, z, G, U, M, self.N, self.K)
        gemm.gemm_bf16_rm(z, Wd, y, M, self.K, self.N)
        return y, (x, z, G, U)

    def backward(self, dy: torch.Tensor, saved):
        x, z, G, U = saved
        M, K, N = x.shape[0], self.K, self.N
        Wg, Wu, Wd = self.weights
        dWd, dz = torch.empty_like(Wd), torch.empty_like(z)
        gemm.gemm_ex("bf16", "rm", "T", "N", N, K, M, 1.0, z, N, 0, dy, K, 0, 0.0, dWd, K, 0)   # z^T dy
        gemm.gemm_ex("bf16", "rm", "N", "T", M, N, K, 1.0, dy, K, 0, Wd, K, 0, 0.0, dz, N, 0)   # dy Wd^T
        dx, dWg, dWu = torch.empty_like(x), torch.empty_like(Wg), torch.empty_like(Wu)
        gemm.gemm_gated_backward("bf16", "silu", x, Wg, Wu, G, U, dz, dx, dWg, dWu, M, N, K)
        return dx, (dWg, dWu, dWd)

    def step(self, grads, rate: float) -> None:
        for master, weight, grad in zip(self.master, self.weights, grads):
            master.sub_(grad.float(), alpha=rate)
            weight.copy_(master)


def tensor_scale(t: torch.Tensor, fmt: str):
    """nv: the largest magnitude maps to 448 * 6; mx has no such scale."""
    return (t.abs().max().float() / 2688).reshape(1) if fmt == "nv" else None


class Linear4:
    """A weight [out, in] in 4 bits, and the product with it."""

    def __init__(self, weight: torch.Tensor, fmt: str):
        self.fmt, (self.out, self.inner) = fmt, weight.shape
        self.scale = tensor_scale(weight, fmt)
        self.Q = torch.empty(gemm.gemm_fp4_code_bytes(self.out, self.inner), dtype=torch.uint8, device="cuda")
        self.S = torch.empty(gemm.gemm_fp4_scale_bytes(fmt, self.out, self.inner), dtype=torch.uint8, device="cuda")
        gemm.gemm_fp4_quantize("bf16", fmt, weight, self.inner, self.scale, self.Q, self.S, self.out, self.inner)

    def dequantized(self) -> torch.Tensor:
        w = torch.empty(self.out, self.inner, dtype=torch.bfloat16, device="cuda")
        gemm.gemm_fp4_dequantize("bf16", self.fmt, self.Q, self.S, self.scale, w, self.inner, self.out, self.inner)
        return w

    def __call__(self, x: torch.Tensor, x_scale) -> torch.Tensor:
        M = x.shape[0]
        y = torch.empty(M, self.out, dtype=torch.bfloat16, device="cuda")
        gemm.gemm_fp4_linear("bf16", self.fmt, x, self.inner, x_scale, self.Q, self.S, self.scale, y, self.out, M,
                             self.out, self.inner)
        return y


class GatedFFN4:
    """The trained block in 4 bits, activation scales taken from a calibration batch."""

    def __init__(self, block: GatedFFN, fmt: str, x: torch.Tensor):
        self.fmt = fmt
        self.gate, self.up, self.down = (Linear4(w.t().contiguous(), fmt) for w in block.weights)
        _, (_, z, _, _) = block.forward(x, save=False)
        self.x_scale, self.z_scale = tensor_scale(x, fmt), tensor_scale(z, fmt)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        z = torch.nn.functional.silu(self.gate(x, self.x_scale)) * self.up(x, self.x_scale)
        return self.down(z, self.z_scale)


def run(tokens: int, width: int, hidden: int, steps: int, fmt: str, seed: int = 0) -> dict:
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    teacher, block = GatedFFN(width, hidden, gen), GatedFFN(width, hidden, gen)
    x = torch.randn(tokens, width, device="cuda", generator=gen).bfloat16()
    target, _ = teacher.forward(x, save=False)
    losses = []
    for _ in range(steps):
        y, saved = block.forward(x, save=True)
        diff = y.float() - target.float()
        losses.append(diff.square().mean())
        _, grads = block.backward((diff * (2.0 / tokens)).bfloat16(), saved)
        block.step(grads, rate=0.2)
    want, _ = block.forward(x, save=False)
    served = GatedFFN4(block, fmt, x)
    got = served(x)
    one = torch.cat([served(x[i:i + 1]) for i in range(min(4, tokens))])
    gemm.gemm_synchronize()
    rel = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())
    return {"losses": [float(v) for v in losses], "error_4bit": rel(got, want),
            "weight_error_4bit": rel(served.down.dequantized(), block.weights[2].t()),
            "token_vs_prompt": rel(one, got[:one.shape[0]])}


def main() -> None:
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--hidden", type=int, default=12288)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--format", choices=("nv", "mx"), default="nv")
    a = p.parse_args()
    r = run(a.tokens, a.width, a.hidden, a.steps, a.format)
    print("loss %.4f -> %.4f over %d steps" % (r["losses"][0], r["losses"][-1], a.steps))
    print("4-bit (%s) output against bf16: %.3f relative; its down weight: %.3f" % (a.format, r["error_4bit"], r["weight_error_4bit"]))
    print("single tokens against the prompt: %.4f" % r["token_vs_prompt"])


if __name__ == "__main__":
    main()
