"""Training steps of a small language model's trunk and head, and its next tokens in FP8.

    python examples/lm_train_step.py [--tokens M] [--width K] [--hidden N] [--layers L] [--vocab V] [--steps S]

Each block adds gated_ffn(norm(h)) to the residual stream h; the head's cross entropy
runs over the whole vocabulary without logits in memory.  Every product, norm, loss and
gradient is the library's; the blocks' matrices are updated with their orthogonalised
momentum, the head and the gains with plain SGD, on FP32 masters.  Serving: the last norm
writes E4M3 rows with their scales, the operand of the FP8 product with the head.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_matrix_multiply_gb300 as gemm  # noqa: E402

EPS = 1e-6


def product(a: torch.Tensor, op_a: str, b: torch.Tensor, op_b: str) -> torch.Tensor:
    """op(a) op(b) of contiguous bf16 matrices."""
    M, K = a.shape if op_a == "N" else a.shape[::-1]
    N = b.shape[1] if op_b == "N" else b.shape[0]
    c = torch.empty(M, N, dtype=a.dtype, device=a.device)
    gemm.gemm_ex("bf16", "rm", op_a, op_b, M, N, K, 1.0, a, a.shape[1], 0, b, b.shape[1], 0, 0.0, c, N, 0)
    return c


class Norm:
    def __init__(self, gain: torch.Tensor):
        self.gain = gain

    def forward(self, x, residual):
        """h = x + residual (x alone without one), norm(h), and what the gradients need."""
        M, K = x.shape
        h = torch.empty_like(x) if residual is not None else None
        y, rstd = torch.empty_like(x), torch.empty(M, device=x.device)
        gemm.gemm_rms_norm("bf16", x, residual, self.gain, EPS, h, y, rstd, M, K)
        return y, (x if h is None else h, rstd)

    def backward(self, saved, dy, dh):
        """The gradient of h (dh: from its other use, updated in place) and of the gains."""
        h, rstd = saved
        M, K = h.shape
        dx = torch.empty_like(h) if dh is None else dh
        dgain = torch.empty(K, device=h.device)
        gemm.gemm_rms_norm_backward("bf16", h, self.gain, rstd, dy, dh, dx, dgain, M, K)
        return dx, dgain


class Model:
    """bf16 weights: blocks of (gain, Wg, Wu [K,N], Wd [N,K]), a last gain, the head [V,K]."""

    def __init__(self, width: int, hidden: int, layers: int, vocab: int, gen: torch.Generator):
        def w(rows, cols, std):
            return torch.randn(rows, cols, device="cuda", generator=gen) * std
        ones = lambda: torch.ones(width, device="cuda")
        self.K, self.N, self.V, self.layers = width, hidden, vocab, layers
        self.embedding = w(vocab, width, 1.0).bfloat16()
        self.master = []
        for _ in range(layers):
            self.master += [ones(), w(width, hidden, width ** -0.5), w(width, hidden, width ** -0.5), w(hidden, width, hidden ** -0.5)]
        self.master += [ones(), w(vocab, width, width ** -0.5)]
        self.momentum = [torch.zeros_like(m) for m in self.master]
        self.sync()

    def sync(self) -> None:
        self.weights = [m.bfloat16() for m in self.master]

    def forward(self, ids: torch.Tensor, targets: torch.Tensor):
        """Each token's loss, and what the gradients need."""
        x, h, saved, M = self.embedding[ids], None, [], len(ids)
        for i in range(self.layers):
            gain, Wg, Wu, Wd = self.weights[4 * i:4 * i + 4]
            y, norm = Norm(gain).forward(x, h)
            z = torch.empty(M, self.N, dtype=x.dtype, device=x.device)
            G, U = (torch.empty(M, self.N, device=x.device) for _ in range(2))
            gemm.gemm_gated("bf16", "silu", y, Wg, Wu, z, G, U, M, self.N, self.K)
            saved.append((norm, y, z, G, U))
            x, h = product(z, "N", Wd, "N"), norm[0]
        y, norm = Norm(self.weights[-2]).forward(x, h)
        loss, lse = torch.empty(M, device=x.device), torch.empty(M, device=x.device)
        gemm.gemm_cross_entropy("bf16", y, self.weights[-1], targets, loss, lse, M, self.V, self.K)
        return loss, (saved, norm, y, lse, targets)

    def backward(self, saved, dloss: torch.Tensor):
        """Gradients of the weights, in their order, and of the embedded tokens."""
        blocks, norm, y, lse, targets = saved
        M, grads = len(targets), []
        dy, dhead = torch.empty_like(y), torch.empty_like(self.weights[-1])
        gemm.gemm_cross_entropy_backward("bf16", y, self.weights[-1], targets, lse, dloss, dy, dhead, M, self.V, self.K)
        dh, dgain = Norm(self.weights[-2]).backward(norm, dy, None)
        grads = [dgain, dhead]
        for i in reversed(range(self.layers)):
            gain, Wg, Wu, Wd = self.weights[4 * i:4 * i + 4]
            norm, y, z, G, U = blocks[i]
            dWd, dz = product(z, "T", dh, "N"), product(dh, "N", Wd, "T")
            dy, dWg, dWu = torch.empty_like(y), torch.empty_like(Wg), torch.empty_like(Wu)
            gemm.gemm_gated_backward("bf16", "silu", y, Wg, Wu, G, U, dz, dy, dWg, dWu, M, self.N, self.K)
            dh, dgain = Norm(gain).backward(norm, dy, dh)
            grads = [dgain, dWg, dWu, dWd] + grads
        return grads, dh

    def step(self, grads, rate: float, decay: float = 0.95) -> None:
        """The blocks' matrices by their orthogonalised momentum, the rest by their gradients."""
        for i, (master, momentum, grad) in enumerate(zip(self.master, self.momentum, grads)):
            if i < 4 * self.layers and i % 4:
                momentum.mul_(decay).add_(grad.float())
                update = momentum.bfloat16()
                M, N = update.shape
                gemm.gemm_orthogonalize("bf16", update, N, update, N, 5, M, N)  # in place
                master.sub_(update.float(), alpha=rate * max(1.0, M / N) ** 0.5)
            else:
                master.sub_(grad.float(), alpha=rate)
        self.sync()

    def next_logits_fp8(self, ids: torch.Tensor) -> torch.Tensor:
        """Half logits of the tokens' successors: the head in E4M3, the last norm's rows too."""
        x, h, M = self.embedding[ids], None, len(ids)
        for i in range(self.layers):
            gain, Wg, Wu, Wd = self.weights[4 * i:4 * i + 4]
            y, (h, _) = Norm(gain).forward(x, h)
            z = torch.empty(M, self.N, dtype=x.dtype, device=x.device)
            gemm.gemm_gated("bf16", "silu", y, Wg, Wu, z, None, None, M, self.N, self.K)
            x = product(z, "N", Wd, "N")
        head, scale = self.weights[-1], self.weights[-1].abs().max().float() / 448
        head8 = (head.float() / scale).to(torch.float8_e4m3fn)
        Q, s = torch.empty(M, self.K, dtype=torch.float8_e4m3fn, device=x.device), torch.empty(M, device=x.device)
        gemm.gemm_rms_norm_e4m3("bf16", x, h, self.weights[-2], EPS, None, Q, s, M, self.K)
        logits = torch.empty(M, self.V, dtype=torch.float16, device=x.device)
        gemm.gemm_e4m3_rowscale(Q, s * scale, head8, logits, M, self.V, self.K)
        return logits


def run(tokens: int, width: int, hidden: int, layers: int, vocab: int, steps: int, seed: int = 0) -> dict:
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    model = Model(width, hidden, layers, vocab, gen)
    follows = torch.randperm(vocab, device="cuda", generator=gen)  # the token after each
    losses = []
    for _ in range(steps):
        ids = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
        targets = torch.where(torch.rand(tokens, device="cuda", generator=gen) < 0.1, -100, follows[ids])  # some rows are padding
        loss, saved = model.forward(ids, targets)
        count = (targets >= 0).sum()
        grads, _ = model.backward(saved, torch.full_like(loss, 1.0) / count)
        model.step(grads, rate=0.02)
        losses.append(loss.sum() / count)
    ids = torch.randint(0, vocab, (16,), device="cuda", generator=gen)
    logits = model.next_logits_fp8(ids)
    gemm.gemm_synchronize()
    return {"losses": [float(v) for v in losses], "logits": logits, "right": int((logits.argmax(1) == follows[ids]).sum())}


def main() -> None:
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--width", type=int, default=1024)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--vocab", type=int, default=32000)
    p.add_argument("--steps", type=int, default=50)
    a = p.parse_args()
    r = run(a.tokens, a.width, a.hidden, a.layers, a.vocab, a.steps)
    print("loss %.3f -> %.3f over %d steps" % (r["losses"][0], r["losses"][-1], a.steps))
    print("next tokens in FP8: %d of 16 right" % r["right"])


if __name__ == "__main__":
    main()
