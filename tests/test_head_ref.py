"""The 64-bit cross entropy against torch's in 64 bits (rows left out among them), and its
gradients against differences."""

import numpy as np
import torch

import head_ref as ref


def test_against_autograd_and_differences():
    rng = np.random.default_rng(0)
    M, N, K = 6, 11, 5
    X, W, d = rng.standard_normal((M, K)), rng.standard_normal((N, K)), rng.standard_normal(M)
    t = np.array([0, 10, 3, -100, 5, 11])
    x, w = torch.tensor(X, requires_grad=True), torch.tensor(W, requires_grad=True)
    tt = torch.tensor(np.where(ref.counts(t, N), t, -100))
    loss = torch.nn.functional.cross_entropy(x @ w.T, tt, ignore_index=-100, reduction="none")
    (loss * torch.tensor(d)).sum().backward()
    got, lse, Z = ref.forward(X, W, t)
    assert np.allclose(got, loss.detach().numpy(), atol=1e-13) and np.allclose(lse, torch.logsumexp(x @ w.T, 1).detach().numpy())
    dX, dW, _ = ref.backward(X, W, t, d)
    assert np.allclose(dX, x.grad.numpy(), atol=1e-13) and np.allclose(dW, w.grad.numpy(), atol=1e-13)
    f = lambda a, b: (ref.forward(a, b, t)[0] * d).sum()
    for i, k in ((0, 0), (5, 1), (3, 2), (4, 4)):
        e = np.zeros_like(X)
        e[i, k] = 1e-6
        assert abs((f(X + e, W) - f(X - e, W)) / 2e-6 - dX[i, k]) < 1e-8
        e = np.zeros_like(W)
        e[2 * i, k] = 1e-6
        assert abs((f(X, W + e) - f(X, W - e)) / 2e-6 - dW[2 * i, k]) < 1e-8
