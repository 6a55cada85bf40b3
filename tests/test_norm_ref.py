"""The 64-bit norm against torch's autograd in 64 bits, and its gradients against differences."""

import numpy as np
import torch

import norm_ref as ref


def test_against_autograd_and_differences():
    rng = np.random.default_rng(0)
    M, K, eps = 4, 37, 1e-3
    H, dY, dH, w = rng.standard_normal((M, K)), rng.standard_normal((M, K)), rng.standard_normal((M, K)), rng.standard_normal(K)
    h, wt = torch.tensor(H, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * wt
    (y * torch.tensor(dY)).sum().backward()
    r, Y = ref.forward(H, w, eps)
    dX, dw = ref.backward(H, w, dY, dH, eps)
    assert np.allclose(Y, y.detach().numpy(), atol=1e-13)
    assert np.allclose(dX - dH, h.grad.numpy(), atol=1e-13) and np.allclose(dw, wt.grad.numpy(), atol=1e-13)
    f = lambda a: (ref.forward(a, w, eps)[1] * dY).sum()
    for i, k in ((0, 0), (3, 36), (1, 20)):
        e = np.zeros_like(H)
        e[i, k] = 1e-6
        assert abs((f(H + e) - f(H - e)) / 2e-6 - (dX - dH)[i, k]) < 1e-8
