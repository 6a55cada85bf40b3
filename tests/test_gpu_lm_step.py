"""The norm, the gated block, the head's loss and the orthogonalised update together, as
examples/lm_train_step.py runs them: gradients against torch's in 64 bits, a captured step,
and the whole example."""

import importlib.util
import os

import pytest
import torch

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(lib):
    spec = importlib.util.spec_from_file_location("lm_train_step", os.path.join(ROOT, "examples", "lm_train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(model, ids, targets, dloss):
    """Loss and gradients by torch's autograd, everything in 64 bits."""
    w = [x.double().requires_grad_() for x in model.weights]
    norm = lambda h, gain: h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * gain
    x = h = model.embedding[ids].double().requires_grad_()
    for i in range(model.layers):
        gain, Wg, Wu, Wd = w[4 * i:4 * i + 4]
        y = norm(h, gain)
        h = h + (torch.nn.functional.silu(y @ Wg) * (y @ Wu)) @ Wd
    z = norm(h, w[-2]) @ w[-1].T
    loss = torch.nn.functional.cross_entropy(z, targets, ignore_index=-100, reduction="none")
    (loss * dloss.double()).sum().backward()
    return loss.detach(), [v.grad for v in w], x.grad


@pytest.mark.parametrize("tokens,width,hidden,layers,vocab", [(70, 64, 136, 2, 300), (300, 264, 512, 2, 1001), (1, 128, 256, 1, 500)])
def test_gradients(example, tokens, width, hidden, layers, vocab):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    model = example.Model(width, hidden, layers, vocab, gen)
    for m in model.master[:4 * layers:4] + [model.master[-2]]:
        m.mul_(1 + 0.2 * torch.randn(m.shape, device="cuda", generator=gen))
    model.sync()
    ids = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
    targets = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
    targets[1::5] = -100
    dloss = torch.rand(tokens, device="cuda", generator=gen) / tokens
    loss, saved = model.forward(ids, targets)
    grads, dx = model.backward(saved, dloss)
    g.gemm_synchronize()
    want_loss, want, want_x = reference(model, ids, targets, dloss)
    # Up to 5 roundings to bf16 a block and way (h, y, z, the block's output; dz, dG, dU, dy,
    # dh), and the head's: at most 24 on a path, each of deviation 2^-8 / sqrt 3 of what it
    # rounds, independent: sqrt(24) 2^-8 / sqrt 3 = 0.011 of the 2-norm, and room of three
    # for what a norm or a gate makes of them.
    tol = 3 * 24 ** 0.5 * 2.0 ** -8 / 3 ** 0.5
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert rel(loss, want_loss) < tol
    for i, (a, b) in enumerate(zip(grads + [dx], want + [want_x])):
        assert rel(a, b) < tol, (i, rel(a, b))


def test_captured_step(example):
    """Forward and backward of the model in one graph: the eager call's bits, on new tokens."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    model = example.Model(128, 264, 2, 700, gen)
    batches = [torch.randint(0, 700, (150,), device="cuda", generator=gen) for _ in range(4)]
    dloss = torch.full((150,), 1 / 150, device="cuda")
    want = []
    for ids, t in (batches[:2], batches[2:]):
        loss, saved = model.forward(ids, t)
        grads, dx = model.backward(saved, dloss)
        want.append([x.clone() for x in [loss, dx, *grads]])
    ids, t = batches[0].clone(), batches[1].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        model.forward(ids, t)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            loss, saved = model.forward(ids, t)
            grads, dx = model.backward(saved, dloss)
        for k in (1, 0, 1):
            ids.copy_(batches[2 * k])
            t.copy_(batches[2 * k + 1])
            graph.replay()
            for a, b in zip([loss, dx, *grads], want[k]):
                assert torch.equal(a, b)
    torch.cuda.synchronize()


def test_example_runs(example):
    r = example.run(tokens=300, width=128, hidden=264, layers=2, vocab=512, steps=4)
    assert all(v == v and v < 20 for v in r["losses"]) and torch.isfinite(r["logits"]).all()
