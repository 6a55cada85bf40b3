"""The 4-bit and gated entry points captured into a CUDA graph: a replay gives what
the calls gave, bit for bit, on new inputs too."""

import pytest
import torch

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    return lib


def captured(call, refill):
    """Outputs of eager calls and of replays of one capture, for two sets of inputs."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()                      # set-up outside the capture
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
        for seed in (1, 2):
            refill(seed)
            want = [t.clone() for t in call()]
            for t in call.outputs:
                t.zero_()
            graph.replay()
            got = [t.clone() for t in call.outputs]
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            assert all(b.float().abs().max() > 0 for b in want)
    g.gemm_set_stream(None)


class Call:
    def __init__(self, run, outputs):
        self.run, self.outputs = run, outputs

    def __call__(self):
        self.run()
        return self.outputs


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_linear(M, fmt):
    N, K = 392, 1040
    x, w = torch.empty(M, K, dtype=BF16, device="cuda"), torch.randn(N, K, dtype=BF16, device="cuda")
    gs = torch.tensor([0.002], device="cuda") if fmt == "nv" else None
    Q = torch.empty(g.gemm_fp4_code_bytes(N, K), dtype=torch.uint8, device="cuda")
    S = torch.empty(g.gemm_fp4_scale_bytes(fmt, N, K), dtype=torch.uint8, device="cuda")
    g.gemm_fp4_quantize("bf16", fmt, w, K, gs, Q, S, N, K)
    torch.cuda.synchronize()
    C = torch.empty(M, N, dtype=BF16, device="cuda")

    def refill(seed):
        x.copy_(torch.randn(M, K, generator=torch.Generator().manual_seed(seed)))

    refill(0)
    captured(Call(lambda: g.gemm_fp4_linear("bf16", fmt, x, K, gs, Q, S, gs, C, N, M, N, K), [C]), refill)


@pytest.mark.parametrize("M", [3, 300])
def test_gated_step(M):
    N, K = 520, 1600   # M = 300: the forward's last wave and dX are split along K
    r = lambda *s: torch.randn(*s, device="cuda").to(BF16)
    X, Wg, Wu, dZ = r(M, K), r(K, N), r(K, N), r(M, N)
    Z, dX, dWg, dWu = (torch.empty_like(t) for t in (dZ, X, Wg, Wu))
    G, U = (torch.empty(M, N, device="cuda") for _ in range(2))

    def run():
        g.gemm_gated("bf16", "gelu", X, Wg, Wu, Z, G, U, M, N, K)
        g.gemm_gated_backward("bf16", "gelu", X, Wg, Wu, G, U, dZ, dX, dWg, dWu, M, N, K)

    captured(Call(run, [Z, G, U, dX, dWg, dWu]),
             lambda seed: X.copy_(torch.randn(M, K, generator=torch.Generator().manual_seed(seed))))
