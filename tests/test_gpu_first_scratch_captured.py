"""A process's first call that takes scratch may be a captured one: its replay gives
what a later call gives.  In processes of their own, since the library's scratch pool
is made once a process."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import sys
import torch
import dense_matrix_multiply_gb300 as g
which = sys.argv[1]
r = lambda *s: torch.randn(*s, device="cuda").bfloat16()
M, N, K = 40, 136, 520
if which == "linear":
    x, w = r(M, K), r(N, K)
    Q = torch.empty(g.gemm_fp4_code_bytes(N, K), dtype=torch.uint8, device="cuda")
    S = torch.empty(g.gemm_fp4_scale_bytes("mx", N, K), dtype=torch.uint8, device="cuda")
    g.gemm_fp4_quantize("bf16", "mx", w, K, None, Q, S, N, K)
    out = [torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")]
    call = lambda: g.gemm_fp4_linear("bf16", "mx", x, K, None, Q, S, None, out[0], N, M, N, K)
else:
    X, Wg, Wu, dZ = r(M, K), r(K, N), r(K, N), r(M, N)
    Z, (G, U) = torch.empty_like(dZ), (torch.empty(M, N, device="cuda") for _ in range(2))
    g.gemm_gated("bf16", "silu", X, Wg, Wu, Z, G, U, M, N, K)      # takes no scratch
    out = [torch.zeros_like(t) for t in (X, Wg, Wu)]
    call = lambda: g.gemm_gated_backward("bf16", "silu", X, Wg, Wu, G, U, dZ, *out, M, N, K)
torch.cuda.synchronize()
s = torch.cuda.Stream()
with torch.cuda.stream(s):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    graph.replay()
    s.synchronize()
    got = [t.clone() for t in out]
    for t in out:
        t.zero_()
    call()
    s.synchronize()
assert all(torch.equal(a, b) and b.float().abs().max() > 0 for a, b in zip(got, out))
g.gemm_synchronize()
print("ok")
"""


@pytest.mark.parametrize("which", ["linear", "backward"])
def test_first_call_with_scratch_is_captured(lib, which):
    r = subprocess.run([sys.executable, "-c", PROGRAM, which], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
