"""A process's first call of the library may be a captured one: the device's set-up
(its status word) is made meanwhile, and the replay gives what a later call gives.
In processes of their own, since that set-up is made once a process."""

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
M, N, K = int(sys.argv[2]), 136, 264
X, W, V = r(M, K), r(K, N), r(K, N)
C = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
Q = torch.zeros(g.gemm_fp4_code_bytes(M, K), dtype=torch.uint8, device="cuda")
S = torch.zeros(g.gemm_fp4_scale_bytes("mx", M, K), dtype=torch.uint8, device="cuda")
out, call = {
    "product": ([C], lambda: g.gemm_bf16_rm(X, W, C, M, N, K)),
    "gated": ([C], lambda: g.gemm_gated("bf16", "silu", X, W, V, C, None, None, M, N, K)),
    "quantize": ([Q, S], lambda: g.gemm_fp4_quantize("bf16", "mx", X, K, None, Q, S, M, K)),
}[which]
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


@pytest.mark.parametrize("which,M", [("product", 4), ("product", 300), ("gated", 4), ("gated", 300), ("quantize", 40)])
def test_first_call_is_captured(lib, which, M):
    r = subprocess.run([sys.executable, "-c", PROGRAM, which, str(M)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
