"""dW of rows off 16 bytes whose last 64 columns hold a row's tail alone, which goes by the
element: the boxes that TMA stores read are not written over, however many tiles a warp
writes one after another."""

import pytest
import torch

from test_gpu_head import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(3, 300001, 65), (1, 200003, 71), (5, 100001, 130), (2, 20001, 1025), (4, 40001, 198)])
def test_boxes_in_turn(lib, M, N, K, dtype):
    """Two to fifteen tiles to a pair of CTAs; the same bits ten times."""
    data = make(M, N, K, dtype, M + N + K, left_out=0.0)
    first = run(dtype, data, M, N, K, want=("dW",))
    check(run(dtype, data, M, N, K), data, dtype)
    for _ in range(9):
        assert torch.equal(run(dtype, data, M, N, K, want=("dW",))["dW"], first["dW"])
