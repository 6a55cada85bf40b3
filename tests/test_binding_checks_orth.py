"""Refusals of gemm_orthogonalize, on the host (no GPU)."""

import pytest
import torch

import dense_matrix_multiply_gb300 as g

A = 1 << 20  # an address that is checked and never read


@pytest.fixture(scope="module", autouse=True)
def built(lib):
    return lib.load()


def refused(*args, match, error=ValueError):
    before = g.gemm_kernel_launches()
    with pytest.raises(error, match=match):
        g.gemm_orthogonalize(*args)
    assert g.gemm_kernel_launches() == before


def test_tensors():
    h = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    refused("bf16", h(3, 8), 8, h(3, 8), 8, 5, 3, 8, match="CUDA device")
    refused("f32", h(3, 8), 8, h(3, 8), 8, 5, 3, 8, match="dtype")
    refused("bf16", h(23), 8, h(3, 8), 8, 5, 3, 8, match="G holds 23")
    refused("bf16", h(3, 8), 8, h(23), 8, 5, 3, 8, match="O holds 23")
    refused("bf16", torch.zeros(3, 8), 8, h(3, 8), 8, 5, 3, 8, match="2-byte elements")
    refused("bf16", h(8, 3).t(), 8, h(3, 8), 8, 5, 3, 8, match="G must have rows")
    refused("bf16", h(3, 8), 8, h(3, 16)[:, ::2], 8, 5, 3, 8, match="O must have rows")
    refused("bf16", h(3, 16)[:, :8], 8, h(3, 8), 8, 5, 3, 8, match="G must have rows")


def test_values():
    bad = lambda *a, match="INVALID", **k: refused("bf16", *a, match=match, error=g.GemmError, **k)
    bad(A, 8, 2 * A, 8, 0, 3, 8)            # no steps
    bad(A, 7, 2 * A, 8, 5, 3, 8)            # leading dimensions
    bad(A, 8, 2 * A, 7, 5, 3, 8)
    bad(0, 8, 2 * A, 8, 5, 3, 8)
    bad(A, 8, 0, 8, 5, 3, 8)
    bad(A + 1, 8, 2 * A, 8, 5, 3, 8)        # off the element
    bad(A, 8, 2 * A, 8, 5, -3, 8)
    bad(A, 8, A + 2, 8, 5, 3, 8, match="ALIAS")
    bad(A, 8, A, 9, 5, 3, 8, match="ALIAS")  # in place with another leading dimension
    bad(A, 8, 2 * A, 8, 5, 3, 8, (float("nan"), 1.0, 1.0), match="INVALID.*coefficients")
    bad(A, 8, 2 * A, 8, 5, 3, 8, (1.0, 1.0, float("inf")), match="INVALID.*coefficients")


def test_nothing_to_do():
    before = g.gemm_kernel_launches()
    g.gemm_orthogonalize("bf16", 0, 8, 0, 8, 5, 0, 8)
    g.gemm_orthogonalize("f16", 0, 1, 0, 1, 5, 8, 0)
    assert g.gemm_last_kernel() == "noop" and g.gemm_kernel_launches() == before
