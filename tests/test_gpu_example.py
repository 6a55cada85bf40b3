"""The example runs the gated block's training and the 4-bit serving together."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_train_then_serve_in_4_bits(lib, fmt):
    path = os.path.join(ROOT, "examples", "ffn_train_then_4bit.py")
    spec = importlib.util.spec_from_file_location("ffn_train_then_4bit", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.run(tokens=300, width=256, hidden=520, steps=30, fmt=fmt)
    assert r["losses"][-1] < 0.5 * r["losses"][0]
    # an E2M1 code is off by 1/8 to 1/4 of its magnitude at most: some 0.1 relative
    # of N(0, 1) weights, and as much of the activations
    assert 0.02 < r["weight_error_4bit"] < 0.2 and r["error_4bit"] < 0.5
    # the same codes through two kernels: FP32 sums in another order, one rounding
    # to bf16 each, and z's codes move where its rounding does
    assert r["token_vs_prompt"] < 0.05
