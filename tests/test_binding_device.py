"""One rule for every entry point of the binding: tensors off the current CUDA device are
refused, and a refused call leaves the thread's stream as it was (no GPU: stand-ins for
tensors, and for torch's current device and streams)."""

import pytest

import dense_matrix_multiply_gb300 as g

M, N, K = 3, 16, 32


class Stand:
    """A contiguous tensor's answers, of `size`-byte elements on a device."""

    def __init__(self, size, device, elements=1 << 12):
        self.size, self.device, self.elements, self.dtype = size, device, elements, f"{size}-byte"
        self.shape = (elements,)

    def element_size(self):
        return self.size

    def is_contiguous(self):
        return True

    def numel(self):
        return self.elements

    def stride(self):
        return (1,)

    def get_device(self):
        return self.device

    def data_ptr(self):
        return 1 << 40

    def storage_offset(self):
        return 0

    def untyped_storage(self):
        return self

    def nbytes(self):
        return self.elements * self.size


def calls(d):
    h, f, b, i = (Stand(n, d) for n in (2, 4, 1, 8))
    return {
        "gemm_f32_rm": (f, f, f, M, N, K),
        "gemm_f16_cm": (h, h, h, M, N, K),
        "gemm_bf16_rm": (h, h, h, M, N, K),
        "gemm_bf16_rm_noalloc": (h, h, h, M, N, K),
        "gemm_bf16_rm_silu_mul": (h, h, h, h, M, N, K),
        "gemm_quantize_rows_e4m3": (h, b, f, M, K),
        "gemm_e4m3_rowscale": (b, f, b, h, M, N, K),
        "gemm_e4m3_rowscale_fused": (h, b, h, M, N, K),
        "gemm_ex": ("f16", "rm", "N", "N", M, N, K, 1.0, h, K, 0, h, N, 0, 0.0, h, N, 0),
        "gemm_fp4_quantize": ("f16", "nv", h, K, f, b, b, M, K),
        "gemm_fp4_dequantize": ("f16", "nv", b, b, f, h, K, M, K),
        "gemm_fp4": ("f16", "nv", b, b, f, b, b, f, h, N, M, N, K),
        "gemm_fp4_linear": ("f16", "nv", h, K, f, b, b, f, h, N, M, N, K),
        "gemm_gated": ("bf16", "silu", h, h, h, h, None, None, M, N, K),
        "gemm_gated_backward": ("bf16", "silu", h, h, h, f, f, h, h, h, h, M, N, K),
        "gemm_rms_norm": ("bf16", h, h, h, 1e-6, h, h, f, M, K),
        "gemm_rms_norm_e4m3": ("bf16", h, h, h, 1e-6, h, b, f, M, K),
        "gemm_rms_norm_backward": ("bf16", h, h, f, h, h, h, f, M, K),
        "gemm_cross_entropy": ("bf16", h, h, i, f, f, M, N, K),
        "gemm_cross_entropy_backward": ("bf16", h, h, i, f, f, h, h, M, N, K),
        "gemm_orthogonalize": ("bf16", h, K, h, K, 5, M, K),
    }


@pytest.fixture
def bound(lib, monkeypatch):
    lib.load()
    monkeypatch.setattr(g, "_raw_device", lambda: 0)
    monkeypatch.setattr(g, "_raw_stream", lambda device: 0x1000 + device)
    g.gemm_set_stream(0x77)
    yield
    g.gemm_set_stream(None)


@pytest.mark.parametrize("name", calls(1))
def test_another_device(bound, name):
    before = g.gemm_kernel_launches()
    with pytest.raises(ValueError, match="tensors on cuda:1, the current device is cuda:0"):
        getattr(g, name)(*calls(1)[name])
    assert g.gemm_get_stream() == 0x77 and g.gemm_kernel_launches() == before


@pytest.mark.parametrize("name", calls(-1))
def test_host_memory(bound, name):
    with pytest.raises(ValueError, match="must live on a CUDA device"):
        getattr(g, name)(*calls(-1)[name])
    assert g.gemm_get_stream() == 0x77


def test_two_devices_and_the_current_one(bound):
    here, there = Stand(4, 0), Stand(4, 1)
    for tensors in ((here, there), (there, here)):
        with pytest.raises(ValueError, match="two devices"):
            g._bind_torch_stream(*tensors)
        with pytest.raises(ValueError, match="two devices"):
            g._take(g.load(), "call", *(("t", t, 4, 1, True) for t in tensors))
        assert g.gemm_get_stream() == 0x77
    g._bind_torch_stream(here, None, 12345)
    assert g.gemm_get_stream() == 0x1000
    g.gemm_set_stream(0x77)
    assert g._take(g.load(), "call", ("t", here, 4, 1, True), ("u", 5, 4, 1, True)) == [1 << 40, 5]
    assert g.gemm_get_stream() == 0x1000
