"""The 4-bit block-scaled operators on the GPU, through the C ABI, against the CPU
reference: codes and scales bit for bit, values read back exactly, products
within fp4_ref.tolerance of 64-bit sums."""

import numpy as np
import pytest
import torch

import fp4_ref as ref

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
GUARD = 0x5A


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def matrix(M, K, dtype, seed, spread=True):
    """16-bit values whose rows (and a few columns) differ in scale."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K))
    if spread:
        x = x * np.exp2(np.arange(M) % 11 - 5)[:, None]
        x[:, ::37] *= 8
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


def scale_of(fmt, a):
    return float(np.float32(a.float().abs().max().item() * 1.047 / 2688)) if fmt == "nv" else None


def dev_scale(s):
    return None if s is None else torch.tensor([s], dtype=torch.float32, device="cuda")


def guarded_bytes(n):
    """n bytes with 512 guard bytes after them."""
    t = torch.full((n + 512,), GUARD, dtype=torch.uint8, device="cuda")
    return t, t[:n]


def quantize(a, fmt, gs, pad=0, off=0):
    """a [M,K] on the host -> device codes, scales (checked for writes past their end)."""
    M, K = a.shape
    ld = K + pad
    big = torch.full((M * ld + off,), 77.0, dtype=a.dtype, device="cuda")
    A = big[off:]
    A.view(M, ld)[:, :K].copy_(a.cuda())
    qb, Q = guarded_bytes(g.gemm_fp4_code_bytes(M, K))
    sb, S = guarded_bytes(g.gemm_fp4_scale_bytes(fmt, M, K))
    name = "bf16" if a.dtype == torch.bfloat16 else "f16"
    g.gemm_fp4_quantize(name, fmt, A, ld, dev_scale(gs), Q, S, M, K)
    g.gemm_synchronize()
    assert (qb[Q.numel():] == GUARD).all() and (sb[S.numel():] == GUARD).all()
    return Q, S


SHAPES = [(1, 1, 0, 0), (1, 4096, 0, 0), (3, 31, 0, 0), (2, 33, 0, 1), (129, 256, 8, 0), (130, 515, 1, 0),
          (64, 1000, 0, 0), (257, 4100, 4, 3), (5, 12288, 0, 0), (300, 96, 0, 0), (40, 1001, 0, 0), (9, 1030, 0, 5),
          (16, 2047, 0, 7), (11, 513, 4, 2), (8, 511, 0, 6)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,pad,off", SHAPES)
def test_quantize_bit_exact_and_read_back(M, K, pad, off, dtype, fmt):
    a = matrix(M, K, dtype, M * 7 + K)
    if M > 4:
        a[2] = 0
        a[3, K // 2] = float("nan")
        a[4, K - 1] = float("-inf")
        a[1] = 2.0 ** -24 if dtype == "f16" else 2.0 ** -130   # subnormal
    finite = torch.where(torch.isfinite(a), a, torch.zeros_like(a))
    gs = scale_of(fmt, finite)
    Q, S = quantize(a, fmt, gs, pad, off)
    code, byte = ref.quantize(fmt, a.float().numpy(), gs)
    got = Q.cpu().numpy().reshape(M, -1)
    want = ref.pack(code)
    # a value rounded to 0 may keep its sign: -0 and 0 are one value
    neg0 = lambda p: np.where(p & 7 == 0, p & 0xF0, p)
    clean = lambda p: neg0(np.where(p & 0x70 == 0, p & 0x0F, p))
    assert np.array_equal(clean(got), clean(want))
    assert np.array_equal(S.cpu().numpy(), ref.tile_scales(fmt, byte, K))
    # read back into a padded matrix
    ld = K + pad
    out = torch.full((M * ld + off,), 77.0, dtype=a.dtype, device="cuda")
    g.gemm_fp4_dequantize(dtype, fmt, Q, S, dev_scale(gs), out[off:], ld, M, K)
    g.gemm_synchronize()
    v = ref.values(fmt, code, byte)                             # exact in FP32
    f32 = v.astype(np.float32) * np.float32(1.0 if gs is None else gs)
    want = torch.from_numpy(f32).to(a.dtype).float().numpy()
    o = out.cpu().float()
    h = o[off:].view(M, ld).numpy()
    assert np.array_equal(h[:, :K], want, equal_nan=True)
    assert (h[:, K:] == 77).all() and (o[:off] == 77).all()


def test_ties_and_signs():
    x = torch.tensor([[4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 6] +
                      [7.5, 0, -0.0, 0.251, -0.251] + [0] * 11], dtype=torch.bfloat16)
    Q, S = quantize(x, "mx", None)
    out = torch.empty(1, 32, dtype=torch.bfloat16, device="cuda")
    g.gemm_fp4_dequantize("bf16", "mx", Q, S, None, out, 32, 1, 32)
    g.gemm_synchronize()
    assert out[0, :21].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, 6, 6, 0, 0, 0.5, -0.5]


def test_nv_underflow_and_saturation():
    x = torch.zeros(3, 32, dtype=torch.bfloat16)
    x[0], x[1], x[2, :16] = 1e-5, 5000.0, 6.0
    Q, S = quantize(x, "nv", None)       # no tensor scale: 1
    out = torch.empty(3, 32, dtype=torch.bfloat16, device="cuda")
    g.gemm_fp4_dequantize("bf16", "nv", Q, S, None, out, 32, 3, 32)
    g.gemm_synchronize()
    o = out.float().cpu()
    assert (o[0] == 0).all() and (o[1] == 2688).all() and (o[2, :16] == 6).all() and (o[2, 16:] == 0).all()


def product(fmt, dtype, M, N, K, seed, ldc_pad=0, c_off=0, linear=False, ldx_pad=0, x_off=0, b_row=None):
    a, b = matrix(M, K, dtype, seed, spread=False), matrix(N, K, dtype, seed + 1, spread=False)
    b = b * K ** -0.5
    ga, gb = scale_of(fmt, a), scale_of(fmt, b)
    if b_row is not None:
        b[b_row, K // 3] = float("nan")
    Qb, Sb = quantize(b, fmt, gb)
    ldc = N + ldc_pad
    big = torch.full((M * ldc + c_off + 64,), 77.0, dtype=DT[dtype], device="cuda")
    C = big[c_off:]
    if linear:
        ldx = K + ldx_pad
        X = torch.full((M * ldx + x_off,), float("nan"), dtype=DT[dtype], device="cuda")
        X[x_off:].view(M, ldx)[:, :K].copy_(a.cuda())
        g.gemm_fp4_linear(dtype, fmt, X[x_off:], ldx, dev_scale(ga), Qb, Sb, dev_scale(gb), C, ldc, M, N, K)
    else:
        Qa, Sa = quantize(a, fmt, ga)
        g.gemm_fp4(dtype, fmt, Qa, Sa, dev_scale(ga), Qb, Sb, dev_scale(gb), C, ldc, M, N, K)
    g.gemm_synchronize()
    o = big.float().cpu().numpy()
    assert (o[:c_off] == 77).all() and (o[c_off + M * ldc:] == 77).all()
    body = o[c_off:c_off + M * ldc].reshape(M, ldc)
    assert (body[:, N:] == 77).all()
    va, vb = ref.values(fmt, *ref.quantize(fmt, a.float().numpy(), ga), ga), ref.values(fmt, *ref.quantize(fmt, b.float().numpy(), gb), gb)
    return body[:, :N].astype(np.float64), va, vb


def check(C, va, vb, dtype, K):
    want = va @ vb.T
    bad = ~np.isfinite(want)
    assert np.array_equal(np.isnan(C), bad)
    tol = ref.tolerance(np.nan_to_num(va), np.nan_to_num(vb), np.nan_to_num(want), dtype, K)
    err = np.where(bad, 0.0, np.abs(C - np.where(bad, 0, want)))
    err = np.where(bad, 0.0, err)
    assert (err <= tol).all(), (err / tol).max()


PRODUCTS = [(1, 1, 1), (1, 8, 16), (3, 5, 33), (128, 128, 256), (256, 256, 256), (256, 512, 1024), (257, 129, 64),
            (100, 72, 4100), (64, 640, 2048), (65, 1001, 96), (640, 264, 288), (16, 1000, 1000), (300, 2050, 544),
            (1024, 1536, 512), (33, 130, 12288), (2, 20000, 128)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(M, N, K, fmt):
    for dtype in ("bf16", "f16"):
        C, va, vb = product(fmt, dtype, M, N, K, M + 3 * N + 5 * K)
        check(C, va, vb, dtype, K)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_linear(M, N, K, fmt):
    for dtype in ("bf16", "f16"):
        C, va, vb = product(fmt, dtype, M, N, K, M + 7 * N + 11 * K, linear=True)
        check(C, va, vb, dtype, K)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", [(512, 12288, 2048), (1600, 5000, 1000), (1601, 5003, 999)])
def test_product_over_several_waves_of_tiles(M, N, K, fmt):
    """192-wide tiles (every second one starts inside a 128-row tile of scales) and
    256-wide ones, several to a cluster, so that both accumulators are used."""
    C, va, vb = product(fmt, "bf16", M, N, K, 13)
    check(C, va, vb, "bf16", K)


@pytest.mark.parametrize("M,N,K,ldc_pad,c_off", [(300, 264, 512, 8, 0), (300, 264, 512, 1, 0), (300, 264, 512, 0, 1),
                                                 (7, 264, 512, 8, 0), (7, 263, 512, 2, 1), (130, 70, 320, 6, 2)])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_strides_and_offsets(M, N, K, ldc_pad, c_off, fmt):
    C, va, vb = product(fmt, "bf16", M, N, K, 5, ldc_pad, c_off)
    check(C, va, vb, "bf16", K)
    C, va, vb = product(fmt, "f16", M, N, K, 6, ldc_pad, c_off, linear=True, ldx_pad=ldc_pad, x_off=c_off)
    check(C, va, vb, "f16", K)


@pytest.mark.parametrize("M", [4, 200])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_nan_block_reaches_only_its_column(M, fmt):
    N, K = 200, 640
    C, va, vb = product(fmt, "bf16", M, N, K, 9, b_row=150)
    assert np.isnan(C[:, 150]).all()
    check(C, va, vb, "bf16", K)


def test_zero_k_and_empty():
    C = torch.full((4, 6), 5.0, dtype=torch.bfloat16, device="cuda")
    g.gemm_fp4("bf16", "mx", None, None, None, None, None, None, C, 6, 4, 5, 0)
    g.gemm_synchronize()
    assert (C[:, :5] == 0).all() and (C[:, 5] == 5).all()
    g.gemm_fp4_linear("bf16", "nv", None, 16, None, None, None, None, C, 6, 0, 5, 16)
    g.gemm_synchronize()


@pytest.mark.parametrize("M", [2, 300])
def test_runs_on_the_callers_stream_and_repeats_bit_for_bit(M):
    N, K, fmt = 512, 2048, "nv"
    a, b = matrix(M, K, "bf16", 1, False).cuda(), matrix(N, K, "bf16", 2, False)
    Qb, Sb = quantize(b, fmt, 0.01)
    gs = dev_scale(0.01)
    outs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x = torch.zeros_like(a)
        torch.cuda._sleep(20_000_000)
        x.copy_(a)              # late on this stream: a call on another one would read zeros
        for _ in range(3):
            C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
            g.gemm_fp4_linear("bf16", fmt, x, K, gs, Qb, Sb, gs, C, N, M, N, K)
            outs.append(C)
    s.synchronize()
    g.gemm_set_stream(None)
    assert outs[0].float().abs().max() > 0
    assert all(torch.equal(outs[0], o) for o in outs[1:])
