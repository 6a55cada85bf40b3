"""The root-mean-square norm with residual on the GPU, through the C ABI, against 64-bit
values within norm_ref's tolerances."""

import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import norm_ref as ref

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
FILL = 77.0
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def make(M, K, dtype, seed, loud=3.0):
    """X, R, w, dY, dH: rows of different loudness."""
    rng = np.random.default_rng(seed)
    rows = np.exp(rng.standard_normal((M, 1)) * loud / 3)
    t = [rng.standard_normal((M, K)), rng.standard_normal((M, K)) * rows, 1 + 0.3 * rng.standard_normal(K),
         rng.standard_normal((M, K)), rng.standard_normal((M, K))]
    return [torch.from_numpy(x.astype(np.float32)).to(DT[dtype]) for x in t]


def guarded(n, dt, off=0):
    """An output of n elements, `off` elements past an aligned base, between guards."""
    b = torch.full((16 + n + 64,), FILL, dtype=torch.float32).to(dt).cuda()
    return b, b[16 + off:16 + off + n]


def untouched(b, n, off):
    h = b.float().cpu()
    assert (h[:16 + off] == FILL).all() and (h[16 + off + n:] == FILL).all()


def placed(x, off=0):
    b = torch.empty(x.numel() + 16, dtype=x.dtype, device="cuda")
    b[off:off + x.numel()].copy_(x.reshape(-1))
    return b[off:off + x.numel()]


def f64(t, *shape):
    return t.double().cpu().numpy().reshape(shape)


def close(got, want, tol, name):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (name, int(bad.sum()), float((np.abs(got - want) / tol).max()))


def summed(X, R):
    return (X.float() + R.float()).to(X.dtype)


def check_forward(dtype, t, M, K, offs=(0,) * 6, w=True):
    X, R, wt = (placed(x, o) for x, o in zip(t[:3], offs[:3]))
    hb, H = guarded(M * K, DT[dtype], offs[3])
    yb, Y = guarded(M * K, DT[dtype], offs[4])
    rb, rstd = guarded(M, torch.float32)
    qb, Q = guarded(M * K, torch.float8_e4m3fn, offs[5])
    sb, scale = guarded(M, torch.float32)
    h2b, H2 = guarded(M * K, DT[dtype], offs[3])
    g.gemm_rms_norm(dtype, X, R, wt if w else None, EPS, H, Y, rstd, M, K)
    g.gemm_rms_norm_e4m3(dtype, X, R, wt if w else None, EPS, H2, Q, scale, M, K)
    g.gemm_synchronize()
    for b, n, o in ((hb, M * K, offs[3]), (yb, M * K, offs[4]), (rb, M, 0), (h2b, M * K, offs[3]), (sb, M, 0)):
        untouched(b, n, o)
    q8 = qb.view(torch.uint8).cpu()  # (77 as E4M3 is 80: compare bytes)
    fill = torch.full((1,), FILL).to(torch.float8_e4m3fn).view(torch.uint8)
    assert (q8[:16 + offs[5]] == fill).all() and (q8[16 + offs[5] + M * K:] == fill).all()
    h = summed(t[0], t[1])
    assert torch.equal(H.cpu().reshape(M, K), h) and torch.equal(H2.cpu().reshape(M, K), h)
    h, wd = h.double().numpy(), t[2].double().numpy() if w else np.ones(K)
    r, y = ref.forward(h, wd, EPS)
    er, ey = ref.forward_error(K)
    close(f64(rstd, M), r, r * er, "rstd")
    close(f64(Y, M, K), y, ref.round_tolerance(y, ey, dtype), "Y")
    s = np.abs(y).max(1) / 448
    close(f64(scale, M), s, s * (ey + 2 * ref.U), "scale")
    v = y / np.where(s > 0, s, 1)[:, None]
    close(f64(Q, M, K), v, ref.e4m3_tolerance(v, ey), "Q")
    return H, rstd


def check_backward(dtype, t, M, K, offs=(0,) * 5, w=True, dH=True):
    h = summed(t[0], t[1])
    H, wt, dY, d = (placed(x, o) for x, o in zip((h, t[2], t[3], t[4]), offs))
    _, rstd = guarded(M, torch.float32)
    g.gemm_rms_norm(dtype, H, None, wt, EPS, None, torch.empty_like(H), rstd, M, K)
    xb, dX = guarded(M * K, DT[dtype], offs[4])
    wb, dw = guarded(K, torch.float32)
    g.gemm_rms_norm_backward(dtype, H, wt if w else None, rstd, dY, d if dH else None, dX, dw, M, K)
    g.gemm_synchronize()
    untouched(xb, M * K, offs[4])
    untouched(wb, K, 0)
    args = (h.double().numpy(), t[2].double().numpy() if w else np.ones(K), t[3].double().numpy(),
            t[4].double().numpy() if dH else np.zeros((M, K)), EPS)
    want_x, want_w = ref.backward(*args)
    tol_x, tol_w = ref.backward_tolerance(*args, dtype)
    close(f64(dX, M, K), want_x, tol_x, "dX")
    close(f64(dw, K), want_w, tol_w, "dw")
    return dX, dw


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 64), (2, 1000), (4, 1001), (7, 1024), (3, 1025), (9, 2048), (6, 2049), (1, 4096),
          (5, 4096), (33, 4097), (3, 8192), (2, 8200), (2, 16384), (3, 16371), (2, 16385), (2, 40000), (1, 70001),
          (300, 1000), (777, 1001), (1300, 520), (2000, 264), (700, 2056)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_forward(M, K, dtype):
    check_forward(dtype, make(M, K, dtype, M + 3 * K), M, K)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_backward(M, K, dtype):
    check_backward(dtype, make(M, K, dtype, M + 5 * K), M, K)


@pytest.mark.parametrize("offs", [(1,) * 6, (3, 3, 3, 3, 3, 3), (1, 0, 0, 0, 0, 0), (0, 5, 0, 0, 0, 0), (0, 0, 1, 0, 0, 0),
                                  (0, 0, 0, 7, 0, 0), (0, 0, 0, 0, 2, 0), (0, 0, 0, 0, 0, 3)])
@pytest.mark.parametrize("M,K", [(5, 1000), (3, 4099), (2, 16400)])
def test_operands_off_16_bytes(M, K, offs):
    t = make(M, K, "bf16", 7)
    check_forward("bf16", t, M, K, offs)
    check_backward("bf16", t, M, K, offs[:5])


@pytest.mark.parametrize("M,K", [(3, 512), (3, 513), (2, 20000)])
def test_without_gain_or_second_gradient(M, K):
    t = make(M, K, "f16", 8)
    check_forward("f16", t, M, K, w=False)
    check_backward("f16", t, M, K, w=False, dH=False)


@pytest.mark.parametrize("M,K", [(7, 1024), (7, 1021), (2, 17000)])
def test_in_place_and_left_out(M, K):
    """H as X or as R, no H, no residual, dX as dH, one gradient alone: the same bits."""
    t = make(M, K, "bf16", 9)
    X, R, w, dY, dH = (x.cuda().reshape(-1) for x in t)
    new = lambda: torch.empty(M * K, dtype=torch.bfloat16, device="cuda")
    H, Y, rstd, Q, scale = new(), new(), torch.empty(M, device="cuda"), new().view(torch.uint8)[:M * K], torch.empty(M, device="cuda")
    g.gemm_rms_norm("bf16", X, R, w, EPS, H, Y, rstd, M, K)
    g.gemm_rms_norm_e4m3("bf16", X, R, w, EPS, None, Q, scale, M, K)
    for which in "XR":
        a, b = X.clone(), R.clone()
        y = new()
        g.gemm_rms_norm("bf16", a, b, w, EPS, a if which == "X" else b, y, None, M, K)
        assert torch.equal(y, Y) and torch.equal(a if which == "X" else b, H)
        a, b, q, s = X.clone(), R.clone(), torch.empty_like(Q), torch.empty_like(scale)
        g.gemm_rms_norm_e4m3("bf16", a, b, w, EPS, a if which == "X" else b, q, s, M, K)
        assert torch.equal(q, Q) and torch.equal(s, scale) and torch.equal(a if which == "X" else b, H)
    y = new()
    g.gemm_rms_norm("bf16", X, R, w, EPS, None, y, None, M, K)
    assert torch.equal(y, Y)
    y = new()
    g.gemm_rms_norm("bf16", H, None, w, EPS, None, y, None, M, K)
    assert torch.equal(y, Y)
    dX, dw = new(), torch.empty(K, device="cuda")
    g.gemm_rms_norm_backward("bf16", H, w, rstd, dY, dH, dX, dw, M, K)
    d, dw2, dx2 = dH.clone(), torch.empty(K, device="cuda"), new()
    g.gemm_rms_norm_backward("bf16", H, w, rstd, dY, d, d, None, M, K)
    g.gemm_rms_norm_backward("bf16", H, w, rstd, dY, dH, None, dw2, M, K)
    assert torch.equal(d, dX) and torch.equal(dw2, dw)
    g.gemm_rms_norm_backward("bf16", H, w, rstd, dY, dH, dx2, dw2, M, K)
    assert torch.equal(dx2, dX) and torch.equal(dw2, dw)  # run to run
    g.gemm_synchronize()


@pytest.mark.parametrize("K", [512, 1027, 20000])
def test_rows_at_the_ends_of_the_range(K):
    """Zeros; squares past FP32's range (bf16); the least normal numbers; a NaN and an
    infinity, which reach their own rows only."""
    rng = np.random.default_rng(3)
    base = rng.standard_normal((6, K)).astype(np.float32)
    for dtype, scales in (("bf16", (0.0, 1e30, 2e38 / np.abs(base[2]).max(), 1e-30, 1.0, 1.0)),
                          ("f16", (0.0, 6e4 / np.abs(base[1]).max(), 1.0, 1e-4, 1.0, 1.0))):
        X = torch.from_numpy(base * np.array(scales, np.float32)[:, None]).to(DT[dtype])
        X[4, K // 2] = float("nan")
        X[5, K - 1] = float("inf")
        w = torch.ones(K, dtype=DT[dtype])
        x, wd = X.cuda().reshape(-1), w.cuda()
        Y, Q = torch.empty_like(x), torch.empty(6 * K, dtype=torch.float8_e4m3fn, device="cuda")
        scale, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
        g.gemm_rms_norm(dtype, x, None, wd, EPS, None, Y, rstd, 6, K)
        g.gemm_rms_norm_e4m3(dtype, x, None, wd, EPS, None, Q, scale, 6, K)
        g.gemm_synchronize()
        h = X.double().numpy()[:4]
        r, y = ref.forward(h, 1.0, EPS)
        er, ey = ref.forward_error(K)
        close(f64(Y, 6, K)[:4], y, ref.round_tolerance(y, ey, dtype), "Y")
        s = np.abs(y).max(1) / 448
        close(f64(scale, 6)[:4], s, s * (ey + 2 * ref.U), "scale")
        v = y / np.where(s > 0, s, 1)[:, None]
        close(f64(Q, 6, K)[:4], v, ref.e4m3_tolerance(v, ey), "Q")
        assert Y.reshape(6, K)[4].isnan().all() and Y.reshape(6, K)[5, K - 1].isnan()
        assert scale[4:].isnan().all()


def test_codes_feed_the_fp8_product():
    """Norm to E4M3, then the row-scaled product: what the norm's values give within the
    codes' half steps, summed, and the product's rounding to half."""
    M, N, K = 70, 136, 512
    t = make(M, K, "f16", 10)
    X, R, w = (x.cuda() for x in t[:3])
    H, Q, scale = torch.empty_like(X), torch.empty(M, K, dtype=torch.uint8, device="cuda"), torch.empty(M, device="cuda")
    W = (torch.randn(N, K, generator=torch.Generator().manual_seed(1)) * 0.05).to(torch.float8_e4m3fn)
    C = torch.empty(M, N, dtype=torch.float16, device="cuda")
    g.gemm_rms_norm_e4m3("f16", X, R, w, EPS, H, Q, scale, M, K)
    g.gemm_e4m3_rowscale(Q, scale, W.view(torch.uint8).cuda(), C, M, N, K)
    g.gemm_synchronize()
    _, y = ref.forward(summed(t[0], t[1]).double().numpy(), t[2].double().numpy(), EPS)
    Wd = W.double().numpy() if hasattr(W, "double") else W.float().double().numpy()
    s = np.abs(y).max(1, keepdims=True) / 448
    tol = (s * ref.e4m3_tolerance(y / s, 1e-5)) @ np.abs(Wd).T + np.abs(y) @ np.abs(Wd).T * 1e-5
    want = y @ Wd.T
    close(f64(C, M, N), want, tol + 2.0 ** -11 * (np.abs(want) + tol) + 2.0 ** -25, "C")


def test_captured_and_replayed():
    """A forward and a backward call in a graph, replayed on new inputs, on a side stream."""
    M, K = 300, 1032
    a, b = make(M, K, "bf16", 20), make(M, K, "bf16", 21)
    bufs = [x.cuda().reshape(-1) for x in a]
    X, R, w, dY, dH = bufs
    H, Y, dX = (torch.empty_like(X) for _ in range(3))
    rstd, dw = torch.empty(M, device="cuda"), torch.empty(K, device="cuda")

    def step():
        g.gemm_rms_norm("bf16", X, R, w, EPS, H, Y, rstd, M, K)
        g.gemm_rms_norm_backward("bf16", H, w, rstd, dY, dH, dX, dw, M, K)
    want = []
    for t in (a, b):
        for x, v in zip(bufs, t):
            x.copy_(v.reshape(-1))
        step()
        want.append([x.clone() for x in (H, Y, dX, dw)])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        for t, w4 in ((a, want[0]), (b, want[1]), (a, want[0])):
            for x, v in zip(bufs, t):
                x.copy_(v.reshape(-1))
            for x in (H, Y, dX, dw):
                x.fill_(FILL)
            graph.replay()
            for x, y in zip((H, Y, dX, dw), w4):
                assert torch.equal(x, y)
    torch.cuda.synchronize()


def test_past_2_31_elements():
    """The last rows of a matrix of more than 2^31 elements: those of a small one."""
    K, M = 4096, (1 << 31) // 4096 + 9
    t = make(16, K, "bf16", 30)
    X = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    X[-16:].copy_(t[1])
    w, dY16 = t[2].cuda(), t[3].cuda()
    Y, rstd = torch.empty_like(X), torch.empty(M, device="cuda")
    g.gemm_rms_norm("bf16", X, None, w, EPS, None, Y, rstd, M, K)
    y16, r16 = torch.empty(16, K, dtype=torch.bfloat16, device="cuda"), torch.empty(16, device="cuda")
    g.gemm_rms_norm("bf16", t[1].cuda(), None, w, EPS, None, y16, r16, 16, K)
    g.gemm_synchronize()
    assert torch.equal(Y[-16:], y16) and torch.equal(rstd[-16:], r16) and not Y[:-16].any()
    dY = Y.zero_()
    dY[-16:].copy_(dY16)
    dX, dw = torch.empty_like(X), torch.empty(K, device="cuda")
    g.gemm_rms_norm_backward("bf16", X, w, rstd, dY, None, dX, dw, M, K)
    dx16 = torch.empty_like(y16)
    g.gemm_rms_norm_backward("bf16", t[1].cuda(), w, r16, dY16, None, dx16, None, 16, K)
    g.gemm_synchronize()
    assert torch.equal(dX[-16:], dx16) and not dX[:-16].any()
    _, want = ref.backward(t[1].double().numpy(), t[2].double().numpy(), t[3].double().numpy(), 0.0, EPS)
    _, tol = ref.backward_tolerance(t[1].double().numpy(), t[2].double().numpy(), t[3].double().numpy(), np.zeros((16, K)), EPS, "bf16")
    close(f64(dw, K), want, tol, "dw")
    del X, Y, dX, dY
    torch.cuda.empty_cache()


def test_no_rows():
    dw = torch.full((8,), FILL, device="cuda")
    z = torch.empty(0, dtype=torch.bfloat16, device="cuda")
    g.gemm_rms_norm_backward("bf16", z, z, None, z, None, None, dw, 0, 8)
    g.gemm_rms_norm("bf16", z, None, z, EPS, None, z, None, 0, 8)
    g.gemm_synchronize()
    assert not dw.any()


FIRST = """
import sys
import torch
import dense_matrix_multiply_gb300 as g
for K in map(int, sys.argv[1:]):
    for name, dt in (("bf16", torch.bfloat16), ("f16", torch.float16)):
        X, w, dY = (torch.randn(n, device="cuda").to(dt) for n in (8 * K, K, 8 * K))
        Y, dX = torch.empty_like(X), torch.empty_like(X)
        rstd, dw = torch.empty(8, device="cuda"), torch.empty(K, device="cuda")
        g.gemm_rms_norm(name, X, None, w, 1e-5, None, Y, rstd, 8, K)
        g.gemm_rms_norm_backward(name, X, w, rstd, dY, None, dX, dw, 8, K)
g.gemm_synchronize()
"""


@pytest.mark.parametrize("sizes", [("256", "8121"), ("8105", "8167")])
def test_first_calls_of_a_process(sizes):
    """Sizes whose shared memory, with what the kernel itself declares, just passes the 48 KB
    that need no leave, before any larger call has asked for it."""
    root = Path(__file__).resolve().parents[1]
    r = subprocess.run([sys.executable, "-c", FIRST, *sizes], cwd=root, capture_output=True, text=True, timeout=180)
    assert r.returncode == 0, r.stderr[-2000:]
