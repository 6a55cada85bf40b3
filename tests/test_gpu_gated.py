"""The gated feed-forward block on the GPU, through the C ABI, against 64-bit values
within gated_ref's tolerances, and its gradients against differences of the
kernel's own forward products."""

import numpy as np
import pytest
import torch

import gated_ref as ref

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
FILL = 77.0


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def make(M, N, K, dtype, seed):
    rng = np.random.default_rng(seed)
    shapes = ((M, K, 1.0), (K, N, 1.5 * K ** -0.5), (K, N, K ** -0.5), (M, N, 1.0))
    t = [torch.from_numpy((rng.standard_normal((a, b)) * s).astype(np.float32)).to(DT[dtype]) for a, b, s in shapes]
    return t, [x.double().numpy() for x in t]


def guarded(rows, cols, dt):
    """A [rows, cols] output with a guard row's worth of elements after it."""
    t = torch.full((rows * cols + 64,), FILL, dtype=dt, device="cuda")
    return t, t[:rows * cols]


def run(dtype, act, t, M, N, K, save=True, grads=True):
    X, Wg, Wu, dZ = (x.cuda() for x in t)
    zb, Z = guarded(M, N, DT[dtype])
    outs = {"Z": (zb, (M, N))}
    G = U = None
    if save:
        gb, G = guarded(M, N, torch.float32)
        ub, U = guarded(M, N, torch.float32)
        outs |= {"G": (gb, (M, N)), "U": (ub, (M, N))}
    g.gemm_gated(dtype, act, X, Wg, Wu, Z, G, U, M, N, K)
    if save and grads:
        xb, dX = guarded(M, K, DT[dtype])
        wb, dWg = guarded(K, N, DT[dtype])
        vb, dWu = guarded(K, N, DT[dtype])
        g.gemm_gated_backward(dtype, act, X, Wg, Wu, G, U, dZ, dX, dWg, dWu, M, N, K)
        outs |= {"dX": (xb, (M, K)), "dWg": (wb, (K, N)), "dWu": (vb, (K, N))}
    g.gemm_synchronize()
    got = {}
    for name, (b, (r, c)) in outs.items():
        h = b.double().cpu().numpy()
        assert (h[r * c:] == FILL).all(), name
        got[name] = h[:r * c].reshape(r, c)
    return got


def close(got, want, tol, name):
    err = np.abs(got - want)
    assert (err <= tol).all(), (name, float((err / tol).max()))


SHAPES = [(1, 8, 8), (1, 64, 128), (1, 1000, 1000), (5, 136, 264), (16, 64, 200), (17, 520, 72), (63, 128, 512),
          (64, 200, 1024), (65, 128, 64), (128, 384, 328), (200, 1000, 136), (257, 264, 520), (333, 1000, 1000),
          (700, 72, 2056), (130, 4104, 64)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward_and_backward(M, N, K, dtype, act):
    t, (X, Wg, Wu, dZ) = make(M, N, K, dtype, M + 3 * N + 7 * K)
    got = run(dtype, act, t, M, N, K)
    Z, G, U = ref.forward(act, X, Wg, Wu)
    tZ, tG, tU = ref.forward_tolerance(act, X, Wg, Wu, dtype)
    close(got["G"], G, tG, "G")
    close(got["U"], U, tU, "U")
    close(got["Z"], Z, tZ, "Z")
    grads = ref.backward(act, X, Wg, Wu, dZ)
    for name, want, tol in zip(("dX", "dWg", "dWu"), grads, ref.backward_tolerance(act, X, Wg, Wu, dZ, dtype)):
        close(got[name], want, tol, name)


@pytest.mark.parametrize("M,N,K", [(600, 5000, 264), (5000, 64, 2056), (512, 5120, 1600), (900, 1000, 1792), (100, 72, 8200),
                                   (800, 700, 136)])
def test_several_waves_of_tiles(M, N, K):
    """More tiles than clusters, forward and dW, then dX: every buffer of the
    kernels is used again and again.  The third: four tiles past a whole wave,
    split along K.  The fourth: dX beside dW, on the few clusters that it
    leaves.  The last two: forward in 64-wide tiles, split along K and whole."""
    t, (X, Wg, Wu, dZ) = make(M, N, K, "bf16", 11)
    got = run("bf16", "silu", t, M, N, K)
    for name, want, tol in zip("ZGU", ref.forward("silu", X, Wg, Wu), ref.forward_tolerance("silu", X, Wg, Wu, "bf16")):
        close(got[name], want, tol, name)
    grads = ref.backward("silu", X, Wg, Wu, dZ)
    for name, want, tol in zip(("dX", "dWg", "dWu"), grads, ref.backward_tolerance("silu", X, Wg, Wu, dZ, "bf16")):
        close(got[name], want, tol, name)


ODD = [(1, 1, 1), (1, 7, 5), (3, 9, 1000), (5, 1001, 8), (65, 129, 333), (64, 255, 33), (200, 1001, 137), (70, 8, 9),
       (333, 1000, 1001)]


@pytest.mark.parametrize("act,dtype", [("silu", "bf16"), ("gelu", "f16")])
@pytest.mark.parametrize("M,N,K", ODD)
def test_sizes_that_are_no_multiples_of_8(M, N, K, dtype, act):
    """Operands through padded copies: the same tolerances, nothing written past the outputs."""
    test_forward_and_backward(M, N, K, dtype, act)


def test_long_products_of_rows_off_128_bytes():
    """X goes to aligned rows first: the same bits as with K filled up with zeros,
    where it does not."""
    M, N, K, K0 = 1400, 4104, 4104, 4160
    (X, Wg, Wu, _), _ = make(M, N, K, "bf16", 13)
    wide = torch.zeros(M, K0, dtype=X.dtype)
    wide[:, :K] = X
    tall = [torch.cat([w, torch.zeros(K0 - K, N, dtype=w.dtype)]) for w in (Wg, Wu)]
    a = run("bf16", "silu", (X, Wg, Wu, X[:1]), M, N, K, grads=False)
    b = run("bf16", "silu", (wide, *tall, X[:1]), M, N, K0, grads=False)
    for n in "ZGU":
        assert np.array_equal(a[n], b[n]), n


@pytest.mark.parametrize("M,N,K", [(3, 72, 40), (100, 264, 128), (100, 263, 127)])
def test_operands_off_16_bytes(M, N, K):
    """Every operand one element past an aligned base: the results of the aligned call, bit for bit."""
    t, _ = make(M, N, K, "bf16", 12)
    want = run("bf16", "gelu", t, M, N, K)

    def off(rows, cols, dt=torch.bfloat16, x=None):
        b = torch.full((rows * cols + 64,), FILL, dtype=dt, device="cuda")
        v = b[1:1 + rows * cols]
        if x is not None:
            v.copy_(x.reshape(-1))
        return b, v

    X, Wg, Wu, dZ = (off(*x.shape, x=x)[1] for x in t)
    outs = {n: off(r, c, d) for n, r, c, d in (("Z", M, N, X.dtype), ("G", M, N, torch.float32), ("U", M, N, torch.float32),
                                              ("dX", M, K, X.dtype), ("dWg", K, N, X.dtype), ("dWu", K, N, X.dtype))}
    o = {n: v for n, (_, v) in outs.items()}
    g.gemm_gated("bf16", "gelu", X, Wg, Wu, o["Z"], o["G"], o["U"], M, N, K)
    g.gemm_gated_backward("bf16", "gelu", X, Wg, Wu, o["G"], o["U"], dZ, o["dX"], o["dWg"], o["dWu"], M, N, K)
    g.gemm_synchronize()
    for n, (b, v) in outs.items():
        assert b[0] == FILL and (b[1 + v.numel():] == FILL).all(), n
        assert np.array_equal(v.double().cpu().numpy(), want[n].reshape(-1)), n


@pytest.mark.parametrize("M,N,K", [(3, 72, 40), (200, 264, 128)])
def test_without_saving_gives_the_same_z(M, N, K):
    t, _ = make(M, N, K, "bf16", 5)
    a, b = run("bf16", "silu", t, M, N, K), run("bf16", "silu", t, M, N, K, save=False)
    assert np.array_equal(a["Z"], b["Z"])


def test_parts_of_the_gradient():
    """Each gradient alone equals the one computed with the others."""
    M, N, K = 150, 136, 264
    t, _ = make(M, N, K, "bf16", 6)
    full = run("bf16", "gelu", t, M, N, K)
    X, Wg, Wu, dZ = (x.cuda() for x in t)
    Z, G, U = torch.empty(M, N, dtype=X.dtype, device="cuda"), *(torch.empty(M, N, device="cuda") for _ in range(2))
    g.gemm_gated("bf16", "gelu", X, Wg, Wu, Z, G, U, M, N, K)
    for name, shape in (("dX", (M, K)), ("dWg", (K, N)), ("dWu", (K, N))):
        out = torch.empty(shape, dtype=X.dtype, device="cuda")
        args = [out if name == n else None for n in ("dX", "dWg", "dWu")]
        g.gemm_gated_backward("bf16", "gelu", X if name != "dX" else None, *((Wg, Wu) if name == "dX" else (None, None)),
                              G, U, dZ, *args, M, N, K)
        g.gemm_synchronize()
        assert np.array_equal(out.double().cpu().numpy(), full[name]), name


def test_order_of_the_weight_gradients_in_memory():
    """dWu below dWg in memory: the batch runs the other way round."""
    M, N, K = 100, 72, 136
    t, (X64, Wg64, Wu64, dZ64) = make(M, N, K, "bf16", 7)
    X, Wg, Wu, dZ = (x.cuda() for x in t)
    Z, G, U = torch.empty(M, N, dtype=X.dtype, device="cuda"), *(torch.empty(M, N, device="cuda") for _ in range(2))
    both = torch.empty(2, K, N, dtype=X.dtype, device="cuda")
    dX = torch.empty(M, K, dtype=X.dtype, device="cuda")
    g.gemm_gated("bf16", "silu", X, Wg, Wu, Z, G, U, M, N, K)
    g.gemm_gated_backward("bf16", "silu", X, Wg, Wu, G, U, dZ, dX, both[1], both[0], M, N, K)
    g.gemm_synchronize()
    want, tol = ref.backward("silu", X64, Wg64, Wu64, dZ64), ref.backward_tolerance("silu", X64, Wg64, Wu64, dZ64, "bf16")
    for got, w, e in zip((dX, both[1], both[0]), want, tol):
        close(got.double().cpu().numpy(), w, e, "swapped")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [8, 96])
def test_gradients_against_differences_of_the_forward_kernel(M, act):
    """<gradient, V> against (L(p + V h) - L(p - V h)) / 2h with L = sum dZ act(G) U, G
    and U from the kernel in FP32.  p on a grid of 2^-4 and V h of 2^-6, exact in
    16 bits.  The difference is off by h^2 / 6 of the third derivative (h = 2^-6:
    under 1 % of the derivatives' size here) and the gradient by its 16-bit
    roundings, whose sum over the elements is a fraction of 2^-8 of |gradient| |V|."""
    N, K = 64, 72
    rng = np.random.default_rng(3)
    grid = lambda r, c, s: np.round(rng.standard_normal((r, c)) * s * 16) / 16
    ops = [grid(M, K, 0.5), grid(K, N, 0.25), grid(K, N, 0.25)]
    dZ = grid(M, N, 1.0)
    to = lambda x: torch.from_numpy(x.astype(np.float32)).to(torch.float16)

    def products(o):
        got = run("f16", act, [to(x) for x in o] + [to(dZ)], M, N, K, grads=False)
        return (dZ * ref.act(act, got["G"])[0] * got["U"]).sum()

    got = run("f16", act, [to(x) for x in ops] + [to(dZ)], M, N, K)
    h = 2.0 ** -6
    for i, name in enumerate(("dX", "dWg", "dWu")):
        V = np.sign(got[name]) * (rng.random(got[name].shape) < 0.02)   # along the gradient: no cancellation
        up, dn = [o.copy() for o in ops], [o.copy() for o in ops]
        up[i] += h * V
        dn[i] -= h * V
        diff = (products(up) - products(dn)) / (2 * h)
        assert diff == pytest.approx((got[name] * V).sum(), rel=0.02), name


def test_large_activations_stay_finite_and_nan_reaches_its_rows():
    M, N, K = 70, 64, 64
    t, _ = make(M, N, K, "bf16", 8)
    t[0][3] = 3e4            # G of some 1e4: saturated activations, no NaN
    t[0][4] = float("nan")
    for act in ("silu", "gelu"):
        for rows in (slice(0, 6), slice(0, 70)):
            m = len(range(*rows.indices(M)))
            got = run("bf16", act, [t[0][rows], t[1], t[2], t[3][rows]], m, N, K)
            ok = np.ones(m, dtype=bool)
            ok[4] = False
            assert np.isfinite(got["Z"][ok]).all() and np.isnan(got["Z"][4]).all()
            assert np.isfinite(got["dX"][ok]).all() and np.isnan(got["dX"][4]).all()
            assert np.isnan(got["dWg"]).all()


def test_empty():
    X = torch.ones(4, 16, dtype=torch.bfloat16, device="cuda")
    Z, G, U = torch.ones(4, 8, dtype=X.dtype, device="cuda"), *(torch.ones(4, 8, device="cuda") for _ in range(2))
    g.gemm_gated("bf16", "silu", None, None, None, Z, G, U, 4, 8, 0)
    g.gemm_synchronize()
    assert (Z == 0).all() and (G == 0).all() and (U == 0).all()
    dW = torch.ones(16, 8, dtype=X.dtype, device="cuda")
    dV = torch.ones(16, 8, dtype=X.dtype, device="cuda")
    g.gemm_gated_backward("bf16", "silu", None, None, None, None, None, None, None, dW, dV, 0, 8, 16)
    g.gemm_synchronize()
    assert (dW == 0).all() and (dV == 0).all()


@pytest.mark.parametrize("M", [4, 300])
def test_runs_on_the_callers_stream_and_repeats_bit_for_bit(M):
    N, K = 264, 512
    t, _ = make(M, N, K, "bf16", 9)
    X0, Wg, Wu, dZ = (x.cuda() for x in t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    with torch.cuda.stream(s):
        X = torch.zeros_like(X0)
        torch.cuda._sleep(20_000_000)
        X.copy_(X0)             # late on this stream: a call on another one would read zeros
        for _ in range(3):
            o = [torch.empty(M, N, dtype=X.dtype, device="cuda"), torch.empty(M, N, device="cuda"),
                 torch.empty(M, N, device="cuda"), torch.empty(M, K, dtype=X.dtype, device="cuda"),
                 torch.empty(K, N, dtype=X.dtype, device="cuda"), torch.empty(K, N, dtype=X.dtype, device="cuda")]
            g.gemm_gated("bf16", "silu", X, Wg, Wu, *o[:3], M, N, K)
            g.gemm_gated_backward("bf16", "silu", X, Wg, Wu, o[1], o[2], dZ, *o[3:], M, N, K)
            outs.append(o)
    s.synchronize()
    g.gemm_set_stream(None)
    assert all(x.float().abs().max() > 0 for x in outs[0])
    for other in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(outs[0], other))


def test_queued_calls_of_mixed_sizes_repeat_bit_for_bit():
    """Forward, backward and 4-bit calls queued without a wait: kernels of one call
    start while the last one's drain, and find its scratch and outputs whole."""
    cases = []
    for i, (M, N, K) in enumerate([(1, 500, 300), (64, 1000, 504), (333, 1000, 1000), (500, 1504, 704), (900, 1000, 1792)]):
        (X, Wg, Wu, dZ), _ = make(M, N, K, "bf16", 20 + i)
        X, Wg, Wu, dZ = (x.cuda() for x in (X, Wg, Wu, dZ))
        Q = torch.empty(g.gemm_fp4_code_bytes(N, K), dtype=torch.uint8, device="cuda")
        S = torch.empty(g.gemm_fp4_scale_bytes("nv", N, K), dtype=torch.uint8, device="cuda")
        g.gemm_fp4_quantize("bf16", "nv", Wg.t().contiguous(), K, None, Q, S, N, K)
        cases.append((M, N, K, X, Wg, Wu, dZ, Q, S))

    def outputs(M, N, K):
        half = lambda r, c: torch.full((r, c), FILL, dtype=torch.bfloat16, device="cuda")
        full = lambda r, c: torch.full((r, c), FILL, device="cuda")
        return [half(M, N), full(M, N), full(M, N), half(M, K), half(K, N), half(K, N), half(M, N)]

    def call(case, o):
        M, N, K, X, Wg, Wu, dZ, Q, S = case
        g.gemm_gated("bf16", "silu", X, Wg, Wu, *o[:3], M, N, K)
        g.gemm_gated_backward("bf16", "silu", X, Wg, Wu, o[1], o[2], dZ, *o[3:6], M, N, K)
        g.gemm_fp4_linear("bf16", "nv", X, K, None, Q, S, None, o[6], N, M, N, K)

    want = []
    for c in cases:
        want.append(outputs(*c[:3]))
        call(c, want[-1])
        g.gemm_synchronize()
    order = [int(i) for i in np.random.default_rng(4).integers(0, len(cases), 60)]
    got = [outputs(*cases[i][:3]) for i in order]
    torch.cuda.synchronize()
    for i, o in zip(order, got):
        call(cases[i], o)
    g.gemm_synchronize()
    for i, o in zip(order, got):
        for k, (x, y) in enumerate(zip(o, want[i])):
            assert torch.equal(x, y), (cases[i][:3], k)
