"""The linear head's softmax cross entropy on the GPU, through the C ABI, against 64-bit
values within head_ref's tolerances."""

import numpy as np
import pytest
import torch

import head_ref as ref

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
FILL = 77.0


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def make(M, N, K, dtype, seed, spread=2.0, left_out=0.2):
    """X, W, targets (some left out, below 0 and past N), dloss of either sign."""
    rng = np.random.default_rng(seed)
    X = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(DT[dtype])
    W = torch.from_numpy((spread * K ** -0.5 * rng.standard_normal((N, K))).astype(np.float32)).to(DT[dtype])
    t = rng.integers(0, N, M)
    gone = rng.random(M) < left_out
    t[gone] = rng.choice([-100, -1, N, -2 ** 63, 2 ** 63 - 1], int(gone.sum()))
    d = (rng.standard_normal(M) / M).astype(np.float32)
    return X, W, torch.from_numpy(t), torch.from_numpy(d)


def guarded(n, dt, off=0):
    b = torch.full((n + 72 + off,), FILL, dtype=dt, device="cuda")
    return b, b[off:off + n]


def placed(x, off=0):
    b = torch.empty(x.numel() + 16, dtype=x.dtype, device="cuda")
    b[off:off + x.numel()].copy_(x.reshape(-1))
    return b[off:off + x.numel()]


def run(dtype, data, M, N, K, off=0, want=("dX", "dW")):
    X, W = (placed(x, off) for x in data[:2])
    t, d = data[2].cuda(), data[3].cuda()
    outs = {"loss": guarded(M, torch.float32) + ((M,),), "lse": guarded(M, torch.float32) + ((M,),)}
    g.gemm_cross_entropy(dtype, X, W, t, outs["loss"][1], outs["lse"][1], M, N, K)
    if want:
        outs |= {"dX": guarded(M * K, DT[dtype], off) + ((M, K),), "dW": guarded(N * K, DT[dtype], off) + ((N, K),)}
        outs = {k: v for k, v in outs.items() if k in ("loss", "lse") or k in want}
        g.gemm_cross_entropy_backward(dtype, X, W, t, outs["lse"][1], d, *(outs[k][1] if k in outs else None for k in ("dX", "dW")),
                                      M, N, K)
    g.gemm_synchronize()
    got = {}
    for k, (b, v, shape) in outs.items():
        o, n = (off if k[0] == "d" else 0), int(np.prod(shape))
        h = b.float().cpu()
        assert (h[:o] == FILL).all() and (h[o + n:] == FILL).all(), k
        got[k] = v.clone().reshape(shape)
    return got


def close(got, want, tol, name):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (name, int(bad.sum()), float((np.abs(got - want) / tol).max()))


def check(got, data, dtype):
    X, W, t, d = (x.double().numpy() if x.is_floating_point() else x.numpy() for x in data)
    loss, lse, _ = ref.forward(X, W, t)
    tl, te = ref.forward_tolerance(X, W, t)
    close(got["loss"], loss, tl, "loss")
    close(got["lse"], lse, te, "lse")
    if "dX" in got:
        dX, dW, _ = ref.backward(X, W, t, d)
        tX, tW = ref.backward_tolerance(X, W, t, d, dtype)
        close(got["dX"], dX, tX, "dX")
        close(got["dW"], dW, tW, "dW")


SHAPES = [(1, 1, 1), (1, 300, 64), (2, 1000, 128), (5, 257, 33), (64, 513, 200), (65, 128, 64), (130, 1001, 137),
          (257, 1000, 264), (300, 2999, 72), (129, 129, 1000), (700, 520, 520), (33, 20000, 40), (1, 33000, 256), (1500, 700, 96)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_loss_and_gradients(M, N, K, dtype):
    data = make(M, N, K, dtype, M + 3 * N + 7 * K, left_out=0.2 if M > 1 else 0.0)
    check(run(dtype, data, M, N, K), data, dtype)


@pytest.mark.parametrize("M", [31, 32, 64, 72, 96, 97, 127, 128, 129])
@pytest.mark.parametrize("N,K", [(257, 520), (21001, 72), (5000, 131)])
def test_rows_up_to_half_a_tile(M, N, K):
    data = make(M, N, K, "bf16", M + N, left_out=0.1)
    check(run("bf16", data, M, N, K), data, "bf16")


@pytest.mark.parametrize("M,N,K,off", [(3, 72, 40, 1), (200, 1000, 264, 3)])
def test_operands_off_16_bytes(M, N, K, off):
    """Every 16-bit operand off an aligned base: the aligned call's bits."""
    data = make(M, N, K, "bf16", 5)
    a, b = run("bf16", data, M, N, K), run("bf16", data, M, N, K, off)
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("M,N", [(1, 1000), (3, 17), (40, 3001), (129, 5000), (7, 8)])
@pytest.mark.parametrize("K,off", [(1, 0), (9, 1), (63, 0), (66, 3), (124, 0), (132, 5), (128, 1), (1001, 7)])
def test_rows_of_the_vocabulary_off_16_bytes(M, N, K, off):
    """Rows of one, two, four or eight alignments, whole tiles and parts of them."""
    data = make(M, N, K, "bf16", M + 3 * N + 7 * K, left_out=0.1 if M > 1 else 0.0)
    check(run("bf16", data, M, N, K, off), data, "bf16")


@pytest.mark.parametrize("K,off", [(1, 3), (2, 0), (2, 1), (2, 7), (4, 0), (4, 1), (4, 3), (6, 5), (7, 2), (12, 7)])
def test_few_hidden_units_off_16_bytes(K, off):
    """Rows shorter than the elements that may lie in front of them."""
    data = make(3, 2000, K, "bf16", K + off)
    check(run("bf16", data, 3, 2000, K, off), data, "bf16")


LARGE_OFF = [(1, 20000, 257, 0), (5, 33001, 131, 1), (3, 8200, 516, 3), (2, 9001, 514, 1), (16, 70001, 67, 0), (70, 72000, 68, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,off", LARGE_OFF)
def test_gradients_of_large_vocabularies_off_16_bytes(M, N, K, off, dtype):
    data = make(M, N, K, dtype, M + N + K, left_out=0.2 if M > 1 else 0.0)
    both = run(dtype, data, M, N, K, off)
    check(both, data, dtype)
    for k in ("dX", "dW"):
        assert torch.equal(run(dtype, data, M, N, K, off, want=(k,))[k], both[k]), k


@pytest.mark.parametrize("K", [57, 130, 1001])
def test_an_infinity_reaches_its_own_row_alone(K):
    """Rows of W that end, or begin, in infinities beside ones that do not: logits of -inf,
    which weigh as much as very small ones -- nothing."""
    M, N = 5, 1500
    X, W, t, d = make(M, N, K, "bf16", K)
    X[:, :8] = X[:, :8].abs() + 0.5
    X[:, -8:] = X[:, -8:].abs() + 0.5
    rows = torch.arange(3, N - 1, 7)
    t[:] = 0
    got = []
    for v in (-np.inf, -30000.0):
        W[rows, -7:] = v
        W[rows[::2], :7] = v
        got.append(run("bf16", (X, W, t, d), M, N, K, want=()))
    for k in ("loss", "lse"):
        assert torch.isfinite(got[0][k]).all()
        assert torch.equal(got[0][k], got[1][k]), k


@pytest.mark.parametrize("spread", [40.0, 300.0])
def test_large_logits(spread):
    data = make(70, 1000, 256, "bf16", 6, spread=spread)
    check(run("bf16", data, 70, 1000, 256), data, "bf16")


@pytest.mark.parametrize("weight", [1.0 / 777, 1.0 / 848, 0.3])
def test_a_common_weight_is_not_rounded(weight):
    """bf16: all rows weigh alike, by what bf16 does not hold (0.0012 to 0.0028 off), and the
    most of dZ is the targets' -weight (1 - p), p 1/4000 or so.  Scaled so that weight is a
    power of two it rounds to -weight for p < 2^-9: the gradients' projections on the right
    ones are 1 + p, 2.5e-4 and the rounding of many independent results, whose mean of 38400
    and more, 2^-9 at most each, is below 1e-4."""
    M, N, K = 300, 4000, 128
    X, W, t, _ = make(M, N, K, "bf16", 11, spread=0.5, left_out=0.0)
    d = torch.full((M,), weight, dtype=torch.float32)
    got = run("bf16", (X, W, t, d), M, N, K)
    dX, dW, _ = ref.backward(*(x.double().numpy() if x.is_floating_point() else x.numpy() for x in (X, W, t, d)))
    for k, want in (("dX", dX), ("dW", dW)):
        have = got[k].double().cpu().numpy()
        assert abs((have * want).sum() / (want * want).sum() - 1) < 5e-4, k


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 2.0 ** 14])
def test_weights_of_the_losses_from_tiny_to_large(scale):
    """Half precision: dZ keeps its precision whatever dloss is (results below half's
    range become its subnormals, or 0)."""
    X, W, t, d = make(60, 900, 64, "f16", 7)
    data = (X, W, t, d * np.float32(scale))
    check(run("f16", data, 60, 900, 64), data, "f16")


def test_rows_left_out_hold_anything():
    """NaN and infinities in rows without a target reach no gradient; lse has them."""
    M, N, K = 200, 700, 136
    X, W, t, d = make(M, N, K, "bf16", 8)
    gone = torch.from_numpy(~ref.counts(t.numpy(), N))
    clean = run("bf16", (X, W, t, d), M, N, K)
    X2, d2 = X.clone(), d.clone()
    X2[gone] = float("nan")
    X2[gone.nonzero()[0, 0]] = float("inf")
    d2[gone] = float("nan")
    got = run("bf16", (X2, W, t, d2), M, N, K)
    for k in ("loss", "dX", "dW"):
        assert torch.equal(got[k], clean[k]), k
    assert not got["dX"][gone.cuda()].any() and not got["loss"][gone.cuda()].any()
    keep = ~gone.cuda()
    assert torch.equal(got["lse"][keep], clean["lse"][keep]) and not torch.isfinite(got["lse"][~keep]).any()


def test_no_row_counts():
    M, N, K = 40, 300, 64
    X, W, t, d = make(M, N, K, "f16", 9)
    got = run("f16", (X, W, torch.full_like(t, -100), d), M, N, K)
    assert not got["loss"].any() and not got["dX"].any() and not got["dW"].any()


def test_infinite_and_nan_logits():
    """A row with a logit of +inf has lse +inf; of -inf, that entry counts for nothing; NaN stays."""
    N, K = 600, 64
    W = torch.zeros(N, K, dtype=torch.bfloat16)
    W[:, 0] = torch.linspace(-1, 1, N)
    W[300, 1] = 1.0
    X = torch.zeros(4, K, dtype=torch.bfloat16)
    X[:, 0] = 1.0
    X[0, 1], X[1, 1], X[2, 1] = 3e38, -3e38, float("nan")
    W[300, 1] = 3e38
    t = torch.tensor([5, 5, 5, 5])
    got = run("bf16", (X, W, t, torch.ones(4)), 4, N, K, want=())
    z = W[:, 0].double()
    rest = torch.logsumexp(z[torch.arange(N) != 300], 0)
    assert got["lse"][0] == float("inf") and got["loss"][0] == float("inf")
    assert abs(float(got["lse"][1]) - float(rest)) < 1e-5
    assert got["lse"][2].isnan() and got["loss"][2].isnan()
    assert abs(float(got["lse"][3]) - float(torch.logsumexp(z, 0))) < 1e-5


def test_one_gradient_alone_and_run_to_run():
    M, N, K = 300, 2000, 200
    data = make(M, N, K, "f16", 10)
    both, again = run("f16", data, M, N, K), run("f16", data, M, N, K)
    for k in both:
        assert torch.equal(both[k], again[k]), k
    for k in ("dX", "dW"):
        assert torch.equal(run("f16", data, M, N, K, want=(k,))[k], both[k]), k
    X, W, t, _ = (x.cuda() for x in data)
    loss = torch.empty(M, device="cuda")
    g.gemm_cross_entropy("f16", X, W, t, loss, None, M, N, K)
    g.gemm_synchronize()
    assert torch.equal(loss, both["loss"])


def sampled(M, N, K, dtype, seed, rows, columns):
    """Large problems: whole rows of loss, lse and dX, whole rows of dW."""
    data = make(M, N, K, dtype, seed, left_out=0.05)
    got = run(dtype, data, M, N, K)
    X, W, t, d = data
    r = np.unique(np.linspace(0, M - 1, rows).astype(int))
    part = (X[r], W, t[r], d[r])
    Xd, Wd, td, dd = X[r].double().numpy(), W.double().numpy(), t[r].numpy(), d[r].double().numpy()
    loss, lse, _ = ref.forward(Xd, Wd, td)
    tl, te = ref.forward_tolerance(Xd, Wd, td)
    close(got["loss"][r], loss, tl, "loss")
    close(got["lse"][r], lse, te, "lse")
    dX, _, _ = ref.backward(Xd, Wd, td, dd)
    if dtype == "f16":  # the scale comes from the largest weight of all rows
        dd = dd.copy()
    tX, _ = ref.backward_tolerance(Xd, Wd, td, dd, dtype)
    if dtype == "f16":
        tX = tX + 2.0 ** -39 * float(d.abs().max()) * np.abs(Wd).sum(0)
    close(got["dX"][r], dX, tX, "dX")
    # dW: lse of every row in 64 bits on the GPU, the chosen columns of dZ
    c = np.unique(np.linspace(0, N - 1, columns).astype(int))
    xg, wg = X.cuda().double(), W.cuda().double()
    every = torch.cat([torch.logsumexp(xg[i:i + 2048] @ wg.T, 1) for i in range(0, M, 2048)])
    ok = ((t >= 0) & (t < N)).cuda()
    P = torch.exp(xg @ wg[c].T - every[:, None])
    hit = t.cuda()[:, None] == torch.from_numpy(c).cuda()
    w8 = torch.where(ok, d.cuda().double(), 0)[:, None]
    dZ = (P - hit.double()) * w8
    want = dZ.T @ torch.where(ok[:, None], xg, 0)
    le = float(ref.logit_error(Xd, Wd).max()) * 2 + float(te.max())
    f = w8.abs() * (P * (le + 1e-5) + 1e-6 * dZ.abs() / w8.abs().clamp(min=1e-300)) + 2.0 ** -39 * float(d.abs().max())
    xa = torch.where(ok[:, None], xg, 0).abs()
    s = (M / 16 + 16) * 2.0 ** -23 * (dZ.abs().T @ xa)
    e = f.T @ xa + s + 8 * ref.ROUND[dtype] / 3 ** 0.5 * ((dZ * dZ).T @ (xa * xa)).sqrt()
    tol = e + ref.ROUND[dtype] * (want.abs() + e) + ref.TINY[dtype]
    off = (got["dW"][c].double() - want).abs()
    assert (off <= tol).all(), ("dW", float((off / tol).max()))


@pytest.mark.parametrize("M,N,K,dtype", [(16500, 9001, 64, "bf16"), (4, 140000, 1001, "bf16"), (40000, 300, 72, "f16"),
                                         (2048, 70001, 128, "f16")])
def test_pieces_of_rows_and_vocabulary(M, N, K, dtype):
    """More than one piece: of dZ, of padded rows of W, of the forward pass's rows, of dX's sums."""
    sampled(M, N, K, dtype, 11, 23, 17)
    torch.cuda.empty_cache()


def test_past_2_31_elements():
    """W of more than 2^31 elements, a few rows: lse and the gradients of its last entries
    equal those of a head without the zeros before them."""
    K, tail, M = 8192, 500, 3
    N = (1 << 31) // K + tail
    X, Wt, t, d = make(M, tail, K, "bf16", 12, left_out=0.0)
    W = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    W[-tail:].copy_(Wt)
    loss, lse, dX = torch.empty(M, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    dW = torch.empty_like(W)
    x, tt = X.cuda(), (t + N - tail).cuda()
    g.gemm_cross_entropy("bf16", x, W, tt, loss, lse, M, N, K)
    g.gemm_cross_entropy_backward("bf16", x, W, tt, lse, d.cuda(), dX, dW, M, N, K)
    g.gemm_synchronize()
    Xd, Wd, td, dd = X.double().numpy(), Wt.double().numpy(), t.numpy(), d.double().numpy()
    Z = Xd @ Wd.T
    want = np.log(np.exp(Z).sum(1) + (N - tail))
    assert np.allclose(lse.cpu().numpy(), want, rtol=1e-5)
    dZ = np.exp(Z - want[:, None])
    dZ[np.arange(M), td] -= 1
    dZ *= dd[:, None]
    for got, ex in ((dX, dZ @ Wd), (dW[-tail:], dZ.T @ Xd)):
        got = got.double().cpu().numpy()
        assert np.linalg.norm(got - ex) <= 0.01 * np.linalg.norm(ex)
    first = (np.exp(-want) * dd) @ Xd  # every entry before the tail has logit 0
    got = dW[[0, N // 2, N - tail - 1]].double().cpu().numpy()
    assert np.linalg.norm(got - first) <= 0.01 * np.linalg.norm(np.tile(first, (3, 1)))
    del W, dW
    torch.cuda.empty_cache()


def test_captured_and_replayed_beside_another_stream():
    """A step in a graph, replayed on new inputs while eager calls run on another stream:
    no scratch is shared."""
    M, N, K = 200, 1500, 136
    a, b = make(M, N, K, "f16", 13), make(M, N, K, "f16", 14)
    want = [run("f16", x, M, N, K) for x in (a, b)]
    bufs = [x.cuda() for x in a]
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dX, dW = torch.empty(M, K, dtype=torch.float16, device="cuda"), torch.empty(N, K, dtype=torch.float16, device="cuda")
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            g.gemm_cross_entropy("f16", bufs[0], bufs[1], bufs[2], loss, lse, M, N, K)
            g.gemm_cross_entropy_backward("f16", bufs[0], bufs[1], bufs[2], lse, bufs[3], dX, dW, M, N, K)
    eb = [x.cuda() for x in b]
    eo = [torch.empty_like(x) for x in (loss, lse, dX, dW)]
    torch.cuda.synchronize()
    for data, w in ((a, want[0]), (b, want[1]), (a, want[0])):
        with torch.cuda.stream(s):
            for x, v in zip(bufs, data):
                x.copy_(v)
            graph.replay()
        with torch.cuda.stream(other):
            g.gemm_cross_entropy("f16", eb[0], eb[1], eb[2], eo[0], eo[1], M, N, K)
            g.gemm_cross_entropy_backward("f16", eb[0], eb[1], eb[2], eo[1], eb[3], eo[2], eo[3], M, N, K)
        torch.cuda.synchronize()
        for k, x in zip(("loss", "lse", "dX", "dW"), (loss, lse, dX, dW)):
            assert torch.equal(x.reshape(w[k].shape), w[k]), k
        for k, x in zip(("loss", "lse", "dX", "dW"), eo):
            assert torch.equal(x.reshape(want[1][k].shape), want[1][k]), k


def test_captured_and_replayed_off_16_bytes():
    """Rows off 16 bytes, a large vocabulary, dW off another way than W: the same bits from a
    graph and beside it."""
    M, N, K = 5, 33001, 131
    a, b = make(M, N, K, "bf16", 15), make(M, N, K, "bf16", 16)
    want = [run("bf16", x, M, N, K) for x in (a, b)]
    bufs = [x.cuda() for x in a]
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dX, (whole, dW) = torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), guarded(N * K, torch.bfloat16, 5)
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            g.gemm_cross_entropy("bf16", bufs[0], bufs[1], bufs[2], loss, lse, M, N, K)
            g.gemm_cross_entropy_backward("bf16", bufs[0], bufs[1], bufs[2], lse, bufs[3], dX, dW, M, N, K)
    eb = [x.cuda() for x in b]
    eo = [torch.empty(n, dtype=dt, device="cuda") for n, dt in ((M, torch.float32), (M, torch.float32), (M * K, torch.bfloat16), (N * K, torch.bfloat16))]
    torch.cuda.synchronize()
    for data, w in ((a, want[0]), (b, want[1])):
        with torch.cuda.stream(s):
            for x, v in zip(bufs, data):
                x.copy_(v)
            graph.replay()
        with torch.cuda.stream(other):
            g.gemm_cross_entropy("bf16", eb[0], eb[1], eb[2], eo[0], eo[1], M, N, K)
            g.gemm_cross_entropy_backward("bf16", eb[0], eb[1], eb[2], eo[1], eb[3], eo[2], eo[3], M, N, K)
        torch.cuda.synchronize()
        for k, x, y in zip(("loss", "lse", "dX", "dW"), (loss, lse, dX, dW), eo):
            assert torch.equal(x.reshape(w[k].shape), w[k]), k
            assert torch.equal(y.reshape(w[k].shape), want[1][k]), k
        h = whole.float()
        assert (h[:5] == FILL).all() and (h[5 + N * K:] == FILL).all()


def test_past_2_31_elements_off_16_bytes():
    """The same of rows off 16 bytes: entries of zeros before the last 500."""
    K, tail, M = 8191, 500, 3
    N = (1 << 31) // K + tail
    X, Wt, t, d = make(M, tail, K, "bf16", 17, left_out=0.0)
    W = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    W[-tail:].copy_(Wt)
    loss, lse, dX = torch.empty(M, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    dW = torch.empty_like(W)
    x, tt = X.cuda(), (t + N - tail).cuda()
    g.gemm_cross_entropy("bf16", x, W, tt, loss, lse, M, N, K)
    g.gemm_cross_entropy_backward("bf16", x, W, tt, lse, d.cuda(), dX, dW, M, N, K)
    g.gemm_synchronize()
    Xd, Wd, td, dd = X.double().numpy(), Wt.double().numpy(), t.numpy(), d.double().numpy()
    Z = Xd @ Wd.T
    want = np.log(np.exp(Z).sum(1) + (N - tail))
    assert np.allclose(lse.cpu().numpy(), want, rtol=1e-5)
    dZ = np.exp(Z - want[:, None])
    dZ[np.arange(M), td] -= 1
    dZ *= dd[:, None]
    for got, ex in ((dX, dZ @ Wd), (dW[-tail:], dZ.T @ Xd)):
        got = got.double().cpu().numpy()
        assert np.linalg.norm(got - ex) <= 0.01 * np.linalg.norm(ex)
    first = (np.exp(-want) * dd) @ Xd
    got = dW[[0, N // 2, N - tail - 1]].double().cpu().numpy()
    assert np.linalg.norm(got - first) <= 0.01 * np.linalg.norm(np.tile(first, (3, 1)))
    del W, dW
    torch.cuda.empty_cache()


def test_pieces_of_rows_off_16_bytes():
    """More than 16384 rows against a vocabulary that is read in place: rows of both pieces."""
    M, N, K = 16400, 540001, 65
    X, W, t, _ = make(M, N, K, "bf16", 18, left_out=0.0)
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    g.gemm_cross_entropy("bf16", X.cuda(), W.cuda(), t.cuda(), loss, lse, M, N, K)
    g.gemm_synchronize()
    rows = torch.tensor([0, 1, 8000, 16383, 16384, 16399])
    Xr, tr = X[rows], t[rows]
    want, wlse, _ = ref.forward(Xr.double().numpy(), W.double().numpy(), tr.numpy())
    tl, te = ref.forward_tolerance(Xr.double().numpy(), W.double().numpy(), tr.numpy())
    close(loss[rows.cuda()], want, tl, "loss")
    close(lse[rows.cuda()], wlse, te, "lse")


def test_empty_sizes():
    """No hidden units: logits of 0; no vocabulary; no rows."""
    t, z = torch.tensor([3, -1, 9], device="cuda"), torch.empty(0, dtype=torch.bfloat16, device="cuda")
    loss, lse = torch.full((3,), FILL, device="cuda"), torch.full((3,), FILL, device="cuda")
    g.gemm_cross_entropy("bf16", z, z, t, loss, lse, 3, 8, 0)
    g.gemm_synchronize()
    assert np.allclose(loss.cpu(), [np.log(8), 0, 0]) and np.allclose(lse.cpu(), np.log(8))
    X, dX = torch.ones(3, 8, dtype=torch.bfloat16, device="cuda"), torch.ones(3, 8, dtype=torch.bfloat16, device="cuda")
    g.gemm_cross_entropy("bf16", X, z, t, loss, lse, 3, 0, 8)
    g.gemm_cross_entropy_backward("bf16", X, z, t, lse, loss, dX, z, 3, 0, 8)
    g.gemm_synchronize()
    assert not loss.any() and (lse == -float("inf")).all() and not dX.any()
    W, dW = torch.ones(4, 8, dtype=torch.bfloat16, device="cuda"), torch.ones(4, 8, dtype=torch.bfloat16, device="cuda")
    e, ti = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    g.gemm_cross_entropy_backward("bf16", z, W, ti, e, e, z, dW, 0, 4, 8)
    g.gemm_synchronize()
    assert not dW.any()
