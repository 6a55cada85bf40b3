"""The orthogonalised update on the GPU, through the C ABI, against 64-bit values within
orth_ref's tolerances."""

import numpy as np
import pytest
import torch

import orth_ref as ref

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
FILL = 77.0


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def make(M, N, dtype, seed, kind="noise"):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, N))
    if kind == "strong":  # eight directions above the noise
        r = min(M, N, 8)
        x = 0.1 * x + rng.standard_normal((M, r)) @ rng.standard_normal((r, N))
    if kind == "fading":  # rows and columns ever weaker
        x *= np.logspace(0, -2, M)[:, None] * np.logspace(0, -1, N)
    return torch.from_numpy((x * 0.01).astype(np.float32)).to(DT[dtype])


def run(dtype, G, steps, off=0, ldg=None, ldo=None, in_place=False, coefficients=ref.QUINTIC):
    """The result, with what lies around and between O's rows checked."""
    M, N = G.shape
    ldg, ldo = ldg or N, ldo or N
    gb = torch.full((M * ldg + 64,), float("nan"), dtype=DT[dtype], device="cuda")
    src = gb[off:off + M * ldg].view(M, ldg)
    src[:, :N] = G.cuda()
    if in_place:
        ob, ldo = gb, ldg
    else:
        ob = torch.full((M * ldo + 64,), FILL, dtype=DT[dtype], device="cuda")
    dst = ob[off:off + M * ldo]
    g.gemm_orthogonalize(dtype, gb[off:off + M * ldg], ldg, dst, ldo, steps, M, N, coefficients)
    g.gemm_synchronize()
    if not in_place:
        around = torch.cat([ob[:off], ob[off + (M - 1) * ldo + N:], dst.view(M, ldo)[:-1, N:].reshape(-1)])
        assert (around == FILL).all()
    return dst.view(M, ldo)[:, :N].clone()


def check(dtype, G, steps, got):
    got, Gd = got.double().cpu().numpy(), G.double().numpy()
    want = ref.orthogonalize(Gd, steps)
    if steps == 1:
        tol = ref.one_step_tolerance(Gd, dtype)
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (int(bad.sum()), float((np.abs(got - want) / tol).max()))
    off, tol = np.linalg.norm(got - want), ref.frobenius_tolerance(Gd, steps, dtype)
    assert off <= tol, (off, tol, np.linalg.norm(want))


SHAPES = [(1, 1), (1, 100), (100, 1), (7, 5), (64, 64), (65, 129), (33, 1000), (1000, 33), (256, 256), (257, 300), (300, 257),
          (520, 520), (513, 1100), (1100, 513)]


@pytest.mark.parametrize("steps", [1, 5])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", SHAPES)
def test_steps(M, N, dtype, steps):
    G = make(M, N, dtype, M + 3 * N, ("noise", "strong", "fading")[(M + N) % 3])
    check(dtype, G, steps, run(dtype, G, steps))


@pytest.mark.parametrize("kind", ["noise", "strong", "fading"])
@pytest.mark.parametrize("steps", [2, 3, 5, 9])
def test_spectra(kind, steps):
    G = make(300, 700, "bf16", 5, kind)
    check("bf16", G, steps, run("bf16", G, steps))


def test_large():
    """More tiles than clusters in every product."""
    G = make(2900, 4100, "bf16", 6, "strong")
    got = run("bf16", G, 2).double()
    a, b, c = ref.QUINTIC
    X = G.cuda().double()
    X = X / X.norm()
    for _ in range(2):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    # as frobenius_tolerance, with |A|_F <= |X|_F |X|_2, |X|_2 <= 1.2, B's values at most 5 and
    # L <= 3.9 (the first step adds no more than the second)
    add = (2 * ref.H / 3 ** 0.5 * (abs(b) + 2 * c * 1.44 + 5) + ref.H * 5) * 1.2 * float(X.norm())
    tol = add * (1 + 3.9) + 2.0 ** -8 * float(X.norm())
    assert float((got - X).norm()) <= tol


@pytest.mark.parametrize("M,N", [(70, 136), (200, 72), (70, 131), (3, 129), (300, 257)])
def test_alignment_and_leading_dimensions(M, N):
    """Rows anywhere: the tight aligned call's bits, nothing but O's elements written."""
    G = make(M, N, "bf16", 7)
    want = run("bf16", G, 5)
    up = (N + 7) // 8 * 8
    for off, ldg, ldo in ((0, up, up), (0, N, up + 8), (1, N, N), (0, N + 3, N + 8), (0, N + 8, N + 5), (8, N + 64, N + 1), (3, N + 1, N + 1)):
        assert torch.equal(run("bf16", G, 5, off, ldg, ldo), want), (off, ldg, ldo)
    assert torch.equal(run("bf16", G, 5, in_place=True), want)
    row = G[:1].cuda().contiguous()
    one, far = torch.empty(N, dtype=torch.bfloat16, device="cuda"), torch.empty(N, dtype=torch.bfloat16, device="cuda")
    g.gemm_orthogonalize("bf16", row.reshape(-1), N, one, N, 5, 1, N)
    g.gemm_orthogonalize("bf16", row.reshape(-1), 1 << 45, far, 1 << 50, 5, 1, N)  # a single row: never stepped by
    g.gemm_synchronize()
    assert torch.equal(one, far)
    assert torch.equal(run("bf16", G, 5, 1, N + 3, in_place=True), want)


@pytest.mark.parametrize("dtype,scales", [("bf16", (1e-30, 1e-3, 1e35)), ("f16", (1e-3, 1.0, 3e5))])
def test_any_magnitude(dtype, scales):
    """The result depends on G's direction only: powers of two give the same bits, and
    squares past FP32's range lose nothing."""
    G = make(90, 130, dtype, 8)
    want = run(dtype, G, 5)
    for s in scales:
        k = 2.0 ** round(np.log2(s))
        scaled = (G.double() * k).to(DT[dtype])
        if torch.equal(scaled.double(), G.double() * k):
            assert torch.equal(run(dtype, scaled, 5), want), s
        else:
            check(dtype, scaled, 5, run(dtype, scaled, 5))


def test_zeros_nan_and_infinities():
    z = torch.zeros(40, 70, dtype=torch.bfloat16)
    assert not run("bf16", z, 5).any()
    for v in (float("nan"), float("inf"), -float("inf")):
        x = make(40, 70, "bf16", 9)
        x[39, 69] = v
        assert run("bf16", x, 5).isnan().all()
    one = torch.zeros(40, 70, dtype=torch.bfloat16)
    one[3, 5] = -1e-38
    got = run("bf16", one, 5).double().cpu().numpy()
    want = ref.orthogonalize(one.double().numpy(), 5)
    assert abs(got[3, 5] - want[3, 5]) <= 0.01 and np.count_nonzero(got) == 1


def test_other_coefficients():
    """The cubic that converges: 1.5 x - 0.5 x^3, to the orthogonal factor itself."""
    G = make(64, 200, "f16", 10)
    got = run("f16", G, 25, coefficients=(1.5, -0.5, 0.0)).double().cpu().numpy()
    U, _, V = np.linalg.svd(G.double().numpy(), full_matrices=False)
    # the last steps' roundings: A and hi in B X (2^-11 each, |b| = 1/2), the result's
    assert np.linalg.norm(got - U @ V) <= (2 * 2.0 ** -11 + 2.0 ** -11) * 8 * 2


def test_run_to_run_and_replayed():
    a, b = make(300, 520, "bf16", 11), make(300, 520, "bf16", 12)
    want = [run("bf16", x, 5) for x in (a, b)]
    assert torch.equal(run("bf16", a, 5), want[0])
    G, O = a.cuda(), torch.empty(300, 520, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            g.gemm_orthogonalize("bf16", G, 520, O, 520, 5, 300, 520)
        for x, w in ((b, want[1]), (a, want[0]), (b, want[1])):
            G.copy_(x)
            O.fill_(FILL)
            graph.replay()
            assert torch.equal(O, w)
    torch.cuda.synchronize()


def test_two_streams_at_once():
    a, b = make(520, 900, "bf16", 13), make(900, 520, "bf16", 14)
    want = [run("bf16", x, 5) for x in (a, b)]
    bufs = [(x.cuda(), torch.empty_like(x, device="cuda"), torch.cuda.Stream()) for x in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, o, s in bufs:
            with torch.cuda.stream(s):
                g.gemm_orthogonalize("bf16", x, x.shape[1], o, x.shape[1], 5, *x.shape)
    torch.cuda.synchronize()
    for (_, o, _), w in zip(bufs, want):
        assert torch.equal(o, w)


def test_long_rows_and_strides_past_2_31():
    """A row stride that takes G past 2^31 elements, and rows of 2^20 elements."""
    ld = (1 << 30) + 64
    big = torch.empty(2 * ld + 200, dtype=torch.bfloat16, device="cuda")
    G = make(3, 200, "bf16", 15)
    for i in range(3):
        big[i * ld:i * ld + 200] = G[i].cuda()
    O = torch.empty(3, 200, dtype=torch.bfloat16, device="cuda")
    g.gemm_orthogonalize("bf16", big, ld, O, 200, 5, 3, 200)
    g.gemm_orthogonalize("bf16", big, ld, big, ld, 5, 3, 200)
    g.gemm_synchronize()
    want = run("bf16", G, 5)
    assert torch.equal(O, want)
    assert all(torch.equal(big[i * ld:i * ld + 200], want[i]) for i in range(3))
    del big
    torch.cuda.empty_cache()
    G = make(2, (1 << 20) + 3, "f16", 16)
    check("f16", G, 5, run("f16", G, 5))
