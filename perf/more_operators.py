"""Cases of the operators around a language model's products: the root-mean-square
norm with the residual's addition (16-bit or E4M3 output, and its gradients), the
softmax cross entropy of a linear head over a large vocabulary with its gradients,
and the orthogonalised update of a weight matrix.

A case is one call (or one training step) as a user's program makes it, on
inputs that `prepare` makes from a seed.  `run` computes it in plain torch
operations (FP32, rounded once), or with the library's kernels where `own` is
set; `exact` evaluates the definitions in 64 bits.

  norm        H = X + R (rounded to the type), Y = w H / sqrt(mean(H^2) + eps)
  norm_e4m3   the same Y as E4M3 codes Q and a scale a row, amax |Y| / 448: Q = E4M3(Y / scale)
  norm_train  the norm, and from dY (of Y) and dH (of H, through the residual) the
              gradients dX (of X and R alike) and dw
  score       cross entropy of targets t under the logits Z = X W^T: lse(Z_i) - Z_i,t_i,
              0 where t_i is no index of the vocabulary; and lse
  head        the same, and dX and dW from the weights dloss of the rows' losses
  orth        G / |G|_F through five steps X <- a X + (b A + c A^2) X, A = X X^T
              (X^T X from the right where G is tall)
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
STEPS = 5
QUINTIC = (3.4445, -4.7750, 2.0315)
LEFT_OUT = -100  # the target of a row that does not count
LOSS_SCALE = {"bf16": 1.0, "f16": 65536.0}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token between two blocks of a model being served
        dict(name="norm_bf16_1x4096", op="norm", dtype="bf16", M=1, K=4096),
        # a decode batch ahead of an 8-bit product
        dict(name="norm_e4m3_f16_32x4096", op="norm_e4m3", dtype="f16", M=32, K=4096),
        # a long prompt ahead of an 8-bit product
        dict(name="norm_e4m3_bf16_8192x4096", op="norm_e4m3", dtype="bf16", M=8192, K=4096),
        # training steps: an odd small one, a long one
        dict(name="norm_train_f16_777x1001", op="norm_train", dtype="f16", M=777, K=1001),
        dict(name="norm_train_bf16_8192x4096", op="norm_train", dtype="bf16", M=8192, K=4096),
        # the log-likelihood of one next token
        dict(name="score_bf16_1x32000x4096", op="score", dtype="bf16", M=1, N=32000, K=4096),
        # training steps of the head: a small one over an odd vocabulary, an ordinary
        # micro-batch, a long one over a large vocabulary
        dict(name="head_f16_333x50257x1000", op="head", dtype="f16", M=333, N=50257, K=1000),
        dict(name="head_bf16_1024x32768x2048", op="head", dtype="bf16", M=1024, N=32768, K=2048),
        dict(name="head_bf16_4096x131072x4096", op="head", dtype="bf16", M=4096, N=131072, K=4096),
        # the update of a small projection, of an odd tall matrix, of the FFN's projection
        dict(name="orth_bf16_512x2048", op="orth", dtype="bf16", M=512, N=2048),
        dict(name="orth_f16_3001x1000", op="orth", dtype="f16", M=3001, N=1000),
        dict(name="orth_bf16_4096x12288", op="orth", dtype="bf16", M=4096, N=12288),
    ]


def _spread(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm_e4m3", "norm_train", "score", "head", "orth"])
    dtype = rng.choice(["bf16", "f16"])
    if op.startswith("norm"):
        return dict(op=op, dtype=dtype, M=_spread(rng, 1, 8192), K=_spread(rng, 64, 8192, rng.choice([1, 8])))
    if op in ("score", "head"):
        M = rng.choice([_spread(rng, 1, 64), _spread(rng, 1, 4096)])
        return dict(op=op, dtype=dtype, M=M, N=_spread(rng, 1000, 131072), K=_spread(rng, 64, 4096, rng.choice([1, 8])))
    M, N = _spread(rng, 32, 4096), _spread(rng, 32, 4096)
    return dict(op=op, dtype=dtype, M=M, N=N) if rng.random() < 0.5 else dict(op=op, dtype=dtype, M=M, N=min(3 * M, 12288))


def work(case):
    op, M = case["op"], case["M"]
    if op == "orth":  # symmetric products: half of their elements
        N = case["N"]
        m, n = min(M, N), max(M, N)
        return {"bytes": 2 * 2 * M * N, "flops": STEPS * (m * m * n + m ** 3 + 2 * m * m * n)}
    K = case["K"]
    if op == "norm":  # X, R, w; H, Y
        return {"bytes": 2 * (4 * M * K + K), "flops": 0}
    if op == "norm_e4m3":  # X, R, w; H, Q, scale
        return {"bytes": 2 * (3 * M * K + K) + M * K + 4 * M, "flops": 0}
    if op == "norm_train":  # X, R, w, dY, dH; H, Y, dX, dw
        return {"bytes": 2 * (7 * M * K + K) + 4 * K, "flops": 0}
    N = case["N"]
    if op == "score":  # X, W, targets; loss, lse
        return {"bytes": 2 * (M * K + N * K) + 16 * M, "flops": 2 * M * N * K}
    return {"bytes": 2 * 2 * (M * K + N * K) + 20 * M, "flops": 6 * M * N * K}


# ------------------------------------------------------------------ inputs
def _normal(shape, std, dtype, gen):
    return (torch.randn(shape, device="cuda", generator=gen) * std).to(dtype)


def _residual_stream(shape, dtype, gen):
    """N(0, 1) rows of different loudness with a few loud channels."""
    x = torch.randn(shape, device="cuda", generator=gen)
    loud = torch.rand(shape[-1], device="cuda", generator=gen) < 0.01
    rows = torch.exp(0.5 * torch.randn(shape[0], 1, device="cuda", generator=gen))
    return (torch.where(loud, x * 8.0, x) * rows).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M = case["op"], case["M"]
    dtype = DTYPES[case["dtype"]]
    st = dict(case)

    def out(*shape, t=dtype):
        return torch.empty(shape, dtype=t, device="cuda")

    if op == "orth":
        # a momentum: a few strong directions, and the rest of them weaker and weaker
        N = case["N"]
        r = min(M, N, 64)
        strong = torch.randn(M, r, device="cuda", generator=gen) * torch.logspace(0, -2, r, device="cuda")
        weak = torch.randn(M, N, device="cuda", generator=gen) * torch.logspace(0, -1, N, device="cuda")
        st["G"] = ((strong @ torch.randn(r, N, device="cuda", generator=gen) + 0.3 * weak) * 1e-4).to(dtype)
        st["G"] = (st["G"].float() * LOSS_SCALE[case["dtype"]]).to(dtype)
        st["O"] = out(M, N)
        return st
    K = case["K"]
    if op.startswith("norm"):
        st["X"] = _normal((M, K), 1.0, dtype, gen)  # a block's output
        st["R"] = _residual_stream((M, K), dtype, gen)
        st["w"] = (1.0 + 0.2 * torch.randn(K, device="cuda", generator=gen)).to(dtype)
        st["H"], st["Y"] = out(M, K), out(M, K)
        if op == "norm_e4m3":
            st["Q"], st["scale"] = out(M, K, t=torch.float8_e4m3fn), out(M, t=torch.float32)
        if op == "norm_train":
            st["dY"], st["dH"] = _normal((M, K), 1.0, dtype, gen), _normal((M, K), 1.0, dtype, gen)
            st["rstd"], st["dX"], st["dw"] = out(M, t=torch.float32), out(M, K), out(K, t=torch.float32)
        return st
    N = case["N"]
    st["W"] = _normal((N, K), 2.0 * K ** -0.5, dtype, gen)
    t = torch.randint(0, N, (M,), device="cuda", generator=gen)
    # a trained head: hidden states lean towards their target's row, some more than others
    lean = torch.rand(M, 1, device="cuda", generator=gen) * 2.0
    st["X"] = (torch.randn(M, K, device="cuda", generator=gen) + lean * st["W"][t].float()).to(dtype)
    padded = torch.rand(M, device="cuda", generator=gen) < 0.05
    padded[0] = False
    st["t"] = torch.where(padded, torch.full_like(t, LEFT_OUT), t)
    st["loss"], st["lse"] = out(M, t=torch.float32), out(M, t=torch.float32)
    if op == "head":
        # the mean over the rows that count (and half precision's loss scale)
        st["dloss"] = (~padded).float() * (LOSS_SCALE[case["dtype"]] / (~padded).sum())
        st["dX"], st["dW"] = out(M, K), out(N, K)
    return st


# ------------------------------------------------------------------ plain form
def _plain_norm(st):
    H = (st["X"].float() + st["R"].float()).to(st["X"].dtype)
    h, w = H.float(), st["w"].float()
    rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    if st["op"] == "norm":
        return {"H": H, "Y": (h * rstd * w).to(H.dtype)}
    if st["op"] == "norm_e4m3":
        # codes next to a border: in 64 bits
        d = H.double()
        y = d / torch.sqrt(d.square().mean(-1, keepdim=True) + EPS) * st["w"].double()
        scale = y.abs().amax(-1, keepdim=True) / 448.0
        q = torch.where(scale > 0, y / scale, torch.zeros_like(y)).clamp(-448.0, 448.0)
        return {"H": H, "Q": q.to(torch.float8_e4m3fn), "scale": scale[:, 0].float()}
    dy, xhat = st["dY"].float(), h * rstd
    wdy = dy * w
    dh = rstd * (wdy - xhat * (wdy * xhat).mean(-1, keepdim=True)) + st["dH"].float()
    return {"H": H, "Y": (xhat * w).to(H.dtype), "dX": dh.to(H.dtype), "dw": (dy * xhat).double().sum(0).float()}


def _plain_head(st):
    X, W, t = st["X"].float(), st["W"].float(), st["t"]
    Z = X @ W.T
    top = Z.amax(-1, keepdim=True)
    E = torch.exp(Z - top)
    total = E.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    counts = (t >= 0) & (t < W.shape[0])
    at = torch.where(counts, t, 0)[:, None]
    loss = torch.where(counts, lse - Z.gather(1, at)[:, 0], 0.0)
    if st["op"] == "score":
        return {"loss": loss, "lse": lse}
    D = E / total
    D.scatter_add_(1, at, torch.full_like(total, -1.0))
    D *= torch.where(counts, st["dloss"], 0.0)[:, None]
    return {"loss": loss, "lse": lse, "dX": (D @ W).to(st["X"].dtype), "dW": (D.T @ X).to(st["X"].dtype)}


def _plain_orth(st):
    a, b, c = QUINTIC
    G = st["G"].float()
    X = G / torch.sqrt(st["G"].double().square().sum()).float()
    X = X.T if X.shape[0] > X.shape[1] else X
    for _ in range(STEPS):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.T if G.shape[0] > G.shape[1] else X).to(st["G"].dtype).contiguous()


# ------------------------------------------------------------------ the library's operators
def _own(st):
    import dense_matrix_multiply_gb300 as gemm

    op, M, dtype = st["op"], st["M"], st["dtype"]
    if op == "orth":
        N = st["N"]
        gemm.gemm_orthogonalize(dtype, st["G"], N, st["O"], N, STEPS, M, N, QUINTIC)
        return st["O"]
    K = st["K"]
    if op == "norm":
        gemm.gemm_rms_norm(dtype, st["X"], st["R"], st["w"], EPS, st["H"], st["Y"], None, M, K)
        return {"H": st["H"], "Y": st["Y"]}
    if op == "norm_e4m3":
        gemm.gemm_rms_norm_e4m3(dtype, st["X"], st["R"], st["w"], EPS, st["H"], st["Q"], st["scale"], M, K)
        return {"H": st["H"], "Q": st["Q"], "scale": st["scale"]}
    if op == "norm_train":
        gemm.gemm_rms_norm(dtype, st["X"], st["R"], st["w"], EPS, st["H"], st["Y"], st["rstd"], M, K)
        gemm.gemm_rms_norm_backward(dtype, st["H"], st["w"], st["rstd"], st["dY"], st["dH"], st["dX"], st["dw"], M, K)
        return {"H": st["H"], "Y": st["Y"], "dX": st["dX"], "dw": st["dw"]}
    N = st["N"]
    gemm.gemm_cross_entropy(dtype, st["X"], st["W"], st["t"], st["loss"], st["lse"], M, N, K)
    if op == "score":
        return {"loss": st["loss"], "lse": st["lse"]}
    gemm.gemm_cross_entropy_backward(dtype, st["X"], st["W"], st["t"], st["lse"], st["dloss"], st["dX"], st["dW"], M, N, K)
    return {"loss": st["loss"], "lse": st["lse"], "dX": st["dX"], "dW": st["dW"]}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    return _plain_orth(state) if op == "orth" else _plain_norm(state) if op.startswith("norm") else _plain_head(state)


# ------------------------------------------------------------------ 64 bits
def _e4m3_64(v):
    """The E4M3 values nearest to v, |v| <= 448: steps of 2^(e - 3), 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3.0)
    return torch.round(v / step) * step  # torch.round: ties to even, as the code's last bit


def _exact_norm(st):
    H = (st["X"].double() + st["R"].double()).to(st["X"].dtype).double()
    w, K = st["w"].double(), st["K"]
    rms = torch.sqrt(torch.einsum("ik,ik->i", H, H) / K + EPS)
    Y = H * w / rms[:, None]
    if st["op"] == "norm":
        return {"H": H, "Y": Y}
    if st["op"] == "norm_e4m3":
        scale = Y.abs().max(1).values / 448.0
        return {"H": H, "Q": _e4m3_64((Y / scale[:, None]).clamp(-448.0, 448.0)), "scale": scale}
    dY = st["dY"].double()
    along = torch.einsum("ik,k,ik->i", dY, w, H)  # of the gradient, on H
    dX = dY * w / rms[:, None] - H * (along / (K * rms ** 3))[:, None] + st["dH"].double()
    return {"H": H, "Y": Y, "dX": dX, "dw": torch.einsum("ik,ik,i->k", dY, H, 1.0 / rms)}


def _exact_head(st):
    X, t, M, N = st["X"].double(), st["t"], st["M"], st["N"]
    step = max(1, (1 << 28) // M)
    pieces = [(v, min(v + step, N)) for v in range(0, N, step)]
    lse = torch.full((M,), -math.inf, dtype=torch.float64, device="cuda")
    for lo, hi in pieces:
        lse = torch.logaddexp(lse, torch.logsumexp(torch.matmul(X, st["W"][lo:hi].double().mT), 1))
    counts = t != LEFT_OUT
    picked = torch.einsum("ik,ik->i", X, st["W"][t.clamp(min=0)].double())
    loss = torch.where(counts, lse - picked, torch.zeros_like(lse))
    if st["op"] == "score":
        return {"loss": loss, "lse": lse}
    weight = torch.where(counts, st["dloss"].double(), torch.zeros_like(lse))
    dX, dW = torch.zeros_like(X), torch.zeros(st["W"].shape, dtype=torch.float64, device="cuda")
    for lo, hi in pieces:
        W = st["W"][lo:hi].double()
        P = torch.exp(torch.matmul(X, W.mT) - lse[:, None])
        P = (P - (t[:, None] == torch.arange(lo, hi, device="cuda")).double()) * weight[:, None]
        dX += torch.matmul(P, W)
        dW[lo:hi] = torch.matmul(P.mT, X)
    return {"loss": loss, "lse": lse, "dX": dX, "dW": dW}


def _exact_orth(st):
    a, b, c = QUINTIC
    X = st["G"].double()
    X = X / torch.linalg.vector_norm(X)
    tall = X.shape[0] > X.shape[1]
    eye = torch.eye(min(X.shape), dtype=torch.float64, device="cuda")
    for _ in range(STEPS):
        A = torch.matmul(X.mT, X) if tall else torch.matmul(X, X.mT)
        P = a * eye + torch.matmul(b * eye + c * A, A)
        X = torch.matmul(X, P) if tall else torch.matmul(P, X)
    return X


def exact(case, seed):
    if case["op"] == "head" and case["M"] * case["N"] * case["K"] > 2.5e12:
        return None  # over 20 seconds
    st = prepare(case, seed)
    op = case["op"]
    return _exact_orth(st) if op == "orth" else _exact_norm(st) if op.startswith("norm") else _exact_head(st)
