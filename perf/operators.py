"""Cases of the 4-bit block-scaled operators and of the gated feed-forward block.

A case is one call (or one training step) as a user's program makes it, on
inputs that `prepare` makes from a seed.  `run` computes it in plain torch
operations (FP32, rounded once), or with the library's kernels where `own` is
set; `exact` evaluates the definitions in 64 bits.

The 4-bit formats.  A row is cut into blocks of consecutive k, each with a scale:
  mx: 32 elements, scale 2^e as an E8M0 byte (e + 127, 255 = NaN),
      e = clamp(floor(log2 amax) - 2, -127, 125);
  nv: 16 elements, E4M3 scale s = e4m3(amax / (6 g)) with an FP32 scale g of the
      whole tensor; the block's step is s g.
Codes are E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign), two to a byte, the even k
in the low half, rows padded to whole groups of 32 elements.  Scale bytes lie in
atoms of 128 rows x 4 blocks (512 bytes: row % 32, row / 32, block), the atoms of
256 k together, row tile after row tile.
"""

import math

import torch

own = False

BLOCK = {"mx": 32, "nv": 16}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # weights read back after quantisation, as a quantisation-aware step or a check of the weights does
        dict(name="roundtrip_mx_bf16_4096x4096", op="roundtrip", fmt="mx", dtype="bf16", M=4096, K=4096),
        # a short batch of odd activations, f16, nv
        dict(name="roundtrip_nv_f16_777x12300", op="roundtrip", fmt="nv", dtype="f16", M=777, K=12300),
        # the product alone, both sides quantised earlier: the large square
        dict(name="product_nv_bf16_8192", op="product", fmt="nv", dtype="bf16", M=8192, N=8192, K=8192),
        # a ragged product: no side a multiple of a tile
        dict(name="product_mx_f16_1000x1001x4100", op="product", fmt="mx", dtype="f16", M=1000, N=1001, K=4100),
        # one token through the FFN's up projection
        dict(name="linear_nv_bf16_1x12288x4096", op="linear", fmt="nv", dtype="bf16", M=1, N=12288, K=4096),
        # a decode batch through the FFN's down projection
        dict(name="linear_mx_bf16_32x4096x12288", op="linear", fmt="mx", dtype="bf16", M=32, N=4096, K=12288),
        # a prompt through the FFN's up projection
        dict(name="linear_nv_bf16_1024x12288x4096", op="linear", fmt="nv", dtype="bf16", M=1024, N=12288, K=4096),
        # one token through the gated projections
        dict(name="gated_silu_bf16_1x12288x4096", op="gated", act="silu", dtype="bf16", M=1, N=12288, K=4096),
        # a prompt of odd length, f16, GELU
        dict(name="gated_gelu_f16_777x11008x4096", op="gated", act="gelu", dtype="f16", M=777, N=11008, K=4096),
        # training steps: a small odd one, an ordinary micro-batch, a long one
        dict(name="train_gelu_f16_333x1000x1000", op="train", act="gelu", dtype="f16", M=333, N=1000, K=1000),
        dict(name="train_silu_bf16_1024x12288x4096", op="train", act="silu", dtype="bf16", M=1024, N=12288, K=4096),
        dict(name="train_silu_bf16_8192x12288x4096", op="train", act="silu", dtype="bf16", M=8192, N=12288, K=4096),
    ]


def _spread(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["roundtrip", "product", "linear", "gated", "train"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "roundtrip":
        return dict(op=op, fmt=rng.choice(["mx", "nv"]), dtype=dtype, M=_spread(rng, 16, 4096), K=_spread(rng, 64, 4096))
    if op == "product":
        return dict(op=op, fmt=rng.choice(["mx", "nv"]), dtype=dtype, M=_spread(rng, 1, 8192), N=_spread(rng, 64, 8192),
                    K=_spread(rng, 64, 8192))
    if op == "linear":
        M = rng.choice([_spread(rng, 1, 64), _spread(rng, 1, 1024)])
        return dict(op=op, fmt=rng.choice(["mx", "nv"]), dtype=dtype, M=M, N=_spread(rng, 256, 12288),
                    K=_spread(rng, 256, 4096))
    act = rng.choice(["silu", "gelu"])
    if op == "gated":
        M = rng.choice([_spread(rng, 1, 64), _spread(rng, 1, 1024)])
        return dict(op=op, act=act, dtype=dtype, M=M, N=_spread(rng, 256, 12288, 8), K=_spread(rng, 256, 4096, 8))
    return dict(op=op, act=act, dtype=dtype, M=_spread(rng, 1, 8192), N=_spread(rng, 256, 12288, 8),
                K=_spread(rng, 256, 4096, 8))


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "roundtrip":  # read A, write codes and scales and the values read back
        return {"bytes": M * K * (2 + 2 + 0.5 + 1.0 / BLOCK[case["fmt"]]), "flops": 0}
    N = case["N"]
    four = 0.5 + 1.0 / BLOCK[case["fmt"]] if "fmt" in case else 0
    if case["op"] == "product":
        return {"bytes": (M + N) * K * four + 2 * M * N, "flops": 2 * M * N * K}
    if case["op"] == "linear":
        return {"bytes": 2 * M * K + N * K * four + 2 * M * N, "flops": 2 * M * N * K}
    fwd = 2 * (M * K + 2 * K * N + M * N)
    if case["op"] == "gated":
        return {"bytes": fwd, "flops": 4 * M * N * K}
    # forward and backward: X, W, dZ read, Z, dX, dW written; the saved G and U are the step's own business
    return {"bytes": fwd + 2 * (M * N + M * K + 2 * K * N), "flops": 12 * M * N * K}


# ------------------------------------------------------------------ inputs
def _activations(shape, dtype, gen):
    """N(0, 1) rows with a few loud channels, as a normalised residual stream has."""
    x = torch.randn(shape, device="cuda", generator=gen)
    loud = torch.rand(shape[-1], device="cuda", generator=gen) < 0.01
    return torch.where(loud, x * 8.0, x).to(dtype)


def _normal(shape, std, dtype, gen):
    return (torch.randn(shape, device="cuda", generator=gen) * std).to(dtype)


def _scale_bytes(fmt, rows, K):
    return (rows + 127) // 128 * ((K + 255) // 256) * (32 * 1024 // BLOCK[fmt])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M, K = case["op"], case["M"], case["K"]
    dtype = DTYPES[case["dtype"]]
    st = dict(case)
    if op == "roundtrip":
        st["A"] = _activations((M, K), dtype, gen)
        st["g"] = _tensor_scale(case["fmt"], st["A"])
        st["Q"] = torch.empty(M, (K + 31) // 32 * 16, dtype=torch.uint8, device="cuda")
        st["S"] = torch.empty(_scale_bytes(case["fmt"], M, K), dtype=torch.uint8, device="cuda")
        st["out"] = torch.empty(M, K, dtype=dtype, device="cuda")
        return st
    N = case["N"]
    if op in ("product", "linear"):
        x = _activations((M, K), dtype, gen)
        w = _normal((N, K), K ** -0.5, dtype, gen)
        st["gx"], st["gw"] = _tensor_scale(case["fmt"], x), _tensor_scale(case["fmt"], w)
        st["Qw"], st["Sw"] = _quantize(case["fmt"], w, st["gw"])
        if op == "product":
            st["Qx"], st["Sx"] = _quantize(case["fmt"], x, st["gx"])
        else:
            st["X"] = x
        st["C"] = torch.empty(M, N, dtype=dtype, device="cuda")
        return st
    st["X"] = _activations((M, K), dtype, gen)
    st["Wg"] = _normal((K, N), K ** -0.5, dtype, gen)
    st["Wu"] = _normal((K, N), K ** -0.5, dtype, gen)
    st["Z"] = torch.empty(M, N, dtype=dtype, device="cuda")
    if op == "train":
        st["dZ"] = _normal((M, N), 1.0, dtype, gen)
        st["G"] = torch.empty(M, N, device="cuda")
        st["U"] = torch.empty(M, N, device="cuda")
        st["dX"] = torch.empty(M, K, dtype=dtype, device="cuda")
        st["dWg"] = torch.empty(K, N, dtype=dtype, device="cuda")
        st["dWu"] = torch.empty(K, N, dtype=dtype, device="cuda")
    return st


def _tensor_scale(fmt, a):
    """nv: calibrated so that the tensor's largest magnitude maps a little below
    448 * 6, as a scale taken from earlier batches does; mx has no such scale."""
    return (a.abs().max().float() * (math.pi / 3.0 / 2688.0)).reshape(1) if fmt == "nv" else None


# ------------------------------------------------------------------ plain form
def _round_e2m1(q):
    """Codes 0 .. 15 of FP32 values: nearest level, ties to the even code."""
    m = q.abs()
    code = (m > 0.25).to(torch.uint8)
    for i, t in enumerate((0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (m >= t).to(torch.uint8) if i % 2 == 0 else (m > t).to(torch.uint8)
    return code + 8 * (q < 0).to(torch.uint8)


def _power_of_two(e):
    """2^e as FP32, built from its bits (2^-127, below the normal range, is 0x400000)."""
    return torch.where(e > -127, (e + 127) << 23, 0x400000).to(torch.int32).view(torch.float32)


def _block_scales(fmt, a, g):
    """FP32 [M, blocks, B] blocks of a (zero padded to 256 k), their scale bytes and steps."""
    B, (M, K) = BLOCK[fmt], a.shape
    x = torch.zeros(M, (K + 255) // 256 * 256, device=a.device)
    x[:, :K] = a.float()
    x = x.reshape(M, -1, B)
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    if fmt == "mx":
        e = (torch.frexp(amax).exponent - 3).clamp(-127, 125)
        e = torch.where(amax > 0, e, -127)
        byte = torch.where(bad, 255, e + 127).to(torch.uint8)
        step = _power_of_two(e)
    else:
        s = (amax / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        byte = torch.where(bad, torch.full_like(s.view(torch.uint8), 127), s.view(torch.uint8))
        step = s.float() * g
    return x, byte, torch.where(bad, torch.zeros_like(step), step)


def _quantize(fmt, a, g):
    """Packed codes [M, ceil(K/32) * 16] and tiled scale bytes."""
    M, K = a.shape
    x, byte, step = _block_scales(fmt, a, g)
    q = torch.where(step[..., None] > 0, x / step[..., None], torch.zeros_like(x))
    code = _round_e2m1(q).reshape(M, -1)[:, : (K + 31) // 32 * 32]
    packed = code[:, 0::2] + 16 * code[:, 1::2]
    tiles = (M + 127) // 128
    full = torch.zeros(tiles * 128, byte.shape[1], dtype=torch.uint8, device=a.device)
    full[:M] = byte
    s = full.reshape(tiles, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)
    return packed.contiguous(), s


def _dequantize(fmt, Q, S, g, M, K):
    """FP32 values [M, K] of packed codes and tiled scale bytes."""
    B = BLOCK[fmt]
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=Q.device)
    v = levels[torch.stack((Q & 15, Q >> 4), -1).reshape(M, -1).int()]
    tiles = (M + 127) // 128
    byte = S.reshape(tiles, -1, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tiles * 128, -1)[:M, : v.shape[1] // B]
    if fmt == "mx":
        s = _power_of_two(byte.int().clamp(max=254) - 127)
        s = torch.where(byte == 255, torch.full_like(s, math.nan), s)
    else:
        s = byte.contiguous().view(torch.float8_e4m3fn).float()
    v = (v.reshape(M, -1, B) * s[..., None]).reshape(M, -1)[:, :K]
    return v * g if fmt == "nv" else v


def _act(act, g):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(act, g):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _plain(st):
    op, M, K = st["op"], st["M"], st["K"]
    dtype = DTYPES[st["dtype"]]
    if op == "roundtrip":
        Q, S = _quantize(st["fmt"], st["A"], st["g"])
        return _dequantize(st["fmt"], Q, S, st["g"], M, K).to(dtype)
    if op in ("product", "linear"):
        if op == "linear":
            Qx, Sx = _quantize(st["fmt"], st["X"], st["gx"])
        else:
            Qx, Sx = st["Qx"], st["Sx"]
        x = _dequantize(st["fmt"], Qx, Sx, st["gx"], M, K)
        w = _dequantize(st["fmt"], st["Qw"], st["Sw"], st["gw"], st["N"], K)
        return (x @ w.T).to(dtype)
    x, wg, wu = st["X"].float(), st["Wg"].float(), st["Wu"].float()
    g, u = x @ wg, x @ wu
    a = _act(st["act"], g)
    z = (a * u).to(dtype)
    if op == "gated":
        return z
    dz = st["dZ"].float()
    du = dz * a
    dg = dz * u * _act_grad(st["act"], g)
    return {"Z": z, "dX": (dg @ wg.T + du @ wu.T).to(dtype), "dWg": (x.T @ dg).to(dtype), "dWu": (x.T @ du).to(dtype)}


# ------------------------------------------------------------------ the library's operators
def _own(st):
    import dense_matrix_multiply_gb300 as gemm

    op, M, K, dtype = st["op"], st["M"], st["K"], st["dtype"]
    if op == "roundtrip":
        gemm.gemm_fp4_quantize(dtype, st["fmt"], st["A"], K, st["g"], st["Q"], st["S"], M, K)
        gemm.gemm_fp4_dequantize(dtype, st["fmt"], st["Q"], st["S"], st["g"], st["out"], K, M, K)
        return st["out"]
    N = st["N"]
    if op == "product":
        gemm.gemm_fp4(dtype, st["fmt"], st["Qx"], st["Sx"], st["gx"], st["Qw"], st["Sw"], st["gw"], st["C"], N, M, N, K)
        return st["C"]
    if op == "linear":
        gemm.gemm_fp4_linear(dtype, st["fmt"], st["X"], K, st["gx"], st["Qw"], st["Sw"], st["gw"], st["C"], N, M, N, K)
        return st["C"]
    if op == "gated":
        gemm.gemm_gated(dtype, st["act"], st["X"], st["Wg"], st["Wu"], st["Z"], None, None, M, N, K)
        return st["Z"]
    gemm.gemm_gated(dtype, st["act"], st["X"], st["Wg"], st["Wu"], st["Z"], st["G"], st["U"], M, N, K)
    gemm.gemm_gated_backward(dtype, st["act"], st["X"], st["Wg"], st["Wu"], st["G"], st["U"], st["dZ"], st["dX"],
                             st["dWg"], st["dWu"], M, N, K)
    return {"Z": st["Z"], "dX": st["dX"], "dWg": st["dWg"], "dWu": st["dWu"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _floor_power64(v):
    """The largest power of two not above v > 0."""
    return v / (2.0 * torch.frexp(v).mantissa)


def _values64(fmt, a, g):
    """The values that the quantised a stands for, from the definition in 64 bits."""
    B, (M, K) = BLOCK[fmt], a.shape
    x = torch.nn.functional.pad(a.double(), (0, -K % B)).reshape(M, -1, B)
    top = x.abs().amax(-1, keepdim=True)
    safe = torch.where(top > 0, top, torch.ones_like(top))
    if fmt == "mx":
        step = (_floor_power64(safe) / 4.0).clamp(min=2.0 ** -127)
    else:
        want = (safe / (6.0 * g.double())).clamp(max=448.0)
        ulp = _floor_power64(want).clamp(min=2.0 ** -6) / 8.0
        step = (torch.round(want / ulp) * ulp).clamp(max=448.0) * g.double()
    step = torch.where(top > 0, step, torch.zeros_like(step))
    q = torch.where(step > 0, x / step, torch.zeros_like(x))
    m = q.abs().clamp(max=6.0)
    grid = torch.where(m < 2.0, 0.5, torch.where(m < 4.0, 1.0, 2.0)).double()
    m = (torch.round(m / grid) * grid).clamp(max=6.0)  # torch.round: ties to even, as the code's last bit
    return (torch.sign(q) * m * step).reshape(M, -1)[:, :K]


def _read64(fmt, Q, S, g, M, K):
    """The same values from stored codes and scale bytes, element by element."""
    dev = Q.device
    k = torch.arange(K, device=dev)
    r = torch.arange(M, device=dev)[:, None]
    code = (Q[:, k // 2].int() >> (4 * (k % 2)).int()) & 15
    mag, sign = code & 7, 1.0 - 2.0 * (code >> 3).double()
    e, f = mag >> 1, (mag & 1).double()
    val = torch.where(e == 0, 0.5 * f, torch.exp2(e.double() - 1.0) * (1.0 + 0.5 * f))
    j = k // BLOCK[fmt]
    atoms = (K + 255) // 256 * 64 // BLOCK[fmt]
    byte = S[((r // 128) * atoms + j // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + j % 4].double()
    if fmt == "mx":
        return sign * val * torch.exp2(byte - 127.0)
    ee, ff = torch.floor(byte / 8.0), byte % 8.0
    s = torch.where(ee == 0, ff * 2.0 ** -9, torch.exp2(ee - 7.0) * (1.0 + ff / 8.0))
    return sign * val * s * g.double()


def exact(case, seed):
    st = prepare(case, seed)
    op, M, K = case["op"], case["M"], case["K"]
    if op == "roundtrip":
        return _values64(case["fmt"], st["A"], st["g"])
    N = case["N"]
    if op in ("product", "linear"):
        fmt = case["fmt"]
        w = _read64(fmt, st["Qw"], st["Sw"], st["gw"], N, K)
        x = _read64(fmt, st["Qx"], st["Sx"], st["gx"], M, K) if op == "product" else _values64(fmt, st["X"], st["gx"])
        return torch.matmul(x, w.mT)
    x, wg, wu = st["X"].double(), st["Wg"].double(), st["Wu"].double()
    G, U = torch.matmul(x, wg), torch.matmul(x, wu)
    if case["act"] == "silu":
        sig = torch.sigmoid(G)
        A, D = G * sig, sig + G * sig * (1.0 - sig)
    else:
        c, c3 = math.sqrt(2.0 / math.pi), 0.044715
        th = torch.tanh(c * G + c * c3 * G ** 3)
        A = 0.5 * G + 0.5 * G * th
        D = 0.5 + 0.5 * th + 0.5 * G * (1.0 - th ** 2) * (c + 3.0 * c * c3 * G ** 2)
    if op == "gated":
        return A * U
    dZ = st["dZ"].double()
    dU, dG = dZ * A, dZ * U * D
    return {"Z": A * U, "dX": torch.matmul(dG, wg.mT) + torch.matmul(dU, wu.mT), "dWg": torch.matmul(x.mT, dG),
            "dWu": torch.matmul(x.mT, dU)}
