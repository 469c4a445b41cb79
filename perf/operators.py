"""The operators of the 8-bit floating-point layer, as they are measured.

Four calls make up an MLP or projection of a transformer whose linear layers hold E4M3 codes
with one power-of-two scale (E8M0 byte) for each block of 128 elements along K:

    norm      h = bf16(x + residual);  y = h * rsqrt(mean(h^2) + eps) * gamma  -> codes, scales
    glu       y = act(gate) [* up] [/ lambda]                                  -> codes, scales
    quantize  y = bf16(x / lambda)  -> codes, scales, and Z = bf16(y L1^T)
    gemm      Y = bf16(dequant(A) dequant(W)^T + Z L2^T + bias)

The block scale is 2^e with the smallest e >= -127 for which max|y| <= 448 * 2^e, so that no
code saturates; the codes are y / 2^e rounded to E4M3.  Scale bytes (e + 127) lie in blocks of
128 rows x 4 groups; the bytes of padding rows and padding groups are 0.
"""
import torch

own = False

G = 128                       # elements per scale
NORM, GLU, QUANT, GEMM = "norm", "glu", "quantize", "gemm"
_MAX_MNK = 4608 * 3072 * 12288
_MAX_ELEMS = 4608 * 12288


def listed():
    return [
        # one token of a conditioning stream through the norm before a projection: latency
        dict(name="norm_one_token", op=NORM, M=1, K=3072, residual=True),
        # a short odd batch, K = 9 groups (a scale block that is not full), no residual
        dict(name="norm_ragged", op=NORM, M=333, K=1152, residual=False),
        # the 4608 image and text tokens of the diffusion transformer before its fused QKV layer
        dict(name="norm_dit", op=NORM, M=4608, K=3072, residual=True),
        # the same width at the largest token count of the layer sweep
        dict(name="norm_batch", op=NORM, M=16384, K=3072, residual=True),
        # a gated SiLU on an odd batch; gate and up are column slices of one wider output
        dict(name="glu_silu_ragged", op=GLU, M=1000, K=2432, act="silu", gated=True, lam=False, pad=384),
        # GELU between MLP-up and MLP-down, with the smoothing factors of the second layer
        dict(name="glu_gelu_dit", op=GLU, M=4608, K=12288, act="gelu", gated=False, lam=True, pad=0),
        # a small batch into a layer that keeps a low-rank branch
        dict(name="quantize_small", op=QUANT, M=77, K=2048, rank=16, lam=True),
        # the QKV layer's input with a rank-32 branch
        dict(name="quantize_dit", op=QUANT, M=4608, K=3072, rank=32, lam=True),
        # one token through the fused QKV layer: the weights are read once
        dict(name="gemm_one_token", op=GEMM, M=1, N=9216, K=3072, rank=0, bias=True),
        # odd sizes: 17 groups along K, half a tile along N
        dict(name="gemm_ragged", op=GEMM, M=300, N=1152, K=2176, rank=16, bias=True),
        # MLP-up of the diffusion transformer with a rank-32 branch
        dict(name="gemm_mlp_up", op=GEMM, M=4608, N=12288, K=3072, rank=32, bias=True),
        # MLP-down, K-heavy, without the branch
        dict(name="gemm_mlp_down", op=GEMM, M=4608, N=3072, K=12288, rank=0, bias=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice([NORM, GLU, QUANT, GEMM, GEMM])
    M = _log_int(rng, 1, 16384)
    K = G * _log_int(rng, 1, 96)
    if op == GEMM:
        N = G * _log_int(rng, 1, 96)
        M = max(1, min(M, _MAX_MNK // (N * K)))
        return dict(op=op, M=M, N=N, K=K, rank=16 * rng.randrange(0, 5), bias=rng.random() < 0.5)
    M = max(1, min(M, _MAX_ELEMS // K))
    if op == NORM:
        return dict(op=op, M=M, K=K, residual=rng.random() < 0.5)
    if op == QUANT:
        return dict(op=op, M=M, K=K, rank=16 * rng.randrange(0, 5), lam=rng.random() < 0.5)
    return dict(op=op, M=max(1, M // 2), K=K, act=rng.choice(["silu", "gelu"]), gated=rng.random() < 0.5,
                lam=rng.random() < 0.5, pad=8 * rng.randrange(0, 64))


# ----------------------------------------------------------------- sizes and the scale layout

def _rows_pad(rows):
    return (rows + 127) // 128 * 128


def _groups_pad(K):
    return (K // G + 3) // 4 * 4


def _scale_bytes(rows, K):
    return _rows_pad(rows) * _groups_pad(K)


def _block(s):
    """Scale bytes [rows][K/128] -> the 128x4 blocked layout, flat; padding is 0."""
    rows, g = s.shape
    rp, gp = _rows_pad(rows), (g + 3) // 4 * 4
    full = torch.zeros((rp, gp), dtype=s.dtype, device=s.device)
    full[:rows, :g] = s
    return full.view(rp // 128, 4, 32, gp // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _unblock(b, rows, K):
    rp, gp = _rows_pad(rows), _groups_pad(K)
    return b.view(rp // 128, gp // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rp, gp)[:rows, : K // G]


def _exponent(a):
    """The smallest e >= -127 with a <= 448 * 2^e (0.875 * 2^9 = 448); -127 for a = 0."""
    m, ex = torch.frexp(a)
    return torch.where(a > 0, torch.clamp(ex - 9 + (m > 0.875), min=-127), -127)


def _pow2(e):
    """2^e in 64 bits for whole e in -1022 .. 1023, exact."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


# ----------------------------------------------------------------- inputs

def _acts(M, K, g, dev):
    """bf16 activations: N(0, 1) with 1 % of the channels 30 times as large."""
    x = torch.randn((M, K), generator=g, device=dev)
    out = torch.rand((K,), generator=g, device=dev) < 0.01
    return torch.where(out, 30.0 * x, x).to(torch.bfloat16)


def _codes(x):
    """A matrix quantized as a weight pack does: uint8 codes [rows][K], scale bytes in blocks."""
    rows, K = x.shape
    xg = x.float().view(rows, K // G, G)
    e = _exponent(xg.abs().amax(2))
    q = (xg.double() * _pow2(-e)[..., None]).float().to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(rows, K), _block((e + 127).to(torch.uint8))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, M, K = case["op"], case["M"], case["K"]
    st = dict(case)
    rank = case.get("rank", 0)
    if op == GEMM:
        N = case["N"]
        st["a_codes"], st["a_scales"] = _codes(_acts(M, K, g, dev))
        st["w_codes"], st["w_scales"] = _codes(0.02 * torch.randn((N, K), generator=g, device=dev))
        st["Z"] = st["L2"] = st["b"] = None
        if rank:
            st["Z"] = torch.randn((M, rank), generator=g, device=dev).to(torch.bfloat16)
            st["L2"] = (0.5 * torch.randn((N, rank), generator=g, device=dev)).to(torch.bfloat16)
        if case["bias"]:
            st["b"] = torch.randn((N,), generator=g, device=dev).to(torch.bfloat16)
        st["Y"] = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        return st
    st["codes"] = torch.empty((M * K,), dtype=torch.uint8, device=dev)
    st["scales"] = torch.empty((_scale_bytes(M, K),), dtype=torch.uint8, device=dev)
    st["lambda"] = st["L1"] = st["Z"] = None
    if case.get("lam"):
        st["lambda"] = torch.exp(torch.randn((K,), generator=g, device=dev))
    if op == NORM:
        st["X"] = _acts(M, K, g, dev)
        st["gamma"] = 1.0 + 0.2 * torch.randn((K,), generator=g, device=dev)
        st["R"] = st["H"] = None
        if case["residual"]:
            st["R"] = _acts(M, K, g, dev)
            st["H"] = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    elif op == GLU:
        wide = _acts(M, K * (2 if case["gated"] else 1) + case["pad"], g, dev)
        st["gate"] = wide[:, case["pad"]: case["pad"] + K]
        st["up"] = wide[:, case["pad"] + K:] if case["gated"] else None
    else:
        st["X"] = _acts(M, K, g, dev)
        if rank:
            st["L1"] = (0.05 * torch.randn((rank, K), generator=g, device=dev)).to(torch.bfloat16)
            st["Z"] = torch.empty((M, rank), dtype=torch.bfloat16, device=dev)
    return st


# ----------------------------------------------------------------- the plain forms

def _quantize(y):
    """Rounded to E4M3 once, in blocks of 128: codes (as their values) and scales (E8M0)."""
    M, K = y.shape
    yg = y.view(M, K // G, G)
    e = _exponent(yg.abs().amax(2))
    # two factors: 2^-e itself leaves the range of 32 bits where e = -127
    half = torch.div(-e, 2, rounding_mode="floor")
    q = yg * torch.exp2(half.float())[..., None] * torch.exp2((-e - half).float())[..., None]
    return q.view(M, K).to(torch.float8_e4m3fn), _block((e + 127).to(torch.uint8)).view(torch.float8_e8m0fnu)


def _act(x, act):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    u = 0.7978845608028654 * (x + 0.044715 * x * x * x)      # tanh form, as x * sigmoid(2u)
    return x / (1.0 + torch.exp(-2.0 * u))


def _dequant(codes, scales, K):
    rows = codes.shape[0]
    s = torch.exp2(_unblock(scales, rows, K).float() - 127.0)
    return (codes.view(torch.float8_e4m3fn).float().view(rows, K // G, G) * s[..., None]).view(rows, K)


def _plain(st):
    op = st["op"]
    if op == NORM:
        h = st["X"]
        if st["R"] is not None:
            h = (h.float() + st["R"].float()).to(torch.bfloat16)
        f = h.float()
        y = f * (1.0 / torch.sqrt((f * f).mean(1, keepdim=True) + 1e-6)) * st["gamma"]
        codes, scales = _quantize(y)
        return [codes, scales] + ([h] if st["R"] is not None else [])
    if op == GLU:
        y = _act(st["gate"].float(), st["act"])
        if st["gated"]:
            y = y * st["up"].float()
        if st["lambda"] is not None:
            y = y / st["lambda"]
        return list(_quantize(y))
    if op == QUANT:
        y = st["X"]
        if st["lambda"] is not None:
            y = (y.float() / st["lambda"]).to(torch.bfloat16)
        y = y.float()
        z = [(y @ st["L1"].float().t()).to(torch.bfloat16)] if st["L1"] is not None else []
        return list(_quantize(y)) + z
    K = st["K"]
    y = _dequant(st["a_codes"], st["a_scales"], K) @ _dequant(st["w_codes"], st["w_scales"], K).t()
    if st["Z"] is not None:
        y = y + st["Z"].float() @ st["L2"].float().t()
    if st["b"] is not None:
        y = y + st["b"].float()
    return [y.to(torch.bfloat16)]


def _framework(st):
    from bit_w4a4_quantized_group_b200 import binding as B
    op = st["op"]
    if op == GEMM:
        B.w4a4_gemm_lowrank_up_t("fp8", st["M"], st["N"], st["K"], st["rank"], st["a_codes"], st["a_scales"], 1.0,
                                 st["w_codes"], st["w_scales"], 1.0, st["Z"], st["L2"], st["b"], st["Y"])
        return [st["Y"]]
    codes, scales = st["codes"], st["scales"]
    if op == NORM:
        B.rmsnorm_quantize_act_t("fp8", st["X"], st["R"], st["gamma"], 1e-6, st["H"], codes, scales)
        extra = st["H"]
    elif op == GLU:
        B.glu_quantize_act_t("fp8", st["act"], st["gate"], st["up"], st["lambda"], codes, scales)
        extra = None
    else:
        B.quantize_act_lowrank_down_t("fp8", st["X"], st["lambda"], 1.0, st["L1"], codes, scales, st["Z"])
        extra = st["Z"]
    out = [codes.view(torch.float8_e4m3fn).view(st["M"], st["K"]), scales.view(torch.float8_e8m0fnu)]
    return out + ([extra] if extra is not None else [])


def run(state):
    return _framework(state) if own else _plain(state)


# ----------------------------------------------------------------- work and the definition in 64 bits

def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    rank = case.get("rank", 0)
    if op == GEMM:
        N = case["N"]
        b = (M + N) * (K + K // G) + 2 * M * N + 2 * rank * (M + N) + (2 * N if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * M * N * (K + rank)}
    b = M * K + M * (K // G)
    if op == NORM:
        b += M * K * (6 if case["residual"] else 2) + 4 * K
        return {"bytes": b, "flops": 5 * M * K}
    b += 4 * K if case["lam"] else 0
    if op == GLU:
        return {"bytes": b + M * K * (4 if case["gated"] else 2), "flops": 10 * M * K}
    return {"bytes": b + 2 * M * K + 2 * rank * (M + K), "flops": 2 * M * K * (rank + 2)}


def _exact_quantize(y):
    """Block exponents by comparison, and y / 2^e before its rounding to E4M3."""
    rows, K = y.shape
    blocks = y.reshape(rows, -1, G)
    top = blocks.abs().max(dim=2).values
    e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -1000) / 448.0))
    e = torch.where(448.0 * torch.exp2(e - 1) >= top, e - 1, e)      # log2 may round either way
    e = torch.where(448.0 * torch.exp2(e) < top, e + 1, e)
    e = e.clamp(min=-127.0)
    r, c = torch.meshgrid(torch.arange(rows, device=y.device), torch.arange(K // G, device=y.device), indexing="ij")
    at = (r // 128 * (_groups_pad(K) // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4
    s = torch.full((_scale_bytes(rows, K),), 2.0 ** -127, dtype=torch.float64, device=y.device)
    s[at.reshape(-1)] = torch.exp2(e).reshape(-1)
    return (blocks * torch.exp2(-e)[:, :, None]).reshape(rows, K), s


def _exact_values(codes, scales, K):
    rows = codes.shape[0]
    r = torch.arange(rows, device=codes.device)[:, None]
    c = torch.arange(K, device=codes.device)[None, :] // G
    at = (r // 128 * (_groups_pad(K) // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4
    i = codes.to(torch.int64)
    man, ex = (i & 7).double(), (i >> 3) & 15
    v = torch.where(ex > 0, (8.0 + man) * torch.exp2(ex.double() - 10.0), man * 2.0 ** -9)
    return torch.where(i > 127, -v, v) * torch.exp2(scales[at].double() - 127.0)


def exact(case, seed):
    st = prepare(case, seed)
    op, K = st["op"], st["K"]
    if op == GEMM:
        y = _exact_values(st["a_codes"], st["a_scales"], K) @ _exact_values(st["w_codes"], st["w_scales"], K).T
        if st["rank"]:
            y += st["Z"].double() @ st["L2"].double().T
        if st["bias"]:
            y += st["b"].double()
        return [y]
    if op == NORM:
        h = st["X"].double()
        if st["residual"]:
            h = (h + st["R"].double()).to(torch.bfloat16).double()
        y = h / torch.sqrt(torch.mean(h ** 2, dim=1, keepdim=True) + 1e-6) * st["gamma"].double()
        codes, scales = _exact_quantize(y)
        return [codes, scales] + ([h] if st["residual"] else [])
    if op == GLU:
        x = st["gate"].double()
        if st["act"] == "silu":
            y = x * torch.sigmoid(x)
        else:
            y = 0.5 * x * (1.0 + torch.tanh((2.0 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3)))
        if st["gated"]:
            y = y * st["up"].double()
        if st["lam"]:
            y = y / st["lambda"].double()
        return list(_exact_quantize(y))
    y = st["X"].double()
    if st["lam"]:
        y = (y / st["lambda"].double()).to(torch.bfloat16).double()
    z = [y @ st["L1"].double().T] if st["rank"] else []
    return list(_exact_quantize(y)) + z
