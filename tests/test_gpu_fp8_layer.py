"""GPU tests of the FP8 layer: its prologue (codes and scales bit for bit), its GEMM against the
product of the same operands in 64 bits, and runs of several operators as a transformer block
uses them.

GEMM tolerance: bf16 rounds by at most 2^-8 of the value; before that the fp32 accumulator takes
one tensor-core sum per 32 (16 for the branch) terms, each off by at most one unit of 2^-23 of
the absolute terms' sum S, and the bias one more.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle as O
from bit_w4a4_quantized_group_b200 import binding as B
from bit_w4a4_quantized_group_b200 import build as BUILD

import fp8_helpers as F
from gpu_helpers import check_device_error, dev_bf16, host_bf16
from layouts import bf16_ulp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    BUILD.build()
    B.load()


# ----------------------------------------------------------------- prologue

@pytest.mark.parametrize("M,K,rank,lam", [
    (1, 128, 0, False), (1, 2048, 16, True), (31, 640, 32, True), (33, 1152, 48, False), (128, 512, 64, True),
    (129, 384, 80, True), (300, 2176, 128, True), (200, 4096, 0, True), (513, 1024, 112, False)])
def test_prologue_codes_and_scales_bit_exact(M, K, rank, lam):
    rng = np.random.default_rng(M + K + rank)
    X = O.bf16_rn(rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.02, 30.0, 1.0))
    X[M // 2, : min(K, 256)] = 0.0
    X[0, 0] = -0.0
    lm = np.exp(rng.standard_normal(K)).astype(np.float32) if lam else None
    L1 = O.bf16_rn(rng.standard_normal((rank, K)) * 0.05) if rank else None
    sz = B.svdq_buffer_sizes("fp8", M, 128, K, rank)
    codes = torch.full((sz.a_codes + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((sz.a_scales + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    Z = torch.full((M, rank), float("nan"), dtype=torch.bfloat16, device="cuda") if rank else None
    B.quantize_act_lowrank_down_t("fp8", dev_bf16(X), None if lm is None else torch.from_numpy(lm).cuda(), 1.0,
                                  dev_bf16(L1) if rank else None, codes, scales, Z)
    check_device_error()
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    assert (c[sz.a_codes:] == 0x5A).all() and (s[sz.a_scales:] == 0x5A).all()
    xh = O.smooth_activations(X, lm)
    ref = F.quantize(xh.astype(np.float64))
    assert np.array_equal(c[: sz.a_codes].reshape(M, K), ref[0])
    assert np.array_equal(F.scales_of(s[: sz.a_scales], M, K), ref[1])
    assert not F.scale_padding_of(s[: sz.a_scales], M, K).any()
    if rank:
        Z64 = xh.astype(np.float64) @ L1.astype(np.float64).T
        S = np.abs(xh.astype(np.float64)) @ np.abs(L1.astype(np.float64)).T
        assert np.all(np.abs(host_bf16(Z) - Z64) <= 2.0 ** -8 * np.abs(Z64) + (K / 16 + 8) * 2.0 ** -23 * S)


# ----------------------------------------------------------------- GEMM

def _operand(rows, K, g, spread):
    """Random E4M3 codes (no NaN) and scale bytes 127 - spread .. 127 + spread, and their values."""
    codes = torch.randint(0, 256, (rows, K), generator=g, device="cuda", dtype=torch.int32)
    codes = torch.where((codes & 127) == 127, codes - 1, codes).to(torch.uint8)
    sb = torch.randint(127 - spread, 128 + spread, (rows, K // 128), generator=g, device="cuda", dtype=torch.int32)
    buf = torch.from_numpy(F.scales_to_buffer(sb.cpu().numpy().astype(np.uint8), K)).cuda()
    val = codes.view(torch.float8_e4m3fn).double().view(rows, K // 128, 128)
    return codes, buf, (val * torch.exp2(sb.double() - 127)[:, :, None]).view(rows, K)


def _gemm(M, N, K, rank, bias, seed=0, spread=3, y_off=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, sa, A = _operand(M, K, g, spread)
    w, sw, W = _operand(N, K, g, spread)
    Z = (20.0 * torch.randn((M, rank), generator=g, device="cuda")).to(torch.bfloat16) if rank else None
    L2 = (20.0 * torch.randn((N, rank), generator=g, device="cuda")).to(torch.bfloat16) if rank else None
    b = (100.0 * torch.randn((N,), generator=g, device="cuda")).to(torch.bfloat16) if bias else None
    buf = torch.full((M * N + y_off + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    Y = buf[y_off: y_off + M * N].view(M, N)
    B.w4a4_gemm_lowrank_up_t("fp8", M, N, K, rank, a, sa, 1.0, w, sw, 1.0, Z, L2, b, Y)
    assert B.svdq_last_launch_count() == 1
    check_device_error()
    assert torch.isnan(buf[:y_off]).all() and torch.isnan(buf[y_off + M * N:]).all()
    ref, S = A @ W.T, A.abs() @ W.abs().T
    if rank:
        ref, S = ref + Z.double() @ L2.double().T, S + Z.double().abs() @ L2.double().abs().T
    if bias:
        ref, S = ref + b.double(), S + b.double().abs()
    err = (Y.double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + (K / 32 + rank / 16 + 1) * 2.0 ** -23 * S
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((err - tol).max()))
    return Y


@pytest.mark.parametrize("M", [1, 2, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 256, 257, 300])
@pytest.mark.parametrize("N,K", [(128, 128), (256, 640), (384, 2176), (1152, 512)])
def test_gemm_few_tokens(M, N, K):
    _gemm(M, N, K, 0, False, seed=M)


@pytest.mark.parametrize("rank", [16, 32, 48, 64, 80, 128])
@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (20, 256, 1152), (77, 384, 1024), (150, 128, 640), (400, 640, 256)])
def test_gemm_branch_and_bias(M, N, K, rank):
    _gemm(M, N, K, rank, True, seed=rank)


@pytest.mark.parametrize("M,N,K,rank", [(2048, 2304, 384, 16), (1024, 3328, 640, 48), (512, 4608, 1152, 0),
                                        (1000, 3456, 128, 32), (4608, 1152, 256, 0), (3000, 6144, 1664, 16),
                                        (1, 9216, 4096, 16), (40, 12288, 512, 0), (5000, 128, 128, 0)])
def test_gemm_many_tiles(M, N, K, rank):
    _gemm(M, N, K, rank, rank > 0, seed=N)


@pytest.mark.parametrize("M,N,K", [(5, 256, 384), (64, 128, 256), (300, 384, 640)])
def test_gemm_output_at_16_bytes(M, N, K):
    _gemm(M, N, K, 16, True, y_off=8)


@pytest.mark.parametrize("M", [1, 3, 100, 300])
def test_gemm_each_scale_byte_reaches_its_group(M):
    """One group at a time carries a value: 9 groups with scales of very different size."""
    K, N = 1152, 256
    a = torch.full((M, K), 0x38, dtype=torch.uint8, device="cuda")        # 1.0
    w = torch.full((N, K), 0x38, dtype=torch.uint8, device="cuda")
    Y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    for grp in range(9):
        sa = np.zeros((M, 9), np.uint8)
        sw = np.zeros((N, 9), np.uint8)
        sa[:, grp] = 120 + grp + np.arange(M) % 3
        sw[:, grp] = 130 - grp + np.arange(N) % 5
        B.w4a4_gemm_lowrank_up_t("fp8", M, N, K, 0, a, torch.from_numpy(F.scales_to_buffer(sa, K)).cuda(), 1.0, w,
                                 torch.from_numpy(F.scales_to_buffer(sw, K)).cuda(), 1.0, None, None, None, Y)
        check_device_error()
        ref = 128.0 * np.exp2(sa[:, grp].astype(float) - 127)[:, None] * np.exp2(sw[:, grp].astype(float) - 127)[None]
        assert np.array_equal(host_bf16(Y).astype(np.float64), ref), grp


def test_gemm_repeats_bit_for_bit():
    for M in (1, 40, 200, 700):
        a, b = _gemm(M, 640, 1152, 32, True, seed=3), _gemm(M, 640, 1152, 32, True, seed=3)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_rows_do_not_depend_on_the_rest_of_the_batch_beyond_rounding():
    """A NaN token stays in its row of Y."""
    M, N, K = 130, 256, 640
    g = torch.Generator(device="cuda").manual_seed(1)
    a, sa, A = _operand(M, K, g, 2)
    w, sw, W = _operand(N, K, g, 2)
    a[7, 100] = 0x7F
    Y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    B.w4a4_gemm_lowrank_up_t("fp8", M, N, K, 0, a, sa, 1.0, w, sw, 1.0, None, None, None, Y)
    check_device_error()
    nan = torch.isnan(Y)
    assert nan[7].all() and int(nan.sum()) == N


# ----------------------------------------------------------------- runs of several operators

def _layer(N, K, rank, seed, lam=True, bias=True):
    from bit_w4a4_quantized_group_b200 import prepare as P
    from bit_w4a4_quantized_group_b200.layer import W4A4LowRankLinear
    rng = np.random.default_rng(seed)
    prep = {"lam": rng.uniform(0.5, 4.0, K).astype(np.float32),
            "R_nk": (rng.standard_normal((N, K)) * 0.02).astype(np.float32),
            "L1_rk": (rng.standard_normal((rank, K)) * 0.05).astype(np.float32),
            "L2_nr": (rng.standard_normal((N, rank)) * 0.05).astype(np.float32), "act_gscale": 1.0}
    b = (rng.standard_normal(N) * 0.1).astype(np.float32) if bias else None
    return W4A4LowRankLinear("fp8", N, K, P.pack("fp8", prep), prep["lam"] if lam else None, 1.0, b), prep, b


@pytest.mark.parametrize("M,N,K,rank", [(1, 256, 640, 16), (150, 384, 1152, 32), (700, 1024, 2048, 0)])
def test_layer_forward(M, N, K, rank):
    lin, prep, b = _layer(N, K, rank, M)
    X = O.bf16_rn(np.random.default_rng(M).standard_normal((M, K)) * 2)
    Y = host_bf16(lin.forward(dev_bf16(X), check=True))
    packed = O.pack_weight("fp8", prep["R_nk"], prep["L1_rk"], prep["L2_nr"])
    ref = O.layer_forward("fp8", X, prep["lam"], 1.0, packed, O.bf16_rn(b))
    # Z may round to the next bf16 (its own test bounds it), so the whole layer is compared by norm:
    # bf16 rounds Y by at most 2^-8 and Z's flips move it by less than that
    assert np.linalg.norm(Y - ref["Y"]) <= 2.0 ** -8 * np.linalg.norm(ref["Y"])
