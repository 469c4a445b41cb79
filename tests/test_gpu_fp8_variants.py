"""Every variant of the FP8 kernels against plain forms, with the variants that the cases have to reach
(svdq_last_variant on a B200's 148 SMs): a rule that chooses otherwise fails here and wants other sizes.
How wide a split K has goes by the clusters that a device holds, which differs between boards of one kind;
those cases name what holds on all of them.

Prologue: codes and scales bit for bit against the same rule in plain torch, all rows; Z in 64 bits.  bf16
rounds Z by at most 2^-8 of its value; before that the fp32 accumulator takes one tensor-core sum per 16
terms and the cluster adds at most 8 partial sums, each off by at most 2^-23 of the absolute terms' sum S.
GEMM, norm and activation: the checks and tolerances of the modules that they come from.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from bit_w4a4_quantized_group_b200 import binding as B
from bit_w4a4_quantized_group_b200 import build as BUILD

import fp8_helpers as F
from gpu_helpers import check_device_error
from test_gpu_fp8_layer import _gemm
from test_gpu_fp8_rows import GLU_DELTA, GLU_FLOOR, NORM_DELTA, _acts, _f64, _glu64, _run_glu, _run_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    BUILD.build()
    B.load()
    assert torch.cuda.get_device_properties(0).multi_processor_count == 148


def _quantize_t(xh):
    """Codes and scale bytes of a bf16 matrix: the smallest e >= -127 with max|x| <= 448 * 2^e."""
    M, K = xh.shape
    g = xh.view(M, K // 128, 128)
    m, ex = torch.frexp(g.abs().amax(2).float())
    e = torch.where(m > 0, (ex - 9 + (m > 0.875)).clamp(min=-127), -127)
    q = torch.ldexp(g.double(), -e[..., None].double()).float().to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(M, K), (e + 127).to(torch.uint8)


# M, K, rank, lambda, and whether K is split: one group and many (rings of two, four and six stages that wrap);
# one wave and several; a last block of 1, 3, 5, 8, 23, ... rows.  Split for certain: few blocks; unsplit for
# certain: one group, or more blocks of 128 rows than two-CTA clusters could be resident.
PROLOGUE = [
    (1, 128, 16, True, False), (300, 256, 32, False, True), (129, 12288, 48, True, True), (2500, 1152, 64, True, True),
    (4608, 3072, 32, True, None), (4599, 4096, 128, False, None), (20001, 1152, 16, True, False), (6003, 2176, 128, False, None),
    (10007, 128, 16, True, False), (10007, 1152, 32, True, False), (16389, 2176, 16, False, False),
    (12005, 4096, 128, True, False), (3001, 384, 32, True, None), (5003, 1152, 16, False, None), (3001, 2176, 32, True, None),
    (7001, 3072, 32, True, None), (9001, 4096, 80, False, None), (2000, 640, 128, True, True)]


@pytest.mark.parametrize("M,K,rank,lam,split", PROLOGUE)
def test_prologue_with_a_branch(M, K, rank, lam, split):
    X = _acts(M, K, M + K + rank)
    X[M // 2, : min(K, 256)] = 0.0
    g = torch.Generator(device="cuda").manual_seed(rank)
    lm = torch.exp(torch.randn((K,), generator=g, device="cuda")) if lam else None
    L1 = (0.05 * torch.randn((rank, K), generator=g, device="cuda")).to(torch.bfloat16)
    sz = B.svdq_buffer_sizes("fp8", M, 128, K, rank)
    codes = torch.full((sz.a_codes + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((sz.a_scales + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    zbuf = torch.full((M * rank + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    Z = zbuf[: M * rank].view(M, rank)
    B.quantize_act_lowrank_down_t("fp8", X, lm, 1.0, L1, codes, scales, Z)
    assert split is None or (B.svdq_last_variant() % 16 > 1) == split
    check_device_error()
    assert (codes[sz.a_codes:] == 0x5A).all() and (scales[sz.a_scales:] == 0x5A).all() and torch.isnan(zbuf[M * rank:]).all()
    xh = X if lm is None else (X.float() / lm).to(torch.bfloat16)
    ref_codes, ref_scales = _quantize_t(xh)
    assert torch.equal(codes[: sz.a_codes].view(M, K), ref_codes)
    sb = scales[: sz.a_scales].cpu().numpy()
    assert np.array_equal(F.scales_of(sb, M, K), ref_scales.cpu().numpy())
    assert not F.scale_padding_of(sb, M, K).any()
    ref, S = xh.double() @ L1.double().T, xh.double().abs() @ L1.double().abs().T
    err = (Z.double() - ref).abs() - (2.0 ** -8 * ref.abs() + (K / 16 + 8) * 2.0 ** -23 * S)
    assert err.max() <= 0, (int((err > 0).sum()), (err > 0).nonzero()[:4].tolist())


def test_prologue_cases_reach_every_variant():
    """128 and 64 rows of a CTA, each with K split and unsplit."""
    seen = set()
    for M, K, rank, _, _ in PROLOGUE:
        X, L1 = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"), torch.zeros((rank, K), dtype=torch.bfloat16, device="cuda")
        sz = B.svdq_buffer_sizes("fp8", M, 128, K, rank)
        B.quantize_act_lowrank_down_t("fp8", X, None, 1.0, L1, torch.empty(sz.a_codes, dtype=torch.uint8, device="cuda"),
                                      torch.empty(sz.a_scales, dtype=torch.uint8, device="cuda"),
                                      torch.empty((M, rank), dtype=torch.bfloat16, device="cuda"))
        rows, ksplit = divmod(B.svdq_last_variant(), 16)
        seen.add((rows, ksplit > 1))
    check_device_error()
    assert seen == {(64, False), (64, True), (128, False), (128, True)}


@pytest.mark.parametrize("M,K,rank", [(10007, 640, 16), (5003, 1152, 32), (4608, 2176, 64)])
def test_prologue_repeats_bit_for_bit(M, K, rank):
    """With a ring that wraps and every CTA of the device busy, several calls in flight."""
    X, L1 = _acts(M, K, 1), _acts(rank, K, 2)
    sz = B.svdq_buffer_sizes("fp8", M, 128, K, rank)
    out = [(torch.zeros(sz.a_codes, dtype=torch.uint8, device="cuda"), torch.zeros(sz.a_scales, dtype=torch.uint8, device="cuda"),
            torch.zeros((M, rank), dtype=torch.bfloat16, device="cuda")) for _ in range(12)]
    for c, s, z in out:
        B.quantize_act_lowrank_down_t("fp8", X, None, 1.0, L1, c, s, z)
    check_device_error()
    for c, s, z in out[1:]:
        assert torch.equal(c, out[0][0]) and torch.equal(s, out[0][1]) and torch.equal(z.view(torch.int16), out[0][2].view(torch.int16))


# token tile, split K or not: several token tiles and a last one of 1, 44, 72, 104 and 128 tokens, with branch
# and bias; tiles that outnumber half the SMs, or all of them, and are not split
@pytest.mark.parametrize("M,N,K,rank,bias,tokens,split", [
    (512, 512, 8192, 0, False, 128, True), (300, 256, 8192, 48, True, 128, True), (128, 384, 4096, 16, True, 128, True),
    (129, 128, 4096, 128, True, 128, True), (200, 512, 4096, 80, False, 128, True), (1000, 128, 8192, 16, True, 128, True),
    (640, 384, 6144, 0, True, 128, True), (65, 384, 2176, 32, True, 128, True), (7, 19200, 512, 16, True, 16, False),
    (30, 19200, 640, 0, True, 32, False), (64, 12288, 1152, 48, True, 64, False), (64, 128, 128, 16, True, 64, False)])
def test_gemm_few_tokens(M, N, K, rank, bias, tokens, split):
    _gemm(M, N, K, rank, bias, seed=M + N)
    got, ksplit = divmod(-B.svdq_last_variant(), 16)
    assert (got, ksplit > 1) == (tokens, split)


@pytest.mark.parametrize("M,N,K,rank,bias,width", [
    (600, 1152, 640, 32, True, 64), (300, 640, 256, 128, True, 64), (800, 1152, 384, 16, True, 64),
    (700, 2304, 640, 48, True, 128), (400, 4608, 640, 16, True, 128), (1024, 2304, 256, 128, True, 128), (512, 4608, 1152, 80, True, 128),
    (1024, 3328, 640, 64, True, 192), (1500, 2304, 640, 128, True, 192),
    (300, 9216, 1152, 16, True, 256), (2048, 2304, 384, 80, True, 256), (1025, 3328, 256, 32, True, 256),
    (2048, 2944, 640, 128, True, 384), (4608, 5888, 2176, 80, True, 384)])
def test_gemm_many_tokens(M, N, K, rank, bias, width):
    _gemm(M, N, K, rank, bias, seed=M + N)
    assert B.svdq_last_variant() == width


@pytest.mark.parametrize("M,K,units", [(1000, 8192, 1), (1100, 4096, 1), (1025, 4224, 2), (1061, 8192, 2), (3, 32768, 2), (3, 32896, 0)])
def test_norm(M, K, units):
    X, R = _acts(M, K, 1), _acts(M, K, 2)
    codes, sb = _run_norm(X, R, None, 1e-6, None)
    B.rmsnorm_quantize_act_t("fp8", X, R, None, 1e-6, None, torch.empty(M * K, dtype=torch.uint8, device="cuda"),
                             torch.empty(F.scale_offsets(M, K, padded=True).size, dtype=torch.uint8, device="cuda"))
    assert B.svdq_last_variant() == units
    F.check_quantized(codes, sb, F.rmsnorm64(_f64((X.float() + R.float()).to(torch.bfloat16)), None, 1e-6), NORM_DELTA)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("lam", [False, True])
@pytest.mark.parametrize("M,K,pairs", [(24011, 640, 4), (12005, 2304, 4), (11983, 2304, 1)])
def test_activation_without_gating(act, lam, M, K, pairs):
    gate = _acts(M, K + 8, M, scale=2.0)[:, 8:]
    lm = torch.linspace(0.25, 4.0, K, device="cuda") if lam else None
    codes, sb = _run_glu(act, gate, None, lm)
    B.glu_quantize_act_t("fp8", act, gate, None, lm, torch.empty(M * K, dtype=torch.uint8, device="cuda"),
                         torch.empty(F.scale_offsets(M, K, padded=True).size, dtype=torch.uint8, device="cuda"))
    assert B.svdq_last_variant() == pairs
    pick = np.r_[0:40, M // 2: M // 2 + 40, M - 40: M]
    F.check_quantized(codes[pick], sb[pick], _glu64(act, gate[torch.from_numpy(pick).cuda()], None, lm), GLU_DELTA, GLU_FLOOR)
    for i in range(0, M, 3001):             # every row: the bytes of small calls, which take one pair per CTA
        part = _run_glu(act, gate[i: i + 3001], None, lm)
        assert np.array_equal(part[0], codes[i: i + 3001]) and np.array_equal(part[1], sb[i: i + 3001])


def test_variant_is_cleared_by_other_calls():
    _gemm(20, 128, 128, 0, False)
    assert B.svdq_last_variant() == -(16 * 32 + 1)
    X = _acts(4, 256, 1)
    sz = B.svdq_buffer_sizes("nvfp4", 4, 128, 256, 0)
    B.quantize_act_lowrank_down_t("nvfp4", X, None, 1.0, None, torch.empty(sz.a_codes, dtype=torch.uint8, device="cuda"),
                                  torch.empty(sz.a_scales, dtype=torch.uint8, device="cuda"), None)
    assert B.svdq_last_variant() == 0
    check_device_error()
