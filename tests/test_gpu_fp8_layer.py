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
                                        (1, 9216, 4096, 16), (40, 12288, 512, 0), (5000, 128, 128, 0),
                                        (2048, 2944, 640, 48), (2000, 2816, 1152, 16), (1800, 3072, 128, 0),
                                        (2048, 4096, 256, 128), (4608, 5888, 2176, 0)])
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


def _weights64(lin):
    N, K = lin.N, lin.K
    return F.dequantize(lin.w_codes.cpu().numpy().reshape(N, K), F.scales_of(lin.w_scales.cpu().numpy(), N, K))


def _fed64(lin, M):
    """The quantized input that the last call left in the layer's workspace, in 64 bits."""
    ws = lin.workspace(M)
    K = lin.K
    return F.dequantize(ws["a_codes"].cpu().numpy().reshape(M, K), F.scales_of(ws["a_scales"].cpu().numpy(), M, K))


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_mlp_block(M, act):
    """Norm with residual -> gate-up layer -> gated activation -> down layer, each operator fed by
    the one before, against 64-bit forms of every step on the operands that the step was given."""
    K, I = 640, 1152
    up, _, bu = _layer(2 * I, K, 0, 3)
    down, _, bd = _layer(K, I, 0, 4)
    rng = np.random.default_rng(M)
    X, R = O.bf16_rn(rng.standard_normal((M, K)) * 2), O.bf16_rn(rng.standard_normal((M, K)))
    gamma = torch.from_numpy(rng.uniform(0.5, 1.5, K).astype(np.float32)).to(torch.bfloat16)
    folded = up.fold_gamma(gamma)
    Xd, Rd = dev_bf16(X), dev_bf16(R)
    H = torch.empty_like(Xd)
    U = up.forward_normed(Xd, Rd, folded, 1e-6, H)
    Y = down.forward_activated(act, U[:, :I], U[:, I:])
    check_device_error()
    h = O.bf16_rn(X.astype(np.float64) + R.astype(np.float64))
    assert np.array_equal(host_bf16(H), h)
    y64 = F.rmsnorm64(h.astype(np.float64), folded.cpu().numpy(), 1e-6)
    F.check_quantized(up.workspace(M)["a_codes"].cpu().numpy().reshape(M, K),
                      F.scales_of(up.workspace(M)["a_scales"].cpu().numpy(), M, K), y64, 2.0 ** -19)

    def gemm_check(lin, got, bias):
        A, W, b = _fed64(lin, M), _weights64(lin), O.bf16_rn(bias).astype(np.float64)
        ref, S = A @ W.T + b, np.abs(A) @ np.abs(W).T + np.abs(b)
        assert np.all(np.abs(host_bf16(got) - ref) <= 2.0 ** -8 * np.abs(ref) + (lin.K / 32 + 1) * 2.0 ** -23 * S)
    gemm_check(up, U, bu)
    u = host_bf16(U).astype(np.float64)
    a64 = F.act64(u[:, :I], act) * u[:, I:] / down.lam.double().cpu().numpy()
    F.check_quantized(down.workspace(M)["a_codes"].cpu().numpy().reshape(M, I),
                      F.scales_of(down.workspace(M)["a_scales"].cpu().numpy(), M, I), a64, 2.0 ** -15, 2.0 ** -110)
    gemm_check(down, Y, bd)


@pytest.mark.parametrize("M", [1, 70, 260])
def test_mlp_block_replays_from_a_graph_and_on_another_stream(M):
    K, I = 640, 1152
    up, _, _ = _layer(2 * I, K, 0, 5)
    down, _, _ = _layer(K, I, 0, 6)
    g = torch.Generator(device="cuda").manual_seed(M)
    folded = up.fold_gamma(torch.ones(K))
    X = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    R = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    H, U, Y = torch.empty_like(X), torch.empty((M, 2 * I), dtype=torch.bfloat16, device="cuda"), torch.empty_like(X)

    def block():
        up.forward_normed(X, R, folded, 1e-6, H, U)
        down.forward_activated("silu", U[:, :I], U[:, I:], Y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    torch.cuda.current_stream().wait_stream(side)
    first = Y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
        block()                                  # twice: each launch may start under the one before
    for i in range(4):
        X.copy_(torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) * (1 + i))
        Y.fill_(float("nan"))
        graph.replay()
        replayed = Y.clone()
        Y.fill_(float("nan"))
        block()
        assert torch.equal(replayed.view(torch.int16), Y.view(torch.int16)), i
    assert torch.isfinite(first).all()
    check_device_error()
    del graph


def test_calls_back_to_back_keep_stream_order():
    """Writers and readers of one workspace in turn, without a wait between: every GEMM reads what the
    call before it wrote, and every writer waits for the GEMM before it."""
    K, N = 1024, 512
    lin, _, _ = _layer(N, K, 0, 8)
    g = torch.Generator(device="cuda").manual_seed(2)
    gamma = lin.fold_gamma(torch.ones(K))
    for M in (1, 100, 400):
        Xs = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) * (i + 1) for i in range(6)]
        ref = []
        for x in Xs:
            ref.append((lin.forward_normed(x, None, gamma), lin.forward_activated("gelu", x), lin.forward(x)))
            torch.cuda.synchronize()
        Ys = [tuple(torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(3)) for _ in Xs]
        for _ in range(5):
            for x, y in zip(Xs, Ys):
                lin.forward_normed(x, None, gamma, Y=y[0])
                lin.forward_activated("gelu", x, Y=y[1])
                lin.forward(x, y[2])
        check_device_error()
        for a, b in zip(ref, Ys):
            for u, v in zip(a, b):
                assert torch.equal(u.view(torch.int16), v.view(torch.int16))


def test_two_streams_at_once():
    """Two layers on two streams, many calls in flight: outputs equal the calls alone."""
    la, _, _ = _layer(640, 1152, 0, 11)
    lb, _, _ = _layer(2304, 640, 16, 12)
    g = torch.Generator(device="cuda").manual_seed(3)
    Xa = torch.randn((33, 1152), generator=g, device="cuda").to(torch.bfloat16)
    Xb = torch.randn((500, 640), generator=g, device="cuda").to(torch.bfloat16)
    ra, rb = la.forward_activated("silu", Xa).clone(), lb.forward(Xb).clone()
    Ya, Yb = torch.empty_like(ra), torch.empty_like(rb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(50):
        with torch.cuda.stream(sa):
            la.forward_activated("silu", Xa, Y=Ya)
        with torch.cuda.stream(sb):
            lb.forward(Xb, Yb)
    check_device_error()
    assert torch.equal(ra.view(torch.int16), Ya.view(torch.int16))
    assert torch.equal(rb.view(torch.int16), Yb.view(torch.int16))


def test_many_repeats_of_long_k_agree():
    """Rings that wrap many times, with every CTA of the device busy: 60 repeats, bit for bit."""
    for M, N, K in ((1, 9216, 4096), (33, 12288, 3072), (100, 3072, 8192), (600, 2304, 4096)):
        g = torch.Generator(device="cuda").manual_seed(M)
        a, sa, _ = _operand(M, K, g, 2)
        w, sw, _ = _operand(N, K, g, 2)
        Y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        first = None
        for i in range(60):
            Y.fill_(float("nan"))
            B.w4a4_gemm_lowrank_up_t("fp8", M, N, K, 0, a, sa, 1.0, w, sw, 1.0, None, None, None, Y)
            if first is None:
                first = Y.clone()
            assert torch.equal(first.view(torch.int16), Y.view(torch.int16)), (M, N, K, i)
        check_device_error()
