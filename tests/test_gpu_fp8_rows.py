"""GPU tests of the row operators with an FP8 output (norm and activation) against plain forms
in 64 bits.

Tolerances: a value may be half an E4M3 step away from a y that differs from the exact one by at
most delta relatively.  delta is the fp32 error of the formula, in units of 2^-24:
  norm  16 elements' squares go through two sums of 8 and an addition, in the looping form up to three
        such sums are added (K <= 40960 here), then 5 + 1 + 5 tree steps: at most 50; halved by the
        square root, plus the divide, the addition of eps, the root and two products: 50 / 2 + 5
        <= 32 = 2^5: 2^-19;
  glu   exp(-t) is 2^a of an argument with at most four roundings, |a| <= 127 wherever the result is
        not below 2^-110: ln 2 * 127 * 4 = 352 units, 4 more for the hardware's 2^a (2^-22), 2 for
        its reciprocal and 4 for the sum and the products, 2 more where two elements share a
        reciprocal, 1 / a = b / (a b) (b's own error cancels): < 512 = 2^9: 2^-15; below that, 2^-110
        absolutely.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from bit_w4a4_quantized_group_b200 import binding as B
from bit_w4a4_quantized_group_b200 import build as BUILD

import fp8_helpers as F
from gpu_helpers import check_device_error

pytestmark = pytest.mark.gpu

NORM_DELTA = 2.0 ** -19
GLU_DELTA, GLU_FLOOR = 2.0 ** -15, 2.0 ** -110


@pytest.fixture(scope="module", autouse=True)
def _lib():
    BUILD.build()
    B.load()


def _acts(M, K, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, K), generator=g, device="cuda") * scale
    x[:, torch.randint(0, K, (max(1, K // 100),), generator=g, device="cuda")] *= 30.0
    return x.to(torch.bfloat16)


def _bufs(M, K, fill=0xA5):
    sz = B.svdq_buffer_sizes("fp8", M, 128, K, 0)
    # a guard behind each buffer shows writes past its end
    return (torch.full((sz.a_codes + 256,), fill, dtype=torch.uint8, device="cuda"),
            torch.full((sz.a_scales + 256,), fill, dtype=torch.uint8, device="cuda"), sz)


def _result(codes, scales, sz, M, K, fill=0xA5):
    check_device_error()
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    assert (c[sz.a_codes:] == fill).all() and (s[sz.a_scales:] == fill).all()
    s = s[: sz.a_scales]
    assert not F.scale_padding_of(s, M, K).any()
    return c[: sz.a_codes].reshape(M, K), F.scales_of(s, M, K)


def _f64(t):
    return t.double().cpu().numpy()


def _run_norm(X, R, gamma, eps, H):
    M, K = X.shape
    codes, scales, sz = _bufs(M, K)
    B.rmsnorm_quantize_act_t("fp8", X, R, gamma, eps, H, codes, scales)
    assert B.svdq_last_launch_count() == 1
    return _result(codes, scales, sz, M, K)


@pytest.mark.parametrize("M,K", [(1, 128), (1, 3072), (2, 640), (127, 1152), (128, 512), (129, 2176), (300, 4096),
                                 (5, 8192), (3, 12288), (4, 16512), (2, 32768), (3, 32896), (2, 40960)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(M, K, residual):
    X = _acts(M, K, M * 7 + K)
    R = _acts(M, K, M + 3 * K) if residual else None
    H = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device="cuda") if residual else None
    g = torch.Generator(device="cuda").manual_seed(K)
    gamma = None if M == 2 else 1 + 0.3 * torch.randn((K,), generator=g, device="cuda")
    codes, sb = _run_norm(X, R, gamma, 1e-6, H)
    h = X if R is None else (X.float() + R.float()).to(torch.bfloat16)
    if residual:
        assert torch.equal(H.view(torch.int16), h.view(torch.int16))
    F.check_quantized(codes, sb, F.rmsnorm64(_f64(h), None if gamma is None else _f64(gamma), 1e-6), NORM_DELTA)


@pytest.mark.parametrize("M,K", [(1024, 128), (1100, 4096), (1025, 4224), (1061, 8192), (1024, 12416)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_many_rows(M, K, residual):
    """Many rows with both launch shapes: one unit of 16 elements per thread, and two for wide rows."""
    X = _acts(M, K, M + K)
    R = _acts(M, K, M + 5 * K) if residual else None
    gamma = torch.linspace(-1.5, 1.5, K, device="cuda")
    codes, sb = _run_norm(X, R, gamma, 1e-6, None)
    h = X if R is None else (X.float() + R.float()).to(torch.bfloat16)
    F.check_quantized(codes, sb, F.rmsnorm64(_f64(h), _f64(gamma), 1e-6), NORM_DELTA)


@pytest.mark.parametrize("K", [3200, 6400, 16384])
def test_norm_bytes_do_not_depend_on_the_batch(K):
    X, R = _acts(1500, K, 41), _acts(1500, K, 42)
    ref = _run_norm(X, R, None, 1e-6, None)
    for lo, hi in ((0, 1), (700, 829), (1499, 1500), (100, 1400)):
        part = _run_norm(X[lo: hi], R[lo: hi], None, 1e-6, None)
        assert np.array_equal(part[0], ref[0][lo: hi]) and np.array_equal(part[1], ref[1][lo: hi])


def test_norm_rows_are_independent_and_may_be_strided():
    M, K = 37, 896
    wide = _acts(M, K + 136, 1)
    X = wide[:, 136:]
    Rw = _acts(M, K + 8, 2)
    R = Rw[:, :K]
    ref = _run_norm(X.contiguous(), R.contiguous(), None, 1e-5, None)
    got = _run_norm(X, R, None, 1e-5, None)
    assert np.array_equal(ref[0], got[0]) and np.array_equal(ref[1], got[1])
    for m in (0, 17, 36):                  # one row at a time gives the same bytes
        one = _run_norm(X[m: m + 1], R[m: m + 1], None, 1e-5, None)
        assert np.array_equal(one[0][0], ref[0][m]) and np.array_equal(one[1][0], ref[1][m])


@pytest.mark.parametrize("K", [1152, 33024])
@pytest.mark.parametrize("where", ["residual", "X"])
def test_norm_in_place(K, where):
    M = 9
    X, R = _acts(M, K, 3), _acts(M, K, 4)
    gamma = torch.linspace(0.5, 1.5, K, device="cuda")
    H = torch.empty_like(X)
    ref = _run_norm(X, R, gamma, 1e-6, H)
    X2, R2 = X.clone(), R.clone()
    got = _run_norm(X2, R2, gamma, 1e-6, R2 if where == "residual" else X2)
    assert np.array_equal(ref[0], got[0]) and np.array_equal(ref[1], got[1])
    assert torch.equal((R2 if where == "residual" else X2).view(torch.int16), H.view(torch.int16))
    assert torch.equal((X2 if where == "residual" else R2).view(torch.int16),
                       (X if where == "residual" else R).view(torch.int16))


def test_norm_sum_not_kept():
    X, R = _acts(6, 512, 5), _acts(6, 512, 6)
    a = _run_norm(X, R, None, 1e-6, None)
    b = _run_norm(X, R, None, 1e-6, torch.empty_like(X))
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_norm_zero_rows_tiny_values_and_nan_rows():
    M, K = 8, 384
    X = _acts(M, K, 7)
    X[1] = 0.0
    X[2] = -0.0
    X[3, 128:256] = 0.0
    X[4] = X[4] * 2.0 ** -100               # squares underflow: eps alone is left
    X[5] = X[5] * 2.0 ** 40
    clean = _run_norm(X, None, None, 1e-6, None)
    F.check_quantized(clean[0], clean[1], F.rmsnorm64(_f64(X), None, 1e-6), NORM_DELTA)
    assert not (clean[0][1] & 0x7F).any() and not clean[1][1].any() and clean[1][3, 1] == 0
    Y = X.clone()
    Y[6, 5] = float("nan")
    dirty = _run_norm(Y, None, None, 1e-6, None)
    keep = [0, 1, 2, 3, 4, 5, 7]
    assert np.array_equal(dirty[0][keep], clean[0][keep]) and np.array_equal(dirty[1][keep], clean[1][keep])
    assert (dirty[0][6] & 0x7F == 0x7F).all()            # the norm of a row with a NaN is NaN


def test_norm_scale_borders():
    """Rows whose norm is 1 make y = gamma: maxima on and next to 448 * 2^e, and E4M3 midpoints."""
    K = 128
    X = torch.ones((1, K), dtype=torch.bfloat16, device="cuda")
    eps = 2.0 ** -60                                   # 1 + eps rounds to 1: rstd is exactly 1
    f = np.float32
    for top, byte in [(448.0, 127), (np.nextafter(f(448), f(999)), 128), (896.0, 128), (447.0, 127), (1.75, 119),
                      (np.nextafter(f(1.75), f(2)), 120), (2.0 ** -119 * 1.75, 0), (2.0 ** -126, 0), (2.0 ** 120, 239)]:
        gamma = torch.zeros(K, device="cuda")
        gamma[5] = float(top)
        codes, sb = _run_norm(X, None, gamma, eps, None)
        assert sb[0, 0] == byte, (top, sb[0, 0])
        ref = F.quantize(_f64(gamma)[None])
        assert np.array_equal(codes, ref[0]) and np.array_equal(sb, ref[1])
    gamma = torch.from_numpy(np.concatenate([[448.0], np.arange(127) * 2.0 ** -10]).astype(f)).cuda()
    codes, _ = _run_norm(X, None, gamma, eps, None)
    assert np.array_equal(codes, F.quantize(_f64(gamma)[None])[0])


def _run_glu(act, gate, up, lam):
    M, K = gate.shape
    codes, scales, sz = _bufs(M, K)
    B.glu_quantize_act_t("fp8", act, gate, up, lam, codes, scales)
    assert B.svdq_last_launch_count() == 1
    return _result(codes, scales, sz, M, K)


def _glu64(act, gate, up, lam):
    y = F.act64(_f64(gate), act)
    if up is not None:
        y = y * _f64(up)
    return y if lam is None else y / _f64(lam)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("lam", [False, True])
@pytest.mark.parametrize("M,K", [(1, 128), (3, 640), (127, 1152), (128, 2048), (130, 2432), (1, 12288)])
def test_glu(act, gated, lam, M, K):
    wide = _acts(M, 2 * K + 24, M + K, scale=2.0)
    gate, up = wide[:, 8: 8 + K], wide[:, 24 + K:] if gated else None
    g = torch.Generator(device="cuda").manual_seed(K)
    lm = torch.exp(torch.randn((K,), generator=g, device="cuda")) if lam else None
    codes, sb = _run_glu(act, gate, up, lm)
    F.check_quantized(codes, sb, _glu64(act, gate, up, lm), GLU_DELTA, GLU_FLOOR)


@pytest.mark.parametrize("act,lam,M,K", [("silu", False, 24011, 640), ("gelu", True, 12005, 2304)])
def test_glu_many_rows(act, lam, M, K):
    """Enough rows that a thread takes several pairs of them, and a last block that is not full."""
    gate = _acts(M, K + 8, 5, scale=2.0)[:, 8:]
    lm = torch.linspace(0.25, 4.0, K, device="cuda") if lam else None
    codes, sb = _run_glu(act, gate, None, lm)
    pick = np.r_[0:40, M // 2: M // 2 + 40, M - 40: M]
    F.check_quantized(codes[pick], sb[pick], _glu64(act, gate[torch.from_numpy(pick).cuda()], None, lm), GLU_DELTA, GLU_FLOOR)
    # every row: the same bytes as the rows in small calls, which take one pair per thread
    for i in range(0, M, 3001):
        part = _run_glu(act, gate[i: i + 3001], None, lm)
        assert np.array_equal(part[0], codes[i: i + 3001]) and np.array_equal(part[1], sb[i: i + 3001])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_over_the_whole_range(act):
    """Every finite bf16 value with |x| <= 2^100 as a gate, each alone in its group."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16)
    x = bits.view(torch.bfloat16)
    x = x[torch.isfinite(x) & (x.float().abs() <= 2.0 ** 100)]
    x = x[: x.numel() // 4 * 4]
    gate = torch.zeros((x.numel() // 4, 512), dtype=torch.bfloat16, device="cuda")
    gate[:, [3, 130, 300, 511]] = x.view(-1, 4)
    codes, sb = _run_glu(act, gate, None, None)
    F.check_quantized(codes, sb, _glu64(act, gate, None, None), GLU_DELTA, GLU_FLOOR)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_gated_beside_every_value(act):
    """Gates over the whole range next to ordinary ones: neighbours share a reciprocal where they can."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16)
    x = bits.view(torch.bfloat16)
    x = x[torch.isfinite(x) & (x.float().abs() <= 2.0 ** 60)]
    x = x[: x.numel() // 4 * 4]
    gate = _acts(x.numel() // 4, 512, 9)
    up = _acts(x.numel() // 4, 512, 10)
    gate[:, [3, 130, 300, 511]] = x.view(-1, 4)
    up[:, [3, 130, 300, 511]] = 2.0 ** -60            # so that the neighbours set the scale
    codes, sb = _run_glu(act, gate, up, None)
    F.check_quantized(codes, sb, _glu64(act, gate, up, None), GLU_DELTA, GLU_FLOOR)


@pytest.mark.parametrize("lam", [False, True])
def test_glu_gated_nan_leaves_its_neighbours(lam):
    M, K = 4, 384
    gate, up = _acts(M, K, 1), _acts(M, K, 2)
    lm = torch.linspace(0.5, 2.0, K, device="cuda") if lam else None
    ref = gate.clone()
    ref[1, 9], ref[2, 200] = 0.0, 0.0
    gate[1, 9], gate[2, 200] = float("nan"), float("nan")
    codes, sb = _run_glu("silu", gate, up, lm)
    assert codes[1, 9] & 0x7F == 0x7F and codes[2, 200] & 0x7F == 0x7F
    codes[1, 9], codes[2, 200] = 0, 0
    F.check_quantized(codes, sb, _glu64("silu", ref, up, lm), GLU_DELTA, GLU_FLOOR)


def test_glu_zero_rows_and_nan_stay_where_they_are():
    M, K = 6, 256
    gate, up = _acts(M, K, 1), _acts(M, K, 2)
    gate[2] = 0.0
    clean = _run_glu("silu", gate, up, None)
    assert not (clean[0][2] & 0x7F).any() and not clean[1][2].any()
    g2 = gate.clone()
    g2[4, 9] = float("nan")
    dirty = _run_glu("silu", g2, up, None)
    assert dirty[0][4, 9] & 0x7F == 0x7F
    dirty[0][4, :128] = clean[0][4, :128]
    dirty[1][4, 0] = clean[1][4, 0]
    assert np.array_equal(dirty[0], clean[0]) and np.array_equal(dirty[1], clean[1])
