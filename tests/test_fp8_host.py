"""The FP8 format on the host (no GPU): buffer sizes, the weight pack against a plain form, the
reference and the PyTorch quantize-dequantize, and every refusal of the FP8 device calls."""
import numpy as np
import pytest
import torch

import oracle as O
from bit_w4a4_quantized_group_b200 import binding as B
from bit_w4a4_quantized_group_b200 import build as BUILD
from bit_w4a4_quantized_group_b200 import prepare as P

import fp8_helpers as F


@pytest.fixture(scope="module", autouse=True)
def lib():
    BUILD.build()
    return B.load()


def test_buffer_sizes():
    s = B.svdq_buffer_sizes("fp8", 300, 640, 1152, 16)      # 9 groups: padded to 12
    assert s.a_codes == 300 * 1152 and s.w_codes == 640 * 1152
    assert s.a_scales == 384 * 12 and s.w_scales == 640 * 12
    assert s.z == 300 * 16 * 2 and s.y == 300 * 640 * 2
    assert B.svdq_buffer_sizes("fp8", 1, 128, 128, 0).a_scales == 128 * 4


def _random(N, K, seed, exp):
    rng = np.random.default_rng(seed)
    R = (rng.standard_t(2.0, (N, K)) * 2.0 ** exp).astype(np.float32)
    R[rng.random((N, K)) < 0.1] = 0.0
    return R


EDGES = np.array([448.0, 448.5, 449.0, 512.0, 1.0, 1.75, np.nextafter(np.float32(1.75), np.float32(2)), 2.0 ** -126,
                  2.0 ** -140, 1e-38, 3.0e38, 0.0, -0.0, -448.0, 2.0 ** -9, 3 * 2.0 ** -10], np.float32)


@pytest.mark.parametrize("N,K,exp", [(128, 128, 0), (256, 640, -20), (128, 1152, 30), (128, 512, -120)])
def test_pack_matches_plain_form(N, K, exp):
    R = _random(N, K, N + K, exp)
    for i, v in enumerate(EDGES):            # groups whose maximum sits at a border of the scale rule
        R[i, :128] = 0.0
        R[i, 3] = v
        R[i, 7] = -v / 3
    got = B.pack_weight_np("fp8", R, None, None)
    codes, sb = F.quantize(R.astype(np.float64))
    assert got["w_gscale"] == 1.0
    assert np.array_equal(got["w_codes"].reshape(N, K), codes)
    assert np.array_equal(F.scales_of(got["w_scales"], N, K), sb)
    assert not F.scale_padding_of(got["w_scales"], N, K).any()
    # no code saturates past half a step, and none is NaN
    assert np.isfinite(F.e4m3_values(codes)).all()
    # the reference and the PyTorch quantize-dequantize of the offline split say the same
    ref = O.quantize("fp8", R)
    assert np.array_equal(ref["codes"], codes) and np.array_equal(ref["scale_bits"], sb)
    assert np.array_equal(P.qdq_weight("fp8", torch.from_numpy(R)).numpy(), F.dequantize(codes, sb))
    assert np.array_equal(O.dequantize("fp8", ref), F.dequantize(codes, sb))


def test_pack_keeps_the_low_rank_factors():
    rng = np.random.default_rng(5)
    R = rng.standard_normal((128, 256)).astype(np.float32)
    L1 = rng.standard_normal((16, 256)).astype(np.float32)
    L2 = rng.standard_normal((128, 16)).astype(np.float32)
    got = B.pack_weight_np("fp8", R, L1, L2)
    ref = O.pack_weight("fp8", R, L1, L2)
    assert np.array_equal((got["L2_bf16"].astype(np.uint32) << 16).view(np.float32), ref["L2_scaled"])
    assert np.array_equal((got["L1_bf16"].astype(np.uint32) << 16).view(np.float32), ref["L1_bf16"])
    with pytest.raises(B.SvdqError):
        B.pack_weight_np("fp8", R, None, None, 2.0)          # FP8 has no tensor scale


def test_split_and_residual_iteration_take_the_format():
    rng = np.random.default_rng(6)
    X = rng.standard_normal((64, 256)).astype(np.float32)
    W = rng.standard_normal((256, 128)) * 0.02
    prep = P.prepare("fp8", X, W, 16, device="cpu", residual_iters=2, early_stop=True)
    packed = P.pack("fp8", prep)
    Q = F.dequantize(packed["w_codes"].reshape(128, 256), F.scales_of(packed["w_scales"], 128, 256))
    assert np.array_equal(Q, P.qdq_weight("fp8", torch.from_numpy(prep["R_nk"])).numpy())


_P = 1 << 20        # an aligned address that is never read: every call below is refused


def _norm(**kw):
    a = dict(fmt="fp8", M=4, K=256, X=_P, ldx=256, residual=_P, ldr=256, gamma=_P, eps=1e-6, H=2 * _P, ldh=256,
             a_codes=_P, a_scales=_P, stream=None)
    a.update(kw)
    return B.svdq_rmsnorm_quantize_act(**a)


@pytest.mark.parametrize("kw", [
    dict(M=0), dict(M=-1), dict(K=0), dict(K=192), dict(X=None), dict(X=_P + 8), dict(ldx=248), dict(ldx=260),
    dict(residual=_P + 2), dict(ldr=128), dict(ldr=257), dict(H=2 * _P + 4), dict(ldh=0), dict(residual=None),
    dict(gamma=_P + 4), dict(eps=0.0), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(eps=1e-42), dict(a_codes=None), dict(a_scales=None), dict(a_codes=_P + 8), dict(a_scales=_P + 1),
    dict(H=_P, ldh=256, X=_P, ldx=264), dict(H=_P, ldh=264), dict(fmt=9),
])
def test_norm_refuses_bad_arguments(kw):
    assert _norm(**kw) == B.SVDQ_ERR_INVALID_ARG
    assert B.svdq_last_launch_count() == 0


def test_norm_refuses_other_formats_and_sizes():
    for fmt in ("nvfp4", "mxfp4", "int4", "w8a8"):
        assert _norm(fmt=fmt) == B.SVDQ_ERR_UNSUPPORTED
    assert _norm(M=1 << 31) == B.SVDQ_ERR_UNSUPPORTED
    assert _norm(K=(1 << 24) + 128, ldx=1 << 25, ldr=1 << 25, ldh=1 << 25) == B.SVDQ_ERR_UNSUPPORTED


def _glu(**kw):
    a = dict(fmt="fp8", act="silu", M=4, K=256, gate=_P, ldg=512, up=_P + 512, ldu=512, lam=_P, a_codes=_P,
             a_scales=_P, stream=None)
    a.update(kw)
    return B.svdq_glu_quantize_act(**a)


@pytest.mark.parametrize("kw", [
    dict(M=0), dict(K=100), dict(act=0), dict(act=3), dict(gate=None), dict(gate=_P + 6), dict(ldg=255),
    dict(ldg=12345), dict(up=_P + 8), dict(ldu=128), dict(lam=_P + 4), dict(a_codes=None), dict(a_scales=None),
    dict(a_scales=_P + 2), dict(a_codes=_P + 2), dict(fmt=0),
])
def test_glu_refuses_bad_arguments(kw):
    assert _glu(**kw) == B.SVDQ_ERR_INVALID_ARG
    assert B.svdq_last_launch_count() == 0


def test_glu_refuses_other_formats():
    for fmt in ("nvfp4", "mxfp4", "int4", "w8a8"):
        assert _glu(fmt=fmt) == B.SVDQ_ERR_UNSUPPORTED


def test_helpers_refuse_mismatched_tensors():
    X = torch.zeros((4, 256), dtype=torch.bfloat16)
    buf = torch.zeros(2048, dtype=torch.uint8)
    with pytest.raises(ValueError):
        B.rmsnorm_quantize_act_t("fp8", X, X[:2], None, 1e-6, None, buf, buf)            # other shape
    with pytest.raises(ValueError):
        B.rmsnorm_quantize_act_t("fp8", X, X.float(), None, 1e-6, None, buf, buf)        # other type
    with pytest.raises(ValueError):
        B.glu_quantize_act_t("fp8", "silu", torch.zeros((256, 4), dtype=torch.bfloat16).t(), None, None, buf, buf)
    with pytest.raises(ValueError):
        B.glu_quantize_act_t("fp8", "silu", X, X[:, :128], None, buf, buf)
    with pytest.raises(KeyError):
        B.glu_quantize_act_t("fp8", "relu", X, None, None, buf, buf, 0)


def test_helpers_refuse_column_vectors_of_another_type_or_length():
    X = torch.zeros((4, 256), dtype=torch.bfloat16)
    for bad in (torch.ones(256, dtype=torch.bfloat16), torch.ones(128), torch.ones(512)[::2], torch.ones(256, dtype=torch.int32)):
        with pytest.raises(ValueError):
            B._column_vector(bad, 256, -1, "gamma")
    assert B._column_vector(None, 256, -1, "gamma") is None
    with pytest.raises(ValueError, match="current CUDA device"):
        B.glu_quantize_act_t("fp8", "silu", X, None, None, X, X, 0)


def test_layer_refuses_to_be_fed_where_it_cannot():
    from bit_w4a4_quantized_group_b200.layer import W4A4LowRankLinear
    rng = np.random.default_rng(0)
    prep = {"lam": np.ones(256, np.float32), "R_nk": rng.standard_normal((128, 256)).astype(np.float32), "act_gscale": 1.0}
    X = torch.zeros((2, 256), dtype=torch.bfloat16)
    for fmt, rank in (("fp8", 16), ("w8a8", 0), ("nvfp4", 0)):
        prep["L1_rk"] = np.zeros((rank, 256), np.float32)
        prep["L2_nr"] = np.zeros((128, rank), np.float32)
        lin = W4A4LowRankLinear(fmt, 128, 256, P.pack(fmt, prep), prep["lam"], 1.0, device="cpu")
        with pytest.raises(ValueError, match="without a low-rank branch"):
            lin.forward_normed(X, None, torch.ones(256))
        with pytest.raises(ValueError, match="without a low-rank branch"):
            lin.forward_activated("silu", X)
    prep["L1_rk"], prep["L2_nr"] = np.zeros((0, 256), np.float32), np.zeros((128, 0), np.float32)
    lam = rng.uniform(0.5, 2, 256).astype(np.float32)
    lin = W4A4LowRankLinear("fp8", 128, 256, P.pack("fp8", prep), lam, 1.0, device="cpu")
    with pytest.raises(ValueError, match="fold_gamma"):
        lin.forward_normed(X, None, None)
    g = torch.from_numpy(rng.uniform(0.5, 2, 256)).to(torch.bfloat16)
    assert torch.equal(lin.fold_gamma(g), g.float() / torch.from_numpy(lam))


def test_hot_calls_convert_arguments_like_ctypes():
    """The extension behind the helpers gives every entry point the arguments that ctypes gives it: the
    same refusal for the same bad argument, position by position, and no call on a wrong type."""
    if B._hot() is B.load():
        pytest.skip("built without Python's headers")
    good = {
        "svdq_quantize_act_lowrank_down": [5, 4, 256, 16, _P, _P, 1.0, _P, _P, _P, _P, None],
        "svdq_w4a4_gemm_lowrank_up": [5, 4, 128, 256, 16, _P, _P, 1.0, _P, _P, 1.0, _P, _P, _P, _P, None],
        "svdq_rmsnorm_quantize_act": [5, 4, 256, _P, 256, _P, 256, _P, 1e-6, 2 * _P, 256, _P, _P, None],
        "svdq_glu_quantize_act": [5, 1, 4, 256, _P, 256, _P, 256, _P, _P, _P, None],
    }
    refused = 0
    for name, args in good.items():
        fast, plain = getattr(B._hot(), name), getattr(B.load(), name)
        for i, v in enumerate(args[:-1]):
            bad = args[:]
            bad[i] = (-1.0 if name == "svdq_rmsnorm_quantize_act" else 3.0) if isinstance(v, float) else v + 4 if v == _P or v == 2 * _P else -3
            a, b = fast(*bad), plain(*bad)
            assert a == b == B.SVDQ_ERR_INVALID_ARG, (name, i, a, b)
            refused += 1
            with pytest.raises(TypeError):
                fast(*(args[:i] + ["x"] + args[i + 1:]))
        with pytest.raises(TypeError):
            fast(*args[:-1])
    assert refused == 50
