"""The activation's stated range at its ends: gates so negative that the reciprocal of 1 + exp(-t) leaves
fp32's normal range, beside an up or a lambda that would bring the product back into it.

Model in 64 bits: f = 1 / ((1 + exp(-t)) lambda), y = gate f up; where 1 + exp(-t) or its product with lambda
is above 2^126, 0 is right as well.  Tolerance: the interface's 2^-15 relatively (four roundings of an
exponent of at most 126: ln 2 * 126 * 4 = 350 units of 2^-24, and about 10 for the hardware's exponential,
its reciprocal and the products: < 2^9).  No input has a denominator within 2^-10 of 2^126, so that the
exponential's own error (below 2^-15) decides nowhere which side a value is on; every product is normal.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from bit_w4a4_quantized_group_b200 import binding as B
from bit_w4a4_quantized_group_b200 import build as BUILD

import fp8_helpers as F
from gpu_helpers import check_device_error, dev_bf16
import oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    BUILD.build()
    B.load()


def _t(x, act):
    return x if act == "silu" else 2.0 * np.sqrt(2.0 / np.pi) * (x + 0.044715 * x ** 3)


def _run(act, gate, up, lam):
    M, K = gate.shape
    sz = B.svdq_buffer_sizes("fp8", M, 128, K, 0)
    codes = torch.full((sz.a_codes,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((sz.a_scales,), 0xA5, dtype=torch.uint8, device="cuda")
    B.glu_quantize_act_t("fp8", act, dev_bf16(gate), None if up is None else dev_bf16(up),
                         None if lam is None else torch.from_numpy(lam).cuda(), codes, scales)
    check_device_error()
    return codes.cpu().numpy().reshape(M, K), F.scales_of(scales.cpu().numpy(), M, K)


def _check(act, gate, up, lam, both_sides=True):
    with np.errstate(over="ignore"):
        d = 1.0 + np.exp(-_t(gate.astype(np.float64), act))
        den = d if lam is None else d * lam.astype(np.float64)
    edge = 2.0 ** 126
    assert np.all(np.abs(np.maximum(d, den) / edge - 1.0) > 2.0 ** -10)
    gone = np.maximum(d, den) > edge
    assert not both_sides or 0.1 < gone.mean() < 0.9
    y = gate / den
    assert np.all(gone | (np.abs(y) >= 2.0 ** -126))
    if up is not None:
        y = y * up.astype(np.float64)
    assert np.all(gone | (np.abs(y) >= 2.0 ** -120)) and np.abs(y).max() < 2.0 ** 127
    codes, sb = _run(act, gate, up, lam)
    y = np.where(gone & ((codes & 0x7F) == 0), 0.0, y)
    F.check_quantized(codes, sb, y, 2.0 ** -15)


def _grid(act, n=64):
    """Gates on both sides of where 1 + exp(-t) reaches 2^126 (t = -87.3), one for each group."""
    lo, hi = (-100.0, -70.0) if act == "silu" else (-11.0, -7.0)
    return O.bf16_rn(np.linspace(lo, hi, n).astype(np.float32))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("exp", [20, 100])
@pytest.mark.parametrize("mixed", [False, True])
def test_very_negative_gates_beside_large_up(act, exp, mixed):
    """mixed: an ordinary gate stands next to each extreme one, with an up that leaves it small."""
    g = np.repeat(_grid(act), 128)[None].repeat(3, 0)
    rng = np.random.default_rng(exp)
    up = O.bf16_rn((np.ldexp(rng.uniform(1.0, 2.0, g.shape), exp) * rng.choice([-1.0, 1.0], g.shape)).astype(np.float32))
    if mixed:
        g[:, 1::2] = O.bf16_rn(rng.uniform(0.5, 2.0, g[:, 1::2].shape).astype(np.float32))
        up[:, 1::2] = np.ldexp(np.float32(1.0), exp - 115)
    _check(act, g, up, None)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("exp", [-100, -20, 30])
def test_very_negative_gates_over_small_and_large_lambda(act, gated, exp):
    g = np.repeat(_grid(act), 128)[None].repeat(2, 0)
    rng = np.random.default_rng(abs(exp))
    lam = np.ldexp(rng.uniform(1.0, 1.9, g.shape[1]), exp).astype(np.float32)
    if exp > 0:                     # the product reaches 2^126 before the exponential does
        g = O.bf16_rn((g * np.float32(0.85)).astype(np.float32)) if act == "silu" else O.bf16_rn((g * np.float32(0.95)).astype(np.float32))
    up = np.ldexp(rng.choice([-1.0, 1.0], g.shape), 60 if exp > 0 else 10).astype(np.float32) if gated else None
    with np.errstate(over="ignore"):
        den = (1.0 + np.exp(-_t(g.astype(np.float64), act))) * np.maximum(lam.astype(np.float64), 1.0)
    near = np.abs(den / 2.0 ** 126 - 1.0) <= 2.0 ** -9          # a gate this close moves away from the edge
    g[near] = _grid(act)[-1]
    if not gated and exp > 0:
        y = np.abs(g) / den
        g[(den < 2.0 ** 126) & (y < 2.0 ** -119)] = _grid(act)[0]       # values that may become 0 either way
    _check(act, g, up, lam)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_values_that_the_range_keeps(act):
    """Without lambda and with |up| <= 2^9 nothing above 2^-110 is lost, whatever the gate."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[torch.isfinite(x) & (x.float().abs() <= 2.0 ** 100)]
    gate = O.bf16_rn(x[: x.numel() // 512 * 512].float().numpy()).reshape(-1, 512)
    up = np.full_like(gate, 512.0)
    codes, sb = _run(act, gate, up, None)
    F.check_quantized(codes, sb, F.act64(gate.astype(np.float64), act) * 512.0, 2.0 ** -15, 2.0 ** -110)
