"""What the FP8 helpers and the layer refuse before any launch (no GPU): tensors whose bits would be
read as another type, or buffers and rows that a call would write or read past the end of."""
import pytest
import torch

from bit_w4a4_quantized_group_b200 import binding as B
from bit_w4a4_quantized_group_b200 import build as BUILD


@pytest.fixture(scope="module", autouse=True)
def lib():
    BUILD.build()
    return B.load()


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32, torch.int16, torch.float64])
def test_row_helpers_read_bf16_alone(dtype):
    """Another type's bits are never read as bf16, whatever the operands agree on among themselves."""
    X = torch.zeros((4, 256), dtype=dtype)
    buf = torch.zeros(2048, dtype=torch.uint8)
    with pytest.raises(ValueError, match="bfloat16"):
        B.rmsnorm_quantize_act_t("fp8", X, X, None, 1e-6, X, buf, buf, 0)
    with pytest.raises(ValueError, match="bfloat16"):
        B.glu_quantize_act_t("fp8", "silu", X, X, None, buf, buf, 0)
    with pytest.raises(ValueError, match="bfloat16"):
        B.glu_quantize_act_t("fp8", "silu", X.to(torch.bfloat16)[0], None, None, buf, buf, 0)      # one row as a vector


@pytest.fixture
def no_launch(monkeypatch):
    """Host tensors pass for those of the current device, and a call that gets as far as the library
    fails the test."""
    class Library:
        def __getattr__(self, name):
            def call(*args):
                raise AssertionError(f"{name} was called")
            return call
    monkeypatch.setattr(B, "_calls", Library())
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: getattr(t, "_dev", 0))
    monkeypatch.setattr(B, "_stream", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: type("Stream", (), {"cuda_stream": 0}))


def _bytes(n, dtype=torch.uint8, dev=0):
    t = torch.zeros(n, dtype=dtype)
    t._dev = dev
    return t


_M, _K = 130, 640
_CODES, _SCALES = _M * _K, 256 * 8
_BAD_BUFFERS = {
    "codes too short": (_bytes(_CODES - 1), _bytes(_SCALES)),
    "scales without the padding rows": (_bytes(_CODES), _bytes(_M * 8)),
    "scales without the padding groups": (_bytes(_CODES), _bytes(256 * 5)),
    "codes of another type": (_bytes(_CODES, torch.int32), _bytes(_SCALES)),
    "scales of another type": (_bytes(_CODES), _bytes(_SCALES, torch.float32)),
    "codes not dense": (_bytes(2 * _CODES)[::2], _bytes(_SCALES)),
    "scales repeated": (_bytes(_CODES), _bytes(1).expand(_SCALES)),
    "codes on another device": (_bytes(_CODES, dev=1), _bytes(_SCALES)),
    "scales on the host": (_bytes(_CODES), _bytes(_SCALES, dev=-1)),
}


@pytest.mark.parametrize("which", sorted(_BAD_BUFFERS))
def test_row_helpers_refuse_buffers_that_do_not_hold_the_outputs(which, no_launch):
    X = torch.zeros((_M, _K), dtype=torch.bfloat16)
    codes, scales = _BAD_BUFFERS[which]
    with pytest.raises(ValueError, match="a_codes, a_scales"):
        B.rmsnorm_quantize_act_t("fp8", X, None, None, 1e-6, None, codes, scales)
    with pytest.raises(ValueError, match="a_codes, a_scales"):
        B.glu_quantize_act_t("fp8", "silu", X, X, None, codes, scales)


def test_row_helpers_take_buffers_of_the_stated_size(no_launch):
    X = torch.zeros((_M, _K), dtype=torch.bfloat16)
    sz = B.svdq_buffer_sizes("fp8", _M, 128, _K, 0)
    assert (sz.a_codes, sz.a_scales) == (_CODES, _SCALES)
    for extra in (0, 64):
        buf = _bytes(_CODES + extra), _bytes(_SCALES + extra)
        with pytest.raises(AssertionError, match="was called"):
            B.rmsnorm_quantize_act_t("fp8", X, None, None, 1e-6, None, *buf)
        with pytest.raises(AssertionError, match="was called"):
            B.glu_quantize_act_t("fp8", "silu", X, None, None, *buf)


def test_row_helpers_take_buffers_of_the_float8_types_that_they_hold(no_launch):
    X = torch.zeros((_M, _K), dtype=torch.bfloat16)
    codes, scales = torch.zeros((_M, _K), dtype=torch.float8_e4m3fn), torch.zeros(_SCALES, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    with pytest.raises(AssertionError, match="was called"):
        B.rmsnorm_quantize_act_t("fp8", X, None, None, 1e-6, None, codes, scales)
    with pytest.raises(AssertionError, match="was called"):
        B.glu_quantize_act_t("fp8", "silu", X, None, None, codes, scales)


def _layer(N, K):
    import numpy as np
    from bit_w4a4_quantized_group_b200 import prepare as P
    from bit_w4a4_quantized_group_b200.layer import W4A4LowRankLinear
    rng = np.random.default_rng(0)
    prep = {"R_nk": rng.standard_normal((N, K)).astype(np.float32), "L1_rk": np.zeros((0, K), np.float32),
            "L2_nr": np.zeros((N, 0), np.float32), "act_gscale": 1.0}
    return W4A4LowRankLinear("fp8", N, K, P.pack("fp8", prep), None, 1.0, device="cpu")


@pytest.mark.parametrize("width", [512, 128, 384])
def test_layer_is_fed_rows_of_its_own_width(width, no_launch):
    """A layer without smoothing has no [K] vector that would show it: the unsliced output of a
    gate-up layer (512 here) once went into a workspace of half its size."""
    lin = _layer(128, 256)
    X = torch.zeros((4, width), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=r"\[M, 256\]"):
        lin.forward_activated("silu", X)
    with pytest.raises(ValueError, match=r"\[M, 256\]"):
        lin.forward_activated("silu", X, X)
    with pytest.raises(ValueError, match=r"\[M, 256\]"):
        lin.forward_normed(X, None, None)
    with pytest.raises(ValueError, match=r"\[M, 256\]"):
        lin.forward_normed(X, X, torch.ones(width), 1e-6, X)
    with pytest.raises(ValueError, match=r"\[M, 256\]"):
        lin.forward_normed(X[:, :64].reshape(256), None, None)


def _calls(lin, X, Y):
    yield lambda: lin.forward(X, Y)
    yield lambda: lin.forward_normed(X, None, None, Y=Y)
    yield lambda: lin.forward_activated("silu", X, Y=Y)


@pytest.mark.parametrize("case", ["short", "float32", "float16", "transposed", "column slice", "expanded", "host", "other device"])
def test_layer_refuses_outputs_that_do_not_hold_its_result(case, no_launch):
    lin = _layer(128, 256)
    X = torch.zeros((4, 256), dtype=torch.bfloat16)
    Y = torch.zeros((4, 128), dtype=torch.bfloat16)
    bad = {"short": Y[:3], "float32": Y.float(), "float16": Y.half(), "transposed": torch.zeros((128, 4), dtype=torch.bfloat16).t(),
           "column slice": torch.zeros((4, 256), dtype=torch.bfloat16)[:, :128], "expanded": Y[:1].expand(4, 128)}.get(case, Y)
    if case in ("host", "other device"):
        bad._dev = -1 if case == "host" else 1
    for call in _calls(lin, X, bad):
        with pytest.raises(ValueError, match="Y: expected"):
            call()
    with pytest.raises(ValueError, match="Y: expected"):
        lin.gemm_only(4, bad)
    for call in _calls(lin, X, torch.zeros((5, 128), dtype=torch.bfloat16)):      # more rows than needed are no fault
        with pytest.raises(AssertionError, match="was called"):
            call()


@pytest.mark.parametrize("case", ["wide", "narrow", "float32", "float16", "transposed", "column slice", "one row as a vector"])
def test_layer_forward_refuses_inputs_that_are_not_its_rows(case, no_launch):
    lin = _layer(128, 256)
    X = torch.zeros((4, 256), dtype=torch.bfloat16)
    bad = {"wide": torch.zeros((4, 512), dtype=torch.bfloat16), "narrow": X[:, :128].contiguous(), "float32": X.float(),
           "float16": X.half(), "transposed": torch.zeros((256, 4), dtype=torch.bfloat16).t(),
           "column slice": torch.zeros((4, 512), dtype=torch.bfloat16)[:, :256], "one row as a vector": X[0]}[case]
    for call in (lambda: lin.forward(bad), lambda: lin.prologue_only(bad)):
        with pytest.raises(ValueError, match="X: expected"):
            call()


def test_layer_refuses_to_launch_on_another_device(no_launch, monkeypatch):
    lin = _layer(128, 256)
    X = torch.zeros((4, 256), dtype=torch.bfloat16)
    Y = torch.zeros((4, 128), dtype=torch.bfloat16)
    elsewhere = X.clone()
    elsewhere._dev = 1
    for call in (lambda: lin.forward(elsewhere), lambda: lin.prologue_only(elsewhere)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    for call in [*_calls(lin, X, Y), lambda: lin.prologue_only(X), lambda: lin.gemm_only(4, Y)]:
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


def test_hot_calls_take_the_streams_that_ctypes_takes():
    """A stream may be a raw handle, None, a c_void_p, or an object with one (torch.cuda.Stream)."""
    import ctypes

    class Stream:
        def __init__(self, p):
            self._as_parameter_ = p

    calls = {"svdq_glu_quantize_act": [5, 1, 0, 256, 1 << 20, 256, None, 0, None, 1 << 20, 1 << 20],     # M = 0: refused
             "svdq_quantize_act_lowrank_down": [5, 0, 256, 0, 1 << 20, None, 1.0, None, 1 << 20, 1 << 20, None]}
    for name, args in calls.items():
        for fn in (getattr(B.load(), name), getattr(B._hot(), name)):
            for stream in (None, 0, 1 << 40, ctypes.c_void_p(None), ctypes.c_void_p(1 << 40), Stream(ctypes.c_void_p(1 << 40)),
                           Stream(1 << 40), Stream(ctypes.c_void_p(None))):
                assert fn(*args, stream) == B.SVDQ_ERR_INVALID_ARG
            for wrong in ("x", 1.5, ctypes.c_int(3), object(), Stream("x")):
                if fn is getattr(B.load(), name) and isinstance(getattr(wrong, "_as_parameter_", wrong), str):
                    continue                       # ctypes takes a text for the address of its characters
                with pytest.raises((TypeError, ctypes.ArgumentError)):
                    fn(*args, wrong)
    assert isinstance(torch.cuda.Stream._as_parameter_, property)


def test_checked_calls_read_the_error_word(no_launch, monkeypatch):
    class Library:
        def __getattr__(self, name):
            return lambda *args: B.SVDQ_OK
    monkeypatch.setattr(B, "_calls", Library())
    words = []
    monkeypatch.setattr(B, "svdq_get_last_device_error", lambda stream: words.pop() if words else (B.SVDQ_OK, 0))
    lin = _layer(128, 256)
    X = torch.zeros((4, 256), dtype=torch.bfloat16)
    for call in (lambda **kw: lin.forward(X, **kw), lambda **kw: lin.forward_normed(X, None, None, **kw),
                 lambda **kw: lin.forward_activated("gelu", X, **kw)):
        words[:] = [(B.SVDQ_ERR_TIMEOUT, 12)]
        with pytest.raises(B.SvdqError, match="site 12"):
            call(check=True)
        assert not words
        words[:] = [(B.SVDQ_ERR_TIMEOUT, 12)]
        call()                                             # unchecked calls leave it for whoever polls it
        assert words and call(check=False) is not None
