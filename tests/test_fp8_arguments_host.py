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
