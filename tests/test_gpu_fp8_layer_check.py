"""check=True of the FP8 layer's calls: a bounded wait that ran out raises instead of returning an output
that nothing vouches for.  The wait that runs out is the self-test's; no kernel is disturbed."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from bit_w4a4_quantized_group_b200 import binding as B
from bit_w4a4_quantized_group_b200 import build as BUILD
from bit_w4a4_quantized_group_b200 import prepare as P
from bit_w4a4_quantized_group_b200.layer import W4A4LowRankLinear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    BUILD.build()
    B.load()


@pytest.mark.parametrize("side_stream", [False, True])
def test_checked_calls_raise_after_a_wait_that_ran_out(side_stream):
    rng = np.random.default_rng(0)
    N, K = 128, 256
    prep = {"R_nk": rng.standard_normal((N, K)).astype(np.float32), "L1_rk": np.zeros((0, K), np.float32),
            "L2_nr": np.zeros((N, 0), np.float32), "act_gscale": 1.0}
    lin = W4A4LowRankLinear("fp8", N, K, P.pack("fp8", prep), None, 1.0)
    X = torch.ones((4, K), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream() if side_stream else torch.cuda.current_stream()):
        for call in (lin.forward, lambda x, check: lin.forward_normed(x, None, None, check=check),
                     lambda x, check: lin.forward_activated("silu", x, check=check)):
            want = call(X, check=True)
            assert B.svdq_selftest_bounded_wait(200_000, torch.cuda.current_stream().cuda_stream) == B.SVDQ_OK
            with pytest.raises(B.SvdqError, match="site 90") as e:
                call(X, check=True)
            assert e.value.status == B.SVDQ_ERR_TIMEOUT
            assert torch.equal(call(X, check=True), want)          # reading the word cleared it
