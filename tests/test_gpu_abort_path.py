"""What a wait that ran out leaves behind, on the self-test kernel (no fault, no hang: every wait is bounded):
the other CTA of the cluster learns of the abort (site 92 otherwise), and both keep their memory for the time that copies and MMAs
on their way might need."""
import pytest

torch = pytest.importorskip("torch")

from bit_w4a4_quantized_group_b200 import binding as B
from bit_w4a4_quantized_group_b200 import build as BUILD

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    BUILD.build()
    B.load()


@pytest.mark.parametrize("limit_ms", [0.01, 2.0, 20.0])
def test_abort_reaches_the_cluster_and_memory_outlives_it(limit_ms):
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    assert B.svdq_get_last_device_error(stream) == (B.SVDQ_OK, 0)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    assert B.svdq_selftest_bounded_wait(int(limit_ms * 1e6), stream) == B.SVDQ_OK
    b.record()
    b.synchronize()
    assert B.svdq_get_last_device_error(stream) == (B.SVDQ_ERR_TIMEOUT, 90)
    # the limit and 1 ms of keeping
    assert limit_ms + 0.95 <= a.elapsed_time(b) < limit_ms + 1000.0
