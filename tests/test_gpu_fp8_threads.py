"""Calls of two Python threads at once, each on a stream of its own: the calls give the interpreter lock away,
so both are inside the library together; first calls of every size among them."""
import threading

import pytest

torch = pytest.importorskip("torch")

from bit_w4a4_quantized_group_b200 import binding as B
from bit_w4a4_quantized_group_b200 import build as BUILD

from gpu_helpers import check_device_error
from test_gpu_fp8_layer import _layer

pytestmark = pytest.mark.gpu


def test_two_threads_at_once():
    BUILD.build()
    B.load()
    sizes = [(1, 256, 640), (40, 384, 1152), (300, 1152, 640), (700, 2304, 640)]
    layers = [[_layer(n, k, r, 7 * i + r)[0] for (_, n, k) in sizes] for i, r in enumerate((16, 0))]
    g = torch.Generator(device="cuda").manual_seed(0)
    xs = [torch.randn((m, k), generator=g, device="cuda").to(torch.bfloat16) for m, _, k in sizes]
    torch.cuda.synchronize()
    out, errors = [[], []], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(30):
                    out[i] = [lin.forward(x) if i == 0 else lin.forward_activated("silu", x) for lin, x in zip(layers[i], xs)]
                    for lin, x in zip(layers[i], xs):
                        lin.prologue_only(x)
            stream.synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    check_device_error()
    for i in range(2):
        for lin, x, got in zip(layers[i], xs, out[i]):
            want = lin.forward(x) if i == 0 else lin.forward_activated("silu", x)
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    check_device_error()
