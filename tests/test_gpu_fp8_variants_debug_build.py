"""The bounds-checking debug build on the FP8 variants of large calls: a clean device error word, and the
release build's outputs and choice of variants (each library in a child process of its own)."""
import os
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(lib, out):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "debug_child_fp8_variants.py"), lib, out],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    return dict(np.load(out))


@pytest.mark.gpu
def test_debug_build_is_clean_and_matches_release(tmp_path):
    from bit_w4a4_quantized_group_b200 import build as BUILD
    dbg = _run(BUILD.build(debug=True), str(tmp_path / "debug.npz"))
    rel = _run(BUILD.build(), str(tmp_path / "release.npz"))
    assert list(dbg["device_error"]) == [0, 0] and list(rel["device_error"]) == [0, 0]
    assert sorted(dbg) == sorted(rel) and len(rel) == 21
    pro = {int(rel[k][0]) for k in rel if k.startswith("prologue") and k.endswith("variant")}
    assert {v // 16 for v in pro} == {64, 128} and 16 * 128 + 1 in pro and 16 * 64 + 1 in pro and any(v % 16 > 1 for v in pro)
    gemm = {int(rel[k][0]) for k in rel if k.startswith("gemm") and k.endswith("variant")}
    assert {v if v > 0 else -(-v // 16) for v in gemm} == {-128, 128, 192, 256}
    for k in rel:
        assert np.array_equal(dbg[k], rel[k]), k
