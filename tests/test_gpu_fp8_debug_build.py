"""The bounds-checking debug build on the FP8 operators: a clean device error word, and the release
build's outputs bit for bit (each library in a child process of its own)."""
import os
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(lib, out):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "debug_child_fp8.py"), lib, out],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    return dict(np.load(out))


@pytest.mark.gpu
def test_debug_build_is_clean_and_matches_release(tmp_path):
    from bit_w4a4_quantized_group_b200 import build as BUILD
    dbg = _run(BUILD.build(debug=True), str(tmp_path / "debug.npz"))
    rel = _run(BUILD.build(), str(tmp_path / "release.npz"))
    assert list(dbg["device_error"]) == [0, 0] and list(rel["device_error"]) == [0, 0]
    assert sorted(dbg) == sorted(rel) and len(rel) > 20
    for k in rel:
        assert np.array_equal(dbg[k], rel[k]), k
