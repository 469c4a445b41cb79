"""A device whose number of SMs cannot be read must give an error status, not a division by it."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_w4a4_quantized_group_b200", "csrc")


def test_the_sm_count_is_checked_before_it_is_used():
    with open(os.path.join(CSRC, "svdq_api.cu"), encoding="utf-8") as f:
        text = f.read()
    calls = [m.start() for m in re.finditer(r"device_sm_count\(\)(?! \{)", text)]
    assert len(calls) == 2                                  # the prologue's and the GEMM's
    for at in calls:
        line, after = text[text.rfind("\n", 0, at): text.find("\n", at)], text[text.find("\n", at):]
        name = re.search(r"const int (\w+) = ", line).group(1)
        assert re.match(rf"\s*if \({name} <= 0\) return SVDQ_ERR_CUDA;", after), line.strip()


def test_what_calls_of_several_threads_share_is_atomic_or_locked():
    """Calls run without the interpreter lock, so that two threads may be in the library at once: what it keeps
    between calls is thread-local, atomic, or behind a mutex or a once flag."""
    allowed = re.compile(r"static (std::atomic<|std::mutex|std::once_flag|constexpr|const |__device__|__global__|void|Seen seen|int n = 0|"
                         r"PFN_cuTensorMapEncodeTiled_v12000 fn)")
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cpp", ".cuh", ".h")):
            continue
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"^\s+static [^\n;({]*[;({=\[]", text, re.M):
            line = m.group().strip()
            assert allowed.match(line) or line.endswith("("), (name, line)
