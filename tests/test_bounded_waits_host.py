"""A bounded wait that a whole warp makes has one result for all its lanes.  Lanes that part at a wait (one
sees the barrier complete just as another's limit runs out) would meet again in instructions that name the
whole warp and have no limit: elect.sync, warp barriers, .aligned forms.  Read from the kernels' sources:
every wait is either the voting form or stands in a block that one lane runs, and a voting one never does.
Or it stands in a role (a block of one kind of warp) that does nothing by whole warps at all."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_w4a4_quantized_group_b200", "csrc")


def _waits(text):
    """(line, name, whether one lane alone runs it) of every wait_bounded* call."""
    text = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), text)
    one_lane = []           # for each open brace: does its block run in one lane?
    out = []
    token = re.compile(r"\{|\}|\b(wait_bounded\w*)\s*\(")
    for m in token.finditer(text):
        if m.group() == "{":
            head = text[max(text.rfind(c, 0, m.start()) for c in ";{}") + 1: m.start()]
            alone = re.search(r"if \((?:[^()]* && )?(?:lane|threadIdx\.x) == 0\)\s*$", head) or re.search(
                r"if \(ptx::elect_one\(\)\)\s*$", head)
            one_lane.append(bool(alone) or (bool(one_lane) and one_lane[-1]))
        elif m.group() == "}":
            one_lane.pop()
        else:
            out.append((text.count("\n", 0, m.start()) + 1, m.group(1), bool(one_lane) and one_lane[-1]))
    assert not one_lane
    return out


def _role_of_single_lanes(text, line):
    """Whether the innermost block `if (warp ...) {` around the line holds no instruction of whole warps."""
    text = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), text)
    at = sum(len(x) + 1 for x in text.split("\n")[: line - 1])
    start = max((m.end() for m in re.finditer(r"if \(warp [^{;]*\) \{", text) if m.end() <= at), default=-1)
    depth, end = 1, start
    while start >= 0 and depth > 0:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
    return start <= at < end and not re.search(
        r"__syncwarp|_sync\(|elect_one|barrier|tmem_|tc_fence|_warp\(", text[start: end])


def test_the_reader_tells_one_lane_from_a_warp():
    src = """
    if (warp == 0) { if (lane == 0) { for (;;) { if (!wait_bounded(a)) break; } } __syncwarp(); }
    else if (warp == 1) { if (wait_bounded_warp(b)) { } // if (lane == 0) {
      wait_bounded(c); if (ok && lane == 0) { wait_bounded_call(d); } if (ptx::elect_one()) { wait_bounded_warp(e); } }
    """
    assert [(n, alone) for _, n, alone in _waits(src)] == [
        ("wait_bounded", True), ("wait_bounded_warp", False), ("wait_bounded", False), ("wait_bounded_call", True),
        ("wait_bounded_warp", True)]
    role = "if (warp < 2) {\n if (!wait_bounded(a)) break;\n mbar_arrive(b);\n }\n else if (warp == 2) {\n wait_bounded(a);\n%s}\n"
    assert _role_of_single_lanes(role % "", 2) and _role_of_single_lanes(role % "__syncwarp();", 2)
    assert _role_of_single_lanes(role % "", 6) and not _role_of_single_lanes(role % "__syncwarp();", 6)


@pytest.mark.parametrize("name", ["gemm_fp8.cu", "gemm_fp8_small.cu", "prologue_fp8.cu", "gemm_int4.cu", "gemm_nvfp4.cu",
                                  "gemm_w8a8.cu", "prologue.cu", "selftest.cu"])
def test_waits_of_whole_warps_are_voted_on(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        text = f.read()
    waits = _waits(text)
    assert waits
    wrong = [(line, n) for line, n, alone in waits if n.endswith("_warp") == alone and not _role_of_single_lanes(text, line)]
    assert not wrong, f"{name}: {wrong}"


def test_barriers_in_aligned_form_gather_the_warp_first():
    """barrier.cluster.*.aligned and bar.sync want all lanes of a warp; a role that branched by lane (a
    producer whose lane 0 starts the copies) may reach them in parts unless it is gathered."""
    found = 0
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r'asm volatile\(\s*"(barrier\.cluster[^"]*\.aligned|bar\.sync)', text):
            body = text[text.rfind("{", 0, m.start()): m.start()]
            assert "__syncwarp();" in body, (name, text.count("\n", 0, m.start()) + 1)
            found += 1
    assert found == 4


def _roles(kernel):
    """(start, end) of the blocks of a kernel's roles: the branches on the warp that hold waits."""
    out, stack = [], []
    for m in re.finditer(r"[{}]", kernel):
        if m.group() == "{":
            head = kernel[max(kernel.rfind(c, 0, m.start()) for c in ";{}") + 1: m.start()]
            chained = bool(re.search(r"\belse\s*$", head)) and bool(out) and kernel[out[-1][1]: m.start()].strip() == "else"
            stack.append((m.end(), chained or bool(re.search(r"if \((warp|first)\b[^{;]*$", head))))
        else:
            start, role = stack.pop()
            if role and not any(r for _, r in stack):
                out.append((start, m.end()))
    return [(a, b) for a, b in out if "wait_bounded" in kernel[a: b]]


@pytest.mark.parametrize("name,roles", [("gemm_fp8.cu", 4), ("gemm_fp8_small.cu", 4), ("prologue_fp8.cu", 3), ("gemm_nvfp4.cu", 4),
                                        ("gemm_w8a8.cu", 3), ("gemm_int4.cu", 4), ("prologue.cu", 2), ("selftest.cu", 1)])
def test_roles_stay_for_their_copies_after_an_abort(name, roles):
    """A role that issues copies or MMAs looks at the abort flag when it ends; one that does not stays where its
    own wait ran out; and so does a wait outside of the roles, before the next barrier."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    starts = [m.start() for m in re.finditer(r"__global__ void ", text)] + [len(text)]
    kernels = [k for k in (text[a: b] for a, b in zip(starts, starts[1:])) if "wait_bounded" in k]
    assert len(kernels) == 1
    kernel = kernels[0][kernels[0].index("{"):]
    kernel = kernel[: re.search(r"\n}\n", kernel).end()]
    found = _roles(kernel)
    assert len(found) == roles
    for a, b in found:
        role = kernel[a: b]
        last = role.rindex("wait_bounded")
        if re.search(r"tma_load|umma_|tmem_cp", role):
            assert re.search(r"end_issuing_role(_of_cta)?\(abort_flag\);", role[last:]), role[:200]
        else:
            assert re.search(r"leave_aborted\(|stay_after_abort\(", role[last:]), role[:200]
    for m in re.finditer(r"wait_bounded", kernel):
        if not any(a <= m.start() < b for a, b in found):
            rest = kernel[m.start():]
            assert rest.index("leave_aborted(abort_flag)") < re.search(r"cluster_|__syncthreads", rest).start()
    # a CTA of the cluster that has ended must not be told: only where all of them meet at the end, always
    tells = re.search(r"leave_aborted\(|end_issuing_role\(", kernel)
    meets = kernel[kernel.rindex("cluster_"):] if "cluster_" in kernel else ""
    assert bool(tells) == (name not in ("prologue.cu", "gemm_int4.cu"))
    if tells:
        line = kernel[: kernel.rindex("cluster_")].split("\n")[-1]
        assert meets.startswith(("cluster_sync();", "cluster_wait();")) and line.strip() in ("ptx::", "if (ks > 1) ptx::"), line
