"""Rules that the exact operators' kernels keep and no run can show to be broken,
read from their source (no GPU needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "adaptive_vector_quantized_b200", "csrc")
FILES = ["cross_few.cu", "cross_few_f32.cu", "cross_join.cu", "cross_simt.cu", "cross_tc.cu", "cross_tc_bwd.cu", "qk_norm.cu"]


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def block(text, at):
    """The braces' content that begins at or after `at`, and where it ends."""
    i = text.index("{", at)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[i:j + 1], j + 1
    raise AssertionError("braces")


def always_at(body, what):
    """Where `what` first stands outside any inner braces, so that every path comes by it; the end if nowhere."""
    depth = 0
    for i, c in enumerate(body):
        depth += {"{": 1, "}": -1}.get(c, 0)
        if depth == 1 and body.startswith(what, i):
            return i
    return len(body)


def functions(text, head):
    """Name and body of every function whose declaration matches `head`."""
    for m in re.finditer(head, text):
        yield m.group("name"), block(text, text.index(")", m.end()))[0]


@pytest.mark.parametrize("name", FILES)
def test_kernels_read_nothing_before_their_wait(name):
    """A dependent launch makes what earlier work on the stream wrote visible at the kernel's own wait, not before."""
    text = source(name)
    parts = dict(functions(text, r"__device__ __forceinline__ void (?P<name>form_\w+)\("))
    reads = re.compile(r"__ldg\(|tma_load|load_tile<|fetch_tile<|load_rows\(|load8\(|key_count\(|key_seen\(|item_of\("
                       r"|key_item\(|row_item\(|lone_key\(|fill_weights<|join_row<|\ba\.(part|delta|lse|lone)\b|\bpart\[")
    kernels = list(functions(text, r"__global__ void __launch_bounds__\([^)]*\)\s*(?P<name>\w+)\("))
    assert kernels
    for kernel, body in kernels:
        used = re.findall(r"(form_\w+)<", body)
        for part in used or [None]:  # in its place, the others left out
            one = re.sub(r"(form_\w+)<[^;]*;", lambda m: parts[part][1:-1] if m.group(1) == part else "", body)
            first = reads.search(one)
            end = first.start() if first else len(one)
            assert always_at(one, "grid_dependency_wait()") < end, (kernel, part, first and first.group())


@pytest.mark.parametrize("name", ["cross_few.cu", "cross_tc.cu", "cross_tc_bwd.cu"])
def test_warps_wait_as_a_whole(name):
    """Where a wait runs out, lanes that each decide for themselves could part before an operation that names all
    32: a wait by lanes stands only where one lane works alone."""
    text = source(name)
    alone = []
    for m in re.finditer(r"if \(lane == 0\) \{", text):
        alone.append((m.start(), block(text, m.start())[1]))
    waits = [m.start() for m in re.finditer(r"guard\.wait\(", text)]
    assert waits and re.search(r"wait_(all|warp)\(guard", text)
    for w in waits:
        assert any(a < w < b for a, b in alone), text[w - 80:w + 60]
