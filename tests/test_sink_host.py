"""Properties of the sink-window and norm + rotation kernels that need no GPU."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_sequence_causal_b200", "csrc")
FILES = ("sink_simt.cu", "sink_decode.cu", "sink_fwd_tc.cu", "sink_fwd_narrow_tc.cu", "sink_bwd_tc.cu", "qk_norm_rope.cu")


def _kernels(text):
    """(name, body) of every kernel definition."""
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\(", text):
        at = depth = text.index("{", text.index(")", m.end()))
        level = 0
        while True:
            level += {"{": 1, "}": -1}.get(text[depth], 0)
            depth += 1
            if level == 0:
                break
        yield m.group(1), re.sub(r"//[^\n]*", "", text[at:depth])


@pytest.mark.parametrize("name", FILES)
def test_nothing_is_read_before_the_dependency_wait(name):
    """Work of earlier kernels is visible only behind grid_dependency_wait(), so no body reads
    lengths, positions or a tensor, and none lets its successor start, ahead of it."""
    with open(os.path.join(CSRC, name)) as f:
        found = list(_kernels(f.read()))
    assert found
    for kernel, body in found:
        assert "grid_dependency_wait();" in body, kernel
        ahead = body[:body.index("grid_dependency_wait();")]
        for word in ("seq_len", "lengths", "positions", ".p)", "partial[", "delta[", "grid_launch_dependents", "atomic"):
            assert word not in ahead, f"{kernel}: {word} before the wait"
