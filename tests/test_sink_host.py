"""Properties of the sink-window and norm + rotation kernels that need no GPU."""

import os
import random
import re
import subprocess

import pytest

from linear_attention_sequence_causal_b200 import build

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


@pytest.fixture(scope="module")
def walk_check(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("walk") / "sink_walk_check")
    subprocess.run([build.nvcc(), "-std=c++17", "-O2", "--expt-relaxed-constexpr", "-I" + CSRC, "-I" + build.INCLUDE, "-o", exe,
                    os.path.join(ROOT, "tests", "sink_walk_check.cu")], check=True)
    return exe


def _walk(exe, cases):
    """cases: (Hq, Hkv, N, w, sinks, d, lengths)."""
    text = "".join(f"{len(ln)} {Hq} {Hkv} {N} {w} {s} {d} {' '.join(map(str, ln))}\n" for Hq, Hkv, N, w, s, d, ln in cases)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(out) == len(cases)
    for case, line in zip(cases, out):
        assert line == "ok", (case, line)


@pytest.mark.parametrize("d", [64, 128])
def test_gradient_units_sum_every_pair_once(walk_check, d):
    """Short sequences of a padded batch: whole chunks of the sinks' pairs are padding."""
    _walk(walk_check, [
        (1, 1, 1100, 64, 4, d, [1100, 300, 130, 0]), (2, 2, 1400, 64, 4, d, [500, 70]), (4, 1, 1500, 40, 33, d, [700, 90]),
        (8, 2, 1100, 1, 64, d, [1099, 129]), (3, 1, 900, 100, 16, d, [900, 101, 100, 99, 1]), (1, 1, 130, 2000, 8, d, [3, 130]),
        (2, 1, 257, 129, 0, d, [257, 255]),
    ])


def test_gradient_units_sum_every_pair_once_on_drawn_shapes(walk_check):
    rng = random.Random(5)
    cases = []
    for _ in range(120):
        Hq, Hkv = rng.choice([(1, 1), (2, 1), (3, 1), (4, 2), (6, 3)])
        N = rng.randint(1, 700)
        cases.append((Hq, Hkv, N, rng.choice([1, 2, 5, 33, 64, 100, 129, 400, 1000]), rng.choice([0, 1, 4, 16, 33, 64]),
                      rng.choice([64, 128]), [rng.randint(0, N) for _ in range(rng.randint(1, 3))]))
    _walk(walk_check, cases)


@pytest.mark.parametrize("name,function", [("sink_fwd_tc.cu", "fwd_rows"), ("sink_fwd_narrow_tc.cu", "narrow_rows"),
                                           ("sink_bwd_tc.cu", "dq_rows"), ("sink_bwd_tc.cu", "dkv_rows")])
def test_row_warps_leave_a_wait_together(name, function):
    """A lane that gave up a wait alone would be missed by its warp's next joint instruction."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    at = text.index(f"void {function}(")
    body = text[at:text.index("\ntemplate <", at)]
    waits = re.findall(r"(\w*wait\w*)\(", body)
    assert {w for w in waits if "bulk" not in w and "tmem" not in w} <= {"fwait_joint", "wait_joint", "wait_warp", "gwait_joint"}
    assert len(waits) > 4
