"""The committed DRAM traffic rows belong to the sources as they are, so that the bench finds them."""

import os
import re

import pytest

import bench


def test_traffic_rows_match_the_sources():
    with open(os.path.join(bench.ROOT, "profiles", "dram_traffic.md")) as f:
        rows = re.findall(r"^\|\s*(\w+)\s*\|\s*([0-9a-f]{12})\s*\|\s*([0-9.eE+]+)\s*\|", f.read(), re.M)
    assert {r[0] for r in rows} == {"la_prefill", "swa_prefill"}
    for kind, digest, size in rows:
        assert bench.kernel_source_hash(kind) == digest, kind
        assert bench.measured_traffic(kind) == pytest.approx(float(size))
