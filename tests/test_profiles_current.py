"""The committed ncu summaries are of the kernel sources as committed: the
bench reports the measured DRAM traffic of its headline workload only then."""
import os
import re

import pytest

import bench

SUMMARIES = ["decode_fp8_b128_s2_h128.md", "decode_fp8_b64_h64.md", "decode_long_sparse_b32_h16.md",
             "launches_fp8_b128_s2_h128.md"]


@pytest.mark.parametrize("name", SUMMARIES)
def test_summary_names_the_current_sources(name):
    text = open(os.path.join(bench.ROOT, "profiles", name)).read()
    assert re.search(r"kernel_source_sha256_16:\s*([0-9a-f]{16})", text).group(1) == bench.kernel_hash()


def test_headline_has_its_measured_traffic():
    assert bench.profiled_traffic("fp8_b128_s2_h128") > 138.4e6 * 2       # the selected KV alone
