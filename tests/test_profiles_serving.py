"""The committed counters of the operators around the paged FP4 cache are of
their kernels' code as committed (comments and spacing aside)."""
import hashlib
import os
import re

import pytest

from fp4_kv_cache_sparse_gb300 import build as lib_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def code_hash(files):
    h = hashlib.sha256()
    for f in files:
        text = open(os.path.join(lib_build.CSRC, f)).read()
        h.update(" ".join(re.sub(r"//[^\n]*", "", text).split()).encode())
    return h.hexdigest()[:16]


@pytest.mark.parametrize("name,kernel", [
    ("page_select.md", "select.cu"), ("kv_append.md", "append.cu"), ("page_means.md", "page_means.cu"),
    ("paged_pair.md", "paged_pair.cu"),
])
def test_counters_name_the_current_code(name, kernel):
    text = open(os.path.join(ROOT, "profiles", name)).read()
    files = re.search(r"^sources: (.*)$", text, re.M).group(1).split(", ")
    assert files[0] == kernel
    assert re.search(r"^code_sha256_16: ([0-9a-f]{16})$", text, re.M).group(1) == code_hash(files)
