"""Kernels launched as programmatic dependents run beside the end of the
stream's previous kernel until griddepcontrol.wait.  What that kernel writes
must not be read by non-coherent loads, which promise that nobody writes it
while this kernel lives and may be moved above the wait: no __ldg, no
ld.global.nc, and no const __restrict__ pointer in the files of these kernels
(page_plan.cu: in the dependent kernel's parameters)."""
import os
import re

import pytest

from fp4_kv_cache_sparse_gb300 import build as lib_build


def source(name):
    text = open(os.path.join(lib_build.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def dependent_kernels(text):
    """(name, parameters) of every kernel whose body waits for the kernel before it."""
    found = []
    for m in re.finditer(r"__global__[^{;]*?\b(\w+_kernel)\s*\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        after = text.index("{", at)
        depth, end = 1, after + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        if "griddepcontrol.wait" in text[after:end]:
            found.append((m.group(1), text[m.end():at]))
    return found


@pytest.mark.parametrize("name,kernels", [
    ("paged.cu", {"paged_decode_kernel", "paged_merge_kernel", "paged_merge_many_kernel"}),
    ("page_plan.cu", {"slot_map_kernel"}),
    ("combine.cu", {"combine_kernel", "rope_fp8_kernel"}),
])
def test_dependent_kernels_read_by_plain_loads(name, kernels):
    text = source(name)
    found = dependent_kernels(text)
    assert {k for k, _ in found} == kernels
    assert "__ldg" not in text and "ld.global.nc" not in text
    for kernel, parameters in found:
        assert not re.search(r"\bconst\b[^,]*__restrict__", parameters), kernel
