"""Row strides of mla_kv_append that no memory has are refused before any launch."""
import ctypes

import pytest

import fp4_kv_cache_sparse_gb300 as mla
from fp4_kv_cache_sparse_gb300 import build as lib_build

A = ctypes.c_void_p(1 << 20)            # aligned fake device address: never dereferenced


@pytest.mark.parametrize("dtype,stride,n", [(0, 1 << 61, 2), (2, (1 << 60) // 8 + 8, 8), (0, (1 << 63) - 8, 2),
                                            (1, 1 << 31, (1 << 31) - 1)])
def test_offsets_past_64_bits(dtype, stride, n):
    lib_build.build()
    assert mla.load().mla_kv_append(mla.KV_FP4_288, dtype, A, stride, n, None, 0, None, A, A, 8, None, None) == 1
