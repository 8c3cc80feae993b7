"""Appending, page means, page selection and shared prefixes without a GPU:
refusals of the C ABI before any launch, planning, and the binding's checks."""
import ctypes

import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla
from fp4_kv_cache_sparse_gb300 import build as lib_build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = ctypes.c_void_p(1 << 20)            # aligned fake device address: never dereferenced
MIS2 = ctypes.c_void_p((1 << 20) + 2)
MIS8 = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return mla.load()


# ---------------------------------------------------------------- append


def _append(lib, fmt=mla.KV_FP4_288, dtype=0, x=A, stride=512, n=4, table=True, off=448, pos=A, slots=A, pool=A, pages=8,
            rope_dim=64, layout=0):
    t = mla.RopeTable(64)
    t.c.rope_dim, t.c.layout = rope_dim, layout
    return lib.mla_kv_append(fmt, dtype, x, stride, n, t.ref if table else None, off, pos, slots, pool, pages, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=mla.KV_BF16), UNSUPPORTED), (dict(fmt=mla.KV_NONE), INVALID), (dict(fmt=9), INVALID), (dict(dtype=3), INVALID),
    (dict(dtype=-1), INVALID), (dict(n=-1), INVALID), (dict(pages=-1), INVALID), (dict(off=-1), INVALID),
    (dict(off=449), INVALID), (dict(off=2 ** 31 - 1), INVALID), (dict(rope_dim=0), INVALID), (dict(rope_dim=65), INVALID),
    (dict(rope_dim=258), INVALID), (dict(layout=2), INVALID), (dict(x=None), INVALID), (dict(slots=None), INVALID),
    (dict(pool=None), INVALID), (dict(pos=None), INVALID), (dict(x=MIS8), INVALID), (dict(pool=MIS8), INVALID),
    (dict(slots=MIS2), INVALID), (dict(pos=MIS2), INVALID), (dict(stride=-512), INVALID), (dict(stride=516), INVALID),
    (dict(dtype=2, stride=514), INVALID), (dict(n=1 << 31), UNSUPPORTED), (dict(n=0, x=None, pos=None), OK),
    (dict(n=0, off=449), INVALID),
])
def test_append_refusals(lib, kw, status):
    assert _append(lib, **kw) == status


def test_append_without_a_table_takes_no_positions(lib):
    assert _append(lib, table=False, pos=None, n=0) == OK
    assert _append(lib, table=False, pos=None, off=511, slots=None) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(pages=-1), INVALID), (dict(n=-1), INVALID), (dict(pool=None), INVALID), (dict(slots=None), INVALID),
    (dict(means=None), INVALID), (dict(pool=MIS8), INVALID), (dict(means=MIS8), INVALID), (dict(slots=MIS2), INVALID),
    (dict(n=1 << 31), UNSUPPORTED), (dict(n=0, pool=None), OK),
])
def test_page_means_refusals(lib, kw, status):
    a = dict(pool=A, pages=8, slots=A, n=4, means=A)
    a.update(kw)
    assert lib.mla_page_means(a["pool"], a["pages"], a["slots"], a["n"], a["means"], None, None) == status


# ---------------------------------------------------------------- binding


def test_binding_refuses_cpu_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    u = torch.zeros(64, 288, dtype=torch.uint8)
    with pytest.raises(ValueError):
        mla.kv_append(torch.zeros(4, 512), i, u, mla.KV_FP4_288)
    with pytest.raises(ValueError):
        mla.page_means(u, i, torch.zeros(1, 528, dtype=torch.uint8))
    with pytest.raises(TypeError):
        mla.kv_append(None, i, u)
