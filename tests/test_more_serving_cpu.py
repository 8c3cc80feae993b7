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


# ---------------------------------------------------------------- selected pages


def _sparse(**kw):
    base = dict(batch=2, seq_len_q=1, h_q=16, max_pages=40, num_pages=100, top_pages=8)
    base.update(kw)
    return mla.PagedSparseProblem.make(**base)


def test_problem_layouts_match_the_header():
    assert ctypes.sizeof(mla.PagedSparseProblem) == 56 and mla.PagedSparseProblem.num_pages.offset == 40
    assert mla.PagedSparseProblem.sm_scale.offset == 52
    assert ctypes.sizeof(mla.PagedSharedProblem) == 48 and mla.PagedSharedProblem.num_pages.offset == 32
    assert mla.PagedSharedProblem.sm_scale.offset == 44


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), INVALID), (dict(seq_len_q=0), INVALID), (dict(h_q=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(top_pages=0), INVALID), (dict(sink_pages=-1), INVALID), (dict(local_pages=0), INVALID),
    (dict(sink_pages=4, local_pages=5), INVALID), (dict(sink_pages=2 ** 31 - 1, local_pages=1), INVALID),
    (dict(sm_scale=float("nan")), INVALID), (dict(kv_format=mla.KV_NONE), INVALID), (dict(kv_format=mla.KV_FP8_528), UNSUPPORTED),
    (dict(head_dim=576), UNSUPPORTED), (dict(page_size=32), UNSUPPORTED), (dict(h_q=129), UNSUPPORTED),
    (dict(max_pages=1 << 25), UNSUPPORTED), (dict(num_pages=1 << 25), UNSUPPORTED), (dict(batch=1 << 26), UNSUPPORTED),
    (dict(top_pages=1 << 25), UNSUPPORTED), (dict(batch=1 << 20, seq_len_q=1 << 12), UNSUPPORTED),
])
def test_sparse_problem_refusals(lib, kw, status):
    parts, ws = ctypes.c_int32(0), ctypes.c_size_t(0)
    p = _sparse(**kw)
    assert lib.mla_paged_sparse_plan(ctypes.addressof(p), 152, ctypes.byref(parts), ctypes.byref(ws)) == status
    assert lib.mla_paged_sparse_decode_fp4(ctypes.addressof(p), A, A, A, A, A, 152, A, 1 << 60, A, A, A, None, None) == status


def test_sparse_argument_checks_before_any_launch(lib):
    p = _sparse()
    parts, ws = mla.paged_sparse_plan(p, 152)
    assert ws >= mla.paged_decode_plan(mla.PagedProblem.make(2, 1, 16, 8, 100), 152)[1] + 2 * 40 * 4

    def call(q=A, kv=A, means=A, table=A, lens=A, nparts=parts, wsp=A, wsb=ws, out=A, lse=A, sel=None):
        return lib.mla_paged_sparse_decode_fp4(ctypes.addressof(p), q, kv, means, table, lens, nparts, wsp, wsb, out, lse, sel,
                                               None, None)

    for name in ("q", "kv", "means", "table", "lens", "out", "lse"):
        assert call(**{name: None}) == INVALID
    for name in ("q", "kv", "means", "out", "wsp"):
        assert call(**{name: MIS8}) == INVALID
    for name in ("table", "lens", "lse", "sel"):
        assert call(**{name: MIS2}) == INVALID
    assert call(nparts=0) == INVALID
    assert call(wsb=ws - 1) == WORKSPACE
    assert call(wsp=None) == WORKSPACE
    assert lib.mla_paged_sparse_plan(None, 152, ctypes.byref(ctypes.c_int32()), ctypes.byref(ctypes.c_size_t())) == INVALID


# ---------------------------------------------------------------- shared prefixes


def _shared(**kw):
    base = dict(batch=4, seq_len_q=1, h_q=16, max_pages=10, max_prefix_pages=50, num_pages=100)
    base.update(kw)
    return mla.PagedSharedProblem.make(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), INVALID), (dict(seq_len_q=0), INVALID), (dict(h_q=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(max_prefix_pages=0), INVALID), (dict(groups=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(sm_scale=float("inf")), INVALID), (dict(kv_format=mla.KV_NONE), INVALID), (dict(kv_format=mla.KV_BF16), UNSUPPORTED),
    (dict(head_dim=576), UNSUPPORTED), (dict(page_size=128), UNSUPPORTED), (dict(h_q=129), UNSUPPORTED),
    (dict(groups=8193), UNSUPPORTED), (dict(max_prefix_pages=1 << 25), UNSUPPORTED), (dict(max_pages=1 << 25), UNSUPPORTED),
    (dict(groups=8192, max_prefix_pages=1 << 18), UNSUPPORTED), (dict(batch=1 << 22, max_prefix_pages=1 << 18), UNSUPPORTED),
])
def test_shared_problem_refusals(lib, kw, status):
    parts, ws = ctypes.c_int32(0), ctypes.c_size_t(0)
    p = _shared(**kw)
    assert lib.mla_paged_shared_plan(ctypes.addressof(p), 152, ctypes.byref(parts), ctypes.byref(ws)) == status
    assert lib.mla_paged_shared_decode_fp4(ctypes.addressof(p), A, A, A, A, A, A, A, 152, A, 1 << 60, A, A, None, None) == status


@pytest.mark.parametrize("kw", [dict(), dict(batch=64, h_q=128, max_prefix_pages=1024)])      # by SMs and by pairs of them
def test_shared_argument_checks_before_any_launch(lib, kw):
    p = _shared(**kw)
    parts, ws = mla.paged_shared_plan(p, 152)
    assert parts == 152

    def call(q=A, kv=A, start=A, ptable=A, plens=A, table=A, lens=A, nparts=parts, wsp=A, wsb=ws, out=A, lse=A):
        return lib.mla_paged_shared_decode_fp4(ctypes.addressof(p), q, kv, start, ptable, plens, table, lens, nparts, wsp, wsb,
                                               out, lse, None, None)

    for name in ("q", "kv", "start", "ptable", "plens", "table", "lens", "out", "lse"):
        assert call(**{name: None}) == INVALID
    for name in ("q", "kv", "out", "wsp"):
        assert call(**{name: MIS8}) == INVALID
    for name in ("start", "ptable", "plens", "table", "lens", "lse"):
        assert call(**{name: MIS2}) == INVALID
    assert call(nparts=0) == INVALID
    assert call(wsb=ws - 1) == WORKSPACE
    assert call(wsp=None) == WORKSPACE


def test_binding_refuses_shapes_and_types():
    i = torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(4, 1, 16, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mla.paged_sparse_decode_fp4(_sparse(), q, i, i, i, i, 1, i, q, i)
    with pytest.raises(ValueError):
        mla.paged_shared_decode_fp4(_shared(), q, i, i, i, i, i, i, 1, i, q, i)
    with pytest.raises(mla.MLAError):
        mla.paged_sparse_plan(_sparse(top_pages=1, sink_pages=1), 152)
    with pytest.raises(mla.MLAError):
        mla.paged_shared_plan(_shared(groups=0), 152)


# ---------------------------------------------------------------- kernels that start early


@pytest.mark.parametrize("name,kernels", [
    ("append.cu", {"kv_append_kernel"}), ("page_means.cu", {"page_means_kernel"}), ("select.cu", {"page_select_kernel"}),
    ("shared_merge.cu", {"shared_merge_kernel", "shared_merge_many_kernel"}), ("paged_pair.cu", {"paged_pair_kernel"}),
])
def test_dependent_kernels_read_by_plain_loads(name, kernels):
    """As test_dependent_loads.py has it: these kernels run beside the end of the one before until griddepcontrol.wait."""
    from test_dependent_loads import dependent_kernels, source
    text = source(name)
    found = dependent_kernels(text)
    assert {k for k, _ in found} == kernels
    assert "__ldg" not in text and "ld.global.nc" not in text
    for kernel, parameters in found:
        assert "__restrict__" not in parameters, kernel
