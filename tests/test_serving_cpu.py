"""The operators around the paged FP4 cache without a GPU: refusals of the C
ABI before any launch, the rotary table against its formulas, planning, and
the binding's checks of its arguments."""
import ctypes
import math

import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla
from fp4_kv_cache_sparse_gb300 import build as lib_build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = ctypes.c_void_p(1 << 20)            # aligned fake device address: never dereferenced
B = ctypes.c_void_p((1 << 20) + 4096)
MIS2 = ctypes.c_void_p((1 << 20) + 2)
MIS4 = ctypes.c_void_p((1 << 20) + 4)
MIS8 = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return mla.load()


# ---------------------------------------------------------------- page plan


def _plan(lib, cached=A, new=A, batch=4, table=A, max_pages=8, free=A, num_pages=64, num_free=A, lens=A, nfo=A, cu=A,
          slots=A, pos=A, max_new=16):
    return lib.mla_page_plan(cached, new, batch, table, max_pages, free, num_pages, num_free, lens, nfo, cu, slots,
                             pos, max_new, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(max_pages=0), INVALID), (dict(num_pages=0), INVALID), (dict(max_new=-1), INVALID),
    (dict(cached=None), INVALID), (dict(new=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
    (dict(num_free=None), INVALID), (dict(lens=None), INVALID), (dict(nfo=None), INVALID), (dict(cu=None), INVALID),
    (dict(slots=None), INVALID), (dict(pos=None), INVALID), (dict(slots=MIS2), INVALID), (dict(table=MIS2), INVALID),
    (dict(batch=8193), UNSUPPORTED), (dict(num_pages=1 << 25), UNSUPPORTED), (dict(max_pages=1 << 25), UNSUPPORTED),
])
def test_page_plan_refusals(lib, kw, status):
    assert _plan(lib, **kw) == status


# ---------------------------------------------------------------- rope


def _table(**kw):
    base = dict(rope_dim=64, theta=10000.0)
    base.update(kw)
    return mla.RopeTable(**base)


def _turns(table):
    """The table's steps as turns per position, signed."""
    return [(s - (1 << 64) if s >= 1 << 63 else s) / 2.0 ** 64 for s in table.c.step[:table.rope_dim // 2]]


def _close_turns(got, freqs):
    # A step is rounded to 2^-64 turns, the double f / (2 pi) to 2^-53 of itself (pow and the divisions: a few of those).
    for g, f in zip(got, freqs):
        want = f / (2 * math.pi)
        assert abs(g - want) <= 2.0 ** -65 + 8 * 2.0 ** -53 * abs(want)


@pytest.mark.parametrize("rd,theta", [(2, 10000.0), (64, 10000.0), (128, 5e5), (256, 1e6), (6, 50.0)])
def test_rope_table_plain_and_linear(rd, theta):
    f = [theta ** (-2.0 * j / rd) for j in range(rd // 2)]
    _close_turns(_turns(_table(rope_dim=rd, theta=theta)), f)
    t = _table(rope_dim=rd, theta=theta, scaling=mla.RopeScaling.linear(8.0))
    _close_turns(_turns(t), [v / 8.0 for v in f])
    assert t.c.factor == 1.0


def test_rope_table_yarn():
    rd, theta, scale, orig = 64, 10000.0, 40.0, 4096
    dim = lambda r: rd * math.log(orig / (r * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rd - 1)
    want = []
    for j in range(rd // 2):
        f, g = theta ** (-2.0 * j / rd), min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        want.append(f * (1 - g) + f / scale * g)
    t = _table(scaling=mla.RopeScaling.yarn(scale, orig))
    _close_turns(_turns(t), want)
    assert want[0] == 1.0 and abs(want[-1] * scale - theta ** (-62.0 / 64)) < 1e-15
    assert abs(t.c.factor - (0.1 * math.log(scale) + 1.0)) <= 2.0 ** -24 * t.c.factor
    assert _table(scaling=mla.RopeScaling.yarn(scale, orig), attention_factor=1.0).c.factor == 1.0


def test_rope_table_from_frequencies_keeps_signs_and_half_turns():
    t = mla.RopeTable(6, freqs=[math.pi, -math.pi / 2, 0.25])
    got = _turns(t)
    assert abs(got[0]) == 0.5 and got[1] == -0.25      # half a turn forward is half a turn back
    _close_turns(got[2:], [0.25])


@pytest.mark.parametrize("kw", [
    dict(rope_dim=0), dict(rope_dim=7), dict(theta=1.0), dict(theta=float("inf")), dict(theta=float("nan")),
    dict(attention_factor=float("inf")), dict(attention_factor=1e300), dict(rope_dim=258),
    dict(scaling=mla.RopeScaling.linear(0.5)), dict(scaling=mla.RopeScaling.linear(float("nan"))),
    dict(scaling=mla.RopeScaling(2, 4.0, 0.0)), dict(scaling=mla.RopeScaling(2, 4.0, 4096, 1.0, 32.0)),
    dict(scaling=mla.RopeScaling(9, 4.0)),
])
def test_rope_table_refusals(kw):
    with pytest.raises(mla.MLAError):
        _table(**kw)


def test_rope_table_frequency_refusals():
    with pytest.raises(mla.MLAError):
        mla.RopeTable(4, freqs=[4.0, 1.0])              # past half a turn a position
    with pytest.raises(mla.MLAError):
        mla.RopeTable(4, freqs=[float("nan"), 1.0])
    with pytest.raises(ValueError):
        mla.RopeTable(4, freqs=[1.0])


def _rope(lib, dtype=0, x=A, xr=4096, xh=512, y=B, yr=4096, yh=512, n=4, heads=8, d=512, off=448, pos=A, table=None):
    t = table or _table()
    return lib.mla_rope(dtype, x, xr, xh, y, yr, yh, n, heads, d, off, pos, t.ref, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(n=-1), INVALID), (dict(heads=0), INVALID),
    (dict(d=0), INVALID), (dict(off=-1), INVALID), (dict(off=449), INVALID), (dict(x=None), INVALID),
    (dict(y=None), INVALID), (dict(pos=None), INVALID), (dict(pos=MIS2), INVALID), (dict(dtype=2, x=MIS2), INVALID),
    (dict(xr=-1), INVALID), (dict(yh=256), INVALID),                       # overlapping heads
    (dict(yr=100, yh=512), INVALID),                                       # overlapping rows
    (dict(x=A, y=A, xr=4096, yr=8192), INVALID),                           # in place with other strides
    (dict(n=1 << 31, yr=4096), UNSUPPORTED), (dict(n=0, x=None, y=None), OK),
])
def test_rope_refusals(lib, kw, status):
    assert _rope(lib, **kw) == status


def test_rope_refuses_a_table_that_is_none(lib):
    t = mla.RopeTable(64)
    t.c.rope_dim = 1000
    assert _rope(lib, table=t) == INVALID
    t.c.rope_dim, t.c.layout = 64, 5
    assert _rope(lib, table=t) == INVALID


# ---------------------------------------------------------------- norm


def _norm(lib, dtype=0, x=A, xs=512, res=None, rs=512, w=A, eps=1e-6, out=None, os_=512, codes=A, cs=528, scales=A,
          ss=528, n=4, d=512):
    return lib.mla_rms_norm_fp8(dtype, x, xs, res, rs, w, eps, out, os_, codes, cs, scales, ss, n, d, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), INVALID), (dict(n=-1), INVALID), (dict(d=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(d=48), UNSUPPORTED), (dict(d=16416, xs=16416), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(x=MIS8), INVALID), (dict(xs=516), INVALID), (dict(w=MIS8), INVALID), (dict(res=MIS8), INVALID),
    (dict(res=A, rs=516), INVALID), (dict(out=A, os_=256), INVALID), (dict(codes=MIS4), INVALID),
    (dict(cs=524), INVALID), (dict(cs=504), INVALID), (dict(ss=8), INVALID), (dict(n=0, x=None), OK),
])
def test_norm_refusals(lib, kw, status):
    assert _norm(lib, **kw) == status


# ---------------------------------------------------------------- paged decode


def _problem(**kw):
    base = dict(batch=2, seq_len_q=1, h_q=16, max_pages=10, num_pages=20)
    base.update(kw)
    return mla.PagedProblem.make(**base)


def test_paged_problem_layout_matches_header():
    assert ctypes.sizeof(mla.PagedProblem) == 48
    assert mla.PagedProblem.num_pages.offset == 32 and mla.PagedProblem.sm_scale.offset == 44


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), INVALID), (dict(seq_len_q=0), INVALID), (dict(h_q=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(num_pages=1 << 25), UNSUPPORTED),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(sm_scale=float("inf")), INVALID), (dict(kv_format=mla.KV_NONE), INVALID),
    (dict(kv_format=mla.KV_FP8_528), UNSUPPORTED), (dict(kv_format=mla.KV_BF16), UNSUPPORTED),
    (dict(head_dim=576), UNSUPPORTED), (dict(page_size=32), UNSUPPORTED), (dict(h_q=129), UNSUPPORTED),
    (dict(max_pages=1 << 25), UNSUPPORTED), (dict(batch=1 << 24, h_q=128), UNSUPPORTED),
])
def test_paged_problem_refusals(lib, kw, status):
    parts, ws = ctypes.c_int32(0), ctypes.c_size_t(0)
    p = _problem(**kw)
    assert lib.mla_paged_decode_plan(ctypes.addressof(p), 152, ctypes.byref(parts), ctypes.byref(ws)) == status
    assert lib.mla_paged_decode_fp4(ctypes.addressof(p), A, A, A, A, 152, A, 1 << 40, A, A, None, None) == status


@pytest.mark.parametrize("sm_scale", [2.4e38, -3.4e38])
def test_paged_problem_refuses_a_scale_that_overflows_in_units_of_ln_2(lib, sm_scale):
    prob = mla.PagedProblem.make(4, 1, 16, 10, 100, sm_scale=sm_scale)
    parts, ws = ctypes.c_int32(), ctypes.c_size_t()
    assert lib.mla_paged_decode_plan(ctypes.byref(prob), 152, ctypes.byref(parts), ctypes.byref(ws)) == INVALID
    prob.sm_scale = math.copysign(2.3e38, sm_scale)
    assert lib.mla_paged_decode_plan(ctypes.byref(prob), 152, ctypes.byref(parts), ctypes.byref(ws)) == 0


def test_paged_decode_argument_checks_before_any_launch(lib):
    p = _problem()
    parts, ws = mla.paged_decode_plan(p, 152)

    def call(q=A, kv=A, table=A, lens=A, nparts=parts, wsp=A, wsb=ws, out=A, lse=A):
        return lib.mla_paged_decode_fp4(ctypes.addressof(p), q, kv, table, lens, nparts, wsp, wsb, out, lse, None, None)

    for name in ("q", "kv", "table", "lens", "out", "lse"):
        assert call(**{name: None}) == INVALID
    for name in ("q", "kv", "out", "wsp"):
        assert call(**{name: MIS8}) == INVALID
    for name in ("table", "lens", "lse"):
        assert call(**{name: MIS2}) == INVALID
    assert call(nparts=0) == INVALID
    assert call(wsb=ws - 1) == WORKSPACE
    assert call(wsp=None) == WORKSPACE


@pytest.mark.parametrize("num_sms", [1, 7, 152])
def test_paged_plan_grows_with_parts_not_with_lengths(num_sms):
    parts, ws = mla.paged_decode_plan(_problem(), num_sms)
    assert 1 <= parts <= num_sms
    assert mla.paged_decode_plan(_problem(max_pages=1000, num_pages=5000), num_sms) == (parts, ws)


# ---------------------------------------------------------------- binding


def test_binding_refuses_a_stream_of_another_device():
    class Stream:
        device_index, cuda_stream = 1, 0

    def never(*args):
        raise AssertionError("the call must not be made")

    with pytest.raises(ValueError, match="stream of device 1"):
        mla._call(never, "mla_rope", 0, Stream())


def test_binding_refuses_cpu_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.rope(torch.zeros(4, 2, 64), i, mla.RopeTable(64))
    with pytest.raises(ValueError):
        mla.page_plan(i, i, i.view(4, 1), i, i, i, i, i, i, i)
    with pytest.raises(ValueError):
        mla.rms_norm_fp8(torch.zeros(4, 64), torch.zeros(64), 1e-6, i, i)
    with pytest.raises(ValueError):
        mla.paged_decode_fp4(_problem(), torch.zeros(2, 1, 16, 512), i, i, i, 1, i, i, i)
    with pytest.raises(TypeError):
        mla.rope(None, i, mla.RopeTable(64))
