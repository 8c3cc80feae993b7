"""mla_rope against rotation in 64 bits.

Tolerance, per element of the pair (a, b) turned by phi: half a step of the
type (eps / 2 of the value, and the type's smallest subnormal), and in fp32
before that: the phase is a 24-bit float of at most half a turn (2^-24 pi),
the steps' and the truncated phase's share is under 2^-30 turns, sine and
cosine are within 2 units in the last place (2^-23 each), the factor, its
product, two products and a sum add 2^-24 each: under 12 * 2^-24 of
factor * (|a| + |b|) in all."""
import math

import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def freqs_of(table):
    return torch.tensor([(s - (1 << 64) if s >= 1 << 63 else s) / 2.0 ** 64 * 2 * math.pi
                         for s in table.c.step[:table.rope_dim // 2]], dtype=torch.float64, device=DEV)


def reference(x, pos, table, interleaved, offset=0, conjugate=False):
    """(result, bound) in 64 bits; the turns are taken from integer arithmetic, not from products of floats."""
    rd, n = table.rope_dim, x.shape[0]
    turns = torch.tensor([[(int(p) * s % (1 << 64)) / 2.0 ** 64 for s in table.c.step[:rd // 2]] for p in pos.tolist()],
                         dtype=torch.float64, device=DEV).view(n, *([1] * (x.dim() - 2)), rd // 2)
    cs, sn = torch.cos(2 * math.pi * turns), torch.sin(2 * math.pi * turns)
    if conjugate:
        sn = -sn
    y, bound = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    part = y[..., offset:offset + rd]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else part.chunk(2, -1)
    f = float(table.c.factor)
    u, v = (a * cs - b * sn) * f, (b * cs + a * sn) * f
    size = (a.abs() + b.abs()) * abs(f)
    info = torch.finfo(x.dtype)
    tiny = info.smallest_normal * info.eps
    tol = [info.eps / 2 * w.abs() + 12 * 2.0 ** -24 * size + tiny for w in (u, v)]
    join = (lambda p, q: torch.stack([p, q], -1).flatten(-2)) if interleaved else (lambda p, q: torch.cat([p, q], -1))
    y[..., offset:offset + rd], bound[..., offset:offset + rd] = join(u, v), join(*tol)
    return y, bound


def inputs(n, h, d, dtype, seed=0, maxpos=200000):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((n, h, d) if h else (n, d), generator=g, device=DEV).to(dtype)
    return x, torch.randint(0, maxpos, (n,), generator=g, device=DEV, dtype=torch.int32)


def check(got, want, bound):
    err = (got.double() - want).abs()
    assert torch.all(err <= bound), float((err - bound).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,h,d,rd,off", [
    (1, 1, 64, 64, 0), (5, 128, 512, 64, 448), (3, 7, 128, 128, 0), (33, 0, 512, 64, 448), (2, 3, 80, 80, 0),
    (9, 2, 78, 78, 0), (4, 3, 37, 10, 3), (4, 2, 37, 10, 27), (17, 1, 2, 2, 0), (300, 5, 96, 32, 32), (7, 2, 256, 256, 0),
    (2, 2, 100, 36, 64)])
def test_matches_64_bits(n, h, d, rd, off, interleaved, dtype):
    x, pos = inputs(n, h, d, dtype, seed=n + d)
    table = mla.RopeTable(rd, interleaved=interleaved, scaling=mla.RopeScaling.yarn(8.0, 4096))
    keep = x.clone()
    want, bound = reference(x, pos, table, interleaved, off)
    out = mla.rope(x, pos, table, offset=off, out=torch.full_like(x, float("nan")))
    check(out, want, bound)
    assert torch.equal(x, keep)
    back, b2 = reference(x, pos, table, interleaved, off, conjugate=True)
    assert mla.rope(x, pos, table, offset=off, conjugate=True) is x          # in place
    check(x, back, b2)
    rest = torch.ones(d, dtype=torch.bool, device=DEV)
    rest[off:off + rd] = False
    assert torch.equal(x[..., rest], keep[..., rest]) and torch.equal(out[..., rest], keep[..., rest])


@pytest.mark.parametrize("interleaved", [True, False])
def test_strided_heads_and_tails_leave_the_rest_alone(interleaved):
    """Heads that are slices of wider rows, in another order, at odd offsets."""
    g = torch.Generator(device=DEV).manual_seed(3)
    table = mla.RopeTable(64, interleaved=interleaved)
    base = torch.randn(6, 40, 200, generator=g, device=DEV).to(torch.bfloat16)
    pos = torch.arange(6, dtype=torch.int32, device=DEV) * 1000 + 7
    for view in (lambda t: t[:, 3:17, 8:136], lambda t: t[:, ::3, 5:133], lambda t: t.transpose(0, 1)[:6, :6, 72:],
                 lambda t: t[:, 1:9, 136:200]):
        whole = base.clone()
        x = view(whole)
        d = x.shape[-1]
        want, bound = reference(x, pos, table, interleaved, d - 64)
        touched = torch.zeros_like(whole, dtype=torch.bool)
        view(touched)[..., d - 64:] = True
        mla.rope(x, pos, table, offset=d - 64)
        check(x, want, bound)
        assert torch.equal(whole[~touched], base[~touched])
        out = torch.zeros(x.shape[1], x.shape[0], d, dtype=x.dtype, device=DEV).transpose(0, 1)
        y0, b0 = reference(view(base), pos, table, interleaved, d - 64)
        check(mla.rope(view(base), pos, table, offset=d - 64, out=out), y0, b0)


@pytest.mark.parametrize("position", [0, 1, 2 ** 24 + 1, 2 ** 31 - 1, -1, -2 ** 31])
def test_far_and_negative_positions_keep_their_angle(position):
    x, _ = inputs(2, 3, 128, torch.float32, seed=5)
    pos = torch.full((2,), position, dtype=torch.int32, device=DEV)
    table = mla.RopeTable(128, theta=500000.0)
    want, bound = reference(x, pos, table, True)
    check(mla.rope(x, pos, table, out=torch.empty_like(x)), want, bound)
    if position == 0:
        assert torch.equal(mla.rope(x, pos, table, out=torch.empty_like(x)), x)


def test_frequencies_match_the_formula():
    """The steps, and so the phases, are those of theta^(-2j/rd): 2^-60 turns a position at most."""
    f = freqs_of(mla.RopeTable(64))
    want = 10000.0 ** (-2.0 * torch.arange(32, dtype=torch.float64, device=DEV) / 64)
    assert torch.all((f - want).abs() <= 1e-15 * want + 2.0 ** -60)


@pytest.mark.parametrize("interleaved", [True, False])
def test_conjugate_is_the_gradient(interleaved):
    """<w, rope(x)> changes with x as conjugate rope(w) says: against differences in 64 bits of the same formula."""
    x, pos = inputs(3, 2, 48, torch.float32, seed=11)
    w, _ = inputs(3, 2, 48, torch.float32, seed=12)
    table = mla.RopeTable(32, interleaved=interleaved, scaling=mla.RopeScaling.yarn(16.0, 2048))
    grad = mla.rope(w, pos, table, offset=8, conjugate=True, out=torch.empty_like(w))
    base, _ = reference(x, pos, table, interleaved, 8)
    for n, h, d in ((0, 0, 0), (0, 1, 8), (1, 0, 9), (2, 1, 23), (1, 1, 24), (0, 0, 39), (2, 0, 47)):
        moved = x.double().clone()
        moved[n, h, d] += 1.0                       # linear in x: a step of one is exact
        y, _ = reference(moved, pos, table, interleaved, 8)
        diff = float(((y - base) * w.double()).sum())
        # As in the bound above, with the pair of w in place of (a, b).
        assert abs(float(grad[n, h, d]) - diff) <= 1e-5 * (1 + abs(diff))


def test_other_streams_and_graphs():
    x, pos = inputs(64, 16, 128, torch.bfloat16, seed=1)
    table = mla.RopeTable(128, interleaved=False)
    want, bound = reference(x, pos, table, False)
    s, out = torch.cuda.Stream(), torch.zeros_like(x)
    torch.cuda.synchronize()
    mla.rope(x, pos, table, out=out, stream=s)
    s.synchronize()
    check(out, want, bound)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mla.rope(x, pos, table, out=out)
    x.normal_()
    g.replay()
    torch.cuda.synchronize()
    want, bound = reference(x, pos, table, False)
    check(out, want, bound)


def test_empty_and_refused():
    table = mla.RopeTable(64)
    x = torch.zeros(0, 4, 64, device=DEV)
    pos = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert mla.rope(x, pos, table) is x
    x, pos = inputs(4, 2, 64, torch.bfloat16)
    with pytest.raises(ValueError):
        mla.rope(x, pos.long(), table)
    with pytest.raises(ValueError):
        mla.rope(x, pos[:3], table)
    with pytest.raises(ValueError):
        mla.rope(x, pos, table, out=x.float())
    with pytest.raises(ValueError):
        mla.rope(x.transpose(1, 2), pos, table)
    with pytest.raises(mla.MLAError):
        mla.rope(x, pos, table, offset=2)
    with pytest.raises(mla.MLAError):
        mla.rope(x[:, :1].expand(4, 2, 64), pos, table)     # heads that share memory, in place
    with pytest.raises(ValueError):
        mla.rope(x.double(), pos, table)


@pytest.mark.parametrize("interleaved", [True, False])
def test_offsets_beyond_32_bits(interleaved):
    """Rows whose element offsets pass 2^31 (4.8 GB of bf16, of which little is touched)."""
    wide = torch.empty(600, 1 << 22, dtype=torch.bfloat16, device=DEV)
    x, pos = inputs(600, 3, 64, torch.bfloat16, seed=21)
    view = wide.as_strided((600, 3, 64), (1 << 22, 128, 1))
    view.copy_(x)
    table = mla.RopeTable(64, interleaved=interleaved)
    check(mla.rope(view, pos, table), *reference(x, pos, table, interleaved))
