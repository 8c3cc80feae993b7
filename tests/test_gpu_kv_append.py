"""mla_kv_append against a plain encoder in 64 bits.

Tolerances.  Rows that do not turn are compared byte for byte (with the
oracle's encoders and with mla_kv_write).  A turned value: the phase is cut to
2^-32 of a turn and rounded to fp32 (2^-24 of an angle of at most pi, 2^-22.3),
sine and cosine are within 2^-22, the factor, the product and the sum round by
2^-24 each, so |y - exact| <= 2^-20 |factor| (|a| + |b|) = delta.  A block's scale must
then be that of some amax within delta of the exact one, and every code the
rounding of some value within delta of the exact one under the scale stored."""
import math

import numpy as np
import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla
import oracle

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
REC = {mla.KV_FP8_528: 528, mla.KV_FP4_288: 288}
ENCODE = {mla.KV_FP8_528: oracle.encode_fp8, mla.KV_FP4_288: oracle.encode_fp4}
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
EPS = 2.0 ** -20


def e4m3(v):
    v = np.abs(v)
    step = np.exp2(np.floor(np.log2(np.maximum(v, 2.0 ** -6))) - 3)
    return np.minimum(np.round(v / step) * step, 448.0)


def e2m1(v):
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 1.0))) - 1)
    return np.clip(np.round(v / step) * step, -6.0, 6.0)


def turned(x, pos, table, offset, factor):
    """Exact y (64 bits) and delta, x [n, 512] float64."""
    pairs = table.rope_dim // 2
    step = np.array(table.c.step[:pairs], dtype=np.uint64)
    phase = pos.astype(np.int64).astype(np.uint64)[:, None] * step[None]      # wraps modulo one turn
    t = phase.astype(np.int64).astype(np.float64) * (2 * math.pi / 2.0 ** 64)
    j = np.arange(pairs)
    a, b = (offset + 2 * j, offset + 2 * j + 1) if table.c.layout == 0 else (offset + j, offset + pairs + j)
    y, delta = x.copy(), np.zeros_like(x)
    y[:, a] = factor * (x[:, a] * np.cos(t) - x[:, b] * np.sin(t))
    y[:, b] = factor * (x[:, b] * np.cos(t) + x[:, a] * np.sin(t))
    delta[:, a] = delta[:, b] = EPS * abs(factor) * (np.abs(x[:, a]) + np.abs(x[:, b]))
    return y, delta


def check_records(rec, y, delta, kv_format):
    n = y.shape[0]
    if kv_format == mla.KV_FP4_288:
        sc = torch.from_numpy(rec[:, 256:].copy()).view(torch.float8_e4m3fn).double().numpy()
        blocks = np.abs(y).reshape(n, 32, 16), delta.reshape(n, 32, 16)
        hi, lo = (blocks[0] + blocks[1]).max(-1), np.maximum(blocks[0] - blocks[1], 0).max(-1)
        tiny = 2.0 ** -23
        assert np.all(sc <= e4m3(hi / 6 * (1 + tiny))) and np.all(sc >= e4m3(lo / 6 * (1 - tiny)))
        data = np.stack([rec[:, :256] & 15, rec[:, :256] >> 4], -1).reshape(n, 512)
        got = LEVELS[data & 7] * np.where(data & 8, -1, 1)
        s = np.repeat(sc, 16, 1)
        live = s > 0
        assert np.all(got[~live] == 0)
        s = np.where(live, s, 1.0)
        ok = (e2m1((y + delta) / s * 1.0) >= got - 0) & (e2m1((y - delta) / s) <= got)
        assert np.all(ok | ~live)
    else:
        e = rec[:, 512:].astype(np.int64) - 127
        a = np.abs(y).reshape(n, 16, 32)
        d = delta.reshape(n, 16, 32)

        def least(v):
            r = np.where(v > 0, np.ceil(np.log2(np.maximum(v, 1e-300) / 448.0)), 0)
            r = np.where((v > 0) & (v * np.exp2(-r) > 448), r + 1, r)
            return np.where((v > 0) & (v * np.exp2(1 - r) <= 448), r - 1, r)
        assert np.all(e <= least((a + d).max(-1))) and np.all(e >= least(np.maximum(a - d, 0).max(-1)))
        got = torch.from_numpy(rec[:, :512].copy()).view(torch.float8_e4m3fn).double().numpy()
        s = np.repeat(np.exp2(e.astype(np.float64)), 32, 1)
        up, down = (y + delta) / s, (y - delta) / s
        assert np.all(np.sign(up) * e4m3(up) >= got) and np.all(np.sign(down) * e4m3(down) <= got)


def latents(n, dtype, seed, width=512, lead=0):
    """Rows of many magnitudes, blocks of zeros and outliers among them, as [n, 512] of a wider row."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, width, generator=g) * torch.exp2(torch.randint(-9, 9, (n, 1), generator=g).float())
    x[:, lead:lead + 16] = 0.0
    x[::3, lead + 40::97] *= 30
    return x.to(dtype).to(DEV)[:, lead:lead + 512]


def append(x, slots, tokens, kv_format, **kw):
    pool = torch.full((tokens, REC[kv_format]), 0xA5, dtype=torch.uint8, device=DEV)
    error = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.kv_append(x, slots, pool, kv_format, error=error, **kw)
    torch.cuda.synchronize()
    return pool.cpu().numpy(), int(error)


@pytest.mark.parametrize("kv_format", list(REC))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_rows_that_do_not_turn_are_the_encoders_bytes(kv_format, dtype):
    n = 333
    x = latents(n, dtype, 3)
    x[5, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 2)      # ties at a scale of 1
    x[6, 16:32] = torch.tensor([0.25, -0.75, 1.25, -1.75, 2.5, -3.5, 5.0, 6.0] * 2) * 0.3125   # and of 5/16
    slots = torch.randperm(64 * 9, generator=torch.Generator().manual_seed(1))[:n].to(torch.int32)
    got, err = append(x, slots.to(DEV), 64 * 9, kv_format)
    want = ENCODE[kv_format](x.double().cpu().numpy())
    assert err == 0 and np.array_equal(got[slots.numpy()], want)
    left = np.setdiff1d(np.arange(64 * 9), slots.numpy())
    assert np.all(got[left] == 0xA5)
    if dtype is torch.bfloat16:
        pool = torch.full((64 * 9, REC[kv_format]), 0xA5, dtype=torch.uint8, device=DEV)
        mla.kv_write(x.contiguous(), slots.to(DEV), pool, kv_format)
        assert np.array_equal(pool.cpu().numpy(), got)


@pytest.mark.parametrize("kv_format", list(REC))
@pytest.mark.parametrize("rd,offset", [(64, 448), (2, 0), (64, 0), (128, 384), (256, 256), (6, 505), (62, 13), (256, 101)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_turned_rows(kv_format, rd, offset, interleaved):
    n = 70
    table = mla.RopeTable(rd, interleaved=interleaved, scaling=mla.RopeScaling.yarn(8.0, 4096) if rd > 2 else None)
    for k, dtype in enumerate([torch.bfloat16, torch.float16, torch.float32]):
        x = latents(n, dtype, rd + offset + k)
        pos = torch.randint(0, 1 << 20, (n,), generator=torch.Generator().manual_seed(k), dtype=torch.int32)
        pos[0], pos[1], pos[2] = 0, 2 ** 31 - 1, -(2 ** 31)
        slots = torch.randperm(128, generator=torch.Generator().manual_seed(k))[:n].to(torch.int32)
        got, err = append(x, slots.to(DEV), 128, kv_format, rope=table, positions=pos.to(DEV), offset=offset)
        y, delta = turned(x.double().cpu().numpy(), pos.numpy(), table, offset, table.c.factor)
        assert err == 0
        check_records(got[slots.numpy()], y, delta, kv_format)


@pytest.mark.parametrize("dtype,width,lead", [(torch.bfloat16, 576, 0), (torch.bfloat16, 1024, 512), (torch.float16, 520, 8),
                                              (torch.float32, 516, 4)])
def test_rows_of_a_wider_projection(dtype, width, lead):
    n = 41
    table = mla.RopeTable(64)
    x = latents(n, dtype, width, width, lead)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    a, _ = append(x, pos, 64, mla.KV_FP4_288, rope=table, positions=pos)
    b, _ = append(x.contiguous(), pos, 64, mla.KV_FP4_288, rope=table, positions=pos)
    assert np.array_equal(a, b)
    same = x[:1].expand(n, 512)                       # one row for all: a stride of 0
    a, _ = append(same, pos, 64, mla.KV_FP8_528, rope=table, positions=pos)
    b, _ = append(same.contiguous(), pos, 64, mla.KV_FP8_528, rope=table, positions=pos)
    assert np.array_equal(a, b)


@pytest.mark.parametrize("kv_format", list(REC))
def test_a_long_list_skips_and_flags(kv_format):
    """More rows than the grid holds at once; -1 and slots outside the pool leave everything else as it was."""
    n, tokens = 30000, 64 * 300
    table = mla.RopeTable(64)
    x = latents(n, torch.bfloat16, 9)
    g = torch.Generator().manual_seed(2)
    slots = torch.full((n,), -1, dtype=torch.int32)
    rows = torch.randperm(n, generator=g)[:tokens - 100]
    slots[rows] = torch.randperm(tokens, generator=g)[:tokens - 100].to(torch.int32)
    pos = torch.randint(0, 100000, (n,), generator=g, dtype=torch.int32)
    got, err = append(x, slots.to(DEV), tokens, kv_format, rope=table, positions=pos.to(DEV))
    assert err == 0
    some = rows[:200]
    y, delta = turned(x[some.to(DEV)].double().cpu().numpy(), pos[some].numpy(), table, 448, 1.0)
    check_records(got[slots[some].numpy()], y, delta, kv_format)
    assert np.all(got[np.setdiff1d(np.arange(tokens), slots.numpy())] == 0xA5)
    bad = slots.clone()
    bad[rows[0]], bad[rows[1]], bad[rows[2]] = tokens, -2, 2 ** 31 - 1
    again, err = append(x, bad.to(DEV), tokens, kv_format, rope=table, positions=pos.to(DEV))
    assert err == mla.DEVERR_BAD_INDEX
    keep = np.setdiff1d(np.arange(tokens), slots[rows[:3]].numpy())
    assert np.array_equal(again[keep], got[keep]) and np.all(again[slots[rows[:3]].numpy()] == 0xA5)


def test_empty_and_single():
    table = mla.RopeTable(64)
    pool = torch.full((64, 288), 0xA5, dtype=torch.uint8, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    mla.kv_append(torch.zeros(0, 512, dtype=torch.bfloat16, device=DEV), none, pool, mla.KV_FP4_288, rope=table, positions=none)
    assert bool((pool == 0xA5).all())
    x = latents(1, torch.bfloat16, 4)
    at = torch.tensor([63], dtype=torch.int32, device=DEV)
    got, err = append(x, at, 64, mla.KV_FP4_288, rope=table, positions=at)
    y, delta = turned(x.double().cpu().numpy(), np.array([63]), table, 448, 1.0)
    check_records(got[63:], y, delta, mla.KV_FP4_288)
    assert np.all(got[:63] == 0xA5)


def test_graph_and_stream():
    """A captured call follows what the buffers hold; a stream of the caller's choice."""
    table = mla.RopeTable(64)
    n = 100
    x, pos = latents(n, torch.bfloat16, 5).clone(), torch.arange(n, dtype=torch.int32, device=DEV)
    pool = torch.zeros(128, 288, dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        mla.kv_append(x, pos, pool, mla.KV_FP4_288, rope=table, positions=pos)
    for k in range(3):
        x.copy_(latents(n, torch.bfloat16, 50 + k))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = append(x, pos, 128, mla.KV_FP4_288, rope=table, positions=pos)
        assert np.array_equal(pool.cpu().numpy()[:n], want[:n])
    other = torch.zeros_like(pool)
    mla.kv_append(x, pos, other, mla.KV_FP4_288, rope=table, positions=pos, stream=s)
    s.synchronize()
    assert torch.equal(other, pool)


def test_pool_beyond_4_gib():
    pages = 250000
    pool = torch.zeros(pages, 64, 288, dtype=torch.uint8, device=DEV)
    x = latents(3, torch.bfloat16, 6)
    at = torch.tensor([pages * 64 - 1, 233017 * 64 + 5, 116509 * 64], dtype=torch.int32, device=DEV)
    mla.kv_append(x, at, pool, mla.KV_FP4_288)
    got = pool.view(-1, 288)[at.long()].cpu().numpy()
    assert np.array_equal(got, oracle.encode_fp4(x.double().cpu().numpy()))
    assert int(pool.view(-1, 288).any(1).sum()) == 3
