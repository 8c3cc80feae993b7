"""mla_kv_append where a pair's dims lie in two blocks of very different size:
what the turn brings from the large dim is all there is of the small one, so
the turn has to be right relative to itself, not to the large dim.

Tolerance.  The phase is exact.  What is left of it behind whole quarters of a
turn rounds to fp32 and is multiplied by a rounded pi, 3 * 2^-24 of itself, and
neither sine nor cosine changes by more of itself there; they are within 2^-23
of themselves; the factor, a product and the sum round by 2^-24 each.  So
|y - exact| <= 8 * 2^-24 |factor| (|a sin| + |b cos|) = delta to first order, with
a percent for the rest, and with cos and sin in turn for the other dim."""
import math

import numpy as np
import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla
from test_gpu_kv_append import append, check_records

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
EPS = 1.01 * 2.0 ** -21


def turned(x, pos, table, offset):
    """Exact y (64 bits) and delta of rows x [n, 512] float64 under a half layout."""
    pairs = table.rope_dim // 2
    step = np.array(table.c.step[:pairs], dtype=np.uint64)
    phase = pos.astype(np.int64).astype(np.uint64)[:, None] * step[None]      # wraps modulo one turn
    # Sine and cosine of a rest of at most an eighth of a turn, so that 64 bits hold them relative to themselves.
    quarters = (phase + np.uint64(1 << 61)) >> np.uint64(62)
    rest = (phase - (quarters << np.uint64(62))).astype(np.int64).astype(np.float64) * (2 * math.pi / 2.0 ** 64)
    s, c = np.sin(rest), np.cos(rest)
    for k in range(4):
        at = quarters % np.uint64(4) == k
        for _ in range(k):
            s[at], c[at] = c[at].copy(), -s[at].copy()
    f = float(np.float32(table.c.factor))
    a, b = x[:, offset:offset + pairs], x[:, offset + pairs:offset + 2 * pairs]
    y, delta = x.copy(), np.zeros_like(x)
    y[:, offset:offset + pairs] = f * (a * c - b * s)
    y[:, offset + pairs:offset + 2 * pairs] = f * (b * c + a * s)
    delta[:, offset:offset + pairs] = EPS * abs(f) * (np.abs(a * c) + np.abs(b * s))
    delta[:, offset + pairs:offset + 2 * pairs] = EPS * abs(f) * (np.abs(b * c) + np.abs(a * s))
    return y, delta


# Frequencies of a whole quarter, a half and none of a turn, and what is next to them.
@pytest.mark.parametrize("around", [0.0, math.pi / 2, -math.pi / 2, math.pi])
@pytest.mark.parametrize("kv_format,low,high", [(mla.KV_FP8_528, -34, -8), (mla.KV_FP4_288, -19, -8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("small", [0.0, 2.0 ** -24])
def test_small_blocks_take_what_the_turn_brings(around, kv_format, low, high, dtype, small):
    n, pairs, offset = 200, 32, 448
    rng = np.random.default_rng(5)
    for exponent in range(low, high):
        small_turns = 2.0 ** exponent * rng.uniform(1, 2, pairs) * np.where(rng.random(pairs) < 0.5, -1, 1)
        freqs = around - np.sign(around) * np.abs(small_turns) if around else small_turns
        table = mla.RopeTable(2 * pairs, interleaved=False, freqs=freqs.tolist(), attention_factor=1.25)
        g = torch.Generator().manual_seed(exponent + 100)
        # FP4 holds no block below 6 * 2^-10: rows as large as its records take, and turns that bring enough of them.
        top = 2000.0 if kv_format == mla.KV_FP4_288 else 16.0
        x = torch.zeros(n, 512)
        big = (torch.rand(n, pairs, generator=g) + 1) / 2 * top * torch.where(torch.rand(n, pairs, generator=g) < 0.5, -1, 1)
        x[:, offset:offset + pairs] = big
        x[:, offset + pairs:] = torch.randn(n, pairs, generator=g) * small
        x[n // 2:] = torch.cat([x[n // 2:, :offset], x[n // 2:, offset + pairs:], x[n // 2:, offset:offset + pairs]], 1)
        x = x.to(dtype)
        pos = torch.randint(1, 6, (n,), generator=g, dtype=torch.int32)
        slots = torch.arange(n, dtype=torch.int32)
        got, err = append(x.to(DEV), slots.to(DEV), 64 * 4, kv_format, rope=table, positions=pos.to(DEV), offset=offset)
        y, delta = turned(x.double().numpy(), pos.numpy(), table, offset)
        assert err == 0
        check_records(got[:n], y, delta, kv_format)
