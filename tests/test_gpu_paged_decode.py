"""mla_paged_decode_fp4 against attention in 64 bits over the same records.

Tolerances.  Scores: 512 products of 16-bit values, exact each, summed in
fp32 by the tensor core in 32 steps of 16 (each step may truncate, 2^-23 of
the running sum of magnitudes): with S = max over tokens of
sm_scale * sum |q_d k_d|, a score is within dx = 64 * 2^-23 * S.  The
exponentials add 2^-22, their fp32 sums 2^-20 in all: so
|lse error| <= dx + 2^-20 (1 + |lse|).  A probability enters the second
product rounded to 16 bits with at least 11 significant bits (2^-11 of
itself), and shifts by 2 dx at most: |out error| <= (2^-11 + 2 dx + 2^-19) *
sum_j p_j |k_j| before the output's own rounding to bf16, 2^-8 of itself."""
import math

import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def decode_records(rec):
    n = rec.shape[0]
    code = torch.stack([rec[:, :256] & 15, rec[:, :256] >> 4], 2).reshape(n, 512).long()
    return E2M1.to(code.device)[code] * rec[:, 256:].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)


def random_records(n, g, top=0x3C):
    """Any e2m1 codes; scales of either sign (the decoder multiplies what is there), zero and subnormal among them."""
    rec = torch.randint(0, 256, (n, 288), generator=g, device=DEV, dtype=torch.int32)
    rec[:, 256:] = torch.randint(0, top, (n, 32), generator=g, device=DEV, dtype=torch.int32)
    rec[::7, 256:] = rec[::7, 256:] % 8             # subnormal scales and zeros
    return rec.to(torch.uint8)


class Case:
    """Sequences over a shuffled pool; whatever no query token may see is 0xFF (NaN scales) and past-the-end table
    entries are wild."""

    def __init__(self, lens, s, h, max_pages=None, seed=0, spare=3, qscale=1.0, records=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.s, self.h = list(lens), s, h
        b = len(lens)
        held = [-(-n // 64) for n in lens]
        self.max_pages = max_pages or max(max(held), 1)
        self.num_pages = max(sum(held) + spare, 1)
        self.kv = torch.full((self.num_pages, 64, 288), 0xFF, dtype=torch.uint8, device=DEV)
        ids = torch.randperm(self.num_pages, generator=g, device=DEV).tolist()
        table = torch.full((b, self.max_pages), -77, dtype=torch.int32)
        table[:, 1::2] = 2 ** 31 - 5
        for r, n in enumerate(lens):
            for k in range(held[r]):
                table[r, k] = ids.pop()
                m = min(64, n - 64 * k)
                rec = (records or random_records)(m, g)
                self.kv[int(table[r, k]), :m] = rec
        self.table = table.to(DEV)
        # Mild scores for most heads; sharper ones for some.
        q = torch.randn(b, s, h, 512, generator=g, device=DEV)
        q *= qscale * torch.exp2(torch.randint(-8, -3, (b, s, h, 1), generator=g, device=DEV).float())
        self.q = q.to(torch.bfloat16)
        self.seq = torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def problem(self, **kw):
        return mla.PagedProblem.make(len(self.lens), self.s, self.h, self.max_pages, self.num_pages, **kw)

    def run(self, num_sms=0, stream=None, **kw):
        dec = mla.PagedFP4Decoder(self.problem(**kw), DEV, num_sms=num_sms)
        dec.workspace.fill_(0xFF)
        out = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:3], float("nan"), device=DEV)
        torch.cuda.synchronize()
        dec(self.q, self.kv, self.table, self.seq, out, lse, stream=stream)
        torch.cuda.synchronize()
        return out, lse, int(dec.error)

    def check(self, out, lse, window=0, sinks=0, sm_scale=None, skip=None):
        scale = 512 ** -0.5 if sm_scale is None else float(torch.tensor(sm_scale, dtype=torch.float32))
        for b, n in enumerate(self.lens):
            k = None
            if n > 0:
                pages = self.table[b, : -(-n // 64)].long()
                ok = (pages >= 0) & (pages < self.num_pages)
                k = decode_records(self.kv[pages.where(ok, 0)].reshape(-1, 288)[:n])
                ok = ok.repeat_interleave(64)[:n]
            j = torch.arange(n, device=DEV)
            for i in range(self.s):
                if skip is not None and i in skip:
                    continue
                at = n - self.s + i
                see = (j <= at) & ((j > at - window) | (j < sinks) if window else torch.ones_like(j, dtype=torch.bool))
                if n:
                    see &= ok
                if not bool(see.any()):
                    assert torch.all(out[b, i] == 0) and not torch.any(torch.signbit(out[b, i].float()))
                    assert torch.all(torch.isneginf(lse[b, i]))
                    continue
                ks, q = k[see], self.q[b, i].double()
                x = q @ ks.T * scale
                dx = 64 * 2.0 ** -23 * (q.abs() @ ks.abs().T * abs(scale)).amax(-1)
                want = torch.logsumexp(x, -1)
                err = (lse[b, i].double() - want).abs()
                tol = dx + 2.0 ** -20 * (1 + want.abs())
                assert torch.all(err <= tol), (b, i, float((err / tol).max()))
                p = torch.softmax(x, -1)
                o = p @ ks
                tol = (2.0 ** -11 + 2 * dx.unsqueeze(-1) + 2.0 ** -19) * (p @ ks.abs()) + 2.0 ** -8 * o.abs()
                err = (out[b, i].double() - o).abs()
                assert torch.all(err <= tol + 1e-30), (b, i, float((err / (tol + 1e-30)).max()))


LENGTHS = [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 200, 256, 257, 1000]


@pytest.mark.parametrize("s,h", [(1, 16), (1, 1), (1, 64), (1, 128), (2, 128), (3, 24), (5, 7), (1, 33), (1, 17), (4, 16),
                                 (7, 100)])
@pytest.mark.parametrize("num_sms", [0, 20])         # (units have fewer rows where parts are plenty)
def test_matches_64_bits_at_every_length(s, h, num_sms):
    c = Case(LENGTHS, s, h, seed=s * 200 + h)
    out, lse, err = c.run(num_sms=num_sms)
    assert err == 0
    c.check(out, lse)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 4), (64, 0), (63, 64), (65, 130), (100, 4), (128, 128),
                                          (300, 5), (5000, 3), (0, 9), (200, 2000), (7, 129)])
@pytest.mark.parametrize("s,h", [(1, 16), (3, 24), (2, 64)])
@pytest.mark.parametrize("num_sms", [0, 20])
def test_windows_and_sinks(window, sinks, s, h, num_sms):
    c = Case([0, 1, 5, 64, 129, 400, 777, 1025], s, h, seed=window + 7 * sinks)
    out, lse, err = c.run(num_sms=num_sms, window=window, sinks=sinks)
    assert err == 0
    c.check(out, lse, window, sinks)


@pytest.mark.parametrize("num_sms", [1, 2, 3, 7, 40, 500])
@pytest.mark.parametrize("s,h", [(1, 16), (1, 40), (2, 128)])
def test_any_number_of_parts(num_sms, s, h):
    c = Case([700, 0, 1, 2500, 130], s, h, seed=num_sms)
    for window, sinks in ((0, 0), (300, 70)):
        out, lse, err = c.run(num_sms=num_sms, window=window, sinks=sinks)
        assert err == 0
        c.check(out, lse, window, sinks)


def test_many_query_tokens_of_one_sequence():
    """The prefill shape: every query token stands at its own position."""
    c = Case([300, 77], 100, 16, seed=3)
    out, lse, err = c.run()
    c.check(out, lse)
    out, lse, err = c.run(window=33, sinks=2)
    assert err == 0
    c.check(out, lse, 33, 2)


@pytest.mark.parametrize("b,h", [(1000, 16), (950, 32), (500, 128)])
@pytest.mark.parametrize("num_sms", [0, 7, 1500])
def test_more_units_than_threads(b, h, num_sms):
    """Units that the threads of a block share several to one; with 1500 parts, one unit to a part."""
    lens = [(37 * r) % 140 if r % 5 else 0 for r in range(b)]
    lens[b // 2] = 900
    c = Case(lens, 1, h, seed=b)
    out, lse, err = c.run(num_sms=num_sms)
    assert err == 0
    c.check(out, lse)


def test_one_long_sequence_is_split_and_merged():
    c = Case([20011], 1, 16, seed=8)
    out, lse, err = c.run()
    assert err == 0
    c.check(out, lse)


def test_maxima_that_grow_from_tile_to_tile():
    """Scores that climb steadily, by far more than any slack, then fall."""
    c = Case([1500], 1, 20, seed=9)
    flat = c.kv[c.table[0].long()].reshape(-1, 288)
    ramp = torch.cat([torch.arange(0, 1000), torch.arange(1000, 500, -1)]).float() / 1000 * 30
    flat[:1500, 256:] = (ramp / 6).to(DEV).unsqueeze(1).to(torch.float8_e4m3fn).view(torch.uint8)
    flat[:1500, :256] = 0x77                        # every value 6 times its scale
    c.kv[c.table[0].long()] = flat.view(-1, 64, 288)
    c.q = torch.full_like(c.q, 0.25)
    c.q[..., ::2] = 0.125
    c.q[:, :, 5] = -c.q[:, :, 5]
    for sms in (0, 1):
        out, lse, err = c.run(num_sms=sms)
        assert err == 0
        c.check(out, lse)


@pytest.mark.parametrize("s,h", [(1, 16), (2, 16), (1, 64), (2, 64)])      # 16, 32, 64 and twice 64 rows
def test_maxima_that_outgrow_the_slack_in_every_tile(s, h):
    """Each tile's scores top the last one's by 12 powers of two and more, so O is rescaled in every tile of every
    unit, between products that add to it: many units at once, the same bits from run to run."""
    b, tiles = 40, 20
    c = Case([tiles * 128 - 7 * r for r in range(b)], s, h, seed=21)
    for r, n in enumerate(c.lens):
        pages = c.table[r, : -(-n // 64)].long()
        flat = c.kv[pages].reshape(-1, 288)
        flat[:n, :8] = 0x77                          # sixes in dims 0 .. 15, under the next larger E4M3 scale in each tile
        flat[:n, 256] = (0x38 + torch.arange(n, device=DEV) // 128).to(torch.uint8)
        c.kv[pages] = flat.view(-1, 64, 288)
    # 12 ln 2 between the scales 1 and 1.125, more between larger ones.
    c.q[..., :16] = 12 * 0.6931471805599453 * 8 / 96 * 512 ** 0.5
    first = c.run()
    assert first[2] == 0
    c.check(*first[:2])
    for _ in range(20):
        out, lse, err = c.run()
        assert err == 0 and torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_large_and_small_queries_and_scales():
    for qscale, top, sm in ((2.0 ** 20, 0x10, 2.0 ** -22), (2.0 ** -60, 0x7F, 1.0), (1e30, 0x30, 1e-31), (1.0, 0x7F, 1e-4)):
        c = Case([130, 7], 2, 18, seed=5, qscale=qscale, records=lambda n, g: random_records(n, g, top))
        out, lse, err = c.run(sm_scale=sm)
        assert err == 0
        c.check(out, lse, sm_scale=sm)


@pytest.mark.parametrize("bits", [16, 20, 23, 25, 26, 27, 28, 29, 31, 40, 100])
@pytest.mark.parametrize("s,h", [(1, 16), (2, 16), (1, 64)])
def test_scores_far_past_what_a_softmax_tells_apart(s, h, bits):
    """Finite queries whose scores reach 2^bits: lse still follows the largest score, out is some average of the
    records, and the largest score's own record (its values have 6 bits, so bf16 holds them) where it leads by more
    than the scores' error on either side."""
    c = Case([700, 128, 1, 2000, 65] * 8, s, h, seed=bits)
    c.q = (c.q.float() * 2.0 ** (bits - 2)).to(torch.bfloat16)
    out, lse, err = c.run()
    assert err == 0 and bool(torch.isfinite(out).all())
    alone = 0
    for b, n in enumerate(c.lens):
        k = decode_records(c.kv[c.table[b, : -(-n // 64)].long()].reshape(-1, 288)[:n])
        for i in range(s):
            at = n - s + i
            if at < 0:
                continue
            ks, q = k[: at + 1], c.q[b, i].double()
            x = q @ ks.T * 512 ** -0.5
            dx = 64 * 2.0 ** -23 * (q.abs() @ ks.abs().T * 512 ** -0.5).amax(-1)
            want = torch.logsumexp(x, -1)
            assert torch.all((lse[b, i].double() - want).abs() <= dx + 2.0 ** -20 * (1 + want.abs()))
            assert torch.all(out[b, i].double().abs() <= ks.abs().amax(0) * (1 + 2.0 ** -7))
            top, arg = x.topk(min(2, at + 1), dim=-1)
            ahead = top[:, 0] - top[:, -1] > 2 * dx + 64 if at else torch.ones(h, dtype=torch.bool, device=DEV)
            # Its weight is 1 within 2^-11, less than half a step of bf16; the others' are below e^-64 each.
            err = (out[b, i].double() - ks[arg[:, 0]]).abs()[ahead]
            assert torch.all(err <= n * math.exp(-64) * ks.abs().max()), float(err.max())
            alone += int(ahead.sum())
    assert alone > len(c.lens) * s * h / (8 if bits > 20 else 40)


@pytest.mark.parametrize("sm_scale", [-0.05, -1.0, 0.0, 1e-30, -3e-38, 1e-44, 2.0])
@pytest.mark.parametrize("s,h", [(1, 16), (3, 24), (1, 64)])
def test_scales_of_either_sign_and_none(s, h, sm_scale):
    """A negative scale turns the order of the scores round; one of 0 or far below any score leaves an average."""
    c = Case([0, 1, 130, 700, 2000], s, h, seed=41)
    for window, sinks in ((0, 0), (150, 70)):
        out, lse, err = c.run(sm_scale=sm_scale, window=window, sinks=sinks)
        assert err == 0
        c.check(out, lse, window, sinks, sm_scale=sm_scale)


def test_a_peak_and_a_long_tail():
    """One token carries most of the mass; the other 40000 each have 2^-22 of its weight, 1 % together."""
    n = 40000
    c = Case([n], 1, 16, seed=6)
    flat = c.kv[c.table[0].long()].reshape(-1, 288)
    flat[:n] = 0
    flat[:n, 256:] = 0x38                            # scale 1
    flat[:n, 8:256] = 0x22                           # ones in dims 16 ..
    flat[12345, :8] = 0x77                           # the peak: sixes in dims 0 .. 15
    flat[12345, 8:256] = 0xAA                        # and minus ones after
    c.kv[c.table[0].long()] = flat.view(-1, 64, 288)
    c.q.zero_()
    c.q[..., :16] = 22 * 0.6931471805599453 / 96 * 512 ** 0.5
    out, lse, err = c.run()
    assert err == 0
    c.check(out, lse)


def test_masked_tail_bytes_do_not_matter():
    """Records past the end are NaN scales here; the same call over zeroed tails gives the same bits."""
    c = Case([1, 65, 190, 500], 2, 30, seed=4)
    a = c.run(window=70, sinks=3)
    for r, n in enumerate(c.lens):
        if n % 64:
            c.kv[int(c.table[r, n // 64]), n % 64:] = 0
    b = c.run(window=70, sinks=3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bad_pages_are_skipped_and_flagged():
    c = Case([300, 64, 640], 2, 16, seed=2)
    good = c.table.clone()
    c.table[0, 1], c.table[0, 4], c.table[1, 0], c.table[2, 3] = -1, c.num_pages, -5, 2 ** 31 - 1
    out, lse, err = c.run()
    assert err == mla.DEVERR_BAD_INDEX
    c.check(out, lse)
    # A page that the window leaves out is not looked at.
    c.table.copy_(good)
    c.table[2, 2] = -9
    out, lse, err = c.run(window=40)
    assert err == 0
    c.check(out, lse, 40)


def test_bad_lengths_count_as_empty_and_are_flagged():
    c = Case([100, 200, 300], 1, 16, seed=2, max_pages=6)
    c.seq[0], c.seq[2] = -3, 385
    out, lse, err = c.run()
    assert err == mla.DEVERR_BAD_LENGTH
    c.lens[0] = c.lens[2] = 0
    c.check(out, lse)


def test_pool_beyond_2_gib():
    """Page ids whose byte offset passes 2^31 and 2^32."""
    pages = 240000                                   # 4.4 GB of records
    pool = torch.empty((pages, 64, 288), dtype=torch.uint8, device=DEV)
    c = Case([500, 70], 2, 16, seed=7)
    ids = [239999, 116508, 116509, 233017, 233016, 5, 150000, 0, 200000, 1]
    new = c.table.clone()
    for r, n in enumerate(c.lens):
        for k in range(-(-n // 64)):
            new[r, k] = ids.pop(0)
            pool[int(new[r, k])] = c.kv[int(c.table[r, k])]
    c.kv, c.table, c.num_pages = pool, new, pages
    out, lse, err = c.run()
    assert err == 0
    c.check(out, lse)


def test_rows_past_the_batch_stay_as_they_were():
    c = Case([90, 130], 3, 24, seed=12)
    out = torch.full((5, 3, 24, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((5, 3, 24), 7.0, device=DEV)
    dec = mla.PagedFP4Decoder(c.problem(), DEV)
    dec(c.q, c.kv, c.table, c.seq, out[:2], lse[:2])
    torch.cuda.synchronize()
    c.check(out[:2], lse[:2])
    assert torch.all(out[2:] == 7) and torch.all(lse[2:] == 7)


def test_same_bits_twice_and_on_another_stream():
    c = Case([3000, 100, 2000], 2, 64, seed=13)
    a = c.run()
    s = torch.cuda.Stream()
    b = c.run(stream=s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_graph_follows_the_lengths_on_the_device():
    c = Case([900, 350], 2, 32, seed=14)
    dec = mla.PagedFP4Decoder(c.problem(window=200, sinks=10), DEV)
    out, lse = dec(c.q, c.kv, c.table, c.seq)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec(c.q, c.kv, c.table, c.seq, out, lse)
    for lens in ([900, 350], [1, 349], [0, 64], [512, 2]):
        c.lens = lens
        c.seq.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        c.check(out, lse, 200, 10)
    assert int(dec.error) == 0


def test_two_decoders_at_once():
    c, d = Case([2500, 900], 1, 64, seed=15), Case([1300, 40, 7], 2, 16, seed=16)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    dc, dd = mla.PagedFP4Decoder(c.problem(), DEV), mla.PagedFP4Decoder(d.problem(), DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        oc = dc(c.q, c.kv, c.table, c.seq, stream=s)
        od = dd(d.q, d.kv, d.table, d.seq, stream=t)
    torch.cuda.synchronize()
    c.check(*oc)
    d.check(*od)


@pytest.mark.parametrize("s,h", [(1, 16), (3, 24), (2, 10)])
def test_nan_records_that_no_row_sees(s, h):
    """A page may hold anything between the sinks and the window: 0 times NaN must not reach a sum."""
    c = Case([400, 130, 1000, 64], s, h, seed=17)
    for b, n in enumerate(c.lens):
        flat = torch.arange(n, device=DEV)
        hidden = flat[(flat >= 4) & (flat <= n - s - 100)]
        pages = c.table[b, hidden // 64].long()
        c.kv[pages, hidden % 64] = 0xFF
    out, lse, err = c.run(window=100, sinks=4)
    assert err == 0
    c.check(out, lse, 100, 4)


@pytest.mark.parametrize("h", [5, 16, 40])
def test_nan_spoils_only_the_rows_that_see_it(h):
    c = Case([200, 65], 3, h, seed=18)
    for b, n in enumerate(c.lens):                   # the last token: seen by the last query token alone
        c.kv[int(c.table[b, (n - 1) // 64]), (n - 1) % 64] = 0xFF
    out, lse, err = c.run()
    assert err == 0
    c.check(out, lse, skip={2})


def test_infinite_query_spoils_only_its_row():
    c = Case([300, 65], 2, 20, seed=19)
    good = c.run()
    q = c.q.clone()
    c.q[0, 1, 3] = float("inf")
    out, lse, err = c.run()
    assert err == 0
    c.q = q
    out[0, 1, 3], lse[0, 1, 3] = good[0][0, 1, 3], good[1][0, 1, 3]
    c.check(out, lse)


def test_captured_behind_a_join_and_a_memset():
    c = Case([700, 65], 1, 32, seed=20)
    dec = mla.PagedFP4Decoder(c.problem(), DEV)
    dec(c.q, c.kv, c.table, c.seq)
    out, lse = torch.empty_like(c.q), torch.empty(2, 1, 32, device=DEV)
    q, seq = torch.zeros_like(c.q), torch.zeros_like(c.seq)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q.copy_(c.q)
        seq.copy_(c.seq)
        torch.cuda.current_stream().wait_stream(side)
        dec(q, c.kv, c.table, seq, out, lse)         # behind two branches
        out.zero_()
        dec(q, c.kv, c.table, seq, out, lse)         # behind a memset
    for _ in range(3):
        q.fill_(float("nan"))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        c.check(out, lse)


def test_binding_refusals():
    c = Case([90], 1, 16)
    dec = mla.PagedFP4Decoder(c.problem(), DEV)
    with pytest.raises(ValueError):
        dec(c.q.float(), c.kv, c.table, c.seq)
    with pytest.raises(ValueError):
        dec(c.q, c.kv[:-1], c.table, c.seq)
    with pytest.raises(ValueError):
        dec(c.q, c.kv, c.table.long(), c.seq)
    with pytest.raises(ValueError):
        dec(c.q[:, :, :8], c.kv, c.table, c.seq)
    with pytest.raises(mla.MLAError):
        mla.paged_decode_fp4(c.problem(), c.q, c.kv, c.table, c.seq, dec.num_parts, dec.workspace[:-16],
                             torch.empty_like(c.q), torch.empty(1, 1, 16, device=DEV))
