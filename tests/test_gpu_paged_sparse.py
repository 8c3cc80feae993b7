"""mla_paged_sparse_decode_fp4: the selection against whole-number arithmetic
(equal, ties included), the attention against 64 bits over the pages selected.

Tolerances of the attention as for mla_paged_decode_fp4: a score within
dx = 64 * 2^-23 * sm_scale * sum |q_d k_d|, |lse error| <= dx + 2^-20 (1 +
|lse|), |out error| <= (2^-11 + 2 dx + 2^-19) sum_j p_j |k_j| and the output's
own rounding to bf16, 2^-8 of itself."""
import math

import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla
from test_gpu_paged_decode import Case, decode_records

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)


def whole_codes(q, sign=1.0):
    """bf16 [h, 512] -> whole numbers [h, 512] and exponents [h], None for rows of zeros (Python arithmetic on exact values)."""
    codes, exps = [], []
    for row in (q.double() * sign):
        top = float(row.abs().max())
        if top == 0:
            codes.append(torch.zeros(512, dtype=torch.int64))
            exps.append(None)
            continue
        e = -120
        while top * 2.0 ** -e > 127:
            e += 1
        codes.append(torch.round(row * 2.0 ** -e).to(torch.int64).cpu())
        exps.append(e)
    return torch.stack(codes), exps


def expected_pages(q, means, ids, last, top, sinks, local, sign=1.0, num_pages=1 << 30):
    """The pages a query token in page `last` attends to; means int8 codes and exponents of all pages on the CPU."""
    total = last + 1
    if total <= top:
        return list(range(total))
    a, exps = whole_codes(q, sign)
    most = max([e for e in exps if e is not None], default=0)
    ok = (ids >= 0) & (ids < num_pages)
    safe = torch.where(ok, ids, 0)
    dots = (a.double() @ means[0][safe].double().T).tolist()      # whole numbers below 2^23: exact
    page_e = means[1][safe].tolist()
    scores = []
    for j in range(total):
        if not bool(ok[j]):
            scores.append(-math.inf)
            continue
        best = max(dots[h][j] * 2.0 ** (max(exps[h] - most, -100) if exps[h] is not None else -100) for h in range(len(exps)))
        scores.append(best * 2.0 ** page_e[j])
    keep = [j for j in range(total) if j < sinks or j > last - local]
    rest = [j for j in range(total) if sinks <= j <= last - local]
    rest.sort(key=lambda j: (-scores[j], j))
    return sorted(keep + rest[:top - len(keep)])


class Sparse(Case):
    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        self.means = torch.full((self.num_pages, 528), 0xA5, dtype=torch.uint8, device=DEV)
        self.refresh()

    def refresh(self):
        slots = torch.arange(63, self.num_pages * 64, 64, dtype=torch.int32, device=DEV)
        mla.page_means(self.kv, slots, self.means)

    def sparse_problem(self, top, sinks, local, **kw):
        return mla.PagedSparseProblem.make(len(self.lens), self.s, self.h, self.max_pages, self.num_pages, top,
                                           sink_pages=sinks, local_pages=local, **kw)

    def run_sparse(self, top, sinks=1, local=1, num_sms=0, stream=None, **kw):
        dec = mla.PagedSparseFP4Decoder(self.sparse_problem(top, sinks, local, **kw), DEV, num_sms=num_sms)
        dec.workspace.fill_(0xFF)
        out = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:3], float("nan"), device=DEV)
        sel = torch.full(self.q.shape[:2] + (top,), -9, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        dec(self.q, self.kv, self.means, self.table, self.seq, out, lse, sel, stream=stream)
        torch.cuda.synchronize()
        return out, lse, sel, int(dec.error)

    def check_sparse(self, got, top, sinks=1, local=1, sm_scale=None, queries=None):
        out, lse, sel = got[:3]
        scale = 512 ** -0.5 if sm_scale is None else sm_scale
        sign = -1.0 if scale < 0 else 1.0
        codes = self.means[:, :512].view(torch.int8).cpu(), self.means[:, 512].long().cpu() - 127
        table = self.table.cpu().long()
        for b, n in enumerate(self.lens):
            for i in range(self.s):
                if queries is not None and (b, i) not in queries:
                    continue
                at = n - self.s + i
                if at < 0:
                    assert torch.all(sel[b, i] == -1)
                    assert torch.all(out[b, i] == 0) and torch.all(torch.isneginf(lse[b, i]))
                    continue
                want = expected_pages(self.q[b, i], codes, table[b], at // 64, top, sinks, local, sign, self.num_pages)
                assert sel[b, i].tolist() == want + [-1] * (top - len(want)), (b, i)
                ids = table[b, want]
                ok = ((ids >= 0) & (ids < self.num_pages)).to(DEV).repeat_interleave(64)
                k = decode_records(self.kv[torch.where((ids >= 0) & (ids < self.num_pages), ids, 0).to(DEV)].reshape(-1, 288))
                m = (len(want) - 1) * 64 + at % 64 + 1
                k, ok = k[:m], ok[:m]
                k = k[ok]
                q = self.q[b, i].double()
                if k.shape[0] == 0:
                    assert torch.all(out[b, i] == 0) and torch.all(torch.isneginf(lse[b, i]))
                    continue
                x = q @ k.T * scale
                dx = 64 * 2.0 ** -23 * (q.abs() @ k.abs().T * abs(scale)).amax(-1)
                ref = torch.logsumexp(x, -1)
                assert torch.all((lse[b, i].double() - ref).abs() <= dx + 2.0 ** -20 * (1 + ref.abs())), (b, i)
                p = torch.softmax(x, -1)
                o = p @ k
                tol = (2.0 ** -11 + 2 * dx.unsqueeze(-1) + 2.0 ** -19) * (p @ k.abs()) + 2.0 ** -8 * o.abs() + 1e-30
                assert torch.all((out[b, i].double() - o).abs() <= tol), (b, i)


LENGTHS = [0, 1, 2, 63, 64, 65, 128, 129, 449, 512, 513, 1000, 2111]


@pytest.mark.parametrize("s,h", [(1, 16), (1, 1), (1, 128), (2, 64), (3, 24), (5, 7), (1, 33), (2, 100)])
@pytest.mark.parametrize("top,sinks,local", [(1, 0, 1), (4, 1, 2), (7, 0, 1), (9, 3, 6), (16, 1, 4), (40, 2, 1)])
def test_lengths_heads_and_budgets(s, h, top, sinks, local):
    c = Sparse(LENGTHS, s, h, seed=s * h + top)
    got = c.run_sparse(top, sinks, local)
    assert got[3] == 0
    c.check_sparse(got, top, sinks, local)


def test_pages_about_something_are_found():
    """A page whose tokens share a direction wins for the head that looks for it."""
    c = Sparse([64 * 40 + 9], 1, 16, seed=3)
    g = torch.Generator(device=DEV).manual_seed(0)
    for page in (5, 17, 30):
        rec = c.kv[int(c.table[0, page])]
        rec[:, 256:] = 0x38
        rec[:, :256] = torch.randint(0, 256, (256,), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
        c.q[0, 0, page % 16] = decode_records(rec[:1])[0].to(torch.bfloat16)
    c.refresh()
    got = c.run_sparse(6, 1, 2)
    c.check_sparse(got, 6, 1, 2)
    assert set((0, 5, 17, 30, 39, 40)) == set(got[2][0, 0].tolist())


def test_ties_go_to_the_lower_page():
    c = Sparse([64 * 50 + 1], 2, 16, seed=5)
    c.table[0, :50] = c.table[0, torch.arange(50, device=DEV) % 3]      # three pages, again and again
    got = c.run_sparse(20, 2, 1)
    c.check_sparse(got, 20, 2, 1)
    c.q.zero_()                                                             # every score 0
    got = c.run_sparse(20, 2, 1)
    c.check_sparse(got, 20, 2, 1)
    assert got[2][0, 0].tolist()[:19] == list(range(19))


@pytest.mark.parametrize("sm_scale", [-0.05, 0.3, 1e-30, 0.0])
def test_scales_of_either_sign(sm_scale):
    c = Sparse([1500, 700], 2, 24, seed=6)
    got = c.run_sparse(5, 1, 1, sm_scale=sm_scale)
    c.check_sparse(got, 5, 1, 1, sm_scale=float(torch.tensor(sm_scale, dtype=torch.float32)))


def test_heads_of_very_different_magnitudes():
    c = Sparse([64 * 30 + 5], 1, 64, seed=7)
    c.q[0, 0] = (c.q[0, 0].float() * torch.exp2(torch.linspace(-125, 100, 64, device=DEV)).unsqueeze(1)).to(torch.bfloat16)
    c.q[0, 0, 10] = 0
    codes = c.run_sparse(8, 0, 1)
    c_means = c.means[:, :512].view(torch.int8).cpu(), c.means[:, 512].long().cpu() - 127
    want = expected_pages(c.q[0, 0], c_means, c.table[0].cpu().long(), 30, 8, 0, 1)
    assert codes[2][0, 0].tolist() == want
    c.q[0, 0] = 3e-38                                                        # exponents at their lower end
    c.q[0, 0, ::2, ::2] = -1e-38
    got = c.run_sparse(8, 0, 1)
    assert got[2][0, 0].tolist() == expected_pages(c.q[0, 0], c_means, c.table[0].cpu().long(), 30, 8, 0, 1)


def test_long_sequences_with_repeated_pages():
    """9000 pages (half a million tokens) out of a small pool, so that scores repeat."""
    c = Sparse([64 * 300], 1, 16, seed=8)
    pages = 9001
    g = torch.Generator(device=DEV).manual_seed(1)
    c.table = c.table[0, torch.randint(0, 300, (1, pages), generator=g, device=DEV)].contiguous()
    c.max_pages, c.lens = pages, [pages * 64 - 3]
    c.seq = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    for top, sinks, local in [(200, 1, 2), (1025, 5, 40), (9000, 0, 1), (9001, 0, 1)]:
        got = c.run_sparse(top, sinks, local)
        assert got[3] == 0
        c.check_sparse(got, top, sinks, local)


def repeated(lens, pool_pages, s, h, seed):
    """Sequences whose pages come out of a small pool, again and again."""
    c = Sparse([64 * pool_pages], s, h, seed=seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    c.max_pages = max(lens) // 64 + 2
    c.lens = list(lens)
    held = c.table[0, :pool_pages]
    c.table = held[torch.randint(0, pool_pages, (len(lens), c.max_pages), generator=g, device=DEV)]
    c.seq = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    c.q = torch.randn(len(lens), s, h, 512, generator=g, device=DEV).to(torch.bfloat16)
    return c


@pytest.mark.parametrize("h,pages,top,sinks,local", [
    (65, 17500, 150, 1, 2),       # more scores than the choice keeps in shared memory
    (65, 12000, 6000, 0, 1),      # room for the scores, not for the list of pages behind them
    (16, 35200, 100, 3, 3),
    (16, 20000, 14000, 0, 2),
    (16, 300, 7, 3, 4),           # nothing left to choose
])
def test_scores_and_lists_of_every_size(h, pages, top, sinks, local):
    c = repeated([pages * 64 - 9], 260, 1, h, seed=pages)
    got = c.run_sparse(top, sinks, local)
    assert got[3] == 0
    c.check_sparse(got, top, sinks, local)


@pytest.mark.parametrize("h", [8, 24, 64, 128])
@pytest.mark.parametrize("num_sms", [0, 1, 7])
def test_many_tiles_and_query_tokens_of_one_block(h, num_sms):
    """Tiles of 128 pages by the dozen, several query tokens a block, short ones in between."""
    c = repeated([64 * 1700 + 3, 5, 64 * 129, 64 * 640 + 63, 0, 64 * 386 + 1], 200, 2, h, seed=h)
    got = c.run_sparse(12, 1, 2, num_sms=num_sms)
    assert got[3] == 0
    c.check_sparse(got, 12, 1, 2)
    again = c.run_sparse(12, 1, 2, num_sms=num_sms)
    assert all(torch.equal(x, y) for x, y in zip(got[:3], again[:3]))


def test_bad_page_ids_are_skipped_and_flagged():
    c = Sparse([64 * 20 + 30, 64 * 12], 1, 16, seed=9)
    c.table[0, 7], c.table[0, 8], c.table[1, 3] = -4, c.num_pages, 2 ** 31 - 1
    got = c.run_sparse(6, 1, 1)
    assert got[3] == mla.DEVERR_BAD_INDEX
    c.check_sparse(got, 6, 1, 1)
    assert not {7, 8} & set(got[2][0, 0].tolist())
    got = c.run_sparse(20, 1, 1)                                             # nothing else is left: chosen, skipped
    assert got[3] == mla.DEVERR_BAD_INDEX
    c.check_sparse(got, 20, 1, 1)


def test_bad_lengths_count_as_empty_and_are_flagged():
    c = Sparse([100, 640, 300], 1, 16, seed=2, max_pages=10)
    c.seq[0], c.seq[2] = -3, 641
    got = c.run_sparse(4)
    assert got[3] == mla.DEVERR_BAD_LENGTH
    c.lens[0] = c.lens[2] = 0
    c.check_sparse(got, 4)


def test_budget_of_everything_is_the_dense_decode():
    c = Sparse([700, 1300, 64], 2, 40, seed=10)
    got = c.run_sparse(c.max_pages)
    out, lse, err = c.run()
    assert got[3] == err == 0
    assert torch.allclose(got[1], lse, atol=1e-5, rtol=1e-6)
    assert torch.all((got[0].float() - out.float()).abs() <= 2.0 ** -7 * out.float().abs() + 1e-3)


@pytest.mark.parametrize("num_sms", [0, 3, 20])
def test_same_bits_on_another_stream_and_any_part_count_selects_alike(num_sms):
    c = Sparse([3000, 100, 2000], 2, 64, seed=13)
    a = c.run_sparse(12, num_sms=num_sms)
    b = c.run_sparse(12, num_sms=num_sms, stream=torch.cuda.Stream())
    for x, y in zip(a[:3], b[:3]):
        assert torch.equal(x, y)
    c.check_sparse(a, 12)


def test_captured_graph_follows_the_lengths_on_the_device():
    c = Sparse([2900, 1350], 2, 32, seed=14)
    dec = mla.PagedSparseFP4Decoder(c.sparse_problem(6, 1, 2), DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = dec(c.q, c.kv, c.means, c.table, c.seq)
    for lens in ([2900, 1350], [70, 0], [1, 1290], [1400, 513]):
        c.seq.copy_(torch.tensor(lens, dtype=torch.int32))
        c.lens = lens
        graph.replay()
        torch.cuda.synchronize()
        c.check_sparse(got, 6, 1, 2)
        assert int(dec.error) == 0


def test_rows_past_the_batch_and_no_selected_output():
    c = Sparse([900, 1300], 2, 24, seed=12)
    p = c.sparse_problem(5, 1, 1)
    parts, ws = mla.paged_sparse_plan(p)
    out = torch.full((4, 2, 24, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((4, 2, 24), 7.0, device=DEV)
    work = torch.full((ws + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    mla.paged_sparse_decode_fp4(p, c.q, c.kv, c.means, c.table, c.seq, parts, work[:ws], out[:2], lse[:2])
    sel = torch.full((4, 2, 5), -9, dtype=torch.int32, device=DEV)
    mla.paged_sparse_decode_fp4(p, c.q, c.kv, c.means, c.table, c.seq, parts, work[:ws], out[:2], lse[:2], selected=sel[:2])
    torch.cuda.synchronize()
    c.check_sparse((out, lse, sel), 5, 1, 1)
    assert torch.all(out[2:] == 7) and torch.all(lse[2:] == 7) and torch.all(sel[2:] == -9)
    assert torch.all(work[ws:] == 0xA5)


def test_pool_beyond_4_gib():
    """The same pages at the far end of a large pool: means, choice and attention as before."""
    c = Sparse([64 * 300 + 5, 900], 1, 24, seed=21)
    want = c.run_sparse(9, 1, 2)
    off, pages, means = 250000, c.num_pages, c.means
    big = torch.zeros(off + pages, 64, 288, dtype=torch.uint8, device=DEV)
    big[off:] = c.kv
    c.kv, c.num_pages = big, off + pages
    c.table = (c.table + off).where((c.table >= 0) & (c.table < pages), c.table)
    c.means = torch.full((c.num_pages, 528), 0xA5, dtype=torch.uint8, device=DEV)
    c.refresh()
    assert torch.equal(c.means[off:], means) and not torch.any(c.means[:off, :512])
    got = c.run_sparse(9, 1, 2)
    assert got[3] == 0
    for x, y in zip(got[:3], want[:3]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("h,num_sms", [(128, 4), (100, 5), (65, 2), (128, 1), (128, 0)])
def test_many_query_tokens_on_few_blocks(h, num_sms):
    """Enough pages a block that pairs of SMs take the selected ones, lengths of every kind among them."""
    c = Sparse(LENGTHS + [64 * 40, 1800, 1] + ([1500] * 40 if num_sms == 0 else []), 2, h, seed=h + num_sms)
    c.q[3] *= 8
    got = c.run_sparse(24, 1, 2, num_sms=num_sms)
    assert got[3] == 0
    c.check_sparse(got, 24, 1, 2)
    again = c.run_sparse(24, 1, 2, num_sms=num_sms, stream=torch.cuda.Stream())
    assert all(torch.equal(x, y) for x, y in zip(got[:3], again[:3]))
