"""mla_paged_shared_decode_fp4 against attention in 64 bits over each group's
prefix and the sequence's own tokens.

Tolerances as for mla_paged_decode_fp4: a score within dx = 64 * 2^-23 *
sm_scale * sum |q_d k_d|, |lse error| <= dx + 2^-20 (1 + |lse|), |out error|
<= (2^-11 + 2 dx + 2^-19) sum_j p_j |k_j| and the output's own rounding to bf16,
2^-8 of itself.  (The merge of the two parts adds a few 2^-24, far inside.)"""
import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla
from test_gpu_paged_decode import Case, decode_records, random_records

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
I32 = torch.int32


@pytest.fixture(params=[1, 9000], ids=["narrow", "wide"], autouse=True)
def width(request):
    """Prefix tables as wide as needed, or so wide that the plan expects long prefixes: pairs of SMs then take 128 rows."""
    Shared.width = request.param
    yield
    Shared.width = 1


class Shared(Case):
    """Own tokens as Case lays them out; prefixes in pages of their own, whatever is past their ends NaN scales."""
    width = 1

    def __init__(self, lens, s, h, start, plens, max_prefix_pages=None, seed=0, **kw):
        super().__init__(lens, s, h, seed=seed, **kw)
        g = torch.Generator(device=DEV).manual_seed(seed + 1)
        self.starts, self.plens = list(start), list(plens)
        held = [-(-n // 64) for n in plens]
        self.max_prefix_pages = max_prefix_pages or max(max(held), Shared.width)
        first = self.num_pages
        extra = torch.full((sum(held) + 1, 64, 288), 0xFF, dtype=torch.uint8, device=DEV)
        self.num_pages += extra.shape[0]
        ids = torch.randperm(extra.shape[0], generator=g, device=DEV).tolist()
        ptable = torch.full((len(plens), self.max_prefix_pages), -77, dtype=I32)
        for r, n in enumerate(plens):
            for k in range(held[r]):
                ptable[r, k] = first + ids.pop()
                m = min(64, n - 64 * k)
                extra[int(ptable[r, k]) - first, :m] = random_records(m, g)
        self.kv = torch.cat([self.kv, extra])
        self.ptable = ptable.to(DEV)
        self.start = torch.tensor(self.starts, dtype=I32, device=DEV)
        self.plen = torch.tensor(self.plens, dtype=I32, device=DEV)

    def shared_problem(self, **kw):
        return mla.PagedSharedProblem.make(len(self.lens), self.s, self.h, self.max_pages, self.max_prefix_pages,
                                           self.num_pages, groups=len(self.plens), **kw)

    def run_shared(self, num_sms=0, stream=None, **kw):
        dec = mla.PagedSharedFP4Decoder(self.shared_problem(**kw), DEV, num_sms=num_sms)
        dec.workspace.fill_(0xFF)
        out = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:3], float("nan"), device=DEV)
        torch.cuda.synchronize()
        dec(self.q, self.kv, self.start, self.ptable, self.plen, self.table, self.seq, out, lse, stream=stream)
        torch.cuda.synchronize()
        return out, lse, int(dec.error)

    def records(self, table, n):
        pages = table[: -(-n // 64)].long()
        ok = (pages >= 0) & (pages < self.num_pages)
        return decode_records(self.kv[pages.where(ok, 0)].reshape(-1, 288)[:n]), ok.repeat_interleave(64)[:n]

    def check_shared(self, out, lse, sm_scale=None, groups=None):
        scale = 512 ** -0.5 if sm_scale is None else float(torch.tensor(sm_scale, dtype=torch.float32))
        starts = self.starts if groups is None else groups
        prefixes = [self.records(self.ptable[g], n) if n > 0 else None for g, n in enumerate(self.plens)]
        for b, n in enumerate(self.lens):
            pre = None
            for g in range(len(self.plens)):
                if starts[g] <= b < starts[g + 1]:
                    pre = prefixes[g]
            own, ok = self.records(self.table[b], n)
            for i in range(self.s):
                at = n - self.s + i
                k = own[: max(at + 1, 0)][ok[: max(at + 1, 0)]]
                if at >= 0 and pre is not None:
                    k = torch.cat([pre[0][pre[1]], k])
                if k.shape[0] == 0:
                    assert torch.all(out[b, i] == 0) and not torch.any(torch.signbit(out[b, i].float()))
                    assert torch.all(torch.isneginf(lse[b, i]))
                    continue
                q = self.q[b, i].double()
                x = q @ k.T * scale
                dx = 64 * 2.0 ** -23 * (q.abs() @ k.abs().T * abs(scale)).amax(-1)
                want = torch.logsumexp(x, -1)
                err = (lse[b, i].double() - want).abs()
                tol = dx + 2.0 ** -20 * (1 + want.abs())
                assert torch.all(err <= tol), (b, i, float((err / tol).max()))
                p = torch.softmax(x, -1)
                o = p @ k
                tol = (2.0 ** -11 + 2 * dx.unsqueeze(-1) + 2.0 ** -19) * (p @ k.abs()) + 2.0 ** -8 * o.abs() + 1e-30
                tol = tol + 2.0 ** -30 * p.amax(-1, keepdim=True) * k.abs().sum(0)
                err = (out[b, i].double() - o).abs()
                assert torch.all(err <= tol), (b, i, float((err / tol).max()))


@pytest.mark.parametrize("plen", [0, 1, 63, 64, 65, 128, 129, 1000, 4097])
@pytest.mark.parametrize("s,h", [(1, 16), (1, 128), (3, 24)])
@pytest.mark.parametrize("num_sms", [0, 5])
def test_one_prefix_for_all(plen, s, h, num_sms):
    c = Shared([1, 5, 64, 0, 129, 300, 2, 77, 200], s, h, [0, 9], [plen], seed=plen + s)
    out, lse, err = c.run_shared(num_sms=num_sms)
    assert err == 0
    c.check_shared(out, lse)


@pytest.mark.parametrize("s,h", [(1, 1), (1, 7), (1, 33), (2, 64), (2, 100), (5, 13)])
@pytest.mark.parametrize("start,plens", [
    ([0, 3, 8], [500, 70]), ([0, 0, 8, 8], [100, 300, 200]),      # empty groups
    ([2, 5, 7], [400, 130]), ([3, 3], [64]),                      # sequences in no group
    ([0, 1, 2, 3, 4, 5, 6, 7, 8], [0, 64, 129, 1, 700, 0, 30, 256]), ([8, 8], [10]),
])
def test_groups(s, h, start, plens):
    c = Shared([30, 200, 0, 64, 1, 128, 513, 9], s, h, start, plens, seed=s * h)
    for sms in (0, 3):
        out, lse, err = c.run_shared(num_sms=sms)
        assert err == 0
        c.check_shared(out, lse)


@pytest.mark.parametrize("num_sms", [1, 2, 7, 40, 500])
@pytest.mark.parametrize("s,h", [(1, 16), (2, 128)])
def test_any_number_of_parts(num_sms, s, h):
    c = Shared([130, 0, 1, 700, 64], s, h, [0, 4, 5], [2500, 900], seed=num_sms)
    out, lse, err = c.run_shared(num_sms=num_sms)
    assert err == 0
    c.check_shared(out, lse)


@pytest.mark.parametrize("b,h,groups", [(700, 16, 1), (600, 16, 300), (150, 128, 4)])
def test_many_sequences(b, h, groups):
    """More units than a block has threads; groups of two sequences each."""
    start = [b * g // groups for g in range(groups + 1)]
    c = Shared([(37 * r) % 140 if r % 5 else 1 for r in range(b)], 1, h, start, [(53 * g) % 400 for g in range(groups)], seed=b)
    out, lse, err = c.run_shared()
    assert err == 0
    c.check_shared(out, lse)


def test_long_prefix_is_split_and_merged():
    c = Shared([40, 3], 1, 16, [0, 2], [20011], seed=8)
    out, lse, err = c.run_shared()
    assert err == 0
    c.check_shared(out, lse)


def test_prefix_and_own_scores_of_very_different_sizes():
    """All the mass in the prefix for some heads, all in the own tokens for others; a negative scale."""
    for sm in (2.0, -1.0, 0.0, 1e-30):
        c = Shared([70, 500, 65], 2, 24, [0, 3], [777], seed=11, qscale=8.0)
        out, lse, err = c.run_shared(sm_scale=sm)
        assert err == 0
        c.check_shared(out, lse, sm_scale=sm)


def test_maxima_that_grow_from_tile_to_tile():
    """Each tile of the prefix tops the last by 12 powers of two and more, so O is rescaled in every one."""
    tiles = 20
    c = Shared([65] * 40, 1, 64, [0, 40], [tiles * 128 - 5], seed=21)
    n = c.plens[0]
    pages = c.ptable[0, : -(-n // 64)].long()
    flat = c.kv[pages].reshape(-1, 288)
    flat[:n, :8] = 0x77
    flat[:n, 256] = (0x38 + torch.arange(n, device=DEV) // 128).to(torch.uint8)
    c.kv[pages] = flat.view(-1, 64, 288)
    c.q[..., :16] = 12 * 0.6931471805599453 * 8 / 96 * 512 ** 0.5
    first = c.run_shared()
    assert first[2] == 0
    c.check_shared(*first[:2])
    for _ in range(10):
        out, lse, err = c.run_shared()
        assert err == 0 and torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_groups_out_of_order_count_as_none():
    for start in ([0, 5, 3], [-1, 2, 6], [0, 2, 7], [2 ** 31 - 1, 0, 0]):
        c = Shared([30, 200, 0, 64, 1, 128], 1, 16, [0, 3, 6], [500, 70], seed=1)
        c.start = torch.tensor(start, dtype=I32, device=DEV)
        out, lse, err = c.run_shared()
        assert err == mla.DEVERR_BAD_METADATA
        c.check_shared(out, lse, groups=[0, 0, 0])


def test_bad_lengths_and_pages_are_flagged():
    c = Shared([30, 200, 60, 64], 2, 16, [0, 2, 4], [500, 300], max_prefix_pages=9, seed=2)
    c.plen[1] = 9 * 64 + 1
    c.seq[0] = -5
    out, lse, err = c.run_shared()
    assert err == mla.DEVERR_BAD_LENGTH
    c.plens[1], c.lens[0] = 0, 0
    c.check_shared(out, lse)
    c = Shared([30, 200, 60, 64], 2, 16, [0, 2, 4], [500, 300], seed=2)
    c.ptable[0, 3], c.ptable[1, 0], c.table[1, 1] = c.num_pages, -1, 2 ** 31 - 1
    out, lse, err = c.run_shared()
    assert err == mla.DEVERR_BAD_INDEX
    c.check_shared(out, lse)


def test_no_prefixes_is_the_paged_decode():
    c = Shared([300, 64, 640], 2, 40, [0, 3], [0], seed=5)
    out, lse, err = c.run_shared()
    want, want_lse, _ = c.run()
    assert err == 0
    assert torch.all((out.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 1e-3)
    assert torch.allclose(lse, want_lse, atol=1e-5, rtol=1e-6)


def test_rows_past_the_batch_and_the_workspace_stay_as_they_were():
    c = Shared([90, 130], 3, 24, [0, 2], [333], seed=12)
    p = c.shared_problem()
    parts, ws = mla.paged_shared_plan(p)
    work = torch.full((ws + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    out = torch.full((5, 3, 24, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((5, 3, 24), 7.0, device=DEV)
    mla.paged_shared_decode_fp4(p, c.q, c.kv, c.start, c.ptable, c.plen, c.table, c.seq, parts, work[:ws], out[:2], lse[:2])
    torch.cuda.synchronize()
    c.check_shared(out[:2], lse[:2])
    assert torch.all(out[2:] == 7) and torch.all(lse[2:] == 7) and torch.all(work[ws:] == 0xA5)


def test_same_bits_twice_and_on_another_stream():
    c = Shared([300, 100, 2000], 2, 64, [0, 2, 3], [3000, 100], seed=13)
    a = c.run_shared()
    b = c.run_shared(stream=torch.cuda.Stream())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_graph_follows_what_is_on_the_device():
    c = Shared([900, 350, 64, 10], 2, 32, [0, 4, 4], [900, 650], seed=14)
    dec = mla.PagedSharedFP4Decoder(c.shared_problem(), DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, lse = dec(c.q, c.kv, c.start, c.ptable, c.plen, c.table, c.seq)
    for lens, start, plens in (([900, 350, 64, 10], [0, 2, 4], [900, 650]), ([0, 1, 64, 3], [1, 1, 3], [130, 5]),
                               ([5, 350, 2, 10], [0, 4, 4], [0, 650])):
        c.seq.copy_(torch.tensor(lens, dtype=I32))
        c.start.copy_(torch.tensor(start, dtype=I32))
        c.plen.copy_(torch.tensor(plens, dtype=I32))
        c.lens, c.starts, c.plens = lens, start, plens
        graph.replay()
        torch.cuda.synchronize()
        c.check_shared(out, lse)
        assert int(dec.error) == 0


@pytest.mark.parametrize("b,s,h", [(9, 1, 128), (3, 4, 100), (40, 1, 33), (129, 1, 1), (1, 2, 128)])
def test_many_rows_over_every_length(b, s, h):
    """Rows that fill blocks of 128 and do not, prefixes around the tiles' and items' ends."""
    for plen in (1, 64, 127, 128, 192, 255, 256, 257, 300, 511, 513, 1025):
        c = Shared([(29 * r + s) % 300 + (r % 7 > 0) for r in range(b)], s, h, [0, b], [plen], seed=plen + h)
        out, lse, err = c.run_shared()
        assert err == 0
        c.check_shared(out, lse)


def test_masses_that_move_between_the_halves_of_an_item():
    """Large scores alternate between the first and the second 128 tokens of an item, so either half of a pair's tokens
    raises the maximum that both share; the same bits from run to run."""
    c = Shared([3, 70, 129, 300] * 8, 1, 64, [0, 32], [256 * 12 - 9], seed=31)
    n = c.plens[0]
    pages = c.ptable[0, : -(-n // 64)].long()
    flat = c.kv[pages].reshape(-1, 288)
    step = torch.arange(n, device=DEV) // 256
    big = ((torch.arange(n, device=DEV) // 128) % 2) == (step % 2)
    flat[:n, :8] = 0x77
    flat[:n, 256] = torch.where(big, 0x38 + step, torch.full_like(step, 0x20)).to(torch.uint8)
    c.kv[pages] = flat.view(-1, 64, 288)
    c.q[..., :16] = 12 * 0.6931471805599453 * 8 / 96 * 512 ** 0.5
    first = c.run_shared()
    assert first[2] == 0
    c.check_shared(*first[:2])
    for _ in range(20):
        out, lse, err = c.run_shared()
        assert err == 0 and torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_nan_records_reach_only_the_rows_that_see_them():
    c = Shared([65, 200, 9, 64], 2, 64, [0, 2, 4], [500, 700], seed=41)
    want = c.run_shared()
    c.kv[int(c.ptable[1, 3]), 5, 256:] = 0x7F           # in the second group's prefix
    out, lse, err = c.run_shared()
    assert err == 0
    assert torch.equal(out[:2], want[0][:2]) and torch.equal(lse[:2], want[1][:2])


@pytest.mark.parametrize("sm_scale", [-0.05, 0.3, 1e-30, 0.0])
@pytest.mark.parametrize("s,h", [(2, 24), (1, 128)])
def test_scales_of_either_sign(sm_scale, s, h):
    c = Shared([300, 64, 1, 129], s, h, [0, 3, 4], [900, 257], seed=51)
    out, lse, err = c.run_shared(sm_scale=sm_scale)
    assert err == 0
    c.check_shared(out, lse, sm_scale=sm_scale)


def test_pool_beyond_4_gib():
    c = Shared([300, 64, 1, 129], 1, 100, [0, 3, 4], [900, 257], seed=52)
    want = c.run_shared()
    off, pages = 250000, c.num_pages
    big = torch.zeros(off + pages, 64, 288, dtype=torch.uint8, device=DEV)
    big[off:] = c.kv
    c.kv, c.num_pages = big, off + pages
    c.table, c.ptable = ((t + off).where((t >= 0) & (t < pages), t) for t in (c.table, c.ptable))
    out, lse, err = c.run_shared()
    assert err == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
