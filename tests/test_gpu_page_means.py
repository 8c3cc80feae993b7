"""mla_page_means against the mean in whole numbers: every byte equal, since
the codes are one rounding of an exact mean."""
from fractions import Fraction

import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla
from test_gpu_paged_decode import decode_records, random_records

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)


def rounded(v):
    """A Fraction to the nearest whole number, halves to even."""
    return round(v)


def mean_record(page):
    """uint8 [64, 288] -> 528 bytes."""
    total = (decode_records(page) * 1024).sum(0)      # whole numbers below 2^28, exact in 64 bits
    ints = [int(v) for v in total.tolist()]
    top = max(abs(v) for v in ints)
    e = 0
    if top:
        e = -60
        while Fraction(top, 65536) / Fraction(2) ** e > 127:
            e += 1
    codes = [rounded(Fraction(v, 65536) / Fraction(2) ** e) for v in ints]
    return torch.tensor([c & 255 for c in codes] + [127 + e] + [0] * 15, dtype=torch.uint8)


def pool_of(pages, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    pool = random_records(pages * 64, g, top=0x7F).view(pages, 64, 288)
    if pages > 3:
        pool[1] = 0                                     # a mean of zeros
        pool[2, :, 256:] = 1                            # the smallest scale: means below one code's step
        pool[2, :, :256] = 0x11
        pool[3, :, 256:] = 0x7E                         # the largest values of one sign: 2688
        pool[3, :, :256] = 0x77
    return pool


@pytest.mark.parametrize("pages", [1, 2, 5, 40])
def test_means_of_every_page(pages):
    pool = pool_of(pages, pages)
    means = torch.full((pages, 528), 0xA5, dtype=torch.uint8, device=DEV)
    slots = (torch.randperm(pages, generator=torch.Generator().manual_seed(0)) * 64 + 63).to(torch.int32).to(DEV)
    mla.page_means(pool, slots, means)
    got = means.cpu()
    for p in range(pages):
        assert torch.equal(got[p], mean_record(pool[p])), p


def test_halves_round_to_even():
    """Sums of exactly half a code's step, of both signs."""
    pool = torch.zeros(1, 64, 288, dtype=torch.uint8, device=DEV)
    pool[0, :, 256:] = 0x38                             # scales of 1
    pool[0, :, 0] = 0x77                                # dims 0 and 1: 6 everywhere, 384 in all: a step of 4
    for d, want in [(2, 1), (4, 3), (6, 5), (8, 7)]:    # sums of 2, 6, 10, 14 in dims 2, 4, 6, 8; minus that in the next
        for t in range(want):
            pool[0, t, d // 2] = 0x4 | (0xC << 4)
    means = torch.zeros(1, 528, dtype=torch.uint8, device=DEV)
    mla.page_means(pool, torch.tensor([63], dtype=torch.int32, device=DEV), means)
    assert torch.equal(means.cpu()[0], mean_record(pool[0]))
    codes = means[0, :10].view(torch.int8).tolist()
    assert codes[:2] == [96, 96] and codes[2:] == [0, 0, 2, -2, 2, -2, 4, -4]


def test_only_completed_pages_are_written():
    pool = pool_of(9, 3)
    means = torch.full((9, 528), 0xA5, dtype=torch.uint8, device=DEV)
    # Page 4 completed, page 5 begun, page 6 all but its last slot, nothing of the others; skipped entries.
    slots = list(range(4 * 64 + 10, 6 * 64 + 20)) + [-1, -1] + list(range(6 * 64, 6 * 64 + 63))
    mla.page_means(pool, torch.tensor(slots, dtype=torch.int32, device=DEV), means)
    got = means.cpu()
    for p in range(9):
        if p in (4, 5):
            assert torch.equal(got[p], mean_record(pool[p]))
        else:
            assert bool((got[p] == 0xA5).all())


def test_bad_slots_are_flagged_and_skipped():
    pool = pool_of(4, 4)
    means = torch.full((5, 528), 0xA5, dtype=torch.uint8, device=DEV)
    error = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = torch.tensor([4 * 64 + 63, -65, 63, 2 ** 31 - 1, -1], dtype=torch.int32, device=DEV)
    mla.page_means(pool, slots, means, num_pages=4, error=error)
    got = means.cpu()
    assert int(error) == mla.DEVERR_BAD_INDEX
    assert torch.equal(got[0], mean_record(pool[0])) and bool((got[1:] == 0xA5).all())


@pytest.mark.parametrize("n", [1, 63, 64, 607, 5000, 400000])
def test_long_lists(n):
    """One request's slots, in a shuffled pool; more entries than the grid takes in one go."""
    pages = n // 64 + 2
    g = torch.Generator(device=DEV).manual_seed(n)
    pool = random_records(pages * 64, g).view(pages, 64, 288)
    ids = torch.randperm(pages, generator=g, device=DEV)
    i = torch.arange(n, device=DEV) + 7
    slots = (ids[i // 64] * 64 + i % 64).to(torch.int32)
    means = torch.full((pages, 528), 0xA5, dtype=torch.uint8, device=DEV)
    mla.page_means(pool, slots, means)
    done = [int(ids[k]) for k in range(pages) if 64 * k + 63 in range(7, n + 7)]
    touched = (means != 0xA5).any(1)
    assert sorted(torch.nonzero(touched).flatten().tolist()) == sorted(done)
    for p in done[:3] + done[-3:]:
        assert torch.equal(means[p].cpu(), mean_record(pool[p]))
    # All of them, in 64-bit torch operations.
    if done:
        at = torch.tensor(done, device=DEV)
        for part in at.split(1000):
            s = decode_records(pool[part].view(-1, 288)).view(-1, 64, 512).sum(1)
            top = s.abs().amax(-1, keepdim=True)
            m, e = torch.frexp(top)
            e = torch.where(m <= 127 / 128, e - 7, e - 6)
            assert torch.equal(means[part, :512].view(torch.int8).double(), torch.round(s * torch.exp2(-e.double())))
            assert torch.equal(means[part, 512].long(), (e - 6 + 127).squeeze(-1).long())


def test_nan_scales_count_as_448():
    pool = torch.zeros(2, 64, 288, dtype=torch.uint8, device=DEV)
    pool[:, :, 0] = 0x32                                # dims 0 and 1: 1 and 1.5
    pool[0, :, 256], pool[1, :, 256] = 0x7F, 0x7E
    means = torch.zeros(2, 528, dtype=torch.uint8, device=DEV)
    mla.page_means(pool, torch.tensor([63, 127], dtype=torch.int32, device=DEV), means)
    assert torch.equal(means[0], means[1]) and int(means[0, 0]) > 0
    pool[0, :, 256], pool[1, :, 256] = 0xFF, 0xFE
    mla.page_means(pool, torch.tensor([63, 127], dtype=torch.int32, device=DEV), means)
    assert torch.equal(means[0], means[1]) and means[0, :1].view(torch.int8).item() < 0


def test_graph_replays_and_same_bytes():
    pool = pool_of(12, 8)
    slots = torch.full((300,), -1, dtype=torch.int32, device=DEV)
    means = torch.zeros(12, 528, dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        mla.page_means(pool, slots, means)
    for p in (3, 7, 11):
        slots.fill_(-1)
        slots[5 * p] = p * 64 + 63
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(means[p].cpu(), mean_record(pool[p]))
    assert int(means.any(1).sum()) == 3
