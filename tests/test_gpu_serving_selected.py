"""Appending, page means, selected pages and shared prefixes as a serving loop
uses them together, eagerly and as captured graphs; and what their kernels read
of a kernel before them that released its dependents early."""
import random

import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla
from test_gpu_early_release import late  # noqa: F401  (a fixture)
from test_gpu_paged_decode import decode_records
from test_gpu_paged_shared import Shared, width  # noqa: F401  (a fixture)
from test_gpu_paged_sparse import Sparse, expected_pages

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
I32 = torch.int32


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("b,h,top,sinks,local", [(4, 16, 4, 1, 1), (3, 40, 3, 0, 2)])
def test_a_loop_that_appends_and_selects(b, h, top, sinks, local, graph):
    """Chunks of prompts and single tokens grow the sequences; every step's new pages get their means; attention over
    what is selected is compared with the records that the loop itself keeps."""
    g = torch.Generator(device=DEV).manual_seed(b)
    max_pages = 14
    pages = b * max_pages
    z = lambda *n: torch.zeros(*n, dtype=I32, device=DEV)  # noqa: E731
    lens, new, table, cu = z(b), z(b), torch.full((b, max_pages), -1, dtype=I32, device=DEV), z(b + 1)
    free, num_free = torch.randperm(pages, generator=g, device=DEV).to(I32), torch.tensor([pages], dtype=I32, device=DEV)
    room = 130 * b
    slots, pos, error = z(room), z(room), z(1)
    projection = torch.zeros(room, 576, dtype=torch.bfloat16, device=DEV)
    latents = projection[:, 32:544]
    q = torch.zeros(b, 1, h, 512, dtype=torch.bfloat16, device=DEV)
    pool = torch.full((pages, 64, 288), 0xFF, dtype=torch.uint8, device=DEV)
    means = torch.full((pages, 528), 0xA5, dtype=torch.uint8, device=DEV)
    rope = mla.RopeTable(64, scaling=mla.RopeScaling.yarn(4.0, 4096))
    dec = mla.PagedSparseFP4Decoder(mla.PagedSparseProblem.make(b, 1, h, max_pages, pages, top, sink_pages=sinks,
                                                                local_pages=local), DEV)
    out, lse = torch.empty_like(q), torch.empty(b, 1, h, device=DEV)
    sel = torch.empty(b, 1, top, dtype=I32, device=DEV)
    stream = torch.cuda.Stream()

    def step():
        mla.page_plan(lens, new, table, free, num_free, lens, num_free, cu, slots, pos, error=error)
        mla.kv_append(latents, slots, pool, mla.KV_FP4_288, rope=rope, positions=pos, error=error)
        mla.page_means(pool, slots, means, error=error)
        dec(q, pool, means, table, lens, out, lse, sel)

    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse)) and torch.all(sel == -1)
    captured = None
    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured, stream=stream):
            step()
    rng = random.Random(b)
    held = [0] * b
    for t in range(60):
        counts = [rng.choice([1, 1, 1, 0, rng.randrange(2, 130)]) for _ in range(b)]
        for r in range(b):
            if held[r] + max(counts[r], 0) > 64 * max_pages - 140:
                counts[r] = -1
        new.copy_(torch.tensor(counts, dtype=I32))
        projection.copy_(torch.randn(room, 576, generator=g, device=DEV) + torch.randn(1, 576, generator=g, device=DEV))
        q.copy_(2 * torch.randn(b, 1, h, 512, generator=g, device=DEV))
        torch.cuda.synchronize()
        if captured is not None:
            captured.replay()
        else:
            with torch.cuda.stream(stream):
                step()
        torch.cuda.synchronize()
        held = [0 if c < 0 else held[r] + c for r, c in enumerate(counts)]
        assert int(error) == 0 and int(dec.error) == 0 and lens.tolist() == held
        if t % 6 != 5:
            continue
        codes = means[:, :512].view(torch.int8).cpu(), means[:, 512].long().cpu() - 127
        # The means that a rebuild of every full page gives are those that the steps left.
        again = torch.full_like(means, 0xA5)
        full = [int(table[r, k]) for r in range(b) for k in range(held[r] // 64)]
        if full:
            mla.page_means(pool, (torch.tensor(full, dtype=I32) * 64 + 63).to(DEV), again)
            assert torch.equal(again[full], means[full])
        for r in range(b):
            m = held[r]
            if m == 0:
                assert torch.all(out[r] == 0) and torch.all(torch.isneginf(lse[r])) and torch.all(sel[r] == -1)
                continue
            ids = table[r].cpu().long()
            want = expected_pages(q[r, 0], codes, ids, (m - 1) // 64, top, sinks, local)
            assert sel[r, 0].tolist() == want + [-1] * (top - len(want))
            k = decode_records(pool[ids[want].to(DEV)].reshape(-1, 288))[: (len(want) - 1) * 64 + (m - 1) % 64 + 1]
            x = q[r, 0].double() @ k.T * 512 ** -0.5
            o = torch.softmax(x, -1) @ k
            assert torch.all((lse[r, 0].double() - torch.logsumexp(x, -1)).abs() <= 1e-3)
            assert torch.all((out[r, 0].double() - o).abs() <= 1e-2 + 1e-2 * o.abs())


def test_samples_of_one_prompt():
    """A prompt appended once, samples of it decoded over its pages and their own: as if each had a copy."""
    g = torch.Generator(device=DEV).manual_seed(5)
    b, h, prompt, own_pages = 6, 32, 777, 4
    prefix_pages = -(-prompt // 64)
    pages = prefix_pages + b * own_pages
    pool = torch.full((pages, 64, 288), 0xFF, dtype=torch.uint8, device=DEV)
    ids = torch.randperm(pages, generator=g, device=DEV).to(I32)
    ptable, table = ids[:prefix_pages].view(1, -1).contiguous(), ids[prefix_pages:].view(b, own_pages).contiguous()
    rope = mla.RopeTable(64)
    at = torch.arange(prompt, dtype=I32, device=DEV)
    mla.kv_append(torch.randn(prompt, 512, generator=g, device=DEV).to(torch.bfloat16), ptable[0, at.long() // 64] * 64 + at % 64,
                  pool, mla.KV_FP4_288, rope=rope, positions=at)
    dec = mla.PagedSharedFP4Decoder(mla.PagedSharedProblem.make(b, 1, h, own_pages, prefix_pages, pages), DEV)
    whole = mla.PagedFP4Decoder(mla.PagedProblem.make(b, 1, h, prefix_pages + 5, pages + b), DEV)
    start, plen = torch.tensor([0, b], dtype=I32, device=DEV), torch.tensor([prompt], dtype=I32, device=DEV)
    lens = torch.zeros(b, dtype=I32, device=DEV)
    for t in range(130):
        slots = table[:, t // 64] * 64 + t % 64
        latents = torch.randn(b, 512, generator=g, device=DEV).to(torch.bfloat16)
        mla.kv_append(latents, slots.contiguous(), pool, mla.KV_FP4_288, rope=rope, positions=lens + prompt)
        lens += 1
        if t not in (0, 40, 63, 64, 129):
            continue
        q = (2 * torch.randn(b, 1, h, 512, generator=g, device=DEV)).to(torch.bfloat16)
        out, lse = dec(q, pool, start, ptable, plen, table, lens)
        # The same tokens as sequences with a copy of the prompt each, laid out in a pool of their own.
        flat = torch.cat([pool[ptable[0].long()].reshape(-1, 288)[:prompt].unsqueeze(0).expand(b, -1, -1),
                          pool[table.long()].reshape(b, -1, 288)[:, : t + 1]], 1)
        n = prompt + t + 1
        copies = torch.full((b, prefix_pages + 5, 64, 288), 0xFF, dtype=torch.uint8, device=DEV)
        copies.view(b, -1, 288)[:, :n] = flat
        one = torch.arange(b * (prefix_pages + 5), dtype=I32, device=DEV).view(b, -1)
        again = mla.PagedFP4Decoder(mla.PagedProblem.make(b, 1, h, prefix_pages + 5, one.numel()), DEV)
        want, want_lse = again(q, copies.view(-1, 64, 288), one, torch.full((b,), n, dtype=I32, device=DEV))
        assert int(dec.error) == 0
        assert torch.all((lse - want_lse).abs() <= 1e-4)
        assert torch.all((out.float() - want.float()).abs() <= 2.0 ** -6 * want.float().abs() + 2.0 ** -9)
    del whole


def test_selected_decode_reads_what_an_early_releasing_kernel_writes(late):  # noqa: F811
    c = Sparse([1700, 65, 0, 1300, 2], 2, 64, seed=31)
    dec = mla.PagedSparseFP4Decoder(c.sparse_problem(6, 1, 1), DEV)
    lens, table = torch.empty_like(c.seq), torch.empty_like(c.table)
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:3], device=DEV)
    sel = torch.empty(5, 2, 6, dtype=I32, device=DEV)
    stream = torch.cuda.Stream()
    for before in (0, 1, 64):
        lens.fill_(before)
        table.fill_(0)
        torch.cuda.synchronize()
        for _ in range(2):
            late(lens, c.seq, table, c.table, stream)
            dec(c.q, c.kv, c.means, table, lens, out, lse, sel, stream=stream)
        torch.cuda.synchronize()
        c.check_sparse((out, lse, sel), 6, 1, 1)
    assert int(dec.error) == 0


def test_shared_decode_reads_what_an_early_releasing_kernel_writes(late):  # noqa: F811
    c = Shared([70, 65, 0, 130, 2], 2, 64, [0, 2, 5], [700, 300], seed=31)
    dec = mla.PagedSharedFP4Decoder(c.shared_problem(), DEV)
    plens, ptable = torch.empty_like(c.plen), torch.empty_like(c.ptable)
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:3], device=DEV)
    stream = torch.cuda.Stream()
    for before in (0, 1, 64):
        plens.fill_(before)
        ptable.fill_(0)
        torch.cuda.synchronize()
        for _ in range(2):
            late(plens, c.plen, ptable, c.ptable, stream)
            dec(c.q, c.kv, c.start, ptable, plens, c.table, c.seq, out, lse, stream=stream)
        torch.cuda.synchronize()
        c.check_shared(out, lse)
    assert int(dec.error) == 0


def test_append_and_means_read_what_an_early_releasing_kernel_writes(late):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(3)
    n = 300
    x = torch.randn(n, 512, generator=g, device=DEV).to(torch.bfloat16)
    slots, pos = torch.arange(n, dtype=I32, device=DEV), torch.arange(n, dtype=I32, device=DEV) * 7
    rope = mla.RopeTable(64)
    want, want_means = torch.zeros(5, 64, 288, dtype=torch.uint8, device=DEV), torch.zeros(5, 528, dtype=torch.uint8, device=DEV)
    mla.kv_append(x, slots, want, mla.KV_FP4_288, rope=rope, positions=pos)
    mla.page_means(want, slots, want_means)
    got, got_means = torch.zeros_like(want), torch.zeros_like(want_means)
    s2, p2 = torch.full_like(slots, -1), torch.zeros_like(pos)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    late(s2, slots, p2, pos, stream)
    mla.kv_append(x, s2, got, mla.KV_FP4_288, rope=rope, positions=p2, stream=stream)
    mla.page_means(got, s2, got_means, stream=stream)
    stream.synchronize()
    assert torch.equal(got, want) and torch.equal(got_means, want_means)
