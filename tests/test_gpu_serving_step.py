"""The operators as a serving loop uses them, one captured graph per step:
pages and slots for the new tokens, the latents' norm and the rotary tail,
the FP4 records into their slots, attention over the sequence's pages; then
the attended rows' own norm.  Requests grow, end and come back over the
steps, and every step is compared with a plain reference."""
import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla
from test_gpu_paged_decode import decode_records
from test_gpu_rms_norm_fp8 import verify

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
I32 = torch.int32


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("b,h,window,sinks", [(5, 16, 0, 0), (3, 40, 70, 4)])
def test_steps_of_a_serving_loop(b, h, window, sinks, graph):
    g = torch.Generator(device=DEV).manual_seed(b)
    max_pages, pages = 6, b * 6
    z = lambda *n: torch.zeros(*n, dtype=I32, device=DEV)  # noqa: E731
    lens, new, table, cu = z(b), z(b), torch.full((b, max_pages), -1, dtype=I32, device=DEV), z(b + 1)
    free, num_free = torch.randperm(pages, generator=g, device=DEV).to(I32), torch.tensor([pages], dtype=I32, device=DEV)
    room = b + 2                                     # padded: the step's spare rows are skipped by their slots
    slots, pos, error = z(room), z(room), z(1)
    latents = torch.zeros(room, 512, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(b, 1, h, 512, dtype=torch.bfloat16, device=DEV)
    qpos = z(b)
    pool = torch.full((pages, 64, 288), 0xFF, dtype=torch.uint8, device=DEV)
    rope = mla.RopeTable(64, scaling=mla.RopeScaling.yarn(4.0, 4096))
    dec = mla.PagedFP4Decoder(mla.PagedProblem.make(b, 1, h, max_pages, pages, window=window, sinks=sinks), DEV)
    weight = (1 + 0.1 * torch.randn(512, generator=g, device=DEV)).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(b, 1, h, device=DEV)
    codes = torch.zeros(b * h, 512, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(b * h, 16, dtype=torch.uint8, device=DEV)
    stream = torch.cuda.Stream()

    def step():
        mla.page_plan(lens, new, table, free, num_free, lens, num_free, cu, slots, pos, error=error)
        mla.rope(latents, pos, rope, offset=448)
        mla.kv_write(latents, slots, pool, mla.KV_FP4_288, error=error)
        mla.rope(q.view(b, h, 512), qpos, rope, offset=448)
        dec(q, pool, table, lens, out, lse)
        mla.rms_norm_fp8(out.view(b * h, 512), weight, 1e-6, codes, scales)

    with torch.cuda.stream(stream):
        step()                                       # nothing new, nothing cached: every row is empty
    stream.synchronize()
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    captured = None
    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured, stream=stream):
            step()
    held = [torch.zeros(0, 288, dtype=torch.uint8, device=DEV) for _ in range(b)]
    import random
    rng = random.Random(b)
    for t in range(150):
        counts = [1 if rng.random() < 0.9 else 0 for _ in range(b)]
        for r in range(b):
            if len(held[r]) > 350 or (len(held[r]) > 0 and rng.random() < 0.01):
                counts[r] = -1
        n = sum(max(c, 0) for c in counts)
        new.copy_(torch.tensor(counts, dtype=I32))
        latents.copy_(torch.randn(room, 512, generator=g, device=DEV))
        q.copy_(2 * torch.randn(b, 1, h, 512, generator=g, device=DEV))
        after = [0 if c < 0 else len(held[r]) + c for r, c in enumerate(counts)]
        qpos.copy_(torch.tensor([max(v - 1, 0) for v in after], dtype=I32))
        torch.cuda.synchronize()
        if captured is not None:
            captured.replay()
        else:
            with torch.cuda.stream(stream):
                step()
        torch.cuda.synchronize()
        assert int(error) == 0 and int(dec.error) == 0
        assert lens.tolist() == after
        assert int((slots >= 0).sum()) == n
        # The records as the writer made them, token by token, in the reference's own lists.
        at = 0
        for r, c in enumerate(counts):
            if c < 0:
                held[r] = held[r][:0]
            for _ in range(max(c, 0)):
                assert int(pos[at]) == len(held[r])
                held[r] = torch.cat([held[r], pool.view(-1, 288)[int(slots[at])].unsqueeze(0)])
                at += 1
        if t % 10 != 9:
            continue
        for r in range(b):
            m = len(held[r])
            if m == 0:
                assert torch.all(out[r] == 0) and torch.all(torch.isneginf(lse[r]))
                continue
            k = decode_records(held[r])
            j = torch.arange(m, device=DEV)
            if window:
                k = k[(j > m - 1 - window) | (j < sinks)]
            x = q[r, 0].double() @ k.T * 512 ** -0.5
            p = torch.softmax(x, -1)
            assert torch.all((lse[r, 0].double() - torch.logsumexp(x, -1)).abs() <= 1e-3)
            o = p @ k
            assert torch.all((out[r, 0].double() - o).abs() <= 1e-2 + 1e-2 * o.abs())
        verify(out.view(b * h, 512), None, weight, 1e-6, codes, scales, None)
