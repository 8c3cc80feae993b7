"""A call that CUDA refuses reports it and leaves no error behind: what the
thread launches next, here or in PyTorch, must not find it and take it for its
own.  The refusal is CUDA's answer to a launch into a capture that a
synchronisation has already spoilt; nothing runs on the GPU."""
import ctypes

import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla
from test_gpu_paged_decode import DEV, Case

pytestmark = pytest.mark.gpu


def runtime():
    mla.load()
    return ctypes.CDLL(next(f for f in open("/proc/self/maps").read().split() if "libcudart.so" in f))


def in_a_spoilt_capture(call):
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        graph.capture_begin()
        with pytest.raises(RuntimeError):
            stream.synchronize()
        assert runtime().cudaPeekAtLastError() == 0   # (PyTorch has taken its own)
        with pytest.raises(mla.MLAError):
            call()
        # Nothing is left for whoever asks next.
        assert runtime().cudaPeekAtLastError() == 0
        with pytest.raises(RuntimeError):
            graph.capture_end()


def paged_decode():
    c = Case([300, 65], 1, 16, seed=33)
    dec = mla.PagedFP4Decoder(c.problem(), DEV)
    out, lse = dec(c.q, c.kv, c.table, c.seq)
    return c, out, lse, lambda: dec(c.q, c.kv, c.table, c.seq, out, lse)


def test_combine_leaves_no_error_behind():
    n, h = 3, 16
    prob = mla.Problem.make(n, 1, h, 128, 2)
    splits = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    o, part = torch.randn(n, h, 512, device=DEV), torch.randn(n, h, device=DEV)
    out, lse = torch.empty(n, 1, h, 512, dtype=torch.bfloat16, device=DEV), torch.empty(n, 1, h, device=DEV)
    torch.cuda.synchronize()
    in_a_spoilt_capture(lambda: mla.combine(prob, splits, o, part, out, lse))
    mla.combine(prob, splits, o, part, out, lse)
    assert torch.equal(out.view(n, h, 512), o.to(torch.bfloat16))


def test_paged_decode_leaves_no_error_behind():
    c, out, lse, call = paged_decode()
    torch.cuda.synchronize()
    in_a_spoilt_capture(call)
    x = torch.ones(4, 2, 64, device=DEV)
    mla.rope(x, torch.zeros(4, dtype=torch.int32, device=DEV), mla.RopeTable(64))       # the next call is its own
    assert torch.all(x == 1)
    out.fill_(float("nan"))
    call()
    c.check(out, lse)
