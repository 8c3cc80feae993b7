"""A caller's kernel that lets its dependents start before it has written the
lengths and tables they read.  The operators' kernels may then be resident
while it still runs; what they read has to be what it wrote.

The kernel here is test-only: it releases its dependents, passes 200 us and
copies lengths and block tables into place."""
import ctypes
import subprocess

import pytest
import torch

from fp4_kv_cache_sparse_gb300 import build as mla_build
from test_gpu_paged_decode import DEV, Case

import fp4_kv_cache_sparse_gb300 as mla

pytestmark = pytest.mark.gpu

SRC = r"""
#include <cstdint>
#include <cuda_runtime.h>

__global__ void copy_late(int32_t* lens, const int32_t* new_lens, int n, int32_t* table, const int32_t* new_table, int m) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  int polls = 0;
  do {
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  } while (t - t0 < 200000 && ++polls < 1000000);
  for (int i = threadIdx.x; i < n; i += blockDim.x) lens[i] = new_lens[i];
  for (int i = threadIdx.x; i < m; i += blockDim.x) table[i] = new_table[i];
}

extern "C" int copy_late_launch(int32_t* lens, const int32_t* new_lens, int n, int32_t* table, const int32_t* new_table,
                                int m, void* stream) {
  copy_late<<<1, 256, 0, static_cast<cudaStream_t>(stream)>>>(lens, new_lens, n, table, new_table, m);
  return static_cast<int>(cudaGetLastError());
}
"""


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    d = tmp_path_factory.mktemp("late")
    src, so = d / "late.cu", d / "liblate.so"
    src.write_text(SRC)
    subprocess.check_call([mla_build.nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17",
                           "-shared", "-Xcompiler", "-fPIC", "-o", str(so), str(src)])
    lib = ctypes.CDLL(str(so))
    lib.copy_late_launch.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int] * 2 + [ctypes.c_void_p]

    def launch(lens, new_lens, table, new_table, stream):
        assert lib.copy_late_launch(lens.data_ptr(), new_lens.data_ptr(), lens.numel(), table.data_ptr(),
                                    new_table.data_ptr(), table.numel(), stream.cuda_stream) == 0
    return launch


@pytest.mark.parametrize("s,h", [(1, 16), (2, 64)])
def test_paged_decode_reads_what_an_early_releasing_kernel_writes(late, s, h):
    c = Case([700, 65, 0, 1300, 2], s, h, seed=31)
    dec = mla.PagedFP4Decoder(c.problem(), DEV)
    lens, table = torch.empty_like(c.seq), torch.empty_like(c.table)
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:3], device=DEV)
    stream = torch.cuda.Stream()
    for before in (0, 1, 64):                          # lengths and pages that were there before
        lens.fill_(before)
        table.fill_(0)
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(2):
            late(lens, c.seq, table, c.table, stream)
            dec(c.q, c.kv, table, lens, out, lse, stream=stream)
        torch.cuda.synchronize()
        c.check(out, lse)
    assert int(dec.error) == 0
