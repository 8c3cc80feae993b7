"""The waits of the paged decode kernel, run out without a GPU fault: a whole
warp's bounded wait gives up after its limit, flags MLA_DEVERR_TIMEOUT and
lets the other warps of the block go on at once; the wait before a block's end
gives up by itself, heeds no other warp's giving up, and returns as soon as
what it waits for has landed.

The kernels here are test-only: they are compiled from this file against the
library's own helpers (mla_device.cuh) with limits of some milliseconds."""
import ctypes
import subprocess

import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla
from fp4_kv_cache_sparse_gb300 import build as mla_build

pytestmark = pytest.mark.gpu

SRC = r"""
#include <cstdint>
#include "mla_device.cuh"

// times[w]: what warp w waited; flags[0]: the abort flag at the end.
// Warp 0 waits on a barrier that nothing arrives on; so does warp 1, with a limit a thousand times longer; warp 2
// waits on one that lane 0 of warp 3 arrives on.
__global__ void warp_waits(unsigned long long* times, int32_t* flags, int32_t* err, unsigned long long limit_ns) {
  __shared__ alignas(8) uint64_t bar[2];
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mla::mbar_init(&bar[0], 1);
    mla::mbar_init(&bar[1], 1);
    abort_flag = 0;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  const uint64_t t0 = mla::global_timer_ns();
  if (warp == 0) mla::mbar_wait_warp(&bar[0], 0, &abort_flag, err, limit_ns);
  if (warp == 1) mla::mbar_wait_warp(&bar[0], 0, &abort_flag, err, 1000 * limit_ns);
  if (warp == 2) mla::mbar_wait_warp(&bar[1], 0, &abort_flag, err, limit_ns);
  if (warp == 3 && (threadIdx.x & 31) == 0) mla::mbar_arrive(&bar[1]);
  if ((threadIdx.x & 31) == 0) times[warp] = mla::global_timer_ns() - t0;
  __syncthreads();
  if (threadIdx.x == 0) flags[0] = abort_flag;
}

// Waits before the end: for a copy that lands (kind 0), for nothing (kind 1).
__global__ void drains(int kind, const int4* src, int4* dst, unsigned long long* times, int32_t* err,
                       unsigned long long limit_ns) {
  __shared__ alignas(128) int4 buf[64];
  __shared__ alignas(8) uint64_t bar;
  if (threadIdx.x == 0) {
    mla::mbar_init(&bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (kind == 0) {
      asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(
                       mla::smem_u32(&bar)),
                   "r"(1024)
                   : "memory");
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                       mla::smem_u32(buf)),
                   "l"(src), "r"(1024), "r"(mla::smem_u32(&bar))
                   : "memory");
    }
  }
  __syncthreads();
  const uint64_t t0 = mla::global_timer_ns();
  mla::mbar_drain(&bar, 0, err, limit_ns);
  if (threadIdx.x == 0) times[0] = mla::global_timer_ns() - t0;
  if (kind == 0) dst[threadIdx.x] = buf[threadIdx.x];
}

extern "C" int warp_waits_launch(unsigned long long* times, int32_t* flags, int32_t* err, unsigned long long limit_ns) {
  warp_waits<<<1, 128>>>(times, flags, err, limit_ns);
  return static_cast<int>(cudaDeviceSynchronize());
}
extern "C" int drains_launch(int kind, const void* src, void* dst, unsigned long long* times, int32_t* err,
                             unsigned long long limit_ns) {
  drains<<<1, 64>>>(kind, static_cast<const int4*>(src), static_cast<int4*>(dst), times, err, limit_ns);
  return static_cast<int>(cudaDeviceSynchronize());
}
"""


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    d = tmp_path_factory.mktemp("waits")
    src, so = d / "waits.cu", d / "libwaits.so"
    src.write_text(SRC)
    subprocess.check_call([mla_build.nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17",
                           "-shared", "-Xcompiler", "-fPIC", "-I", mla_build.CSRC, "-o", str(so), str(src)])
    lib = ctypes.CDLL(str(so))
    p, n = ctypes.c_void_p, ctypes.c_ulonglong
    lib.warp_waits_launch.argtypes = [p, p, p, n]
    lib.drains_launch.argtypes = [ctypes.c_int, p, p, p, p, n]
    return lib


def cuda(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def test_a_warp_that_gives_up_flags_it_and_frees_the_others(waits):
    times, flags, err = cuda(4, dtype=torch.int64), cuda(1, dtype=torch.int32), cuda(1, dtype=torch.int32)
    assert waits.warp_waits_launch(times.data_ptr(), flags.data_ptr(), err.data_ptr(), 2_000_000) == 0
    t = times.tolist()
    assert int(err) == mla.DEVERR_TIMEOUT and int(flags) == 1
    assert 2_000_000 <= t[0] < 500_000_000
    assert t[1] < 500_000_000                         # not its own two seconds
    assert t[2] < 2_000_000                           # its barrier was arrived on


@pytest.mark.parametrize("kind", [0, 1])
def test_the_wait_before_the_end(waits, kind):
    src = torch.arange(256, dtype=torch.int32, device="cuda")
    dst, times, err = torch.zeros_like(src), cuda(1, dtype=torch.int64), cuda(1, dtype=torch.int32)
    assert waits.drains_launch(kind, src.data_ptr(), dst.data_ptr(), times.data_ptr(), err.data_ptr(), 5_000_000) == 0
    if kind == 0:
        assert int(err) == 0 and torch.equal(src, dst) and int(times) < 5_000_000
    else:
        assert int(err) == mla.DEVERR_TIMEOUT and 5_000_000 <= int(times) < 500_000_000
