// api.cu -- the C ABI (include/mla.h): argument validation, work planning
// and kernel launches.  No allocation, no host synchronisation.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "../../include/mla.h"
#include "mla_internal.h"

namespace mla {

// Shape checks shared by every entry point.
mla_status_t validate_problem(const mla_problem_t* p) {
  if (p == nullptr) return MLA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->seq_len_q < 1 || p->topk < 1 || p->extra_topk < 0 || p->h_q < 1) return MLA_ERR_INVALID_ARG;
  if (p->num_pages < 1) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(p->sm_scale)) return MLA_ERR_INVALID_ARG;
  // The record format decides the kernel: FP4 only as the extra cache, no bf16 cache.
  if (p->kv_format == MLA_KV_FP4_288 || p->kv_format == MLA_KV_BF16) return MLA_ERR_UNSUPPORTED;
  if (p->kv_format != MLA_KV_FP8_528) return MLA_ERR_INVALID_ARG;
  if (p->head_dim != MLA_HEAD_DIM || p->page_size != MLA_PAGE_SIZE || p->num_kv_heads != 1)
    return MLA_ERR_UNSUPPORTED;
  if (!(p->h_q == 16 || p->h_q == 32 || p->h_q == 64 || p->h_q == 128)) return MLA_ERR_UNSUPPORTED;
  if (p->extra_topk > 0) {
    if (p->extra_kv_format == MLA_KV_BF16 || p->extra_kv_format == MLA_KV_FP8_528) return MLA_ERR_UNSUPPORTED;
    if (p->extra_kv_format != MLA_KV_FP4_288) return MLA_ERR_INVALID_ARG;
    if (p->extra_num_pages < 1) return MLA_ERR_INVALID_ARG;
  }
  const int64_t nq = static_cast<int64_t>(p->batch) * p->seq_len_q;
  const int64_t T = (p->topk + 127) / 128 + (static_cast<int64_t>(p->extra_topk) + 127) / 128;
  if (nq * T >= (int64_t(1) << 31) || nq * p->h_q >= (int64_t(1) << 31)) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

// Shape part of the plan plus the workspace layout for a given part count.
Plan plan_for_parts(const mla_problem_t* p, int num_parts) {
  Plan pl{};
  pl.nh = p->h_q < 64 ? p->h_q : 64;
  pl.n_hg = p->h_q / pl.nh;
  pl.Tm = (p->topk + 127) / 128;
  pl.Te = (p->extra_topk + 127) / 128;
  pl.T = pl.Tm + pl.Te;
  const int64_t nq = static_cast<int64_t>(p->batch) * p->seq_len_q;
  pl.G = nq * pl.T;
  pl.num_parts = num_parts;
  pl.S = num_parts > 0 ? (pl.G + num_parts - 1) / num_parts : 0;
  pl.max_splits = nq + num_parts;
  pl.ws_o_bytes = static_cast<size_t>(pl.max_splits) * p->h_q * MLA_HEAD_DIM * sizeof(float);
  pl.ws_o_bytes = (pl.ws_o_bytes + 255) & ~size_t(255);
  pl.ws_bytes = pl.ws_o_bytes + static_cast<size_t>(pl.max_splits) * p->h_q * sizeof(float);
  return pl;
}

namespace {

constexpr int kMaxDevices = 64;
int g_sm_count[kMaxDevices] = {0};
std::mutex g_sm_mutex;

// A call that CUDA refused: its error is reported here and does not stay with
// the thread, where the next launch's check would take it for its own.
mla_status_t cuda_failed() {
  (void)cudaGetLastError();
  return MLA_ERR_CUDA;
}

mla_status_t device_sm_count(int* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cuda_failed();
  if (dev >= 0 && dev < kMaxDevices) {
    std::lock_guard<std::mutex> lock(g_sm_mutex);
    if (g_sm_count[dev] == 0) {
      int n = 0;
      if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return cuda_failed();
      g_sm_count[dev] = n;
    }
    *out = g_sm_count[dev];
    return MLA_OK;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return cuda_failed();
  *out = n;
  return MLA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Balanced partition: about one part per SM for each head group (a CTA
// fills an SM), never more parts than work items.
Plan make_plan(const mla_problem_t* p, int num_sms) {
  Plan pl = plan_for_parts(p, 1);
  int64_t target = num_sms / pl.n_hg;
  if (target < 1) target = 1;
  if (target > pl.G) target = pl.G;
  const int64_t S = (pl.G + target - 1) / target;
  pl = plan_for_parts(p, static_cast<int>((pl.G + S - 1) / S));
  pl.S = S;
  return pl;
}

// The 128-head cluster kernel runs 128-head problems without an extra
// cache; every other shape runs on the swap-AB kernel.
bool uses_pair_kernel(const mla_problem_t* problem) { return problem->h_q == 128 && problem->extra_topk == 0; }

int element_bytes(int32_t dtype) { return dtype == MLA_FP32 ? 4 : (dtype == MLA_BF16 || dtype == MLA_FP16 ? 2 : 0); }

constexpr float kLog2e = 1.4426950408889634f;

bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

mla_status_t validate_paged(const mla_paged_problem_t* p) {
  if (p == nullptr) return MLA_ERR_INVALID_ARG;
  if (p->batch < 1 || p->seq_len_q < 1 || p->h_q < 1 || p->max_pages < 1 || p->num_pages < 1 || p->window < 0 ||
      p->sinks < 0 || !std::isfinite(p->sm_scale * kLog2e))
    return MLA_ERR_INVALID_ARG;
  if (p->kv_format == MLA_KV_FP8_528 || p->kv_format == MLA_KV_BF16) return MLA_ERR_UNSUPPORTED;
  if (p->kv_format != MLA_KV_FP4_288) return MLA_ERR_INVALID_ARG;
  if (p->head_dim != MLA_HEAD_DIM || p->page_size != MLA_PAGE_SIZE || p->h_q > 128) return MLA_ERR_UNSUPPORTED;
  // Positions, rows and tiles are counted in 32 bits.
  const int64_t most = int64_t(1) << 31, rows = static_cast<int64_t>(p->seq_len_q) * p->h_q;
  if (static_cast<int64_t>(p->max_pages) * MLA_PAGE_SIZE >= most - 256 || rows * p->batch >= most ||
      static_cast<int64_t>(p->batch) * p->max_pages >= most || p->num_pages >= most / MLA_PAGE_SIZE)
    return MLA_ERR_UNSUPPORTED;
  const int64_t units = p->batch * ((rows + 15) / 16);
  // Tiles and a unit's own cost, rounded up to whole parts.
  if (units * ((p->max_pages + 1) / 2 + 4) >= most - (1 << 16)) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

// Where the decode kernels write the fused epilogue's FP8 records of query
// tokens that have one split.
struct RopeOut {
  uint8_t* out;
  const int32_t* positions;
  RopeFreqs freqs;
};

}  // namespace

// Validation and the decode kernel's launch, shared by the bf16 and the
// FP8 output calls.  With rope, query tokens of one split are written as FP8
// records there instead of to out (which may then be null); *pout receives
// the parameters.
mla_status_t decode_launch(const mla_problem_t* problem, const void* q, const void* kv, const int32_t* indices,
                           const void* extra_kv, const int32_t* extra_indices, const int32_t* d_sched,
                           const int32_t* d_num_splits, int32_t num_parts, void* workspace, size_t workspace_bytes,
                           uint16_t* out, float* lse, int32_t* d_error, const RopeOut* rope, mla_stream_t stream,
                           DecodeParams* pout) {
  mla_status_t st = validate_problem(problem);
  if (st != MLA_OK) return st;
  if (q == nullptr || kv == nullptr || indices == nullptr || d_sched == nullptr || d_num_splits == nullptr ||
      lse == nullptr)
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(indices) & 3u))
    return MLA_ERR_INVALID_ARG;
  if (problem->extra_topk > 0) {
    if (extra_kv == nullptr || extra_indices == nullptr || !aligned16(extra_kv) ||
        (reinterpret_cast<uintptr_t>(extra_indices) & 3u))
      return MLA_ERR_INVALID_ARG;
  }
  // The part ranges live in d_sched (checked on the device); the host needs
  // only the part count for the grid and the workspace layout.
  Plan pl = plan_for_parts(problem, num_parts);
  if (num_parts < 1 || num_parts > pl.G) return MLA_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < pl.ws_bytes) return MLA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return MLA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int nq = problem->batch * problem->seq_len_q;

  DecodeParams& p = *pout;
  p = DecodeParams{};
  p.q = static_cast<const uint16_t*>(q);
  p.kv = static_cast<const uint8_t*>(kv);
  p.idx = indices;
  p.xkv = problem->extra_topk > 0 ? static_cast<const uint8_t*>(extra_kv) : nullptr;
  p.xidx = problem->extra_topk > 0 ? extra_indices : nullptr;
  p.sched = d_sched;
  p.num_splits = d_num_splits;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.ws_o_bytes);
  p.ws_splits_cap = pl.max_splits;
  p.out = out;
  p.lse = lse;
  p.d_error = d_error;
  p.nq = nq;
  p.h_q = problem->h_q;
  p.n_hg = pl.n_hg;
  p.topk = problem->topk;
  p.xtopk = problem->extra_topk;
  p.Tm = pl.Tm;
  p.T = pl.T;
  const int64_t cap = int64_t(1) << 31;
  p.pool_tokens = problem->num_pages * MLA_PAGE_SIZE < cap ? problem->num_pages * MLA_PAGE_SIZE : cap;
  p.xpool_tokens = problem->extra_topk > 0
                       ? (problem->extra_num_pages * MLA_PAGE_SIZE < cap ? problem->extra_num_pages * MLA_PAGE_SIZE
                                                                          : cap)
                       : 0;
  p.scale_log2 = problem->sm_scale * 1.4426950408889634f;
  if (rope != nullptr) {
    p.rope_out = rope->out;
    p.positions = rope->positions;
    p.rope = rope->freqs;
  }

  const int grid = pl.num_parts * pl.n_hg;
  cudaError_t e;
  if (uses_pair_kernel(problem)) {
    // All 128 heads on the MMA's M dimension, the latent dims split over a
    // 2-CTA cluster (same part count and SM budget as two 64-head groups).
    e = launch_decode_pair(p, pl.num_parts, s);
  } else {
    switch (pl.nh) {
      case 64: e = launch_decode<64>(p, grid, s); break;
      case 32: e = launch_decode<32>(p, grid, s); break;
      default: e = launch_decode<16>(p, grid, s); break;
    }
  }
  if (e != cudaSuccess) return cuda_failed();
  return MLA_OK;
}

}  // namespace mla

using namespace mla;

extern "C" {

const char* mla_status_string(mla_status_t s) {
  switch (s) {
    case MLA_OK: return "ok";
    case MLA_ERR_INVALID_ARG: return "invalid argument";
    case MLA_ERR_UNSUPPORTED: return "unsupported problem";
    case MLA_ERR_WORKSPACE: return "workspace too small";
    case MLA_ERR_CUDA: return "CUDA error";
    case MLA_ERR_TIMEOUT: return "timeout";
  }
  return "unknown status";
}

mla_status_t mla_get_metadata(const mla_problem_t* problem, int32_t num_sms, int32_t* d_sched,
                              int32_t* d_num_splits, int32_t* num_parts_out, size_t* workspace_bytes_out,
                              mla_stream_t stream) {
  mla_status_t st = validate_problem(problem);
  if (st != MLA_OK) return st;
  if (num_parts_out == nullptr || workspace_bytes_out == nullptr || num_sms < 0) return MLA_ERR_INVALID_ARG;
  if ((d_sched == nullptr) != (d_num_splits == nullptr)) return MLA_ERR_INVALID_ARG;
  if (num_sms == 0) {
    st = device_sm_count(&num_sms);
    if (st != MLA_OK) return st;
  }
  const Plan pl = make_plan(problem, num_sms);
  *num_parts_out = pl.num_parts;
  *workspace_bytes_out = pl.ws_bytes;
  if (d_sched == nullptr) return MLA_OK;
  const int nq = problem->batch * problem->seq_len_q;
  if (launch_metadata(pl, nq, d_sched, d_num_splits, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return cuda_failed();
  return MLA_OK;
}

mla_status_t mla_sparse_decode(const mla_problem_t* problem, const void* q, const void* kv, const int32_t* indices,
                               const void* extra_kv, const int32_t* extra_indices, const int32_t* d_sched,
                               const int32_t* d_num_splits, int32_t num_parts, void* workspace,
                               size_t workspace_bytes, void* out, float* lse, int32_t* d_error,
                               mla_stream_t stream) {
  mla_status_t st = validate_problem(problem);
  if (st != MLA_OK) return st;
  if (out == nullptr || !aligned16(out)) return MLA_ERR_INVALID_ARG;
  DecodeParams p{};
  st = decode_launch(problem, q, kv, indices, extra_kv, extra_indices, d_sched, d_num_splits, num_parts, workspace,
                     workspace_bytes, static_cast<uint16_t*>(out), lse, d_error, nullptr, stream, &p);
  if (st != MLA_OK) return st;
  if (num_parts > 1) {
    // Only query tokens with more than one split have partials to merge: a
    // grid over parts visits just those (at most one per part) and is the
    // smaller grid when parts are fewer than query tokens; otherwise one warp
    // per row, the kernel skipping one-split rows.
    const int32_t* by_part = num_parts < p.nq ? d_sched : nullptr;
    if (launch_combine(d_num_splits, p.ws_o, p.ws_lse, p.out, lse, p.nq, problem->h_q, true, by_part, num_parts,
                       p.T, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
      return cuda_failed();
  }
  return MLA_OK;
}

mla_status_t mla_sparse_decode_rope_fp8(const mla_problem_t* problem, const void* q, const void* kv,
                                        const int32_t* indices, const void* extra_kv, const int32_t* extra_indices,
                                        const int32_t* d_sched, const int32_t* d_num_splits, int32_t num_parts,
                                        void* workspace, size_t workspace_bytes, const int32_t* positions,
                                        float rope_theta, void* out_fp8, float* lse, int32_t* d_error,
                                        mla_stream_t stream) {
  mla_status_t st = validate_problem(problem);
  if (st != MLA_OK) return st;
  if (out_fp8 == nullptr || positions == nullptr || (reinterpret_cast<uintptr_t>(positions) & 3u) ||
      (reinterpret_cast<uintptr_t>(out_fp8) & 3u))
    return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(rope_theta) || !(rope_theta > 1.f)) return MLA_ERR_INVALID_ARG;
  RopeOut ro{};
  ro.out = static_cast<uint8_t*>(out_fp8);
  ro.positions = positions;
  for (int j = 0; j < 32; ++j) ro.freqs.f[j] = std::pow(static_cast<double>(rope_theta), -2.0 * j / 64.0);
  // The decode kernels write the records of one-split query tokens
  // themselves; only split tokens go through the workspace to the merge.
  DecodeParams p{};
  st = decode_launch(problem, q, kv, indices, extra_kv, extra_indices, d_sched, d_num_splits, num_parts, workspace,
                     workspace_bytes, nullptr, lse, d_error, &ro, stream, &p);
  if (st != MLA_OK) return st;
  if (launch_rope_fp8(d_num_splits, p.ws_o, p.ws_lse, positions, ro.freqs, ro.out, lse, p.nq, problem->h_q, true,
                      num_parts < p.nq ? d_sched : nullptr, num_parts, p.T,
                      reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return cuda_failed();
  return MLA_OK;
}

mla_status_t mla_combine(const mla_problem_t* problem, const int32_t* d_num_splits, const float* o_partial,
                         const float* lse_partial, void* out, float* lse, mla_stream_t stream) {
  mla_status_t st = validate_problem(problem);
  if (st != MLA_OK) return st;
  if (d_num_splits == nullptr || o_partial == nullptr || lse_partial == nullptr || out == nullptr || lse == nullptr)
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(o_partial) || !aligned16(out) || (reinterpret_cast<uintptr_t>(lse_partial) & 3u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MLA_ERR_INVALID_ARG;
  const int nq = problem->batch * problem->seq_len_q;
  if (launch_combine(d_num_splits, o_partial, lse_partial, static_cast<uint16_t*>(out), lse, nq, problem->h_q,
                     false, nullptr, 0, 0, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return cuda_failed();
  return MLA_OK;
}

mla_status_t mla_dequantize(int32_t kv_format, const void* records, int64_t n, void* out, mla_stream_t stream) {
  if (kv_format != MLA_KV_FP8_528 && kv_format != MLA_KV_FP4_288) {
    return kv_format == MLA_KV_BF16 ? MLA_ERR_UNSUPPORTED : MLA_ERR_INVALID_ARG;
  }
  if (n < 0 || (n > 0 && (records == nullptr || out == nullptr))) return MLA_ERR_INVALID_ARG;
  if (n > 0 && (!aligned16(records) || !aligned16(out))) return MLA_ERR_INVALID_ARG;
  if (n * 32 >= (int64_t(1) << 40)) return MLA_ERR_UNSUPPORTED;
  if (launch_dequant(kv_format, static_cast<const uint8_t*>(records), n, static_cast<uint16_t*>(out),
                     reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return cuda_failed();
  return MLA_OK;
}

mla_status_t mla_kv_write(int32_t kv_format, const void* latents, const int32_t* slots, int64_t n, void* pool,
                          int64_t num_pages, int32_t* d_error, mla_stream_t stream) {
  if (kv_format != MLA_KV_FP8_528 && kv_format != MLA_KV_FP4_288) {
    return kv_format == MLA_KV_BF16 ? MLA_ERR_UNSUPPORTED : MLA_ERR_INVALID_ARG;
  }
  if (n < 0 || num_pages < 0) return MLA_ERR_INVALID_ARG;
  if (n == 0) return MLA_OK;
  if (latents == nullptr || slots == nullptr || pool == nullptr) return MLA_ERR_INVALID_ARG;
  if (!aligned16(latents) || !aligned16(pool) || (reinterpret_cast<uintptr_t>(slots) & 3u) != 0)
    return MLA_ERR_INVALID_ARG;
  if (n * MLA_HEAD_DIM >= (int64_t(1) << 40)) return MLA_ERR_UNSUPPORTED;
  const int64_t cap = int64_t(1) << 31;
  const int64_t pool_tokens = num_pages * MLA_PAGE_SIZE < cap ? num_pages * MLA_PAGE_SIZE : cap;
  if (launch_kv_write(kv_format, static_cast<const uint16_t*>(latents), slots, n, static_cast<uint8_t*>(pool),
                      pool_tokens, d_error, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return cuda_failed();
  return MLA_OK;
}

mla_status_t mla_page_plan(const int32_t* cached_lens, const int32_t* new_lens, int32_t batch, int32_t* block_table,
                           int32_t max_pages, int32_t* free_pages, int32_t num_pages, const int32_t* num_free,
                           int32_t* seq_lens, int32_t* num_free_out, int32_t* cu_new, int32_t* slots,
                           int32_t* positions, int32_t max_new, int32_t* d_error, mla_stream_t stream) {
  if (batch < 0 || max_pages < 1 || num_pages < 1 || max_new < 0) return MLA_ERR_INVALID_ARG;
  if (batch > kPlanMaxBatch || static_cast<int64_t>(num_pages) * MLA_PAGE_SIZE >= (int64_t(1) << 31) ||
      static_cast<int64_t>(max_pages) * MLA_PAGE_SIZE >= (int64_t(1) << 31))
    return MLA_ERR_UNSUPPORTED;
  if (free_pages == nullptr || num_free == nullptr || num_free_out == nullptr || cu_new == nullptr)
    return MLA_ERR_INVALID_ARG;
  if (batch > 0 && (cached_lens == nullptr || new_lens == nullptr || block_table == nullptr || seq_lens == nullptr))
    return MLA_ERR_INVALID_ARG;
  if (max_new > 0 && (slots == nullptr || positions == nullptr)) return MLA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(cached_lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(block_table), static_cast<const void*>(free_pages),
                        static_cast<const void*>(num_free), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(num_free_out), static_cast<const void*>(cu_new),
                        static_cast<const void*>(slots), static_cast<const void*>(positions)})
    if (!aligned_to(p, 4)) return MLA_ERR_INVALID_ARG;
  if (launch_page_plan(cached_lens, new_lens, batch, block_table, max_pages, free_pages, num_pages, num_free, seq_lens,
                       num_free_out, cu_new, slots, positions, max_new, d_error,
                       reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return cuda_failed();
  return MLA_OK;
}

mla_status_t mla_rope_table_from_freqs(mla_rope_table_t* table, int32_t rope_dim, int32_t layout, const double* freqs,
                                       double factor) {
  if (table == nullptr || freqs == nullptr || rope_dim < 2 || (rope_dim & 1) != 0) return MLA_ERR_INVALID_ARG;
  if (layout != MLA_ROPE_INTERLEAVED && layout != MLA_ROPE_HALF) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(factor) || !std::isfinite(static_cast<float>(factor))) return MLA_ERR_INVALID_ARG;
  if (rope_dim > MLA_ROPE_MAX_DIM) return MLA_ERR_UNSUPPORTED;
  const double pi = 3.14159265358979323846;
  for (int j = 0; j < rope_dim / 2; ++j)
    if (!(std::fabs(freqs[j]) <= pi)) return MLA_ERR_INVALID_ARG;
  table->rope_dim = rope_dim;
  table->layout = layout;
  table->factor = static_cast<float>(factor);
  for (int j = 0; j < MLA_ROPE_MAX_DIM / 2; ++j) {
    // Turns in [-1/2, 1/2] as a 64-bit fraction; half a turn wraps to -2^63,
    // the same phase.  |turns| * 2^64 < 2^63 is representable, else +-2^63.
    const double turns = j < rope_dim / 2 ? freqs[j] / (2.0 * pi) : 0.0;
    const double scaled = std::nearbyint(std::ldexp(turns, 64));
    table->step[j] = std::fabs(scaled) >= 9223372036854775808.0
                         ? uint64_t(1) << 63
                         : static_cast<uint64_t>(static_cast<int64_t>(scaled));
  }
  return MLA_OK;
}

mla_status_t mla_rope_table(mla_rope_table_t* table, int32_t rope_dim, int32_t layout, double theta, int32_t scaling,
                            double scale, double original_len, double beta_fast, double beta_slow, double factor) {
  if (rope_dim < 2 || (rope_dim & 1) != 0) return MLA_ERR_INVALID_ARG;
  if (rope_dim > MLA_ROPE_MAX_DIM) return MLA_ERR_UNSUPPORTED;
  if (!std::isfinite(theta) || !(theta > 1.0)) return MLA_ERR_INVALID_ARG;
  if (scaling != MLA_ROPE_PLAIN && scaling != MLA_ROPE_LINEAR && scaling != MLA_ROPE_YARN) return MLA_ERR_INVALID_ARG;
  if (scaling != MLA_ROPE_PLAIN && (!std::isfinite(scale) || !(scale >= 1.0))) return MLA_ERR_INVALID_ARG;
  double lo = 0.0, hi = 0.0;
  if (scaling == MLA_ROPE_YARN) {
    if (!std::isfinite(original_len) || !(original_len > 0.0) || !std::isfinite(beta_fast) || !(beta_slow > 0.0) ||
        !(beta_fast >= beta_slow))
      return MLA_ERR_INVALID_ARG;
    const double two_pi = 2.0 * 3.14159265358979323846;
    const auto dim_of = [&](double turns) {
      return rope_dim * std::log(original_len / (turns * two_pi)) / (2.0 * std::log(theta));
    };
    lo = std::fmax(std::floor(dim_of(beta_fast)), 0.0);
    hi = std::fmin(std::ceil(dim_of(beta_slow)), rope_dim - 1.0);
  }
  double f[MLA_ROPE_MAX_DIM / 2];
  for (int j = 0; j < rope_dim / 2; ++j) {
    f[j] = std::pow(theta, -2.0 * j / rope_dim);
    if (scaling == MLA_ROPE_LINEAR) f[j] /= scale;
    if (scaling == MLA_ROPE_YARN) {
      const double g = std::fmin(std::fmax((j - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      f[j] = f[j] * (1.0 - g) + f[j] / scale * g;
    }
  }
  return mla_rope_table_from_freqs(table, rope_dim, layout, f, factor);
}

mla_status_t mla_rope(int32_t dtype, const void* x, int64_t x_row_stride, int64_t x_head_stride, void* y,
                      int64_t y_row_stride, int64_t y_head_stride, int64_t n, int32_t heads, int32_t head_dim,
                      int32_t offset, const int32_t* positions, const mla_rope_table_t* table, int32_t conjugate,
                      mla_stream_t stream) {
  const int bytes = element_bytes(dtype);
  if (bytes == 0 || table == nullptr || n < 0 || heads < 1 || head_dim < 1 || offset < 0) return MLA_ERR_INVALID_ARG;
  if (table->rope_dim < 2 || table->rope_dim > MLA_ROPE_MAX_DIM || (table->rope_dim & 1) != 0 ||
      (table->layout != MLA_ROPE_INTERLEAVED && table->layout != MLA_ROPE_HALF) || !std::isfinite(table->factor))
    return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(offset) + table->rope_dim > head_dim) return MLA_ERR_INVALID_ARG;
  if (x_row_stride < 0 || x_head_stride < 0 || y_row_stride < 0 || y_head_stride < 0) return MLA_ERR_INVALID_ARG;
  if (n == 0) return MLA_OK;
  if (x == nullptr || y == nullptr || positions == nullptr || !aligned_to(x, bytes) || !aligned_to(y, bytes) ||
      !aligned_to(positions, 4))
    return MLA_ERR_INVALID_ARG;
  if (x == y && (x_row_stride != y_row_stride || x_head_stride != y_head_stride)) return MLA_ERR_INVALID_ARG;
  // The heads of y must not overlap one another: one of the two strides is
  // the outer one and clears everything inside it.
  const bool rows_outer = n == 1 || y_row_stride >= y_head_stride * (heads - 1) + head_dim;
  const bool heads_outer = heads == 1 || y_head_stride >= y_row_stride * (n - 1) + head_dim;
  if (!((rows_outer && (heads == 1 || y_head_stride >= head_dim)) ||
        (heads_outer && (n == 1 || y_row_stride >= head_dim))))
    return MLA_ERR_INVALID_ARG;
  if (n >= (int64_t(1) << 31) || head_dim > (1 << 20) || heads > (1 << 20)) return MLA_ERR_UNSUPPORTED;
  const RopeParams p{x, y, x_row_stride, x_head_stride, y_row_stride, y_head_stride, n, heads, head_dim, offset,
                     positions, conjugate != 0};
  if (launch_rope(dtype, p, *table, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return cuda_failed();
  return MLA_OK;
}

mla_status_t mla_rms_norm_fp8(int32_t dtype, const void* x, int64_t x_stride, const void* residual,
                              int64_t residual_stride, const void* weight, float eps, void* residual_out,
                              int64_t residual_out_stride, void* codes, int64_t codes_stride, void* scales,
                              int64_t scales_stride, int64_t n, int32_t dim, int32_t* d_error, mla_stream_t stream) {
  const int bytes = element_bytes(dtype);
  if (bytes == 0 || n < 0 || dim < 1 || !std::isfinite(eps) || eps < 0.f) return MLA_ERR_INVALID_ARG;
  if (dim % 32 != 0 || dim > 16384 || n >= (int64_t(1) << 31)) return MLA_ERR_UNSUPPORTED;
  if (n == 0) return MLA_OK;
  if (x == nullptr || weight == nullptr || codes == nullptr || scales == nullptr) return MLA_ERR_INVALID_ARG;
  const auto rows_ok = [&](const void* p, int64_t stride, bool written) {
    return aligned16(p) && stride >= 0 && (stride * bytes) % 16 == 0 && (!written || n == 1 || stride >= dim);
  };
  if (!rows_ok(x, x_stride, false) || !aligned16(weight)) return MLA_ERR_INVALID_ARG;
  if (residual != nullptr && !rows_ok(residual, residual_stride, false)) return MLA_ERR_INVALID_ARG;
  if (residual_out != nullptr && !rows_ok(residual_out, residual_out_stride, true)) return MLA_ERR_INVALID_ARG;
  if (!aligned_to(codes, 8) || codes_stride % 8 != 0 || (n > 1 && (codes_stride < dim || scales_stride < dim / 32)))
    return MLA_ERR_INVALID_ARG;
  NormParams p{};
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.residual_out = residual_out;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  p.x_row = x_stride;
  p.residual_row = residual_stride;
  p.residual_out_row = residual_out_stride;
  p.codes_row = codes_stride;
  p.scales_row = scales_stride;
  p.n = n;
  p.dim = dim;
  p.eps = eps;
  p.d_error = d_error;
  if (launch_rms_norm_fp8(dtype, p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return cuda_failed();
  return MLA_OK;
}

mla_status_t mla_paged_decode_plan(const mla_paged_problem_t* problem, int32_t num_sms, int32_t* num_parts_out,
                                   size_t* workspace_bytes_out) {
  mla_status_t st = validate_paged(problem);
  if (st != MLA_OK) return st;
  if (num_parts_out == nullptr || workspace_bytes_out == nullptr || num_sms < 0 || num_sms > (1 << 16))
    return MLA_ERR_INVALID_ARG;
  if (num_sms == 0) {
    st = device_sm_count(&num_sms);
    if (st != MLA_OK) return st;
  }
  const PagedPlan pl = paged_plan(problem, num_sms);
  *num_parts_out = pl.num_parts;
  *workspace_bytes_out = pl.ws_bytes;
  return MLA_OK;
}

mla_status_t mla_paged_decode_fp4(const mla_paged_problem_t* problem, const void* q, const void* kv,
                                  const int32_t* block_table, const int32_t* seq_lens, int32_t num_parts,
                                  void* workspace, size_t workspace_bytes, void* out, float* lse, int32_t* d_error,
                                  mla_stream_t stream) {
  const mla_status_t st = validate_paged(problem);
  if (st != MLA_OK) return st;
  if (q == nullptr || kv == nullptr || block_table == nullptr || seq_lens == nullptr || out == nullptr ||
      lse == nullptr)
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv) || !aligned16(out) || !aligned_to(block_table, 4) || !aligned_to(seq_lens, 4) ||
      !aligned_to(lse, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_parts < 1 || num_parts > (1 << 16)) return MLA_ERR_INVALID_ARG;
  const PagedPlan pl = paged_plan(problem, num_parts);
  if (workspace == nullptr || workspace_bytes < pl.ws_bytes) return MLA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return MLA_ERR_INVALID_ARG;
  PagedParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.kv = static_cast<const uint8_t*>(kv);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.ws_o_bytes);
  p.ws_info = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + pl.ws_o_bytes + pl.ws_lse_bytes);
  p.d_error = d_error;
  p.batch = problem->batch;
  p.s = problem->seq_len_q;
  p.h = problem->h_q;
  p.rows = problem->seq_len_q * problem->h_q;
  p.max_pages = problem->max_pages;
  p.window = problem->window;
  p.sinks = problem->sinks;
  p.num_pages = problem->num_pages;
  p.scale_log2 = problem->sm_scale * kLog2e;
  if (launch_paged_decode(p, pl, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return cuda_failed();
  return MLA_OK;
}

}  // extern "C"
