// mla_internal.h -- host/device interface between the C-ABI layer and the
// kernels of the library (not installed, not part of the ABI).
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/mla.h"

namespace mla {

// Everything the decode kernel reads, resolved by the host layer.
// Output-side rotary frequencies of the fused epilogue: freqs[j] =
// theta^(-2j/64) for the pair (448 + 2j, 449 + 2j).
struct RopeFreqs {
  double f[32];
};

struct DecodeParams {
  const uint16_t* q;        // bf16 [nq][h_q][512]
  const uint8_t* kv;        // FP8 records
  const int32_t* idx;       // [nq][topk]
  const uint8_t* xkv;       // FP4 records (extra cache) or null
  const int32_t* xidx;      // [nq][xtopk] or null
  const int32_t* sched;     // [num_parts][8]
  const int32_t* num_splits;  // [nq + 1]
  float* ws_o;              // [ws_splits_cap][h_q][512]
  float* ws_lse;            // [ws_splits_cap][h_q]
  int64_t ws_splits_cap;
  uint16_t* out;            // bf16 [nq][h_q][512]
  float* lse;               // [nq][h_q]
  int32_t* d_error;         // nullable
  int nq, h_q, n_hg, topk, xtopk, Tm, T;
  int64_t pool_tokens, xpool_tokens;
  float scale_log2;         // sm_scale * log2(e)
  // Fused output epilogue written by the decode kernel itself for query
  // tokens of one split: null, or [nq][h_q][528] FP8 records after the
  // conjugate rotary embedding at positions[qidx].
  uint8_t* rope_out;
  const int32_t* positions;
  RopeFreqs rope;
};

// Work plan derived from the problem shape and the SM count.
struct Plan {
  int nh;          // heads per CTA (16, 32 or 64)
  int n_hg;        // head groups = h_q / nh
  int Tm, Te, T;   // tiles per query token: main, extra, total
  int64_t G;       // total (query token, tile) items
  int64_t S;       // items per part
  int num_parts;
  int64_t max_splits;
  size_t ws_o_bytes, ws_bytes;
};

// Shape checks shared by every entry point (MLA_OK or the status to return).
mla_status_t validate_problem(const mla_problem_t* p);

// Shape part of the plan plus the workspace layout (ws_bytes) for a given
// part count; the one definition of the workspace size.
Plan plan_for_parts(const mla_problem_t* p, int num_parts);

template <int NH>
cudaError_t launch_decode(const DecodeParams& p, int grid, cudaStream_t stream);
int decode_smem_bytes(int nh);

// 128 heads, FP8 main cache only: a 2-CTA cluster per part splitting the latent dims.
cudaError_t launch_decode_pair(const DecodeParams& p, int num_parts, cudaStream_t stream);
int decode_pair_smem_bytes();

cudaError_t launch_metadata(const Plan& plan, int nq, int32_t* d_sched, int32_t* d_num_splits, cudaStream_t stream);

// Merge of split partials.  With sched (the decode's part schedule, T
// tiles per query token) only the rows of query tokens that have several
// splits are visited, every other row having been written by the decode
// kernel; without it every row is (skip_single then skips one-split rows).
cudaError_t launch_combine(const int32_t* d_num_splits, const float* o_part, const float* lse_part, uint16_t* out,
                           float* lse, int nq, int h_q, bool skip_single, const int32_t* sched, int num_parts, int T,
                           cudaStream_t stream);

// Merge of each query token's split partials (with skip_single, only tokens
// of more than one split), conjugate rotary embedding of dims 448..511 and
// the cast to 528-byte FP8 records.
cudaError_t launch_rope_fp8(const int32_t* d_num_splits, const float* o_part, const float* lse_part,
                            const int32_t* positions, const RopeFreqs& freqs, uint8_t* out, float* lse, int nq,
                            int h_q, bool skip_single, const int32_t* sched, int num_parts, int T,
                            cudaStream_t stream);

cudaError_t launch_dequant(int kv_format, const uint8_t* records, int64_t n, uint16_t* out, cudaStream_t stream);

cudaError_t launch_kv_write(int kv_format, const uint16_t* latents, const int32_t* slots, int64_t n, uint8_t* pool,
                            int64_t pool_tokens, int32_t* d_error, cudaStream_t stream);

// Requests of one page plan: their prefix sums live in shared memory.
constexpr int kPlanMaxBatch = 8192;
cudaError_t launch_page_plan(const int32_t* cached_lens, const int32_t* new_lens, int batch, int32_t* block_table,
                             int max_pages, int32_t* free_pages, int num_pages, const int32_t* num_free,
                             int32_t* seq_lens, int32_t* num_free_out, int32_t* cu_new, int32_t* slots,
                             int32_t* positions, int max_new, int32_t* d_error, cudaStream_t stream);

// Rotary positions; strides in elements, checked by the caller.
struct RopeParams {
  const void* x;
  void* y;
  int64_t x_row, x_head, y_row, y_head, n;
  int heads, head_dim, offset;
  const int32_t* positions;
  bool conjugate;
};
cudaError_t launch_rope(int dtype, const RopeParams& p, const mla_rope_table_t& table, cudaStream_t stream);

// New tokens' latents, turned on the way into their records; row stride in elements.
struct AppendParams {
  const void* latents;
  const int32_t* positions;  // null when nothing turns
  const int32_t* slots;
  uint8_t* pool;
  int64_t row_stride, n, pool_tokens;
  int offset;
  int32_t* d_error;          // nullable
};
cudaError_t launch_kv_append(int kv_format, int dtype, const AppendParams& p, const mla_rope_table_t& table,
                             cudaStream_t stream);

cudaError_t launch_page_means(const uint8_t* pool, int64_t pool_tokens, const int32_t* slots, int64_t n, uint8_t* means,
                              int32_t* d_error, cudaStream_t stream);

// RMS norm with the residual's addition to FP8 blocks; strides in elements.
struct NormParams {
  const void* x;
  const void* residual;  // nullable
  const void* weight;
  void* residual_out;    // nullable
  uint8_t* codes;
  uint8_t* scales;
  int64_t x_row, residual_row, residual_out_row, codes_row, scales_row, n;
  int dim;
  float eps;
  int32_t* d_error;      // nullable
};
cudaError_t launch_rms_norm_fp8(int dtype, const NormParams& p, cudaStream_t stream);

// Attention over a paged FP4 cache.
struct PagedParams {
  const uint16_t* q;           // bf16 [batch * rows][512]
  const uint8_t* kv;           // FP4 records
  const int32_t* block_table;  // [batch][max_pages]
  const int32_t* seq_lens;     // [batch]
  uint16_t* out;               // bf16 [batch * rows][512]
  float* lse;                  // [batch * rows]
  float* ws_o;
  float* ws_lse;
  int32_t* ws_info;
  int32_t* d_error;            // nullable
  int batch, s, h, rows;       // rows = s * h query rows of a sequence
  int max_pages, window, sinks;
  bool info_by_unit;           // ws_info has an entry for each unit, not for each part
  int64_t num_pages;
  float scale_log2;            // sm_scale * log2(e)
};
struct PagedPlan {
  int nr;          // query rows a CTA works on: 16, 32 or 64
  int groups;      // row groups of a sequence
  int num_parts;
  int units;       // shared prefixes: numbers of units
  bool pair;       // shared prefixes by pairs of SMs: a unit is 128 rows, a part is a pair
  size_t ws_o_bytes, ws_lse_bytes, ws_bytes;
};
PagedPlan paged_plan(const mla_paged_problem_t* p, int num_parts);
cudaError_t launch_paged_decode(const PagedParams& p, const PagedPlan& plan, cudaStream_t stream);

// The same for sequences in groups that share a prefix: partials of all units,
// then their merge, which writes the outputs.
struct SharedParams : PagedParams {
  // Units 0 .. batch * groups - 1 are those of the sequences'
  // own tokens; those of group g's rows over its prefix begin at batch * groups +
  // floor(group_start[g] * rows / nr) + g.  ws_info has an entry for each unit
  // and, behind them, the number of groups that count (0: they were not in order).
  const int32_t* group_start;  // [num_groups + 1]
  const int32_t* prefix_table; // [num_groups][max_prefix_pages]
  const int32_t* prefix_lens;  // [num_groups]
  int num_groups, max_prefix_pages, units;
};
PagedPlan shared_plan(const mla_paged_shared_problem_t* p, int num_parts);
cudaError_t launch_shared_decode(const SharedParams& p, const PagedPlan& plan, cudaStream_t stream);
cudaError_t launch_shared_merge(const SharedParams& p, const PagedPlan& plan, cudaStream_t stream);
cudaError_t launch_shared_pair(const SharedParams& p, const PagedPlan& plan, cudaStream_t stream);

// Which pages each query token attends to: scores of the pages' means, and the
// best of them as block tables and lengths of one-token sequences.
struct SelectParams {
  const uint16_t* q;           // bf16 [batch * s * h][512]
  const uint8_t* means;        // [num_pages][MLA_MEAN_BYTES]
  const int32_t* block_table;  // [batch][max_pages]
  const int32_t* seq_lens;     // [batch]
  float* scores;               // [batch * s][max_pages]
  int32_t* sel_table;          // [batch * s][top]: page ids
  int32_t* sel_lens;           // [batch * s]
  int32_t* selected;           // [batch * s][top]: pages of the sequence, nullable
  int32_t* d_error;            // nullable
  int batch, s, h, max_pages, top, sinks, local, num_parts;
  int64_t num_pages;
  float sign;                  // that of the softmax scale
};
cudaError_t launch_page_select(const SelectParams& p, cudaStream_t stream);

// cuTensorMapEncodeTiled from the driver, looked up once (thread-safe
// static initialization); nullptr if the driver does not offer it.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn tensor_map_encoder() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeTiledFn>(f) : EncodeTiledFn{nullptr};
  }();
  return fn;
}

// A kernel's dynamic shared memory limit, set once per device: the attribute
// belongs to the current device's context, so bit d of `done` records device
// d (devices past 63 set it on every call).
inline cudaError_t max_dynamic_smem_once(std::atomic<uint64_t>& done, const void* kernel, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit != 0) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

}  // namespace mla
