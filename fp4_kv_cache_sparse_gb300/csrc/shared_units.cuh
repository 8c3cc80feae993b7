// shared_units.cuh -- blocks of query rows over a prefix that a group of
// sequences shares (SharedParams, mla_internal.h), for the kernels that walk them.
#pragma once

#include "mla_device.cuh"
#include "mla_internal.h"
#include "mla_tensor.cuh"

namespace mla {

// The first prefix unit of group g, counted from the first of all.
__device__ __forceinline__ int prefix_unit(const SharedParams& p, int nr, int g) {
  return load_i32(p.group_start + g) * p.rows / nr + g;
}

// Prefix unit v: NR rows of a group, whichever sequences they belong to.  Numbers
// that fall between two groups, and groups without a prefix, have len 0.
struct PrefixUnit {
  int group, row0, nrows;  // row0 counts from the batch's first row
  int len;                 // tokens of the prefix
  bool bad;                // a length that cannot be
};
template <int NR>
__device__ __forceinline__ PrefixUnit prefix_unit_at(const SharedParams& p, int v, int num_groups) {
  PrefixUnit t{};
  if (num_groups == 0) return t;
  int g = 0;  // the last group whose units begin at or before v
  for (int n = num_groups; n > 1;) {
    const int half = n / 2;
    if (prefix_unit(p, NR, g + half) <= v) g += half;
    n -= half;
  }
  const int from = load_i32(p.group_start + g) * p.rows, to = load_i32(p.group_start + g + 1) * p.rows;
  const int len = load_i32(p.prefix_lens + g), k = v - prefix_unit(p, NR, g);
  t.bad = len < 0 || len > p.max_prefix_pages * kPage;
  t.group = g;
  t.row0 = from + k * NR;
  t.nrows = min(NR, to - t.row0);
  t.len = t.bad || k < 0 || t.nrows <= 0 ? 0 : len;
  return t;
}

// How many groups count: none if their starts are not in order.  For a whole CTA
// of `threads` threads; flags the latter once.
__device__ __forceinline__ int groups_in_order(const SharedParams& p, int tid, int threads, bool flags) {
  bool wrong = false;
  for (int g = tid; g <= p.num_groups; g += threads) {
    const int at = load_i32(p.group_start + g);
    wrong = wrong || at < 0 || at > p.batch || (g > 0 && at < load_i32(p.group_start + g - 1));
  }
  const bool none = __syncthreads_or(wrong);
  if (flags && tid == 0) {
    p.ws_info[static_cast<int64_t>(p.units) * 4] = none ? 0 : p.num_groups;
    if (none && p.d_error) atomicOr(p.d_error, MLA_DEVERR_BAD_METADATA);
  }
  return none ? 0 : p.num_groups;
}

}  // namespace mla
