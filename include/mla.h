/*
 * mla.h -- C ABI of the GB300 (sm_103a) token-sparse MLA decode library.
 *
 * The sparse decode, in three calls: the tile-scheduler metadata (computed
 * once before a decode loop), the decode step itself, and the merge of
 * split-KV partial results.  Beside it the operators that a serving step over
 * a paged FP4 cache needs: the cache writer, page and slot planning, rotary
 * positions, the residual norm with its FP8 cast, and attention over the pages.
 * Sources for what the sparse decode computes (page title, section):
 *   "flops/flashmla-decode-fp8-fp4-kv" -- "Arithmetic intensity" (the 528-byte
 *       FP8 and 288-byte FP4 token records, scales inlined in each record) and
 *       "Workarounds" (indices tensor (batch, seq_len_q, topk) of
 *       page_block*64+offset entries; metadata computed once before the decode
 *       loop; split decoding with num_splits);
 *   "deepseek-ai/FlashMLA" -- "How to use it" (metadata first, then one decode
 *       call per generation step; output plus log-sum-exp) and "Key technical
 *       details" (data followed by per-token scales; -1 entries ignored);
 *   "flops/attn-mla-kernel-support-matrix" -- "notes" (decode takes FP8 or
 *       FP4 caches only; bf16 KV is not supported).
 *
 * Conventions for every call:
 *   - Pointers named d_* and every tensor argument are DEVICE pointers; the
 *     problem descriptor and the *_out arguments are HOST pointers.
 *   - All tensors are dense, row-major, contiguous (but where a call takes
 *     strides), owned by the caller; the library allocates nothing and keeps no
 *     state between calls except a per-device cache of the SM count.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and returns without synchronising the host.
 *   - The return status reports argument validation and launch errors only;
 *     on any status other than MLA_OK nothing was enqueued.  Problems found
 *     in device data are reported through the optional device error word.
 */
#ifndef MLA_H
#define MLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st* mla_stream_t; /* same type as cudaStream_t */

typedef enum {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size, inconsistent metadata size */
  MLA_ERR_UNSUPPORTED = 2,   /* a legal problem outside what the kernels implement */
  MLA_ERR_WORKSPACE = 3,     /* workspace smaller than the plan or metadata call reported */
  MLA_ERR_CUDA = 4,          /* a CUDA runtime call or a launch failed */
  MLA_ERR_TIMEOUT = 5        /* reserved for host-side waits; device timeouts use MLA_DEVERR_TIMEOUT */
} mla_status_t;

/* KV cache record formats ("Arithmetic intensity" of the FP8/FP4 KV page). */
enum {
  MLA_KV_NONE = 0,
  MLA_KV_FP8_528 = 1,  /* 512 B e4m3 (dim order) + 16 B e8m0 scales, one per 32 dims */
  MLA_KV_FP4_288 = 2,  /* 256 B e2m1 (even dim in the low nibble) + 32 B e4m3 scales, one per 16 dims */
  MLA_KV_BF16 = 3      /* named only to be rejected: decode does not take a bf16 cache */
};

/* Bits OR-ed into the optional device error word. */
enum {
  MLA_DEVERR_BAD_INDEX = 1,     /* an index was < -1 or >= num_pages*64; that entry was skipped */
  MLA_DEVERR_TIMEOUT = 2,       /* a bounded on-chip wait gave up; outputs are undefined */
  MLA_DEVERR_BAD_METADATA = 4,  /* scheduler metadata inconsistent with the problem; work skipped */
  MLA_DEVERR_NO_ROOM = 8,       /* page plan: not enough free pages, or more new tokens than slots */
  MLA_DEVERR_BAD_LENGTH = 16    /* a request length is negative or past its block table row */
};

#define MLA_HEAD_DIM 512
#define MLA_PAGE_SIZE 64
#define MLA_SCHED_INTS 8   /* int32 words per scheduler entry */

/* Problem descriptor (host memory). */
typedef struct {
  int32_t batch;           /* b >= 1 */
  int32_t seq_len_q;       /* s >= 1, query tokens per sequence (e.g. 2 for speculative decode) */
  int32_t h_q;             /* query heads: 16, 32, 64 or 128 */
  int32_t head_dim;        /* must be 512 (the shared latent width) */
  int32_t num_kv_heads;    /* must be 1: one latent vector per token serves every head as K and V */
  int32_t topk;            /* main indices per query token, >= 1 */
  int32_t extra_topk;      /* extra-cache indices per query token; 0 = no extra cache */
  int64_t num_pages;       /* pages in the main pool (bounds check of indices) */
  int64_t extra_num_pages; /* pages in the extra pool */
  int32_t page_size;       /* must be 64 */
  int32_t kv_format;       /* must be MLA_KV_FP8_528 */
  int32_t extra_kv_format; /* MLA_KV_FP4_288 when extra_topk > 0, else MLA_KV_NONE */
  float sm_scale;          /* softmax scale applied to q.k, e.g. 1/sqrt(512) */
} mla_problem_t;

/*
 * Tile-scheduler metadata, computed once before a decode loop
 * ("Workarounds": "Tile-scheduler metadata computed once before the decode
 * loop rather than per step"; "How to use it", step 3).
 *
 * Work is the list of (query token, tile) pairs, a tile being up to 128
 * consecutive index slots of one query token (main slots first, then extra
 * slots).  The list is cut into num_parts contiguous, balanced parts, one per
 * CTA group; a query token whose tiles fall into several parts is decoded as
 * several splits that are merged afterwards ("Split decoding with
 * num_splits").  The partition depends only on the problem shape and the SM
 * count, never on index values, so one result serves every step.
 *
 *   num_sms              SMs to plan for; 0 = query the current device.
 *   d_sched              device int32[num_parts][MLA_SCHED_INTS], written.
 *   d_num_splits         device int32[batch*seq_len_q + 1], written: the
 *                        exclusive prefix of per-query split counts.
 *   num_parts_out        host, required: number of parts.
 *   workspace_bytes_out  host, required: bytes of device workspace that
 *                        mla_sparse_decode needs for split partials.
 * Query mode: with d_sched == NULL and d_num_splits == NULL only the two
 * host outputs are filled and nothing is enqueued.
 */
mla_status_t mla_get_metadata(const mla_problem_t* problem, int32_t num_sms,
                              int32_t* d_sched, int32_t* d_num_splits,
                              int32_t* num_parts_out, size_t* workspace_bytes_out,
                              mla_stream_t stream);

/*
 * One sparse decode step ("How to use it", step 3; "Arithmetic intensity";
 * "Workarounds").  For every query token (b, s) and head h, over the tokens
 * T named by the valid entries of indices[b][s][:] (main cache) and
 * extra_indices[b][s][:] (extra cache), each token t contributing its decoded
 * 512-dim latent k_t as both key and value:
 *     x_t = sm_scale * <q[b,s,h,:], k_t>
 *     lse[b,s,h] = ln sum_{t in T} exp(x_t)
 *     out[b,s,h,:] = sum_{t in T} exp(x_t - lse) * k_t      (rounded to bf16)
 * one softmax over main and extra tokens together.  With no valid token the
 * output is +0 and lse is -inf.
 *
 *   q              bf16 [batch][seq_len_q][h_q][512], 16-byte aligned.
 *   kv             uint8 [num_pages][64][528] FP8 records, 16-byte aligned.
 *   indices        int32 [batch][seq_len_q][topk]; entry = page*64 + offset,
 *                  -1 = skip.  Entries < -1 or >= num_pages*64 are skipped
 *                  and flagged (MLA_DEVERR_BAD_INDEX).
 *   extra_kv       uint8 [extra_num_pages][64][288] FP4 records, or NULL.
 *   extra_indices  int32 [batch][seq_len_q][extra_topk], or NULL.
 *   d_sched, d_num_splits, num_parts   from mla_get_metadata for this problem
 *                  (same shape fields and SM count).
 *   workspace      device scratch of at least workspace_bytes (the value
 *                  mla_get_metadata reported); contents need no initialisation.
 *   out            bf16 [batch][seq_len_q][h_q][512].
 *   lse            float [batch][seq_len_q][h_q], natural logarithm.
 *   d_error        device int32 or NULL; error bits are OR-ed into it (the
 *                  caller clears it).
 * Rejections: a main cache that is not MLA_KV_FP8_528 (an FP4 cache is valid
 * only as the extra cache, a bf16 cache not at all), head_dim != 512,
 * page_size != 64, num_kv_heads != 1, unsupported h_q -> MLA_ERR_UNSUPPORTED.
 * Split partials are merged by an internal launch of the combine kernel on
 * the same stream.  Calls that share a workspace must not overlap.
 * out and workspace must be 16-byte aligned (MLA_ERR_INVALID_ARG otherwise).
 * Alignment beyond the minimum: with q 32-byte aligned (any allocator's
 * default), the 128-head kernel loads the query rows in 32-byte pieces; at
 * 16 bytes it uses 16-byte pieces, with identical results.
 */
mla_status_t mla_sparse_decode(const mla_problem_t* problem,
                               const void* q, const void* kv, const int32_t* indices,
                               const void* extra_kv, const int32_t* extra_indices,
                               const int32_t* d_sched, const int32_t* d_num_splits, int32_t num_parts,
                               void* workspace, size_t workspace_bytes,
                               void* out, float* lse, int32_t* d_error,
                               mla_stream_t stream);

/*
 * The decode step with the fused output epilogue ("deepseek-ai/FlashMLA",
 * "What it is": the conjugate RoPE on the output side and the final cast to
 * FP8, outputs ready for a downstream FP8 einsum; "flops/attn-mla-kernel-
 * support-matrix", "notes": qk_rope_head_dim = 64).  Same inputs and LSE as
 * mla_sparse_decode; instead of the bf16 output, each (query token, head)
 * row is
 *   1. the attention output o (fp32, before any rounding),
 *   2. turned on its rotary part -- dims 448..511 as 32 interleaved pairs
 *      (448 + 2j, 449 + 2j) -- by the conjugate rotation: pair j by
 *      -pos * rope_theta^(-2j/64), (a, b) -> (a cos + b sin, b cos - a sin),
 *      pos = positions[b][s],
 *   3. cast to a 528-byte FP8 record in the cache's own format (512 E4M3FN
 *      bytes in dim order, then one e8m0 scale per 32 dims, the writer's
 *      rule: the least power of two 2^e with block amax * 2^-e <= 448, each
 *      value rounded to nearest even).
 *   positions   int32 [batch][seq_len_q] (device): each query token's position.
 *   rope_theta  the rotary base (> 1), e.g. 10000.
 *   out_fp8     uint8 [batch][seq_len_q][h_q][528] (device, 4-byte aligned).
 * The workspace must be at least what mla_get_metadata reports.  With 128
 * heads and no extra cache, the decode kernel writes the records of query
 * tokens that have one split itself and only tokens of several splits pass
 * through the workspace to the merge kernel (the same arithmetic either
 * way); for other shapes every query token's result passes through it on
 * its way to the epilogue in the merge kernel.  Rejections and errors as for
 * mla_sparse_decode; a null positions or out_fp8, or a theta that is not
 * finite and > 1, is MLA_ERR_INVALID_ARG.
 */
mla_status_t mla_sparse_decode_rope_fp8(const mla_problem_t* problem,
                                        const void* q, const void* kv, const int32_t* indices,
                                        const void* extra_kv, const int32_t* extra_indices,
                                        const int32_t* d_sched, const int32_t* d_num_splits, int32_t num_parts,
                                        void* workspace, size_t workspace_bytes,
                                        const int32_t* positions, float rope_theta,
                                        void* out_fp8, float* lse, int32_t* d_error,
                                        mla_stream_t stream);

/*
 * Merge of split-KV partial results ("Workarounds": split decoding with
 * num_splits).  For query token q its splits are
 * num_splits[q] .. num_splits[q+1]-1; split i of head h carries its own
 * normalised output o_partial[i][h][:] and its natural-log lse_partial[i][h]:
 *     L = ln sum_i exp(lse_i);   out = sum_i exp(lse_i - L) * o_i   (bf16)
 * Splits with lse = -inf weigh nothing; if all are -inf the result is +0 and
 * -inf.  A query token with one split is copied.
 *   d_num_splits  int32 [batch*seq_len_q + 1] prefix (device).
 *   o_partial     float [total_splits][h_q][512] (device).
 *   lse_partial   float [total_splits][h_q] (device).
 *   out, lse      as in mla_sparse_decode.
 */
mla_status_t mla_combine(const mla_problem_t* problem, const int32_t* d_num_splits,
                         const float* o_partial, const float* lse_partial,
                         void* out, float* lse, mla_stream_t stream);

/*
 * Dequantize whole cache records to bf16 with the decode kernel's own
 * in-register dequantization ("Arithmetic intensity": e4m3 x e8m0 per 32
 * dims for FP8; e2m1 x e4m3 per 16 dims for FP4).  Every decoded value is
 * exactly representable in bf16, so the result is exact.
 *   kv_format  MLA_KV_FP8_528 or MLA_KV_FP4_288.
 *   records    uint8 [n][528 or 288] (device, 16-byte aligned).
 *   out        bf16 [n][512] (device).
 */
mla_status_t mla_dequantize(int32_t kv_format, const void* records, int64_t n, void* out,
                            mla_stream_t stream);

/*
 * Decode without a caller-provided workspace.  The pages have no counterpart
 * to this entry point; it exists for callers that may not allocate device
 * memory at call time -- a plugin or hook inside another runtime that hands
 * it only input and output buffers, or a serving loop whose device memory is
 * all reserved up front by its own pool and which may not call cudaMalloc on
 * its per-step path.
 *
 * Same arguments and result as mla_sparse_decode minus the workspace: the
 * split partials go to a fixed array of MLA_NOALLOC_SCRATCH_BYTES that every
 * device loading this library holds until the process exits.  Every call
 * looks up that array's address on the current device (a host-side query, so
 * the address stays right after a device reset); the first lookup on a device
 * also loads the library's device code there, so make the first call before
 * any stream capture.  The problem is validated first (MLA_ERR_INVALID_ARG /
 * MLA_ERR_UNSUPPORTED as for mla_sparse_decode); then MLA_ERR_WORKSPACE, with
 * nothing enqueued, when the problem's workspace (the bytes mla_get_metadata
 * reports for it) exceeds MLA_NOALLOC_SCRATCH_BYTES.  All calls share the one
 * array: calls that overlap on the GPU race and must be serialised by the
 * caller (one stream).  Allocates nothing.
 */
#define MLA_NOALLOC_SCRATCH_BYTES (128u * 1024u * 1024u)
mla_status_t mla_sparse_decode_noalloc(const mla_problem_t* problem,
                                       const void* q, const void* kv, const int32_t* indices,
                                       const void* extra_kv, const int32_t* extra_indices,
                                       const int32_t* d_sched, const int32_t* d_num_splits, int32_t num_parts,
                                       void* out, float* lse, int32_t* d_error,
                                       mla_stream_t stream);

/*
 * KV-cache writer: quantize new tokens' latents into records and store each
 * at its slot of the paged pool -- the step that fills the cache the decode
 * reads ("Arithmetic intensity": 528-byte FP8 records, e4m3 data plus one
 * e8m0 scale per 32 values; 288-byte FP4 records, e2m1 data with the even
 * index in the low nibble plus one e4m3 scale per 16 values).  Block scales:
 * FP8 uses 2^e for the least e with amax * 2^-e <= 448 (scale byte 127 + e;
 * 127 for an all-zero block; e clamped to [-127, 127]); FP4 uses amax / 6
 * rounded to E4M3FN (a zero scale stores all-zero data).  Every element rounds
 * to nearest, ties to even, saturating at the format's largest finite value.
 *   kv_format  MLA_KV_FP8_528 or MLA_KV_FP4_288.
 *   latents    bf16 [n][512] (device, 16-byte aligned), finite values.
 *   slots      int32 [n] (device): page * 64 + offset; -1 = skip.  Slots
 *              < -1 or >= num_pages * 64 are skipped and flagged
 *              (MLA_DEVERR_BAD_INDEX).
 *   pool       uint8 [num_pages][64][528 or 288] (device, 16-byte aligned);
 *              only the addressed records are written.  Two tokens with the
 *              same slot race.
 *   d_error    device int32 or NULL, as in mla_sparse_decode.
 */
mla_status_t mla_kv_write(int32_t kv_format, const void* latents, const int32_t* slots, int64_t n, void* pool,
                          int64_t num_pages, int32_t* d_error, mla_stream_t stream);

/*
 * Block tables and slot maps of a paged pool, built on the device from
 * request lengths: where mla_kv_write puts each new token, which pages
 * mla_paged_decode_fp4 reads, and which position mla_rope turns it to.  One
 * call per step and no host synchronisation, so a captured graph replays it.
 *
 * Request r holds cached_lens[r] = c tokens in the first ceil(c / 64) entries
 * of its block table row and appends new_lens[r] = n tokens:
 *   n >= 0  it takes ceil((c + n) / 64) - ceil(c / 64) pages from the top of
 *           the free stack, in request order (its first new page is the topmost
 *           one left), and they follow its held pages in its row.  New token i
 *           has position p = c + i and slot 64 * row[p / 64] + p % 64.
 *   n = -1  the request has ended: its held pages go back onto the stack (in
 *           request and row order, all before any page is taken); its length
 *           becomes 0 and its row is left as it is.
 * The tokens are packed in request order: those of r at cu_new[r] ..
 * cu_new[r + 1] - 1 of slots and positions.  Entries from cu_new[batch] on to
 * max_new get slot -1 (which mla_kv_write skips) and position 0.
 *
 *   cached_lens, new_lens  int32 [batch].
 *   block_table   int32 [batch][max_pages]; only entries of pages taken are written.
 *   free_pages    int32 [num_pages]: the stack of free page ids, top last.
 *   num_free      int32 [1]: how many there are.
 *   seq_lens      int32 [batch], written: c + n (may be cached_lens itself).
 *   num_free_out  int32 [1], written (may be num_free itself).
 *   cu_new        int32 [batch + 1], written.
 *   slots, positions  int32 [max_new], written to the end.
 *   d_error       device int32 or NULL; bits are OR-ed into it.
 * The call refuses as a whole -- tables, stack and lengths stay as they are,
 * cu_new is all 0 and every slot -1 -- when a length is negative or past
 * 64 * max_pages (MLA_DEVERR_BAD_LENGTH), when pages or slots do not suffice
 * (MLA_DEVERR_NO_ROOM), or when num_free lies outside [0, num_pages] or more
 * pages come back than the stack holds (MLA_DEVERR_BAD_METADATA).  A page id
 * outside [0, num_pages) gives its tokens slot -1 and MLA_DEVERR_BAD_INDEX; one
 * that an ended request gives back is flagged likewise and goes onto the stack.
 * batch is at most 8192 and num_pages * 64 below 2^31 (MLA_ERR_UNSUPPORTED).
 * Apart from the two pairs named, no buffer may overlap another.
 */
mla_status_t mla_page_plan(const int32_t* cached_lens, const int32_t* new_lens, int32_t batch,
                           int32_t* block_table, int32_t max_pages,
                           int32_t* free_pages, int32_t num_pages, const int32_t* num_free,
                           int32_t* seq_lens, int32_t* num_free_out, int32_t* cu_new,
                           int32_t* slots, int32_t* positions, int32_t max_new,
                           int32_t* d_error, mla_stream_t stream);

/* Element types of activations. */
enum { MLA_BF16 = 0, MLA_FP16 = 1, MLA_FP32 = 2 };

/*
 * Rotary positions.  A table holds, for each of the rope_dim / 2 pairs, the
 * turns per position as a 64-bit fixed-point fraction: position times step,
 * modulo 2^64, is the exact phase at any int32 position, so far positions
 * lose nothing and no cosine table is read.
 */
enum { MLA_ROPE_INTERLEAVED = 0, MLA_ROPE_HALF = 1 };     /* pairs (2j, 2j+1), or (j, j + rope_dim/2) */
enum { MLA_ROPE_PLAIN = 0, MLA_ROPE_LINEAR = 1, MLA_ROPE_YARN = 2 };
#define MLA_ROPE_MAX_DIM 256
typedef struct {
  int32_t rope_dim;          /* even, 2 .. MLA_ROPE_MAX_DIM */
  int32_t layout;            /* MLA_ROPE_INTERLEAVED or MLA_ROPE_HALF */
  float factor;              /* on the rotated dims (the attention factor of long contexts), finite */
  uint64_t step[MLA_ROPE_MAX_DIM / 2];
} mla_rope_table_t;

/*
 * Fill a table (host only) from frequencies f_j in radians per position:
 * step_j = f_j / (2 pi) * 2^64, |f_j| <= pi.  mla_rope_table computes
 * f_j = theta^(-2j / rope_dim) and scales it for contexts past original_len:
 *   MLA_ROPE_LINEAR  f_j / scale.
 *   MLA_ROPE_YARN    f_j (1 - g_j) + f_j / scale * g_j with the ramp
 *                    g_j = clamp((j - lo) / max(hi - lo, 0.001), 0, 1), where
 *                    dim(r) = rope_dim ln(original_len / (2 pi r)) / (2 ln theta),
 *                    lo = max(floor(dim(beta_fast)), 0),
 *                    hi = min(ceil(dim(beta_slow)), rope_dim - 1).
 * factor is taken as given (YaRN models commonly use 0.1 ln(scale) + 1).
 */
mla_status_t mla_rope_table(mla_rope_table_t* table, int32_t rope_dim, int32_t layout, double theta,
                            int32_t scaling, double scale, double original_len, double beta_fast, double beta_slow,
                            double factor);
mla_status_t mla_rope_table_from_freqs(mla_rope_table_t* table, int32_t rope_dim, int32_t layout,
                                       const double* freqs, double factor);

/*
 * y = x with dims offset .. offset + rope_dim - 1 of every head turned:
 * pair (a, b) at position p -> factor * (a cos - b sin, b cos + a sin) of the
 * angle p f_j, computed in fp32 and rounded once.  The other dims are copied
 * (out of place) or left (in place).  With conjugate != 0 the angle is
 * negated: the transpose, which takes a gradient of y to the gradient of x.
 *   x, y      dtype [n][heads][head_dim] with element strides row_stride and
 *             head_stride (the last dim dense), element aligned; y may be x
 *             itself with the same strides (in place) and must not overlap
 *             it otherwise.
 *   positions int32 [n].
 * Rows that start on 16-byte boundaries and ranges that are whole 16-byte
 * pieces move in 16-byte accesses, others element by element.
 */
mla_status_t mla_rope(int32_t dtype, const void* x, int64_t x_row_stride, int64_t x_head_stride, void* y,
                      int64_t y_row_stride, int64_t y_head_stride, int64_t n, int32_t heads, int32_t head_dim,
                      int32_t offset, const int32_t* positions, const mla_rope_table_t* table, int32_t conjugate,
                      mla_stream_t stream);

/*
 * New tokens into the paged pool with their rotary positions applied on the
 * way: mla_rope on dims offset .. offset + rope_dim - 1 of each latent and
 * mla_kv_write of the result, in one pass and with one rounding, that to the
 * record (the turned values are fp32 in between).
 *   kv_format  MLA_KV_FP8_528 or MLA_KV_FP4_288; records as mla_kv_write makes them.
 *   dtype      MLA_BF16, MLA_FP16 or MLA_FP32.
 *   latents    dtype [n][512], rows row_stride elements apart, each 16-byte
 *              aligned (so the rows of a wider projection serve); finite values,
 *              finite after the turn in fp32 too.
 *   table      the rotary table, or NULL: nothing turns (positions is then
 *              not read and may be NULL).
 *   positions  int32 [n] (device); those of skipped rows are not used.
 *   slots, pool, num_pages, d_error   as in mla_kv_write: -1 skips a row, other
 *              slots outside the pool are skipped and flagged, only the
 *              addressed records are written, two rows with the same slot race.
 * Rows of 16 bits without a table give the bytes that mla_kv_write gives.
 */
mla_status_t mla_kv_append(int32_t kv_format, int32_t dtype, const void* latents, int64_t row_stride, int64_t n,
                           const mla_rope_table_t* table, int32_t offset, const int32_t* positions,
                           const int32_t* slots, void* pool, int64_t num_pages, int32_t* d_error, mla_stream_t stream);

/*
 * The means of full pages in 8 bits, by which mla_paged_sparse_decode_fp4 selects
 * pages.  Tokens are appended in order, so a page is full when its last slot is
 * written: every slot of the list that is the last one of its page (slot % 64 ==
 * 63) has that page's mean computed from its 64 FP4 records; other entries do
 * nothing.  So the slots of a step (mla_page_plan's) keep the means up to date,
 * and a list of last slots makes those of a cache that was filled before.
 * A mean is a record of MLA_MEAN_BYTES: 512 int8 codes, the byte 127 + e, 15
 * zeros.  With the exact mean m and the least e that gives max |m_d| 2^-e <= 127
 * (e = 0 for a mean of zeros), code d is m_d 2^-e rounded to nearest even: no
 * other rounding.  A NaN scale in a record counts as 448 (of its sign).
 *   pool     uint8 [num_pages][64][288] FP4 records, 16-byte aligned.
 *   slots    int32 [n] (device); -1 = skip, others outside the pool are skipped
 *            and flagged (MLA_DEVERR_BAD_INDEX).
 *   means    uint8 [num_pages][MLA_MEAN_BYTES], 16-byte aligned; only those of
 *            the pages named are written.
 *   d_error  device int32 or NULL.
 */
#define MLA_MEAN_BYTES 528
mla_status_t mla_page_means(const void* pool, int64_t num_pages, const int32_t* slots, int64_t n, void* means,
                            int32_t* d_error, mla_stream_t stream);

/*
 * Root-mean-square norm with the residual's addition, cast to FP8 blocks:
 *     s = x + residual        (fp32; residual may be NULL)
 *     residual_out = s        (rounded to dtype; may be residual itself, NULL to drop it)
 *     v = s / sqrt(mean(s^2) + eps) * weight          (fp32 throughout)
 * and per 32 values of v the least power of two 2^e with amax * 2^-e <= 448
 * (scale byte 127 + e; 127 for an all-zero block; e >= -127), each value
 * rounded to the nearest E4M3FN.  The norm is taken of the unrounded sum.
 * codes and scales have row strides of their own, so with dim 512, codes = r
 * and scales = r + 512 at stride 528 the rows have the form of FP8 records
 * (mla_dequantize reads them; mla_rope and mla_kv_write take 16-bit rows, so a
 * latent is rotated and written from those).  Outputs overlap no input but as
 * said, and not one another.
 *   x, residual, residual_out, weight  dtype; rows at element strides, each
 *             row 16-byte aligned (weight [dim], 16-byte aligned).
 *   codes     uint8, rows 8-byte aligned; scales uint8 [n][dim / 32].
 *   dim       a multiple of 32, at most 16384 (MLA_ERR_UNSUPPORTED otherwise).
 *   d_error   device int32 or NULL; bits are OR-ed into it (MLA_DEVERR_TIMEOUT
 *             when a row's copy did not arrive: that row is not written, nor
 *             are those that its block has not asked for by then).
 * Infinities and NaN in a row make that row's codes undefined, and so does a
 * mean(s^2) + eps that fp32 cannot hold (0, as of a row of zeros with eps = 0,
 * or a sum of squares past 3.4e38); no other row.
 */
mla_status_t mla_rms_norm_fp8(int32_t dtype, const void* x, int64_t x_stride, const void* residual,
                              int64_t residual_stride, const void* weight, float eps, void* residual_out,
                              int64_t residual_out_stride, void* codes, int64_t codes_stride, void* scales,
                              int64_t scales_stride, int64_t n, int32_t dim, int32_t* d_error, mla_stream_t stream);

/*
 * Attention over the pages of a cache held in 4 bits: every query token sees
 * the tokens of its own sequence, all of them or a window and the first few.
 */
typedef struct {
  int32_t batch;        /* b >= 1 */
  int32_t seq_len_q;    /* s >= 1: the last s tokens of each sequence are the query tokens */
  int32_t h_q;          /* query heads, 1 .. 128 */
  int32_t head_dim;     /* must be 512 */
  int32_t page_size;    /* must be 64 */
  int32_t max_pages;    /* entries of a block table row; a table no wider than the sequences need is faster
                           for short ones, as the plan knows their lengths by it */
  int32_t window;       /* tokens seen back from the query token, itself included; 0 = all */
  int32_t sinks;        /* the first tokens of a sequence, seen whatever the window */
  int64_t num_pages;    /* pages in the pool (bounds check of the block table) */
  int32_t kv_format;    /* must be MLA_KV_FP4_288 */
  float sm_scale;       /* softmax scale applied to q.k, finite in units of ln 2 too (|sm_scale| < 2.35e38) */
} mla_paged_problem_t;

/* Host-only planning: the part count (num_sms = 0 asks the current device) and the workspace bytes. */
mla_status_t mla_paged_decode_plan(const mla_paged_problem_t* problem, int32_t num_sms, int32_t* num_parts_out,
                                   size_t* workspace_bytes_out);

/*
 * One attention step.  Query token i of sequence b stands at position
 * p = seq_lens[b] - s + i and sees the cached tokens j <= p with
 * window == 0, j > p - window or j < sinks; over those, with latents k_j,
 *     lse = ln sum_j exp(sm_scale <q, k_j>),  out = sum_j exp(sm_scale <q, k_j> - lse) k_j.
 * A query token that sees nothing (an empty sequence, p < 0) gets +0 and -inf.
 *   q            bf16 [batch][s][h_q][512], 16-byte aligned, finite.
 *   kv           uint8 [num_pages][64][288] FP4 records, 16-byte aligned.
 *                Records that no query token of a sequence sees are never used, whatever
 *                bytes they hold; a NaN scale in one makes the rows that see it
 *                undefined, no other.
 *   block_table  int32 [batch][max_pages]: page ids; entries past ceil(len / 64), and
 *                those of pages that window and sinks leave out, are not read.
 *                The tokens of a page id outside [0, num_pages) are skipped
 *                and flagged (MLA_DEVERR_BAD_INDEX).
 *   seq_lens     int32 [batch] (device), the query tokens included; negative or past
 *                64 * max_pages: treated as 0 and flagged (MLA_DEVERR_BAD_LENGTH).
 *   num_parts, workspace, workspace_bytes   as mla_paged_decode_plan says; the
 *                workspace is 16-byte aligned and needs no initialisation.
 *                Calls that share one must not overlap.
 *   out          bf16 [batch][s][h_q][512], 16-byte aligned;  lse  float [batch][s][h_q].
 *   d_error      device int32 or NULL.
 */
mla_status_t mla_paged_decode_fp4(const mla_paged_problem_t* problem, const void* q, const void* kv,
                                  const int32_t* block_table, const int32_t* seq_lens, int32_t num_parts,
                                  void* workspace, size_t workspace_bytes, void* out, float* lse, int32_t* d_error,
                                  mla_stream_t stream);

/*
 * Attention of each query token over a few pages of its sequence, which a cheap
 * score of the pages' means selects: long contexts at the cost of top_pages.
 */
typedef struct {
  int32_t batch;        /* b >= 1 */
  int32_t seq_len_q;    /* s >= 1: the last s tokens of each sequence are the query tokens */
  int32_t h_q;          /* query heads, 1 .. 128 */
  int32_t head_dim;     /* must be 512 */
  int32_t page_size;    /* must be 64 */
  int32_t max_pages;    /* entries of a block table row */
  int32_t top_pages;    /* pages a query token attends to at most, >= 1 */
  int32_t sink_pages;   /* the first pages, always among them, >= 0 */
  int32_t local_pages;  /* the query token's own page and those before it, always among them, >= 1 */
  int64_t num_pages;    /* pages in the pool (bounds check of the block table) */
  int32_t kv_format;    /* must be MLA_KV_FP4_288 */
  float sm_scale;       /* as in mla_paged_problem_t */
} mla_paged_sparse_problem_t; /* sink_pages + local_pages <= top_pages */

/* Host-only planning, as mla_paged_decode_plan.  The workspace holds a float for each (query token, table entry). */
mla_status_t mla_paged_sparse_plan(const mla_paged_sparse_problem_t* problem, int32_t num_sms, int32_t* num_parts_out,
                                   size_t* workspace_bytes_out);

/*
 * One attention step.  Query token i of sequence b stands at position
 * p = seq_lens[b] - s + i, in page c = p / 64.  It attends to the tokens j <= p
 * of the selected pages: all of 0 .. c if they are at most top_pages, otherwise
 *   0 .. sink_pages - 1,  c - local_pages + 1 .. c,  and of the pages between
 *   them (all full) those with the highest scores, top_pages in all; equal
 *   scores go to the lower page.
 * A page's score is the largest of its heads' <q_h, mean of the page> (smallest
 * for a negative sm_scale), from 8-bit codes of both: with e_h the least exponent
 * (at least -120) that gives max |q_hd| 2^-e_h <= 127, a_hd = q_hd 2^-e_h rounded
 * to nearest even and a mean's codes c_d and exponent e (mla_page_means),
 *     score = max_h  2^max(e_h - max_g e_g, -100) * sum_d a_hd c_d  * 2^e,
 * g over the rows that are not all 0.  That is exact in fp32, so the selection
 * does not depend on the order of any sum.
 *   q, kv, block_table, seq_lens, out, lse   as in mla_paged_decode_fp4, as are
 *                rows that see nothing and what is flagged.  A page id outside the
 *                pool scores minus infinity; its tokens are skipped.
 *   means        uint8 [num_pages][MLA_MEAN_BYTES], 16-byte aligned; read for
 *                the full pages of the block tables that are scored.
 *   selected     int32 [batch][s][top_pages] or NULL, written: the pages of the
 *                sequence each query token attends to, ascending, -1 after the last.
 *   num_parts, workspace, workspace_bytes   as mla_paged_sparse_plan says,
 *                16-byte aligned; calls that share a workspace must not overlap.
 */
mla_status_t mla_paged_sparse_decode_fp4(const mla_paged_sparse_problem_t* problem, const void* q, const void* kv,
                                         const void* means, const int32_t* block_table, const int32_t* seq_lens,
                                         int32_t num_parts, void* workspace, size_t workspace_bytes, void* out,
                                         float* lse, int32_t* selected, int32_t* d_error, mla_stream_t stream);

/*
 * Attention for a batch whose sequences share long prefixes (a system prompt, a
 * document, the prompt of many samples): each group of consecutive sequences has
 * one prefix, whose records are read and decoded once for all rows of the group,
 * and every sequence goes on with pages of its own.
 */
typedef struct {
  int32_t batch;            /* b >= 1 */
  int32_t seq_len_q;        /* s >= 1: the last s tokens of each sequence are the query tokens */
  int32_t h_q;              /* query heads, 1 .. 128 */
  int32_t head_dim;         /* must be 512 */
  int32_t page_size;        /* must be 64 */
  int32_t groups;           /* prefixes, 1 .. MLA_MAX_PREFIX_GROUPS */
  int32_t max_prefix_pages; /* entries of a prefix table row */
  int32_t max_pages;        /* entries of a block table row (own pages); tables no wider than the sequences need are faster */
  int64_t num_pages;        /* pages in the pool (bounds check of the tables) */
  int32_t kv_format;        /* must be MLA_KV_FP4_288 */
  float sm_scale;           /* as in mla_paged_problem_t */
} mla_paged_shared_problem_t;
#define MLA_MAX_PREFIX_GROUPS 8192

/* Host-only planning, as mla_paged_decode_plan.  The workspace holds fp32 outputs of every query row twice. */
mla_status_t mla_paged_shared_plan(const mla_paged_shared_problem_t* problem, int32_t num_sms, int32_t* num_parts_out,
                                   size_t* workspace_bytes_out);

/*
 * One attention step.  Sequences group_start[g] .. group_start[g + 1] - 1 share
 * prefix g; sequences in no group have none.  Query token i of sequence b stands
 * at position p = seq_lens[b] - s + i of its own tokens; it sees the own tokens
 * j <= p and, if p >= 0, the whole prefix, all under one softmax:
 *     lse = ln sum_j exp(sm_scale <q, k_j>),  out = sum_j exp(sm_scale <q, k_j> - lse) k_j.
 * A query token with p < 0 (padding) gets +0 and -inf.
 *   q, kv, out, lse   as in mla_paged_decode_fp4.
 *   group_start  int32 [groups + 1], ascending from >= 0 to <= batch; groups may
 *                be empty.  Otherwise no sequence has a prefix (MLA_DEVERR_BAD_METADATA).
 *   prefix_table int32 [groups][max_prefix_pages]: page ids; entries past
 *                ceil(prefix_lens[g] / 64) are not read.
 *   prefix_lens  int32 [groups], any length (the last page may be part full);
 *                negative or past 64 * max_prefix_pages: treated as 0 and
 *                flagged (MLA_DEVERR_BAD_LENGTH).
 *   block_table  int32 [batch][max_pages]: the sequences' own pages.
 *   seq_lens     int32 [batch]: their own tokens, the query tokens included, the
 *                prefix not; bad lengths as in mla_paged_decode_fp4.
 * Page ids outside the pool: their tokens are skipped and flagged
 * (MLA_DEVERR_BAD_INDEX).  num_parts, workspace, workspace_bytes and d_error as in
 * mla_paged_decode_fp4, from mla_paged_shared_plan.
 */
mla_status_t mla_paged_shared_decode_fp4(const mla_paged_shared_problem_t* problem, const void* q, const void* kv,
                                         const int32_t* group_start, const int32_t* prefix_table,
                                         const int32_t* prefix_lens, const int32_t* block_table,
                                         const int32_t* seq_lens, int32_t num_parts, void* workspace,
                                         size_t workspace_bytes, void* out, float* lse, int32_t* d_error,
                                         mla_stream_t stream);

/* Static description of a status code. */
const char* mla_status_string(mla_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* MLA_H */
