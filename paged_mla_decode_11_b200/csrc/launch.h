// Internal launch entry points of the kernels behind the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "pagedmla.h"

namespace pagedmla {

// Records an error for mla_last_error_string() on this thread and returns `code`.
int record_error(int code, const char *msg);

// Raises a kernel's dynamic shared-memory limit once per (kernel, device), so that
// launches inside CUDA-graph capture make no attribute calls.
cudaError_t set_smem_once(const void *kernel, int bytes);

// lengths_are_offsets: seqlens holds batch + 1 offsets (a CSR row_ptr) and length b is
// seqlens[b + 1] - seqlens[b]
cudaError_t launch_metadata(const int32_t *seqlens, int batch, int ovh, int num_parts, int32_t *tile_md,
                            int32_t *num_splits, cudaStream_t stream, bool lengths_are_offsets = false);
cudaError_t launch_decode_mma(const CUtensorMap &map, const DecodeParams &p, cudaStream_t stream);
cudaError_t launch_decode_mma16(const CUtensorMap &kv_map, const CUtensorMap &q_map, const DecodeParams &p,
                                cudaStream_t stream);
// Token-level sparse decode, up to 16 query heads per latent head and query token (p.row_ptr,
// p.col_idx, p.sq_fold set; p.batch / p.s_q / p.R describe query tokens as sequences).
cudaError_t launch_decode_sparse16(const CUtensorMap &q_map, const DecodeParams &p, cudaStream_t stream);
// The 64-row tcgen05 kernel takes more than 16 rows per latent head.
bool wide_supported(int R, int g);
cudaError_t launch_decode_wide(const CUtensorMap &kv_map, const DecodeParams &p, cudaStream_t stream);
// The CTA-pair tcgen05 kernel takes whole 128-row blocks whose 64-row halves are (position,
// head) rectangles: g a multiple or a divisor of 64.
bool pair_supported(int R, int g);
cudaError_t launch_decode_pair(const CUtensorMap &kv_map, const CUtensorMap &q_map, const DecodeParams &p,
                               int q_box_heads, cudaStream_t stream);
cudaError_t launch_decode_tc_narrow(const CUtensorMap &kv_map, const CUtensorMap &q_map,
                                    const DecodeParams &p, cudaStream_t stream);
cudaError_t launch_decode_fp8(const CUtensorMap &k8_map, const CUtensorMap &scale_map, const CUtensorMap &q_map,
                              const DecodeParams &p, cudaStream_t stream);
// The CTA-pair kernel over the FP8 cache, any number of query rows per latent head.
cudaError_t launch_decode_fp8_pair(const CUtensorMap &k8_map, const CUtensorMap &page_map, const CUtensorMap &half_map,
                                   const DecodeParams &p, const float *k_scale, int64_t num_pages, cudaStream_t stream);
cudaError_t launch_combine(const int32_t *num_splits, int batch, int s_q, int h_q, int h_kv,
                           const float *lse_accum, const float *o_accum, __nv_bfloat16 *out,
                           float *lse, cudaStream_t stream, int sq_fold = 1);
cudaError_t launch_merge(const __nv_bfloat16 *o_parts, const float *lse_parts, int n_parts, int batch, int s_q,
                         int h_q, __nv_bfloat16 *out, float *lse, cudaStream_t stream);
cudaError_t launch_absorb_q(const __nv_bfloat16 *q_nope, int64_t n_row, int64_t n_head, const __nv_bfloat16 *q_rope,
                            int64_t r_row, int64_t r_head, const __nv_bfloat16 *w_uk, __nv_bfloat16 *q_out, int T,
                            int H, cudaStream_t stream);
cudaError_t launch_absorb_out(const __nv_bfloat16 *o_lat, int64_t l_row, int64_t l_head, const __nv_bfloat16 *w_uv,
                              __nv_bfloat16 *out, int T, int H, cudaStream_t stream);

// Rotary positions (rope.cu); strides in elements, the tile sizes are the launcher's.
constexpr int kRopeMaxPairs = 512;
struct RopeParams {
  const void *x;
  void *out;
  int64_t x_t, x_h, o_t, o_h;
  int64_t tokens;
  int heads, width, pairs;
  const void *positions;
  const double *inv_freq;
  float magnitude;
  bool pos64, inverse, copy_front;  // copy_front: the columns in front are to be copied (out is not x)
  int tile_tokens, tile_heads;
};
cudaError_t launch_rope(RopeParams p, int dtype, bool half, cudaStream_t stream);

// Cache write and read-back (cache.cu).
cudaError_t launch_cache_slots(const int32_t *row_ptr, const int32_t *seqlens, int batch, const int32_t *block_table,
                               int64_t bt_stride, int bt_width, int64_t num_pages, int64_t tokens, int64_t *slots,
                               int32_t *positions, cudaStream_t stream);
struct CacheWriteParams {
  const void *latent, *rope;
  int64_t l_t, l_h, r_t, r_h;
  int64_t tokens;
  int h_kv;
  const void *weight;       // nullptr: no norm
  float eps;
  const void *positions;
  const double *inv_freq;   // nullptr: rope columns as they are
  float magnitude;
  bool pos64, half;
  const int64_t *slots;
  void *cache;
  float *scale;             // nullptr: a bf16 cache
  int64_t num_slots;
};
cudaError_t launch_cache_write(const CacheWriteParams &p, int dtype, cudaStream_t stream);
struct CacheReadParams {
  const void *cache;
  const float *scale;       // nullptr: a bf16 cache
  int64_t num_slots;
  int64_t tokens;
  int h_kv;
  const int64_t *slots;
  __nv_bfloat16 *out;
  int64_t o_t, o_h;
};
cudaError_t launch_cache_read(const CacheReadParams &p, cudaStream_t stream);

// Verification of drafted tokens (verify.cu).
struct VerifyParams {
  const void *target, *draft;  // draft nullptr: drafts chosen with certainty
  int64_t t_b, t_s, d_b, d_s;  // element strides of their batch and position dims
  int batch, drafts, vocab;
  const int32_t *tokens;
  const float *uniform, *uniform_new;
  const int32_t *num_drafts;   // nullptr: all of them
  int32_t *accepted, *out;
  unsigned long long wait_ns;  // limit of a device-side wait
  int missing;                 // sums expected beyond those that are sent (the self-test: 1)
};
cudaError_t launch_verify(const VerifyParams &p, int dtype, cudaStream_t stream);

cudaError_t launch_watchdog_selftest(int *status, unsigned long long timeout_ns,
                                     cudaStream_t stream);

}  // namespace pagedmla
