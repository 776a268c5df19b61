// Filling the paged latent cache and reading it back.
//
// Write, per (token, latent head) row: the 512 latent columns c are normalised,
//   c_k = x_k * w_k / sqrt(mean(x^2) + eps)                         (when a weight is given)
// the 64 rope columns are turned by their position (rope.cuh; when positions are given), and
// the 576 columns go to the row's slot (page * 64 + offset): rounded to bf16, or as E4M3 codes
// with one fp32 scale, scale = max|row| / 448 (1 for a row of zeros) and code = row / scale
// rounded to nearest.  The codes are taken from the fp32 row, not from its bf16 rounding.
//
// Read: the rows of listed slots, in list order, as bf16 (codes times their scale).
//
// Both move each byte once and are bound by HBM.  Rows with a slot outside the pool are skipped
// by the write and read as zeros.
#include <cuda_fp8.h>

#include "launch.h"
#include "rope.cuh"

namespace pagedmla {

// ------------------------------------------------------------------------------------
// Slots and positions of a step's new tokens.
// ------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
    cache_slots_kernel(const int32_t *__restrict__ row_ptr, const int32_t *__restrict__ seqlens, int batch,
                       const int32_t *__restrict__ block_table, int64_t bt_stride, int bt_width, int64_t num_pages,
                       int64_t tokens, int64_t *__restrict__ slots, int32_t *__restrict__ positions) {
  const int64_t t = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  grid_launch_dependents();
  grid_dependency_wait();
  if (t >= tokens) return;
  int64_t slot = -1;
  int32_t pos = 0;
  if (t >= __ldcg(row_ptr) && t < __ldcg(row_ptr + batch)) {
    int lo = 0, hi = batch;  // the last b with row_ptr[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (__ldcg(row_ptr + mid) <= t) lo = mid; else hi = mid;
    }
    // the sequence's new tokens are the last of its cache entries
    const int64_t at = int64_t(__ldcg(seqlens + lo)) - (__ldcg(row_ptr + lo + 1) - t);
    if (at >= 0 && at / kPage < bt_width) {
      const int64_t page = __ldcg(block_table + lo * bt_stride + at / kPage);
      if (page >= 0 && page < num_pages) {
        slot = page * kPage + at % kPage;
        pos = int32_t(at);
      }
    }
  }
  slots[t] = slot;
  positions[t] = pos;
}

cudaError_t launch_cache_slots(const int32_t *row_ptr, const int32_t *seqlens, int batch, const int32_t *block_table,
                               int64_t bt_stride, int bt_width, int64_t num_pages, int64_t tokens, int64_t *slots,
                               int32_t *positions, cudaStream_t stream) {
  return launch_early(cache_slots_kernel, dim3(unsigned((tokens + 255) / 256)), dim3(256), 0, stream, row_ptr, seqlens,
                      batch, block_table, bt_stride, bt_width, num_pages, tokens, slots, positions);
}

// ------------------------------------------------------------------------------------
// Write: one warp per row.  Lane l holds 16 latent columns in 16-byte accesses of neighbouring
// lanes, and pair l of the rope columns, so the norm, the scale and the rotation need no shared
// memory: two warp reductions per row.
// ------------------------------------------------------------------------------------
constexpr int kWriteWarps = 8;

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

template <typename T, bool kFp8>
__global__ void __launch_bounds__(kWriteWarps * 32) cache_write_kernel(const CacheWriteParams p) {
  constexpr int VEC = 16 / sizeof(T), NV = 16 / VEC;  // NV accesses of VEC columns per lane
  using V = Pack<T, VEC>;
  const int lane = threadIdx.x % 32;
  const int64_t row = int64_t(blockIdx.x) * kWriteWarps + threadIdx.x / 32;
  grid_launch_dependents();
  grid_dependency_wait();
  if (row >= p.tokens * p.h_kv) return;
  const int64_t t = p.h_kv == 1 ? row : row / p.h_kv;
  const int h = int(row - t * p.h_kv);
  const int64_t slot = __ldcg(reinterpret_cast<const long long *>(p.slots) + t);
  const T *lat = static_cast<const T *>(p.latent) + t * p.l_t + h * p.l_h;
  const T *rp = static_cast<const T *>(p.rope) + t * p.r_t + h * p.r_h;
  V in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = load_cg(reinterpret_cast<const V *>(lat + (i * 32 + lane) * VEC));
  const int c0 = p.half ? lane : 2 * lane, c1 = p.half ? lane + 32 : c0 + 1;  // this lane's rope pair
  float r0, r1;
  if (p.half) {
    r0 = to_float(load_cg(rp + c0));
    r1 = to_float(load_cg(rp + c1));
  } else {
    const Pack<T, 2> pr = load_cg(reinterpret_cast<const Pack<T, 2> *>(rp + c0));
    r0 = to_float(pr.v[0]);
    r1 = to_float(pr.v[1]);
  }
  if (p.inv_freq) {
    const float2 w = rope_cos_sin(load_position(p.positions, p.pos64, t), __ldg(p.inv_freq + lane), p.magnitude, false);
    const float y0 = r0 * w.x - r1 * w.y;
    r1 = r0 * w.y + r1 * w.x;
    r0 = y0;
  }
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = to_float(in[i / VEC].v[i % VEC]);
  if (p.weight) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = rsqrtf(ss * (1.f / kDV) + p.eps);
    const T *w = static_cast<const T *>(p.weight);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const V wv = *reinterpret_cast<const V *>(w + (i * 32 + lane) * VEC);  // a model parameter
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[i * VEC + k] *= inv * to_float(wv.v[k]);
    }
  }
  if (slot < 0 || slot >= p.num_slots) return;
  const int64_t dst_row = slot * p.h_kv + h;
  if constexpr (!kFp8) {
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.cache) + dst_row * kD;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t w[VEC / 2];
#pragma unroll
      for (int k = 0; k < VEC / 2; ++k) w[k] = pack_bf16x2(v[i * VEC + 2 * k], v[i * VEC + 2 * k + 1]);
      if constexpr (VEC == 8)
        *reinterpret_cast<uint4 *>(dst + (i * 32 + lane) * VEC) = make_uint4(w[0], w[1], w[2], w[3]);
      else
        *reinterpret_cast<uint2 *>(dst + (i * 32 + lane) * VEC) = make_uint2(w[0], w[1]);
    }
    if (p.half) {
      dst[kDV + c0] = __float2bfloat16_rn(r0);
      dst[kDV + c1] = __float2bfloat16_rn(r1);
    } else {
      *reinterpret_cast<uint32_t *>(dst + kDV + c0) = pack_bf16x2(r0, r1);
    }
  } else {
    // E4M3 has no infinity: infinities and NaN become NaN codes and do not enter the scale
    const float kNaN = __int_as_float(0x7fffffff);
    float amax = 0.f;
    auto see = [&](float &x) {
      const float a = fabsf(x);
      if (a <= 3.402823466e38f)
        amax = fmaxf(amax, a);
      else
        x = kNaN;
    };
#pragma unroll
    for (int i = 0; i < 16; ++i) see(v[i]);
    see(r0);
    see(r1);
    // non-negative floats order as their bit patterns
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    float scale = amax / 448.f;
    if (scale == 0.f) scale = 1.f;
    // true quotients: inputs of few bits often lie exactly in the middle of two codes, where a
    // product with 1 / scale would round to the wrong side
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] /= scale;
    r0 /= scale;
    r1 /= scale;
    uint8_t *dst = static_cast<uint8_t *>(p.cache) + dst_row * kD;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t w[VEC / 4];
#pragma unroll
      for (int k = 0; k < VEC / 4; ++k)
        w[k] = uint32_t(e4m3x2(v[i * VEC + 4 * k], v[i * VEC + 4 * k + 1])) |
               uint32_t(e4m3x2(v[i * VEC + 4 * k + 2], v[i * VEC + 4 * k + 3])) << 16;
      if constexpr (VEC == 8)
        *reinterpret_cast<uint2 *>(dst + (i * 32 + lane) * VEC) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t *>(dst + (i * 32 + lane) * VEC) = w[0];
    }
    const uint16_t r = e4m3x2(r0, r1);
    if (p.half) {
      dst[kDV + c0] = uint8_t(r);
      dst[kDV + c1] = uint8_t(r >> 8);
    } else {
      *reinterpret_cast<uint16_t *>(dst + kDV + c0) = r;
    }
    if (lane == 0) p.scale[h * p.num_slots + slot] = scale;
  }
}

template <typename T>
static cudaError_t launch_cache_write_typed(const CacheWriteParams &p, cudaStream_t stream) {
  const int64_t rows = p.tokens * p.h_kv;
  const dim3 grid(unsigned((rows + kWriteWarps - 1) / kWriteWarps));
  return p.scale ? launch_early(cache_write_kernel<T, true>, grid, dim3(kWriteWarps * 32), 0, stream, p)
                 : launch_early(cache_write_kernel<T, false>, grid, dim3(kWriteWarps * 32), 0, stream, p);
}

cudaError_t launch_cache_write(const CacheWriteParams &p, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case MLA_DTYPE_BF16: return launch_cache_write_typed<__nv_bfloat16>(p, stream);
    case MLA_DTYPE_F16: return launch_cache_write_typed<__half>(p, stream);
    default: return launch_cache_write_typed<float>(p, stream);
  }
}

// ------------------------------------------------------------------------------------
// Read: 288 threads are four rows of 72 threads, each thread eight columns of a row (a 16-byte
// store; a 16- or 8-byte load) of kRows / 4 rows, all loads issued before the first store.
// ------------------------------------------------------------------------------------
constexpr int kReadThreads = 4 * (kD / 8);

__device__ __forceinline__ uint32_t e4m3x2_scaled(uint16_t codes, float scale) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(codes, __NV_E4M3);  // exact
  const float2 f = __half22float2(__half2(h));
  return pack_bf16x2(f.x * scale, f.y * scale);
}

template <bool kFp8, int kRows>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const CacheReadParams p) {
  constexpr int N = kRows / 4;
  const int c = threadIdx.x % (kD / 8), r0 = threadIdx.x / (kD / 8);
  const int64_t first = int64_t(blockIdx.x) * kRows + r0, rows = p.tokens * p.h_kv;
  grid_launch_dependents();
  grid_dependency_wait();
  uint4 data[N];
  float scale[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t row = first + 4 * i;
    data[i] = make_uint4(0u, 0u, 0u, 0u);
    scale[i] = 0.f;
    if (row < rows) {
      const int64_t t = p.h_kv == 1 ? row : row / p.h_kv;
      const int h = int(row - t * p.h_kv);
      const int64_t slot = __ldcg(reinterpret_cast<const long long *>(p.slots) + t);
      if (slot >= 0 && slot < p.num_slots) {
        const int64_t src = (slot * p.h_kv + h) * (kD / 8) + c;
        if constexpr (kFp8) {
          const uint2 u = __ldcg(static_cast<const uint2 *>(p.cache) + src);
          data[i].x = u.x;
          data[i].y = u.y;
          scale[i] = __ldcg(p.scale + h * p.num_slots + slot);
        } else {
          data[i] = __ldcg(static_cast<const uint4 *>(p.cache) + src);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t row = first + 4 * i;
    if (row < rows) {
      const int64_t t = p.h_kv == 1 ? row : row / p.h_kv;
      const int h = int(row - t * p.h_kv);
      uint4 o = data[i];
      if constexpr (kFp8)
        o = make_uint4(e4m3x2_scaled(uint16_t(data[i].x), scale[i]), e4m3x2_scaled(uint16_t(data[i].x >> 16), scale[i]),
                       e4m3x2_scaled(uint16_t(data[i].y), scale[i]), e4m3x2_scaled(uint16_t(data[i].y >> 16), scale[i]));
      *reinterpret_cast<uint4 *>(p.out + t * p.o_t + h * p.o_h + 8 * c) = o;
    }
  }
}

template <bool kFp8>
static cudaError_t launch_cache_read_typed(const CacheReadParams &p, cudaStream_t stream) {
  const int64_t rows = p.tokens * p.h_kv;
  if (rows <= 4 * 296) return launch_early(cache_read_kernel<kFp8, 4>, dim3(unsigned((rows + 3) / 4)), dim3(kReadThreads), 0, stream, p);
  return launch_early(cache_read_kernel<kFp8, 16>, dim3(unsigned((rows + 15) / 16)), dim3(kReadThreads), 0, stream, p);
}

cudaError_t launch_cache_read(const CacheReadParams &p, cudaStream_t stream) {
  return p.scale ? launch_cache_read_typed<true>(p, stream) : launch_cache_read_typed<false>(p, stream);
}

}  // namespace pagedmla
