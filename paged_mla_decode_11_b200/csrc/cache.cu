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
// Both move each byte once, so HBM bounds a long call and the launch a short one.  Rows with a slot
// outside the pool are skipped by the write and read as zeros.
//
// Measured (B200, calls, scattered slots): write of 64 rows 3.6 us (bf16, 1.9 in a graph) and 3.7 us (FP8,
// 2.1); of 65,521 rows into the FP8 cache (114 MB) 25.7 us, 0.68 of the copy rate, and into the bf16 cache
// (151 MB) 28.8 us, 0.80.  Read of 7,777 bf16 rows (18 MB) 3.8 us; of 65,521 FP8 rows (114 MB) 20.4 us, 0.85
// of the copy rate.  Slots of 64 tokens 2.5 us and of 65,521 (1.3 MB) 3.1 us in a graph: launch and round trips.
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
// memory: two warp reductions per row.  A long call is bound by the row's arithmetic, a
// chain of two reductions and the conversions (about 270 instructions a row, issue slots 57% busy, fixed
// latencies the main stall), not by its bytes: a warp therefore takes
// several rows, keeps the weight and its pair's frequency in registers while cp.async brings the next
// rows to shared memory; products run two to an instruction; and a row is divided by its scale with
// one division (below).  65,521 rows: 43 us with a warp per row and 18 divisions, 34 us with rows in a
// loop and the next one in registers, 24.5 us with the ring (25.2 us four rows deep, 30 us at 8 blocks
// an SM, whose 64 registers spill).
// ------------------------------------------------------------------------------------
constexpr int kWriteWarps = 4, kWriteBlocks = 7;  // warps a block, blocks an SM
constexpr int kWriteAhead = 3;                     // rows of a warp in shared memory

__device__ __forceinline__ uint32_t e4m3x2(float2 v) { return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3); }

// Two neighbouring elements.
__device__ __forceinline__ float2 pair_to_float(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_to_float(uint32_t w, __half) { return __half22float2(*reinterpret_cast<__half2 *>(&w)); }

// Rows on their way to a warp: a ring of kWriteAhead rows in shared memory, filled by cp.async.
template <typename T>
struct WriteRing {
  static constexpr int VEC = 16 / sizeof(T), NV = 16 / VEC;          // a lane's 16-byte accesses of a row
  static constexpr int kRow = kD * sizeof(T);                        // bytes
  static constexpr int kWarp = kWriteAhead * kRow;
  static constexpr int kSmem = kWriteWarps * kWarp;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A lane's 16 columns, 16 bytes at a time from `words` (shared memory or parameters).
template <typename T>
__device__ __forceinline__ void widen16(const uint4 *words, int lane, float2 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < WriteRing<T>::NV; ++i) {
    const uint4 raw = words[i * 32 + lane];
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (sizeof(T) == 4) {
      v[2 * i] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
      v[2 * i + 1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[4 * i + k] = pair_to_float(w[k], T());
    }
  }
}

template <typename T, bool kFp8, bool kNorm>
__global__ void __launch_bounds__(kWriteWarps * 32, kWriteBlocks) cache_write_kernel(const CacheWriteParams p) {
  using Ring = WriteRing<T>;
  constexpr int VEC = Ring::VEC, NV = Ring::NV;
  extern __shared__ __align__(16) uint8_t write_smem[];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int h = blockIdx.y;
  const int64_t step = int64_t(gridDim.x) * kWriteWarps;
  int64_t t = int64_t(blockIdx.x) * kWriteWarps + warp;
  grid_launch_dependents();
  grid_dependency_wait();
  if (t >= p.tokens) return;
  uint8_t *ring = write_smem + warp * Ring::kWarp;
  const uint32_t ring_at = smem_u32(ring);

  // the source of the next copy, moved on by a step each time
  int64_t copy_t = t;
  const T *lat = static_cast<const T *>(p.latent) + t * p.l_t + h * p.l_h + lane * VEC;
  const T *rp = static_cast<const T *>(p.rope) + t * p.r_t + h * p.r_h + lane * VEC;
  const int64_t lat_step = step * p.l_t, rope_step = step * p.r_t;
  auto copy_row = [&](int stage) {
    if (copy_t < p.tokens) {
      const uint32_t dst = ring_at + stage * Ring::kRow + lane * 16;
#pragma unroll
      for (int i = 0; i < NV; ++i) copy16(dst + i * 512, lat + i * 32 * VEC);
      if (lane < 64 / VEC) copy16(dst + kDV * sizeof(T), rp);
      copy_t += step;
      lat += lat_step;
      rp += rope_step;
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kWriteAhead - 1; ++i) copy_row(i);

  const int c0 = p.half ? lane : 2 * lane, c1 = p.half ? lane + 32 : c0 + 1;  // this lane's rope pair
  float2 weight[8];
  if constexpr (kNorm) widen16<T>(static_cast<const uint4 *>(p.weight), lane, weight);
  const double turns = p.inv_freq ? rope_turns(__ldg(p.inv_freq + lane)) : 0.0;
  const uint32_t row_columns = uint32_t(p.h_kv) * kD;  // of a token in the cache
  const uint32_t head_columns = uint32_t(h) * kD;
  float *scales = p.scale + h * p.num_slots;
  uint32_t slots = 0;  // of rows t + lane * step for 32 rows, checked (slots are below 2^31; ~0: skip)
  double places = 0.0;
  for (int it = 0, stage = 0; t < p.tokens; t += step, ++it, stage = stage + 1 == kWriteAhead ? 0 : stage + 1) {
    if (it % 32 == 0) {
      const int64_t mine = t + lane * step;
      slots = ~0u;
      if (mine < p.tokens) {
        const int64_t s = __ldcg(reinterpret_cast<const long long *>(p.slots) + mine);
        if (s >= 0 && s < p.num_slots) slots = uint32_t(s);
        if (p.inv_freq) places = load_position(p.positions, p.pos64, mine);
      }
    }
    __syncwarp();  // every lane has read the stage that is filled next
    copy_row(stage == 0 ? kWriteAhead - 1 : stage - 1);
    copies_wait<kWriteAhead - 1>();
    __syncwarp();
    const uint32_t slot = __shfl_sync(0xffffffffu, slots, it % 32);
    const double pos = __shfl_sync(0xffffffffu, places, it % 32);
    if (slot == ~0u) continue;
    const T *row = reinterpret_cast<const T *>(ring + stage * Ring::kRow);
    float2 v[8];
    widen16<T>(reinterpret_cast<const uint4 *>(row), lane, v);
    float2 r = make_float2(to_float(row[kDV + c0]), to_float(row[kDV + c1]));
    if (p.inv_freq) {
      const float2 w = rope_cos_sin(pos, turns, p.magnitude, false);
      r = make_float2(r.x * w.x - r.y * w.y, r.x * w.y + r.y * w.x);
    }
    float inv = 1.f;  // of the latent columns: v * inv is the row (applied below)
    if constexpr (kNorm) {
      float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) s2 = fma2(v[i], v[i], s2);
      float ss = s2.x + s2.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      inv = rsqrtf(ss * (1.f / kDV) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], weight[i]);
    }
    const uint64_t at = uint64_t(slot) * row_columns + head_columns;
    if constexpr (!kFp8) {
      if constexpr (kNorm)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], make_float2(inv, inv));
      __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.cache) + at;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        uint32_t w[VEC / 2];
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) w[k] = pack_bf16x2(v[i * VEC / 2 + k].x, v[i * VEC / 2 + k].y);
        if constexpr (VEC == 8)
          *reinterpret_cast<uint4 *>(dst + (i * 32 + lane) * VEC) = make_uint4(w[0], w[1], w[2], w[3]);
        else
          *reinterpret_cast<uint2 *>(dst + (i * 32 + lane) * VEC) = make_uint2(w[0], w[1]);
      }
      if (p.half) {
        dst[kDV + c0] = __float2bfloat16_rn(r.x);
        dst[kDV + c1] = __float2bfloat16_rn(r.y);
      } else {
        *reinterpret_cast<uint32_t *>(dst + kDV + c0) = pack_bf16x2(r.x, r.y);
      }
    } else {
      // largest magnitude of the row; fmaxf passes over NaN, which become NaN codes by themselves
      float lmax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) lmax = fmaxf(lmax, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
      // non-negative floats order as their bit patterns
      auto warp_max = [](float m) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))); };
      float amax = warp_max(fmaxf(lmax * inv, fmaxf(fabsf(r.x), fabsf(r.y))));
      const bool finite = amax <= 3.402823466e38f;
      if (!finite) {
        // E4M3 has no infinity: infinities become NaN codes too and do not enter the scale
        amax = 0.f;
        auto see = [&](float &x, float f) {
          const float m = fabsf(x * f);
          if (m <= 3.402823466e38f)
            amax = fmaxf(amax, m);
          else
            x = __int_as_float(0x7fffffff);
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          see(v[i].x, inv);
          see(v[i].y, inv);
        }
        see(r.x, 1.f);
        see(r.y, 1.f);
        amax = warp_max(amax);
      }
      float scale = amax / 448.f;
      if (scale == 0.f) scale = 1.f;
      const float y = 1.f / scale;
      if (!finite || amax < 1e-24f) {  // 1 / scale, or a rest below, could leave the normal range
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = make_float2(v[i].x * inv / scale, v[i].y * inv / scale);
        r = make_float2(r.x / scale, r.y / scale);
      } else if constexpr (kNorm) {
        // within 2^-21 of the quotient: another code only where that lies so close to the middle of two
        const float f = inv * y;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], make_float2(f, f));
        r = mul2(r, make_float2(y, y));
      } else {
        // Rows as given hold values of few bits, whose quotients often lie exactly in the middle of two
        // codes; a product with 1 / scale would round many of those to the wrong side.  With y the
        // correctly rounded 1 / b and q = a y, the rest a - q b is exact in an FMA and q + y (a - q b)
        // is the correctly rounded quotient (P. Markstein, "Computation of elementary functions on the
        // IBM RISC System/6000 processor", 1990).
        const float2 y2 = make_float2(y, y), nb = make_float2(-scale, -scale);
        auto quotient = [&](float2 a) {
          const float2 q = mul2(a, y2);
          return fma2(fma2(q, nb, a), y2, q);
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = quotient(v[i]);
        r = quotient(r);
      }
      uint8_t *dst = static_cast<uint8_t *>(p.cache) + at;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) w[k] = e4m3x2(v[i * VEC / 2 + 2 * k]) | e4m3x2(v[i * VEC / 2 + 2 * k + 1]) << 16;
        if constexpr (VEC == 8)
          *reinterpret_cast<uint2 *>(dst + (i * 32 + lane) * VEC) = make_uint2(w[0], w[1]);
        else
          *reinterpret_cast<uint32_t *>(dst + (i * 32 + lane) * VEC) = w[0];
      }
      const uint32_t rc = e4m3x2(r);
      if (p.half) {
        dst[kDV + c0] = uint8_t(rc);
        dst[kDV + c1] = uint8_t(rc >> 8);
      } else {
        *reinterpret_cast<uint16_t *>(dst + kDV + c0) = uint16_t(rc);
      }
      if (lane == 0) scales[slot] = scale;
    }
  }
}

template <typename T, bool kFp8>
static cudaError_t launch_cache_write_typed(const CacheWriteParams &p, cudaStream_t stream) {
  // one row a warp while the rows fit on the chip at once, then a resident grid
  const int64_t resident = std::max(148 * kWriteBlocks / p.h_kv, 1);
  const dim3 grid(unsigned(std::min((p.tokens + kWriteWarps - 1) / kWriteWarps, resident)), unsigned(p.h_kv));
  constexpr int kSmem = WriteRing<T>::kSmem;
  return p.weight ? launch_early(cache_write_kernel<T, kFp8, true>, grid, dim3(kWriteWarps * 32), kSmem, stream, p)
                  : launch_early(cache_write_kernel<T, kFp8, false>, grid, dim3(kWriteWarps * 32), kSmem, stream, p);
}

cudaError_t launch_cache_write(const CacheWriteParams &p, int dtype, cudaStream_t stream) {
  const bool fp8 = p.scale != nullptr;
  switch (dtype) {
    case MLA_DTYPE_BF16:
      return fp8 ? launch_cache_write_typed<__nv_bfloat16, true>(p, stream) : launch_cache_write_typed<__nv_bfloat16, false>(p, stream);
    case MLA_DTYPE_F16:
      return fp8 ? launch_cache_write_typed<__half, true>(p, stream) : launch_cache_write_typed<__half, false>(p, stream);
    default:
      return fp8 ? launch_cache_write_typed<float, true>(p, stream) : launch_cache_write_typed<float, false>(p, stream);
  }
}

// ------------------------------------------------------------------------------------
// Read: a warp takes four rows, 4 x 72 units of eight columns (a 16-byte store; a 16- or 8-byte
// load): nine units a lane, all loads issued before the first store.
// ------------------------------------------------------------------------------------
constexpr int kReadWarps = 4, kReadRows = 4, kReadUnits = kD / 8;

__device__ __forceinline__ uint32_t e4m3x2_scaled(uint16_t codes, float scale) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(codes, __NV_E4M3);  // exact
  const float2 f = __half22float2(__half2(h));
  return pack_bf16x2(f.x * scale, f.y * scale);
}

template <bool kFp8>
__global__ void __launch_bounds__(kReadWarps * 32) cache_read_kernel(const CacheReadParams p) {
  constexpr int N = kReadRows * kReadUnits / 32;
  const int lane = threadIdx.x % 32;
  const int64_t first = (int64_t(blockIdx.x) * kReadWarps + threadIdx.x / 32) * kReadRows, rows = p.tokens * p.h_kv;
  grid_launch_dependents();
  grid_dependency_wait();
  if (first >= rows) return;
  // lane l (mod 4) keeps row first + l: its place in the cache (-1: none), in out, and its scale
  const int64_t mine = first + lane % kReadRows;
  int64_t src = -1, dst = -1;
  float scale = 0.f;
  if (mine < rows) {
    const int64_t t = p.h_kv == 1 ? mine : mine / p.h_kv;
    const int h = int(mine - t * p.h_kv);
    dst = t * p.o_t + h * p.o_h;
    const int64_t slot = __ldcg(reinterpret_cast<const long long *>(p.slots) + t);
    if (slot >= 0 && slot < p.num_slots) {
      src = (slot * p.h_kv + h) * kReadUnits;
      if (kFp8) scale = __ldcg(p.scale + h * p.num_slots + slot);
    }
  }
  uint4 data[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int u = lane + 32 * i, r = u / kReadUnits;
    const int64_t at = __shfl_sync(0xffffffffu, src, r);
    data[i] = make_uint4(0u, 0u, 0u, 0u);
    if (at >= 0) {
      if constexpr (kFp8) {
        const uint2 c = __ldcg(static_cast<const uint2 *>(p.cache) + at + u - r * kReadUnits);
        data[i].x = c.x;
        data[i].y = c.y;
      } else {
        data[i] = __ldcg(static_cast<const uint4 *>(p.cache) + at + u - r * kReadUnits);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int u = lane + 32 * i, r = u / kReadUnits;
    const int64_t to = __shfl_sync(0xffffffffu, dst, r);
    uint4 o = data[i];
    if constexpr (kFp8) {
      const float s = __shfl_sync(0xffffffffu, scale, r);
      o = make_uint4(e4m3x2_scaled(uint16_t(data[i].x), s), e4m3x2_scaled(uint16_t(data[i].x >> 16), s),
                     e4m3x2_scaled(uint16_t(data[i].y), s), e4m3x2_scaled(uint16_t(data[i].y >> 16), s));
    }
    if (to >= 0) *reinterpret_cast<uint4 *>(p.out + to + 8 * (u - r * kReadUnits)) = o;
  }
}

cudaError_t launch_cache_read(const CacheReadParams &p, cudaStream_t stream) {
  const int64_t rows = p.tokens * p.h_kv;
  const dim3 grid(unsigned((rows + kReadWarps * kReadRows - 1) / (kReadWarps * kReadRows)));
  return p.scale ? launch_early(cache_read_kernel<true>, grid, dim3(kReadWarps * 32), 0, stream, p)
                 : launch_early(cache_read_kernel<false>, grid, dim3(kReadWarps * 32), 0, stream, p);
}

}  // namespace pagedmla
