// Rotary angles, shared by the rotary kernel and the cache writer, and the element types
// their inputs may have.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace pagedmla {

// A pair's frequency in turns per position.
__device__ __forceinline__ double rope_turns(double inv_freq) { return inv_freq * 0.15915494309189533577; }  // 1 / (2 pi)

// (cos, sin) of position * frequency, times the magnitude.  The turns are counted and reduced in
// fp64: at position 10^6 the angle of the fastest pair is 10^6 radians, and an fp32 product would
// be off by up to 0.03.  The reduced half turn in [-1, 1] goes to sincospif, so the angle's total
// error stays near 10^-7 at any position (of up to 2^50 turns).
__device__ __forceinline__ float2 rope_cos_sin(double position, double turns_per_position, float magnitude, bool inverse) {
  const double turns = position * turns_per_position;
  constexpr double kRound = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to a whole number
  const double whole = __dadd_rn(__dadd_rn(turns, kRound), -kRound);
  float s, c;
  sincospif(2.f * float(turns - whole), &s, &c);
  s *= magnitude;
  return make_float2(c * magnitude, inverse ? -s : s);
}

// Positions, slots, activations and cache rows may come from the kernel just before, which may
// still have been running when this one started: they are read through L2 (ld.global.cg).
__device__ __forceinline__ double load_position(const void *positions, bool is64, int64_t i) {
  return is64 ? double(__ldcg(static_cast<const long long *>(positions) + i))
              : double(__ldcg(static_cast<const int *>(positions) + i));
}

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// N elements of T moved as one access (16 bytes, or a single element).
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

template <int kBytes>
struct WordOf;
template <>
struct WordOf<2> { using type = unsigned short; };
template <>
struct WordOf<4> { using type = unsigned int; };
template <>
struct WordOf<8> { using type = uint2; };
template <>
struct WordOf<16> { using type = uint4; };

// One access of a value's own size and alignment through L2.
template <typename V>
__device__ __forceinline__ V load_cg(const V *ptr) {
  using W = typename WordOf<sizeof(V)>::type;
  const W w = __ldcg(reinterpret_cast<const W *>(ptr));
  return *reinterpret_cast<const V *>(&w);
}

// The same as a streaming store (evicted from L2 first): results larger than L2 then do not push out
// inputs that are still to be read.
template <typename V>
__device__ __forceinline__ void store_cs(V *ptr, const V &v) {
  using W = typename WordOf<sizeof(V)>::type;
  __stcs(reinterpret_cast<W *>(ptr), *reinterpret_cast<const W *>(&v));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
  return d;
}

}  // namespace pagedmla
