// Rotary positions: of every (token, head) row x[0 .. width), the last 2n columns are n pairs,
// and pair i is turned by the angle a = position * inv_freq[i]:
//   y0 = m (x0 cos a - x1 sin a),   y1 = m (x0 sin a + x1 cos a)
// (m: the magnitude of scaled frequencies; inverse: a -> -a, which is also the gradient, the
// transposed map).  Pairs are columns (2i, 2i + 1) or, in the half layout, (i, i + n).  The
// columns in front of them pass through.
//
// Every element is read and written once, so HBM bounds the kernel.  A block takes a tile of
// tokens x heads: it computes the angles of its tokens once into shared memory (fp64, so a
// per-element angle would cost more than the memory traffic) and shares them over the tile's
// heads.  A thread moves 16 bytes of each member of its pairs at a time; when a size, stride or
// address is not a multiple of that it moves one pair at a time.  Columns are rotated in fp32
// and rounded once.
//
// Measured (B200): 128 tokens x 128 heads x 64 bf16 columns (4.2 MB) 2.8 us in a graph, 4.1 as a call;
// 4,093 x 128 x 192 (402 MB) 67.8 us in a graph, 69.5 as a call, 0.88 of the copy rate; moved one element
// at a time 257 x 16 x 600 (9.9 MB) 16.9 us.  The large size took 77 us
// with ordinary stores (results push inputs out of L2), 97 us with blocks of 512 threads and 86 us with
// two units a thread (64 registers, fewer blocks).
#include "launch.h"
#include "rope.cuh"

namespace pagedmla {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxAngles = 1024;  // per block (8 KB of shared memory)

// Each unit is VEC pairs, two accesses of VEC elements.  A tile has one of them a thread, or the units
// of a single row where those are more: with kRopeMaxPairs pairs moved one at a time two a thread.  The
// units are read first, so that the angles are computed while they are on their way.
template <int VEC>
constexpr int kRopeUnits = (kRopeMaxPairs / VEC + kRopeThreads - 1) / kRopeThreads;

template <typename T, bool kHalf, int VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  static_assert(kRopeMaxPairs <= kRopeMaxAngles, "the angles of one token fit");
  constexpr int kUnits = kRopeUnits<VEC>;
  __shared__ float2 cs[kRopeMaxAngles];
  using V = Pack<T, VEC>;
  const int64_t t0 = int64_t(blockIdx.x) * p.tile_tokens;
  const int h0 = blockIdx.y * p.tile_heads;
  const int nt = int(min(int64_t(p.tile_tokens), p.tokens - t0)), nh = min(p.tile_heads, p.heads - h0);
  const int n = p.pairs, units = n / VEC;
  const int front = p.width - 2 * n;  // columns that pass through
  grid_launch_dependents();
  grid_dependency_wait();
  const T *x = static_cast<const T *>(p.x);
  T *out = static_cast<T *>(p.out);
  const int total = nt * nh * units;
  V a[kUnits], b[kUnits];
  auto place = [&](int i, int &lt, int &h, int &u, int &c0, int &c1) {
    const int r = i / units;
    u = i - r * units;
    lt = r / nh;
    h = h0 + r - lt * nh;
    c0 = front + (kHalf ? u * VEC : 2 * u * VEC);
    c1 = kHalf ? c0 + n : c0 + VEC;
  };
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int i = threadIdx.x + k * kRopeThreads;
    if (i < total) {
      int lt, h, u, c0, c1;
      place(i, lt, h, u, c0, c1);
      const T *src = x + (t0 + lt) * p.x_t + h * p.x_h;
      a[k] = load_cg(reinterpret_cast<const V *>(src + c0));
      b[k] = load_cg(reinterpret_cast<const V *>(src + c1));
    }
  }
  if (p.copy_front) {
    const int fv = front / VEC, all = nt * nh * fv;
#pragma unroll 4
    for (int i = threadIdx.x; i < all; i += kRopeThreads) {
      const int r = i / fv, c = (i - r * fv) * VEC;
      const int64_t t = t0 + r / nh;
      const int h = h0 + r % nh;
      store_cs(reinterpret_cast<V *>(out + t * p.o_t + h * p.o_h + c),
               load_cg(reinterpret_cast<const V *>(x + t * p.x_t + h * p.x_h + c)));
    }
  }
  for (int i = threadIdx.x; i < nt * n; i += kRopeThreads)
    cs[i] = rope_cos_sin(load_position(p.positions, p.pos64, t0 + i / n), rope_turns(__ldg(p.inv_freq + i % n)),
                         p.magnitude, p.inverse);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int i = threadIdx.x + k * kRopeThreads;
    if (i >= total) break;
    int lt, h, u, c0, c1;
    place(i, lt, h, u, c0, c1);
    const float2 *w = cs + lt * n + u * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      // pair j of the unit: members a[j], b[j], or neighbours of the 2 VEC columns of a and b
      T &m0 = kHalf ? a[k].v[j] : (2 * j < VEC ? a[k].v[2 * j] : b[k].v[2 * j - VEC]);
      T &m1 = kHalf ? b[k].v[j] : (2 * j + 1 < VEC ? a[k].v[2 * j + 1] : b[k].v[2 * j + 1 - VEC]);
      const float x0 = to_float(m0), x1 = to_float(m1);
      m0 = from_float<T>(x0 * w[j].x - x1 * w[j].y);
      m1 = from_float<T>(x0 * w[j].y + x1 * w[j].x);
    }
    T *dst = out + (t0 + lt) * p.o_t + h * p.o_h;
    store_cs(reinterpret_cast<V *>(dst + c0), a[k]);
    store_cs(reinterpret_cast<V *>(dst + c1), b[k]);
  }
}

template <typename T, bool kHalf>
static cudaError_t launch_rope_typed(const RopeParams &p, bool wide, cudaStream_t stream) {
  constexpr int kVec = 16 / sizeof(T);
  const dim3 grid(unsigned((p.tokens + p.tile_tokens - 1) / p.tile_tokens),
                  unsigned((p.heads + p.tile_heads - 1) / p.tile_heads));
  return wide ? launch_early(rope_kernel<T, kHalf, kVec>, grid, dim3(kRopeThreads), 0, stream, p)
              : launch_early(rope_kernel<T, kHalf, 1>, grid, dim3(kRopeThreads), 0, stream, p);
}

cudaError_t launch_rope(RopeParams p, int dtype, bool half, cudaStream_t stream) {
  const int size = dtype == MLA_DTYPE_F32 ? 4 : 2, vec = 16 / size;
  auto multiple = [&](int64_t v) { return v % vec == 0; };
  const bool wide = multiple(p.pairs) && multiple(p.width) && multiple(p.x_t) && multiple(p.x_h) && multiple(p.o_t) &&
                    multiple(p.o_h) && reinterpret_cast<uintptr_t>(p.x) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
  // a tile of heads, then of tokens, of one unit a thread, but of a row at least
  const int units = wide ? p.pairs / vec : p.pairs;
  p.tile_heads = std::max(1, std::min(p.heads, kRopeThreads / units));
  p.tile_tokens = std::max(1, std::min(kRopeThreads / (units * p.tile_heads), kRopeMaxAngles / p.pairs));
  switch (dtype) {
    case MLA_DTYPE_BF16:
      return half ? launch_rope_typed<__nv_bfloat16, true>(p, wide, stream)
                  : launch_rope_typed<__nv_bfloat16, false>(p, wide, stream);
    case MLA_DTYPE_F16:
      return half ? launch_rope_typed<__half, true>(p, wide, stream) : launch_rope_typed<__half, false>(p, wide, stream);
    default:
      return half ? launch_rope_typed<float, true>(p, wide, stream) : launch_rope_typed<float, false>(p, wide, stream);
  }
}

}  // namespace pagedmla
