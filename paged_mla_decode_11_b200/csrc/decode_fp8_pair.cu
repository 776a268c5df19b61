// Paged MLA decode over an FP8 latent cache for more than 16 query rows per latent head, on CTA
// pairs (tcgen05 cta_group::2, kind::f8f6f4).  Cache format and results as in decode_fp8.cu: the
// row a token contributes is k_scale * e4m3(code).
//
// Both products run on the codes as they are, without widening them, by splitting the other
// operand into two 8-bit terms whose sum keeps it:
//   q = 2^-a (q_hi + q_lo)    a the row's own power of two (largest |q| in [128, 256)), q_hi the
//                             nearest E4M3 value and q_lo, E4M3, the rest.  A bf16 value has 8
//                             significant bits and E4M3 4, in steps of 2^-9 at least: the sum is exact
//                             from 2^-2 on, for every |q| of 2^-9 of the row's largest, and below off by
//                             at most 2^-10, 2^-17 of the largest
//   P s = 2^u (v_hi + v_lo)  s the key's scale, u the row's own: its largest P s so far is in [2^6, 2^8]
//                             units.  v_hi is the nearest E4M3 value, v_lo the rest in E5M2.  For v in
//                             [2^k, 2^(k+1)) the rest is at most 2^(k-4) and E5M2's half step below that
//                             2^(k-8): within 2^-8 of the value, as a bf16 rounding of P is, while
//                             v >= 2^-6 (and 2^-11, as both start from v in f16); below, within 2^-14,
//                             that is 2^-20 of the row's largest.  (A
//                             unit of the largest scale alone would let a key of no weight in the row,
//                             such as a row of zeros, which the writer stores with scale 1, push all
//                             others below 2^-14)
// so S = (q_hi K^T + q_lo K^T) 2^-a s and O = v_hi V + v_lo V take twice the products at twice the
// bf16 rate, on half the bytes.  Sums are fp32 in tensor memory.
//
// One CTA pair takes 128 query rows (64 per CTA; rows past R are masked).  Per group of two pages
// (128 keys), as in decode_pair.cu: CTA c of the pair loads page c of the group whole; S has
// M = 128 rows and N = 128 keys, row r's scores for the first page on lane r of tensor memory and
// for the second on lane 64 + r.  After the score, CTA 0 holds value columns 0-255 and CTA 1 columns
// 256-511 of both pages: each loads the partner page's half (an L2 hit) over blocks it no longer
// needs, at the offsets where its partner keeps the same keys.  O has N = 256 value columns, twice.
//
// A page of codes takes 40 KB of shared memory (five blocks of 64 tokens x 128 columns), so three
// groups fit beside the query instead of the bf16 kernel's two, and three score buffers beside the
// output in tensor memory: the partner's load and the softmax of a group hide behind the next two
// groups' scores.
//
// Measured (B200): 128 sequences x 128 heads x 4,096 tokens 155 us in short runs (941 TFLOP/s of the
// formula's flops) and 179 us under the sustained power cap (SM clock 1.6 GHz), where the products'
// energy sets the clock; 198 us with plan and combine; the bf16 kernel takes 195 to 205 us.  A group takes
// about 3,640 cycles, of which its products are issued in 2,280.  What is waited for is the way round of a
// ring stage, 10,800 cycles for the three groups in flight: page load 2,500, score 1,820, softmax 2,700 (of
// which rescaling O takes 770 in two groups of three), the issuing warp's turn 1,320, PV and the producer's
// turn 2,480.
// Kept on the way from 284 us with plan and combine: eight softmax warps instead of four, issue warps
// that run converged so that descriptors stay uniform (an MMA issued from a divergent lane took 100
// cycles instead of 45), barriers polled together, six query loaders that split ahead, output rows
// transposed between lanes before they are stored, the A tile of PV kept in the operand buffer for its
// second half and the scales in registers (sustained, with the combine, 193.8 to 191.6 to 190.5 us).  Measured slower: register splits for the loaders (setmaxnreg,
// which spilled), all warps loading the first query, one-lane polls, an L2 prefetch, a fixed order of
// score and PV with blocking waits (206), barriers polled between the MMAs (204), score and PV issued
// by two warps (198), paired fp32 arithmetic in the softmax (194.5), looped instead of unrolled MMAs (198).
// The unit of v by row (see above) costs 2.7% against one of the largest scale (with plan and combine, in
// turn, 170.8 -> 175.4 us; 33 ragged sequences of two tokens 68.0 -> 71.2); rescaling O takes 4% of either.
// The score's maxima and the largest P s exchanged one after the other took 180.2, both behind a barrier
// that tells whether any thread needs them 178.8 to 211.
//
// Shared memory (per CTA, 8 KB blocks of 64 rows x 128 bytes, 128-byte swizzle):
//   ring: 3 stages x 6 slots: slots 0-4 the own page's column blocks; after the score CTA 0 reloads
//         slots 2-3 with the partner page's blocks 0-1 and CTA 1 slots 0-1 with its blocks 2-3; slot
//         4 (rope, free after the score) takes v_hi and slot 5 v_lo (64 rows x 128 keys)
//   query: q_hi column blocks 0-3, q_lo blocks 0-3, and one block of both rope halves
// Tensor memory (512 columns): O (value halves at 0 and 128), S at 256, 320 and 384.
//
// Warp roles (both CTAs):
//   warp 0      producer: own pages and the group's key scales, the partner page's value half (an L2
//               prefetch of the pages ahead measured slower: 162 against 153 us)
//   warp 1      tensor-memory owner; in CTA 0 the MMA issuer (one thread)
//   warps 2-9   softmax, O rescale and epilogue: lane l of sub-partition q owns row (32 q + l) mod 64
//               and half q / 2 (keys of that page; value columns 256 (q / 2) + 0..255), of which the
//               two warps of a sub-partition take 32 keys and 128 columns each.  Splitting P is the
//               longest stage: one warp per sub-partition took 3.0 us a group, against 1.6 us of MMAs
//   warps 10-15 query loaders: 11 rows each (9 the last), split into q_hi and q_lo and held in registers
//               until the previous query tile is free
// Every wait is bounded.
#include <cuda_fp8.h>

#include "launch.h"

namespace pagedmla {

namespace {

struct FpPair {
  static constexpr int kThreads = 512;
  static constexpr int BM = 64;                  // query rows per CTA
  static constexpr int kStages = 3;
  static constexpr int kBlock = 64 * 128;        // bytes of a block
  static constexpr int kPageBlocks = 5;          // column blocks of a page (the last one half filled)
  static constexpr int kSlots = kPageBlocks + 1;
  static constexpr int kLoaders = 6, kLoadRows = 11;  // warps, and query rows of a warp
  static constexpr int kQScales = 8;             // row-scale buffers, by piece
  static constexpr int kOffRing = 0;
  static constexpr int kOffQ = kOffRing + kStages * kSlots * kBlock;
  static constexpr int kOffX = kOffQ + 9 * kBlock;            // row-max exchange [2][4][64], row sums [4][64]
  static constexpr int kOffSc = kOffX + (8 + 4) * 64 * 4;     // key scales [stage][128]
  static constexpr int kOffQSc = kOffSc + kStages * 128 * 4;  // row scales [8][64]
  enum {
    FULL = 0, VFULL = FULL + kStages, EMPTY = VFULL + kStages, SFULL = EMPTY + kStages, SFREE = SFULL + kStages,
    PFULL = SFREE + kStages, SCALES = PFULL + kStages, QSC = SCALES + kStages, OFULL = QSC + kQScales,
    OFREE = OFULL + 1, QFULL = OFREE + 1, QFREE = QFULL + 1, FINAL = QFREE + 1, NBARS = FINAL + 1
  };
  static constexpr int kOffBar = kOffQSc + kQScales * 64 * 4;
  static constexpr int kOffTmem = kOffBar + NBARS * 8;
  static constexpr int kOffAbort = kOffTmem + 8;
  static constexpr int kSmemBytes = kOffAbort + 8 + 1024;     // + slack for 1 KB alignment
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kTmemO = 0;          // value halves v at 128 v
  static constexpr uint32_t kTmemS = 256;        // score buffers at 256 + 64 stage
  static constexpr uint32_t kOwnBytes = kPageBlocks * kBlock;  // a page (its last block's fill counts)
  static constexpr uint32_t kHalfVBytes = 2 * kBlock;          // half of a page's values
  static_assert(kOffQ % 1024 == 0, "swizzled tiles need 1 KB alignment");
  static_assert(kTmemS + 64 * kStages <= kTmemCols, "tensor memory");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// ------------------------------------------------------------------------------------
// CTA-pair helpers.
// ------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Cluster address of the same shared-memory offset in CTA 0 of the pair.
__device__ __forceinline__ uint32_t map_cta0(uint32_t local) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(local));
  return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// TMA load into this CTA's shared memory, its bytes counted on a barrier of CTA 0.
__device__ __forceinline__ void load_for_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar_cluster, int c0, int c1,
                                              int c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

// The same of a page's value columns (page_map: all four blocks; half_map: columns 256 half + 0..255;
// both over columns of a block, tokens, blocks, latent heads), stored block after block.
__device__ __forceinline__ void load_blocks_for_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar_cluster,
                                                     int token, int head, int half, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(0), "r"(token), "r"(2 * half), "r"(head),
      "l"(policy)
      : "memory");
}

// Instruction descriptor of kind::f8f6f4 with fp32 D and E4M3 B; A is E4M3, or E5M2 (a_e5m2).
__device__ constexpr uint32_t idesc_f8(int M, int N, bool a_e5m2, bool b_mn_major) {
  return (1u << 4) | (uint32_t(a_e5m2) << 7) | (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
}

// The issuing warp runs converged and one elected lane (the same each time) issues: descriptors
// that are uniform over the warp stay in uniform registers.
__device__ __forceinline__ void mma_f8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Two products of one A tile, d0 by b0 and d1 by b1: the first keeps A in the tensor cores' operand
// buffer for the second, which saves a third of its reads of shared memory.
__device__ __forceinline__ void mma_f8_pair_twice(uint32_t d0, uint32_t d1, uint64_t a, uint64_t b0, uint64_t b1,
                                                  uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %6, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f8f6f4.collector::a::fill [%0], %2, %3, %5, p;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f8f6f4.collector::a::lastuse [%1], %2, %4, %5, p;\n\t}" ::"r"(d0),
      "r"(d1), "l"(a), "l"(b0), "l"(b1), "r"(idesc), "r"(acc)
      : "memory");
}

// Arrive once on the barrier at this offset in both CTAs when all tcgen05 work issued so far by
// the elected lane is done.
__device__ __forceinline__ void commit_both(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\t.reg .pred e;\n\tmov.b16 m, 3;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void tmem_store32(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
      "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
      "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
      : "memory");
}

// Element k of lane l of each group of N neighbouring lanes becomes element l of lane k.
template <int N>
__device__ __forceinline__ void transpose_lanes(uint4 (&u)[N], int lane) {
#pragma unroll
  for (int d = 1; d < N; d <<= 1) {
    const bool upper = (lane & d) != 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(i & d)) {
        uint4 &a = u[i], &b = u[i | d];
        const uint4 send = upper ? a : b;
        uint4 got;
        got.x = __shfl_xor_sync(0xffffffffu, send.x, d);
        got.y = __shfl_xor_sync(0xffffffffu, send.y, d);
        got.z = __shfl_xor_sync(0xffffffffu, send.z, d);
        got.w = __shfl_xor_sync(0xffffffffu, send.w, d);
        if (upper)
          a = got;
        else
          b = got;
      }
  }
}

__device__ __forceinline__ bool all_lanes(bool v) { return __all_sync(0xffffffffu, v); }
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }  // -126 <= e <= 127

// Two values as 8-bit codes (low byte first), and the values of two E4M3 codes.
__device__ __forceinline__ uint32_t to_e4m3x2(__half2 v) {
  return __nv_cvt_halfraw2_to_fp8x2(__half2_raw(v), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t to_e5m2x2(__half2 v) {
  return __nv_cvt_halfraw2_to_fp8x2(__half2_raw(v), __NV_SATFINITE, __NV_E5M2);
}
__device__ __forceinline__ __half2 from_e4m3x2(uint32_t codes) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(codes), __NV_E4M3));
}

// Largest magnitude of eight bf16 values, as its bits (non-negative values order as integers).
__device__ __forceinline__ uint32_t bf16_top(const uint4 &u) {
  const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// A query row's power of two, 2^(7 - (e - 127)) for the biased exponent e of its largest value; a
// row with an infinity or NaN becomes NaN.
__device__ __forceinline__ float row_up(int e) { return e == 255 ? __int_as_float(0x7fffffff) : pow2(134 - e); }

// Eight bf16 values times `up` as E4M3 codes (x, y), and the codes of the rest (z, w).  Between
// 2^-16 and 256 the scaled values are f16 values (smaller ones are off by at most 2^-25).
__device__ __forceinline__ uint4 split_q(const uint4 &u, float up) {
  const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
  uint32_t h[4], lw[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2 x = __floats2half2_rn(__uint_as_float(w4[k] << 16) * up, __uint_as_float(w4[k] & 0xffff0000u) * up);
    h[k] = to_e4m3x2(x);
    lw[k] = to_e4m3x2(__hsub2(x, from_e4m3x2(h[k])));
  }
  return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, lw[0] | lw[1] << 16, lw[2] | lw[3] << 16);
}

// Four values as E4M3 codes, and the rests in E5M2 (through f16: 2^-11 of the value).
__device__ __forceinline__ void split_v(const float (&v)[4], uint32_t &hi, uint32_t &lo) {
  const __half2 x0 = __floats2half2_rn(v[0], v[1]), x1 = __floats2half2_rn(v[2], v[3]);
  const uint32_t h0 = to_e4m3x2(x0), h1 = to_e4m3x2(x1);
  hi = h0 | h1 << 16;
  lo = to_e5m2x2(__hsub2(x0, from_e4m3x2(h0))) | to_e5m2x2(__hsub2(x1, from_e4m3x2(h1))) << 16;
}

// ------------------------------------------------------------------------------------
// Pieces of a part and their groups of two pages.
// ------------------------------------------------------------------------------------
struct Piece {
  int L, t0, t1, ntiles, ngroups;  // the last group may hold one page
};

// One sequence piece of a part, trimmed to the keys the pair's 128 rows can see.
__device__ __forceinline__ Piece piece_of(const DecodeParams &p, const PartCursor &pc, int seq, int prow0) {
  Piece w;
  w.L = p.seqlens[seq];
  w.t0 = seq == pc.bi ? pc.bt : 0;
  w.t1 = seq == pc.ei ? pc.et : w.L;
  if (p.causal) {
    const int last_row = min(p.R - 1, prow0 + 2 * FpPair::BM - 1);
    w.t1 = min(w.t1, w.L - (p.s_q - 1 - last_row / p.g));
  }
  w.ntiles = w.t1 > w.t0 ? (w.t1 - w.t0 + kPage - 1) / kPage : 0;
  w.ngroups = (w.ntiles + 1) / 2;
  return w;
}

// Walks a part's groups in order, with its stage of the ring and that stage's phase.
struct Groups {
  int seq, j, ntiles, ngroups, t0;
  int count, stage, phase;
  bool done;

  __device__ __forceinline__ void seek(const DecodeParams &p, const PartCursor &pc, int prow0, int from) {
    for (seq = from; part_has(pc, seq); ++seq) {
      const Piece w = piece_of(p, pc, seq, prow0);
      if (w.ngroups > 0) {
        j = 0;
        ntiles = w.ntiles;
        ngroups = w.ngroups;
        t0 = w.t0;
        done = false;
        return;
      }
    }
    done = true;
  }
  __device__ __forceinline__ void start(const DecodeParams &p, const PartCursor &pc, int prow0) {
    count = stage = phase = 0;
    seek(p, pc, prow0, pc.bi);
  }
  __device__ __forceinline__ void next(const DecodeParams &p, const PartCursor &pc, int prow0) {
    ++count;
    if (++stage == FpPair::kStages) {
      stage = 0;
      phase ^= 1;
    }
    if (++j == ngroups) seek(p, pc, prow0, seq + 1);
  }
  // The group's two pages; a lone last page stands for both (its second half is masked).  Numbers
  // outside the pool are moved into it: TMA would fill their pages, but scales are plain copies.
  __device__ __forceinline__ void pages(const DecodeParams &p, int num_pages, int &a, int &b) const {
    const int32_t *row = p.block_table + int64_t(seq) * p.bt_stride + t0 / kPage;
    a = min(max(row[2 * j], 0), num_pages - 1);
    b = min(max(row[min(2 * j + 1, ntiles - 1)], 0), num_pages - 1);
  }
};

}  // namespace

// The pair is the cluster's x dimension (grid x = the CTAs of the 128-row blocks, y = parts, z =
// latent heads).
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(FpPair::kThreads, 1)
    decode_fp8_pair_kernel(const __grid_constant__ CUtensorMap k8_map, const __grid_constant__ CUtensorMap page_map,
                           const __grid_constant__ CUtensorMap half_map, const DecodeParams p, const float *__restrict__ k_scale, int num_pages) {
  using T = FpPair;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = int(cta_rank());
  const int part = blockIdx.y, kvh = blockIdx.z;
  const int prow0 = int(blockIdx.x / 2) * 2 * T::BM;  // first row of the pair's 128-row block
  const int crow0 = prow0 + rank * T::BM;             // first row of this CTA
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + T::kOffBar;
  auto bar = [&](int i) { return bar0 + 8u * uint32_t(i); };
  auto bar_cta0 = [&](int i) { return map_cta0(bar(i)); };  // barriers both CTAs arrive on live in CTA 0
  volatile int *abort = reinterpret_cast<volatile int *>(smem + T::kOffAbort);
  const uint32_t sQ = sbase + T::kOffQ;
  auto slot = [&](int st, int k) { return sbase + uint32_t(T::kOffRing + (st * T::kSlots + k) * T::kBlock); };
  float *xmax = reinterpret_cast<float *>(smem + T::kOffX);  // [2 parity][4 key quarters][64 rows]
  float *xsum = xmax + 8 * 64;                                // [4 key quarters][64 rows]
  float *qscale = reinterpret_cast<float *>(smem + T::kOffQSc);
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < T::kStages; ++i) {
      mbar_init(bar(T::FULL + i), 1);
      mbar_init(bar(T::VFULL + i), 1);
      mbar_init(bar(T::EMPTY + i), 1);
      mbar_init(bar(T::SFULL + i), 1);
      mbar_init(bar(T::SFREE + i), 16);
      mbar_init(bar(T::PFULL + i), 16);
      mbar_init(bar(T::SCALES + i), 1);
    }
    for (int i = 0; i < T::kQScales; ++i) mbar_init(bar(T::QSC + i), T::kLoaders);
    mbar_init(bar(T::OFULL), 1);
    mbar_init(bar(T::OFREE), 16);
    mbar_init(bar(T::QFULL), 2 * T::kLoaders);
    mbar_init(bar(T::QFREE), 1);
    mbar_init(bar(T::FINAL), 1);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + T::kOffTmem),
                 "r"(T::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  pair_sync();  // both CTAs' barriers are initialised before any cross-CTA arrive
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + T::kOffTmem);
  grid_dependency_wait();  // the plan comes from the scheduler kernel just before
  const PartCursor pc = load_part(p.tile_md, part);
  const unsigned long long lim_ns = p.watchdog_ns;

  if (warp == 0) {
    // ------------------------- producer (one warp in both CTAs) -------------------------
    // The warp runs converged; one instruction issues a step's copies from several lanes.
    if (lane == 0) {
      prefetch_tensormap(&k8_map);
      prefetch_tensormap(&page_map);
      prefetch_tensormap(&half_map);
    }
    // pages are read by both CTAs of the pair (the second time from L2)
    const uint64_t policy = l2_evict_normal_policy();
    const float *scales = k_scale + int64_t(kvh) * num_pages * kPage;
    Groups wa, wb;  // own pages, partner value halves
    wa.start(p, pc, prow0);
    wb = wa;
    bool ok = true;
    unsigned long long idle_since = 0;
    uint32_t spins = 0;
    while (ok && (!wa.done || wb.count < wa.count)) {
      bool progressed = false;
      // the partner page's value half of a group, once its score is done
      if (wb.count < wa.count && all_lanes(mbar_test_wait(bar(T::SFULL + wb.stage), wb.phase))) {
        int pa, pb;
        wb.pages(p, num_pages, pa, pb);
        if (lane == 0) {
          if (leader) mbar_arrive_expect_tx(bar(T::VFULL + wb.stage), 2 * T::kHalfVBytes);
          load_blocks_for_pair(slot(wb.stage, leader ? 2 : 0), &half_map, bar_cta0(T::VFULL + wb.stage),
                               (leader ? pb : pa) * kPage, kvh, leader ? 0 : 1, policy);
        }
        __syncwarp();
        wb.next(p, pc, prow0);
        progressed = true;
      }
      // the own page and the scales of a group, once the products of the stage's last group are done
      if (!progressed && !wa.done &&
          (wa.count < T::kStages || all_lanes(mbar_test_wait(bar(T::EMPTY + wa.stage), wa.phase ^ 1)))) {
        int pa, pb;
        wa.pages(p, num_pages, pa, pb);
        const int phys = leader ? pa : pb, st = wa.stage;
        if (lane == 0) {
          if (leader) mbar_arrive_expect_tx(bar(T::FULL + st), 2 * T::kOwnBytes);
          mbar_arrive_expect_tx(bar(T::SCALES + st), 512);
        }
        __syncwarp();
        if (lane == 0)
          load_blocks_for_pair(slot(st, 0), &page_map, bar_cta0(T::FULL + st), phys * kPage, kvh, 0, policy);
        else if (lane == 1)
          load_for_pair(slot(st, 4), &k8_map, bar_cta0(T::FULL + st), 512, kvh, phys * kPage, policy);
        else if (lane < 4)
          bulk_load_hint(sbase + T::kOffSc + st * 512 + (lane - 2) * 256, scales + int64_t(lane == 2 ? pa : pb) * kPage, 256,
                         bar(T::SCALES + st), policy);
        __syncwarp();
        wa.next(p, pc, prow0);
        progressed = true;
      }
      if (progressed) {
        idle_since = 0;
      } else if (__nanosleep(32), (++spins & 15u) == 0) {
        const unsigned long long now = global_ns();
        if (*abort) {
          ok = false;
        } else if (idle_since == 0) {
          idle_since = now;
        } else if (now - idle_since > lim_ns) {
          *abort = 1;
          if (lane == 0) report_timeout(p.status);
          ok = false;
        }
        ok = all_lanes(ok);
      }
    }
    // Every copy issued lands before the CTAs exit: the scales on this CTA's barriers, the pages
    // of both CTAs on CTA 0's (CTA 1 leaves after CTA 0: the final cluster barrier).  The last
    // group of each stage is the one to wait for.
    if (lane == 0) {
      int never = 0;
      for (int i = 1; i <= T::kStages; ++i) {
        const int ga = wa.count - i, gb = wb.count - i;
        if (ga >= 0) {
          mbar_wait(bar(T::SCALES + ga % T::kStages), (ga / T::kStages) & 1, &never, p.status, lim_ns);
          if (leader) mbar_wait(bar(T::FULL + ga % T::kStages), (ga / T::kStages) & 1, &never, p.status, lim_ns);
        }
        if (leader && gb >= 0) mbar_wait(bar(T::VFULL + gb % T::kStages), (gb / T::kStages) & 1, &never, p.status, lim_ns);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      // ------------------------- MMA issuer (CTA 0, one warp) -------------------------
      // The score of a group needs its pages in both CTAs (FULL), the query tile (QFULL) and its
      // score buffer read (SFREE); its PV needs both CTAs' v tiles (PFULL) and partner halves
      // (VFULL), and at a piece's first group the previous epilogue (OFREE).  Scores run up to
      // kStages groups ahead of PV; when both are ready the score goes first until it is two groups
      // ahead.  A poll of shared memory takes some 200 cycles beside the MMAs' operand reads, so the
      // barriers of a step are polled together, and none of them again once it has been seen.
      const uint32_t idesc_qk = idesc_f8(128, 128, false, false);
      const uint32_t idesc_hi = idesc_f8(128, 256, false, true), idesc_lo = idesc_f8(128, 256, true, true);
      Groups wq, wv;
      wq.start(p, pc, prow0);
      wv = wq;
      int qpiece = 0, vpiece = 0;
      bool qk_ready = false, pv_ready = false, ok = true;
      unsigned long long idle_since = 0;
      uint32_t spins = 0;
      while (ok && !wv.done) {
        bool q1 = true, q2 = true, q3 = true, v1 = true, v2 = true, v3 = true;
        const bool poll_qk = !qk_ready && !wq.done && wq.count < wv.count + T::kStages;
        const bool poll_pv = !pv_ready && wv.count < wq.count;
        if (poll_qk) {
          q1 = mbar_test_wait(bar(T::FULL + wq.stage), wq.phase);
          if (wq.count >= T::kStages) q2 = mbar_test_wait(bar(T::SFREE + wq.stage), wq.phase ^ 1);
          if (wq.j == 0) q3 = mbar_test_wait(bar(T::QFULL), qpiece & 1);
        }
        if (poll_pv) {
          v1 = mbar_test_wait(bar(T::PFULL + wv.stage), wv.phase);
          v2 = mbar_test_wait(bar(T::VFULL + wv.stage), wv.phase);
          if (wv.j == 0 && vpiece > 0) v3 = mbar_test_wait(bar(T::OFREE), (vpiece - 1) & 1);
        }
        if (poll_qk) qk_ready = all_lanes(q1 && q2 && q3);
        if (poll_pv) pv_ready = all_lanes(v1 && v2 && v3);
        if (qk_ready && (!pv_ready || wq.count < wv.count + 2)) {
          tc_fence_after();
          const int st = wq.stage;
          const uint32_t d = tmem + T::kTmemS + 64 * st;
          const uint64_t kb = smem_desc_sw128(slot(st, 0), 16, 1024), qa = smem_desc_sw128(sQ, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < kD / 32; ++kk) {
            const int cb = kk >> 2, in = (kk & 3) * 32;
            // descriptors step by (byte offset >> 4) in their address field
            const uint64_t b = kb + uint64_t((cb * T::kBlock + in) >> 4);
            const uint64_t hi = uint64_t((cb < 4 ? cb * T::kBlock + in : 8 * T::kBlock + in) >> 4);
            const uint64_t lo = uint64_t((cb < 4 ? (4 + cb) * T::kBlock + in : 8 * T::kBlock + 64 + in) >> 4);
            mma_f8_pair(d, qa + hi, b, idesc_qk, kk > 0 ? 1u : 0u);
            mma_f8_pair(d, qa + lo, b, idesc_qk, 1u);
          }
          commit_both(bar(T::SFULL + st));
          if (wq.j + 1 == wq.ngroups) {
            commit_both(bar(T::QFREE));  // the query tile may be replaced
            ++qpiece;
          }
          wq.next(p, pc, prow0);
          qk_ready = false;
          idle_since = 0;
        } else if (pv_ready) {
          tc_fence_after();
          const int st = wv.stage;
          const bool first = wv.j == 0;
          // a lone last page: the second page's keys are masked (v = 0), skip their products
          const int halves = (2 * wv.j + 1 < wv.ntiles) ? 2 : 1;
          const uint64_t hi = smem_desc_sw128(slot(st, 4), 16, 1024), lo = smem_desc_sw128(slot(st, 5), 16, 1024);
          const uint64_t vb = smem_desc_sw128(slot(st, 0), T::kBlock, 1024);
          for (int h = 0; h < halves; ++h)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              const uint64_t a = uint64_t((h * 64 + ks * 32) >> 4);
              const uint64_t b0 = vb + uint64_t((2 * h * T::kBlock + ks * 4096) >> 4), b1 = b0 + uint64_t(T::kBlock >> 4);
              const uint32_t o = tmem + T::kTmemO, acc = (!first || h > 0 || ks > 0) ? 1u : 0u;
              mma_f8_pair_twice(o, o + 128, hi + a, b0, b1, idesc_hi, acc);
              mma_f8_pair_twice(o, o + 128, lo + a, b0, b1, idesc_lo, 1u);
            }
          commit_both(bar(T::EMPTY + st));
          if (wv.j + 1 == wv.ngroups) {
            commit_both(bar(T::OFULL));
            ++vpiece;
          }
          wv.next(p, pc, prow0);
          pv_ready = false;
          idle_since = 0;
        } else if ((++spins & 15u) == 0) {
          const unsigned long long now = global_ns();
          if (*abort) {
            ok = false;
          } else if (idle_since == 0) {
            idle_since = now;
          } else if (now - idle_since > lim_ns) {
            *abort = 1;
            if (lane == 0) report_timeout(p.status);
            ok = false;
          }
          ok = all_lanes(ok);
        }
      }
      commit_both(bar(T::FINAL));
    }
    __syncwarp();
    // all tensor-core work (issued by CTA 0, writing both CTAs' tensor memory) is complete before
    // either CTA releases its tensor memory
    if (lane == 0) {
      int never = 0;
      mbar_wait(bar(T::FINAL), 0, &never, p.status, lim_ns);
    }
    __syncwarp();
  } else if (warp < 10) {
    // ------------------------- softmax / O rescale / epilogue -------------------------
    const int q = warp & 3;                 // tensor-memory sub-partition of this warp
    const int lrow = (32 * q + lane) & 63;  // row within the CTA's 64
    const int hf = q >> 1;                  // 0: first page's keys, values 0-255; 1: second page, 256-511
    const int quarter = 2 * hf + (warp - 2) / 4;  // this warp's 32 of the group's keys
    const int col0 = 128 * ((warp - 2) / 4);      // and its 128 of the half's 256 columns
    const int row = crow0 + lrow;
    const bool active = row < p.R;
    const int s_row = row / p.g, h_row = kvh * p.g + row % p.g;
    const uint32_t lanes = tmem + (uint32_t(32 * q) << 16);
    const int xbar = 1 + (q & 1);           // named barrier of the four warps sharing rows
    const uint32_t sfree = bar_cta0(T::SFREE), pfull = bar_cta0(T::PFULL), ofree = bar_cta0(T::OFREE);
    int g = 0, st = 0, phase = 0, last_st = 0, last_phase = 0, qs = 0;
    bool ok = true;
    for (int seq = pc.bi; part_has(pc, seq); ++seq) {
      const Piece w = piece_of(p, pc, seq, prow0);
      const int ns0 = split_base(p.num_splits, seq);
      const int nsplit = split_base(p.num_splits, seq + 1) - ns0;
      const int ord = seq == pc.bi ? pc.bord : 0;
      const int64_t acc_row = (int64_t(ns0 + ord) * p.h_kv + kvh) * p.R + row;
      __nv_bfloat16 *out_row = p.out + ((int64_t(seq) * p.s_q + s_row) * p.h_q + h_row) * kDV + hf * 256 + col0;
      float *acc_out = p.o_accum + acc_row * kDV + hf * 256 + col0;
      float *lse_row = p.lse + (int64_t(seq) * p.h_q + h_row) * p.s_q + s_row;
      if (w.ngroups == 0) {
        // no visible key in this piece: zero output (or partial) and lse = -inf
        if (active) {
          if (nsplit == 1) {
            for (int i = 0; i < 16; ++i) reinterpret_cast<uint4 *>(out_row)[i] = make_uint4(0u, 0u, 0u, 0u);
            if (quarter == 0) *lse_row = -INFINITY;
          } else {
            for (int i = 0; i < 32; ++i) reinterpret_cast<float4 *>(acc_out)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (quarter == 0) p.lse_accum[acc_row] = -INFINITY;
          }
        }
        continue;
      }
      // rows past R and rows without a visible key get v = 0 (every key masked)
      const int lim = active ? min(w.t1, p.causal ? w.L - (p.s_q - 1 - s_row) : w.L) : -1;
      ok = all_lanes(ok && mbar_wait(bar(T::QSC + (qs & (T::kQScales - 1))), (qs / T::kQScales) & 1, abort, p.status, lim_ns));
      // score of raw products to log2 units: 2^-a of the row and the softmax scale
      // (kept above 0, so that a masked score stays -inf)
      const float rowf = fmaxf(qscale[(qs & (T::kQScales - 1)) * 64 + lrow] * p.scale_log2, 1.2e-38f);
      float m_used = -INFINITY, l = 0.f;  // of this thread's quarter of the row's keys: maximum, sum of P
      float unit = -INFINITY;             // log2 of the row's unit of v and O
      for (int j = 0; j < w.ngroups; ++j, ++g) {
        ok = all_lanes(ok && mbar_wait(bar(T::SCALES + st), phase, abort, p.status, lim_ns));
        const float4 *sc4 = reinterpret_cast<const float4 *>(smem + T::kOffSc + st * 512);
        const int key0 = w.t0 + 128 * j + 32 * quarter;
        float ks[32];  // the scales of this warp's keys, read while the score is still running
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 s = sc4[8 * quarter + i];
          ks[4 * i] = s.x, ks[4 * i + 1] = s.y, ks[4 * i + 2] = s.z, ks[4 * i + 3] = s.w;
        }
        ok = all_lanes(ok && mbar_wait(bar(T::SFULL + st), phase, abort, p.status, lim_ns));
        tc_fence_after();
        float sv[32];
        if (ok) tmem_ld32(lanes + T::kTmemS + 64 * st + 32 * (quarter & 1), sv);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(sfree + 8u * st);
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 32; ++i) sv[i] *= ks[i];
        // keys at or past this row's limit get -inf, and no scale: that of a slot that is no key may be
        // anything (only partial groups need the test)
        if (__any_sync(0xffffffffu, key0 + 32 > lim)) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (key0 + i >= lim) {
              sv[i] = -INFINITY;
              ks[i] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) m4[i & 3] = fmaxf(m4[i & 3], sv[i]);
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * rowf;
        // The quarter's own running maximum, refreshed when it grows by more than 2 (log2 units).  P is
        // taken a quarter of its size: it stays below 1, and P s below the scale
        const float m_new = mx > m_used + 2.f ? mx : m_used;
        l *= m_new > m_used ? fast_exp2(m_used - m_new) : 1.f;
        m_used = m_new;
        const float nbase = m_used == -INFINITY ? 0.f : -2.f - m_used;
        float s4[4] = {0.f, 0.f, 0.f, 0.f}, t4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float e = fast_exp2(fmaf(sv[i], rowf, nbase));
          s4[i & 3] += e;
          sv[i] = e * ks[i];
          if (i & 1) t4[(i >> 1) & 3] = fmaxf(t4[(i >> 1) & 3], fmaxf(fabsf(sv[i - 1]), fabsf(sv[i])));
        }
        // The quarters share the unit of v, which follows the row's largest P s: exchange those.  It is
        // refreshed when that leaves 2^8 units, which E4M3 still holds, and then put at 2^6.  A unit is at
        // least 2^-118 of the largest P, which holds scales down to 2^-110 and keeps f finite
        const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        float *xm = xmax + (g & 1) * 4 * 64 + lrow;
        xm[quarter * 64] = m_used + fmaxf(2.f + fast_log2(top), -112.f);
        named_bar_sync(xbar, 128);
        l += (s4[0] + s4[1]) + (s4[2] + s4[3]);
        const float row_top = fmaxf(fmaxf(xm[0], xm[64]), fmaxf(xm[128], xm[192]));
        const bool need = row_top > unit + 8.f;
        float alpha = 1.f;
        if (need) {
          alpha = fast_exp2(unit - (row_top - 6.f));
          unit = row_top - 6.f;
        }
        const bool rescale = j > 0 && __any_sync(0xffffffffu, need);
        const float f = m_used == -INFINITY ? 0.f : fast_exp2(m_used + 2.f - unit);
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v[4] = {sv[4 * i] * f, sv[4 * i + 1] * f, sv[4 * i + 2] * f, sv[4 * i + 3] * f};
          split_v(v, hi[i], lo[i]);
        }
        // O may be rescaled once the previous group's PV has completed (its commit arrives on EMPTY
        // of that group's stage; that barrier is at most one phase behind)
        if (rescale) {
          ok = all_lanes(ok && mbar_wait(bar(T::EMPTY + last_st), last_phase, abort, p.status, lim_ns));
          if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int c0 = col0; c0 < col0 + 128; c0 += 32) {
              float v[32];
              tmem_ld32(lanes + T::kTmemO + c0, v);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] *= alpha;
              tmem_store32(lanes + T::kTmemO + c0, v);
            }
            tmem_st_wait();
          }
        }
        if (ok) {
          // the two terms of v into their tiles: 32 keys are two 16-byte chunks of a row
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(slot(st, 4) + sw128(lrow, 2 * quarter + c)),
                         "r"(hi[4 * c]), "r"(hi[4 * c + 1]), "r"(hi[4 * c + 2]), "r"(hi[4 * c + 3])
                         : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(slot(st, 5) + sw128(lrow, 2 * quarter + c)),
                         "r"(lo[4 * c]), "r"(lo[4 * c + 1]), "r"(lo[4 * c + 2]), "r"(lo[4 * c + 3])
                         : "memory");
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(pfull + 8u * st);
        last_st = st;
        last_phase = phase;
        if (++st == T::kStages) {
          st = 0;
          phase ^= 1;
        }
      }

      // ---- epilogue: O / l -> output (or fp32 split partial), natural-log LSE ----
      // (the buffer of the next group's maxima, last read before the barrier of the last group)
      float *xm = xmax + (g & 1) * 4 * 64 + lrow;
      xm[quarter * 64] = m_used;
      xsum[quarter * 64 + lrow] = l;
      named_bar_sync(xbar, 128);
      const float m_row = fmaxf(fmaxf(xm[0], xm[64]), fmaxf(xm[128], xm[192]));
      float l_row = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // a quarter without a visible key has no sum, or that of a row of NaN
        const float l_i = xsum[64 * i + lrow], m_i = xm[64 * i];
        l_row += m_i == -INFINITY ? l_i : l_i * fast_exp2(m_i - m_row);
      }
      ok = all_lanes(ok && mbar_wait(bar(T::OFULL), qs & 1, abort, p.status, lim_ns));
      tc_fence_after();
      if (ok) {
        const float inv = l_row > 0.f ? fast_exp2(unit - m_row - 2.f) / l_row : (l_row == 0.f ? 0.f : l_row);
        const int64_t out_off = out_row - p.out;
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 32) {
          float v[32];
          tmem_ld32(lanes + T::kTmemO + col0 + c0, v);
          // a lane holds 32 columns of its own row; transposed over groups of lanes, a store covers
          // whole 64- or 128-byte stretches of a row instead of 16 bytes of 32 rows
          if (nsplit == 1) {
            uint4 u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              u[k] = make_uint4(pack_bf16x2(v[8 * k] * inv, v[8 * k + 1] * inv),
                                pack_bf16x2(v[8 * k + 2] * inv, v[8 * k + 3] * inv),
                                pack_bf16x2(v[8 * k + 4] * inv, v[8 * k + 5] * inv),
                                pack_bf16x2(v[8 * k + 6] * inv, v[8 * k + 7] * inv));
            transpose_lanes(u, lane);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int from = (lane & ~3) + k;  // the lane whose row u[k] is of
              const int64_t off = __shfl_sync(0xffffffffu, out_off, from);
              if (row - lane + from < p.R) *reinterpret_cast<uint4 *>(p.out + off + c0 + 8 * (lane & 3)) = u[k];
            }
          } else {
            uint4 u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              u[k] = make_uint4(__float_as_uint(v[4 * k] * inv), __float_as_uint(v[4 * k + 1] * inv),
                                __float_as_uint(v[4 * k + 2] * inv), __float_as_uint(v[4 * k + 3] * inv));
            transpose_lanes(u, lane);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int from = (lane & ~7) + k;
              if (row - lane + from < p.R)
                *reinterpret_cast<uint4 *>(acc_out + int64_t(from - lane) * kDV + c0 + 4 * (lane & 7)) = u[k];
            }
          }
        }
        if (active && quarter == 0) {
          const float lse_v = l_row == 0.f ? -INFINITY : (m_row + 2.f + fast_log2(l_row)) * 0.69314718055994531f;
          if (nsplit == 1)
            *lse_row = lse_v;
          else
            // a maximum over partials would pass over a NaN; +inf makes the merged row NaN
            p.lse_accum[acc_row] = lse_v == lse_v ? lse_v : INFINITY;
        }
      }
      tc_fence_before();
      // the row-sum slots are rewritten by the next piece only after all four warps have read them
      named_bar_sync(xbar, 128);
      if (lane == 0) arrive_cluster(ofree);
      ++qs;
    }
  } else {
    // ------------------------- query loaders -------------------------
    // Lane l holds 16-byte chunks l and l + 32 (8 columns each) of every row of the warp, and of the
    // rope columns (chunk 64 + l mod 8) those of rows l / 8 + 4 i.
    constexpr int N = T::kLoadRows, NR = (N + 3) / 4;
    static_assert(T::kLoaders * N >= T::BM && N <= 16, "every row has a loader, a row scale per half warp");
    const int row0 = (warp - 10) * N;
    // the row whose offset and scale this lane keeps; rows past R stand for the last one (masked later)
    const int my_x = row0 + (lane & 15), my_row = min(crow0 + my_x, p.R - 1);
    const bool mine = (lane & 15) < N && my_x < T::BM;
    const int64_t my_off = int64_t(my_row / p.g) * p.q_ss + int64_t(kvh * p.g + my_row % p.g) * p.q_sh;
    const uint32_t qfull = bar_cta0(T::QFULL);
    auto chunk_of = [&](const __nv_bfloat16 *base, int i, int c) {  // chunk c of row row0 + i
      return __ldcg(reinterpret_cast<const uint4 *>(base + __shfl_sync(0xffffffffu, my_off, i)) + c);
    };
    auto put = [&](int block, int x, int byte, uint32_t u, uint32_t v) {
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(sQ + block * T::kBlock + sw128(x, byte >> 4) + (byte & 8)),
                   "r"(u), "r"(v)
                   : "memory");
    };
    int qs = 0;
    bool ok = true;
    for (int seq = pc.bi; part_has(pc, seq); ++seq) {
      if (piece_of(p, pc, seq, prow0).ngroups == 0) continue;
      const __nv_bfloat16 *base = p.q + int64_t(seq) * p.q_sb;
      uint4 r[NR], a[N][2];
#pragma unroll
      for (int i = 0; i < NR; ++i) r[i] = chunk_of(base, lane / 8 + 4 * i, 64 + lane % 8);
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) a[i][c] = chunk_of(base, i, lane + 32 * c);
      int my_e = 8;  // biased exponent of this lane's row's largest value
#pragma unroll
      for (int i = 0; i < N; ++i) {
        uint32_t m = max(bf16_top(a[i][0]), bf16_top(a[i][1]));
        if (lane / 8 == i % 4) m = max(m, bf16_top(r[i / 4]));
        m = __reduce_max_sync(0xffffffffu, m);
        if ((lane & 15) == i) my_e = max(int(m >> 7), 8);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float up = row_up(__shfl_sync(0xffffffffu, my_e, i));
        a[i][0] = split_q(a[i][0], up);
        a[i][1] = split_q(a[i][1], up);
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) r[i] = split_q(r[i], row_up(__shfl_sync(0xffffffffu, my_e, lane / 8 + 4 * i)));
      if (qs > 0) ok = all_lanes(ok && mbar_wait(bar(T::QFREE), (qs - 1) & 1, abort, p.status, lim_ns));
      if (ok) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (row0 + i < T::BM) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int col = 8 * (lane + 32 * c);
              put(col / 128, row0 + i, col % 128, a[i][c].x, a[i][c].y);
              put(4 + col / 128, row0 + i, col % 128, a[i][c].z, a[i][c].w);
            }
          }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int in = lane / 8 + 4 * i, byte = 8 * (lane % 8);
          if (in < N && row0 + in < T::BM) {
            put(8, row0 + in, byte, r[i].x, r[i].y);
            put(8, row0 + in, 64 + byte, r[i].z, r[i].w);
          }
        }
        if (lane < 16 && mine)
          qscale[(qs & (T::kQScales - 1)) * 64 + my_x] = my_e == 255 ? __int_as_float(0x7fffffff) : pow2(my_e - 134);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(T::QSC + (qs & (T::kQScales - 1))));
        arrive_cluster(qfull);
      }
      ++qs;
    }
  }
  grid_launch_dependents();
  tc_fence_before();
  __syncthreads();
  pair_sync();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(T::kTmemCols) : "memory");
  pair_sync();
}

cudaError_t launch_decode_fp8_pair(const CUtensorMap &k8_map, const CUtensorMap &page_map, const CUtensorMap &half_map, const DecodeParams &p, const float *k_scale,
                                   int64_t num_pages, cudaStream_t stream) {
  using T = FpPair;
  cudaError_t e = set_smem_once(reinterpret_cast<const void *>(decode_fp8_pair_kernel), T::kSmemBytes);
  if (e != cudaSuccess) return e;
  const unsigned pairs = unsigned((p.R + 2 * T::BM - 1) / (2 * T::BM));
  return launch_early(decode_fp8_pair_kernel, dim3(2 * pairs, p.num_parts, p.h_kv), dim3(T::kThreads), T::kSmemBytes,
                      stream, k8_map, page_map, half_map, p, k_scale, int(num_pages));
}

}  // namespace pagedmla
