// Verification of drafted tokens (speculative sampling) against the target's probabilities.
//
// For one sequence with drafts d_0 .. d_{n-1}, target rows p_0 .. p_n and draft rows q_0 ..
// q_{n-1} over a vocabulary of V, given uniform numbers u_i and u':
//   d_i is accepted while u_i q_i(d_i) < p_i(d_i); let r be the number accepted.
//   The next token is drawn from w = max(p_r - q_r, 0) when r < n, else from w = p_n, by
//   inverting its distribution: the lowest j whose running sum of w exceeds u' * sum(w).
// With the accepted drafts the tokens then follow the target's distribution exactly.  (A draft
// without probabilities was chosen with certainty: q is 1 at it and 0 elsewhere.)
//
// Only the sampled row of p and of q is read in full, once, so HBM bounds large batches and the
// latency of a few dependent reads small ones.  A cluster of CTAs takes a sequence: each CTA a
// contiguous range of the vocabulary, each of its warps a contiguous segment.  The segments'
// sums go to every CTA of the cluster through distributed shared memory, every CTA finds the
// segment that holds the wanted point, and the CTA that owns it reads it again (from L2) and
// scans it.  Sums are
// fp64: a point of the distribution falls between running sums 1/V apart, and fp32 sums over
// 10^5 entries are off by a good part of that.  The order of the sums is fixed by the launch
// shape, without atomics.
//
// Measured (B200, graphs and calls alike): 64 sequences x 3 drafts x 131,072 fp32 entries (50 MB)
// 13.6 us, of which the acceptance takes 2.1, the sums 5 to 6, the exchange and search 1.5 and the last
// scan 2.2 us; one sequence x 32,003 bf16 entries 6.1 us, a chain of four memory round trips.  The first
// took 25 us with two conversions to fp64 an entry, loads in registers and cluster barriers.
#include <cooperative_groups.h>

#include "launch.h"
#include "rope.cuh"

namespace pagedmla {

constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32, kVerifyMaxCluster = 8;
constexpr int kVerifyAhead = 4;  // 512-byte pieces of a warp's rows on their way

// The weight of a token; what is not a finite positive number has none.
__device__ __forceinline__ double verify_weight(float p, float q) {
  const double w = double(p) - double(q);
  return w > 0.0 && w <= 3.5e38 ? w : 0.0;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Inclusive running sum over the lanes.
__device__ __forceinline__ double warp_scan(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

constexpr int kSumsLate = -2;  // in the place of a segment: the sums have not arrived

struct SegmentAt {
  int segment;    // -1: nothing has weight
  double before;  // running sum in front of it
  double point;   // what the running sum has to exceed
};

// The segment that holds the wanted point, found by one warp: lane l sums `per` neighbouring segments;
// the first lane whose running sum exceeds the point has it.  A point at or past the total (u' of 1 or
// more) takes the last segment that holds anything.
__device__ __forceinline__ SegmentAt find_segment(const double *sums, int segments, float uniform, int lane) {
  const int per = (segments + 31) / 32, g0 = min(lane * per, segments), g1 = min(g0 + per, segments);
  double mine = 0.0;
#pragma unroll 1
  for (int g = g0; g < g1; ++g) mine += sums[g];
  const double upto = warp_scan(mine, lane);
  const double point = double(uniform) * __shfl_sync(0xffffffffu, upto, 31);
  const unsigned some = __ballot_sync(0xffffffffu, mine > 0.0), over = __ballot_sync(0xffffffffu, mine > 0.0 && upto > point);
  SegmentAt at = {-1, 0.0, over ? point : INFINITY};
  if (some == 0) return at;
  const int from = over ? __ffs(over) - 1 : 31 - __clz(some);
  double run = __shfl_sync(0xffffffffu, upto - mine, from);
#pragma unroll 1
  for (int g = from * per; g < min(from * per + per, segments); ++g) {
    const double w = sums[g];
    if (w > 0.0) {
      at.segment = g;
      at.before = run;
      if (run + w > point) break;
    }
    run += w;
  }
  return at;
}

// Store 8 bytes at the same place of CTA `rank` of the cluster, counted by its barrier.
__device__ __forceinline__ void send_to_cta(double value, uint32_t local, uint32_t barrier, int rank) {
  uint32_t at, bar;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(local), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(barrier), "r"(rank));
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(at),
               "l"(__double_as_longlong(value)), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void verify_copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// VEC: elements of an access.  16 bytes when rows and strides allow it: these go through a ring in
// shared memory (cp.async), deep enough to keep HBM busy with few registers; every lane reads back
// what it copied itself.  Otherwise one element at a time.
template <typename T, int VEC>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const VerifyParams p) {
  namespace cg = cooperative_groups;
  using V = Pack<T, VEC>;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int seq = blockIdx.x / C, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  extern __shared__ __align__(16) uint8_t verify_ring[];
  // The segments' sums of the whole cluster, and of this CTA; a second set for the draw from p itself.
  // They are exchanged by counted stores that only warp 0 waits for: a cluster barrier in their place
  // makes every warp acquire at cluster scope, after which the SM's shuffles took 250 cycles each (64 x
  // 131,072 fp32: 16.0 us against 13.5, also where only warp 0's wait is in the way).
  __shared__ double all_sum[2][kVerifyMaxCluster * kVerifyWarps];
  __shared__ double own_sum[kVerifyWarps];
  __shared__ uint64_t s_full[2];
  __shared__ double warp_total[kVerifyWarps];
  __shared__ double s_before, s_point;
  __shared__ float s_uniform;
  __shared__ int s_accepted, s_segment, s_found, s_last;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_arrive_expect_tx(smem_u32(&s_full[i]), uint32_t((C * kVerifyWarps + p.missing) * sizeof(double)));
    }
    fence_barrier_init();
  }
  cluster.barrier_arrive();  // every CTA's barriers are ready before a store to it
  grid_launch_dependents();
  grid_dependency_wait();

  // What needs no other value first is read at once: the drafts' probabilities are the second round
  // trip to memory, the sampled row the third.
  int n = p.num_drafts ? __ldcg(p.num_drafts + seq) : p.drafts;
  const T *target = static_cast<const T *>(p.target) + seq * p.t_b;
  const T *draft = p.draft ? static_cast<const T *>(p.draft) + seq * p.d_b : nullptr;
  const int32_t *tokens = p.tokens + int64_t(seq) * p.drafts;
  if (warp == 0) {
    int r = 0;
    for (;; r += 32) {
      const int i = r + lane;
      bool good = true;
      if (i < p.drafts) {
        const int tok = __ldcg(tokens + i);
        const double u = __ldcg(p.uniform + int64_t(seq) * p.drafts + i);
        good = false;
        if (tok >= 0 && tok < p.vocab) {
          const double pt = to_float(load_cg(target + i * p.t_s + tok));
          const double qt = draft ? double(to_float(load_cg(draft + i * p.d_s + tok))) : 1.0;
          good = u * qt < pt;
        }
      }
      const unsigned bad = __ballot_sync(0xffffffffu, !good || i >= min(n, p.drafts));  // the n-th place ends it
      if (bad) {
        r += __ffs(bad) - 1;
        break;
      }
    }
    if (lane == 0) s_accepted = r;
  } else if (tid == 32) {
    s_uniform = fmaxf(__ldcg(p.uniform_new + seq), 0.f);
    s_found = 0x7fffffff;
    s_last = -1;
  }
  cluster.barrier_wait();
  __syncthreads();
  n = max(0, min(n, p.drafts));
  const int r = s_accepted;
  const T *prow = target + r * p.t_s;
  const T *qrow = r < n && draft ? draft + r * p.d_s : nullptr;
  const int sure = r < n && !draft ? __ldcg(tokens + r) : -1;  // q = 1 at this token

  // segment g = rank * kVerifyWarps + warp covers columns [g * len, (g + 1) * len)
  const int segments = C * kVerifyWarps;
  const int len = ((p.vocab + segments - 1) / segments + VEC - 1) / VEC * VEC;
  auto begin_of = [&](int g) { return int(min(int64_t(g) * len, int64_t(p.vocab))); };
  bool subtract = r < n;
  for (int round = 0;; ++round) {
    const int lo = begin_of(rank * kVerifyWarps + warp), hi = begin_of(rank * kVerifyWarps + warp + 1);
    const bool both = subtract && qrow;
    const int one_at = subtract ? sure : -1;
    auto weight_at = [&](int j) {
      return verify_weight(to_float(load_cg(prow + j)), both ? to_float(load_cg(qrow + j)) : j == one_at ? 1.f : 0.f);
    };
    // A lane's sum.  With q' = min(p, q) the weight is p - q': its rounding d goes to the fp64 sum (the
    // conversion runs at a sixteenth of the fp32 rate, so there is one of them), and the rest
    // (p - d) - q', exact in fp32 and below 2^-24 d, to an fp32 sum that is off by less than 2^-43 of the
    // whole.  NaN and infinities show in the sum and are sorted out below.
    double sum = 0.0;
    float rest = 0.f;
    auto add = [&](float pj, float qj) {
      const float q1 = fminf(pj, qj), d = pj - q1;
      sum += double(d);
      rest += (pj - d) - q1;
    };
    if constexpr (VEC > 1) {
      uint8_t *ring = verify_ring + (warp * kVerifyAhead * 2 * 32 + lane) * 16;
      const uint32_t ring_at = smem_u32(ring);
      const int whole = lo + (hi - lo) / VEC * VEC;
      int next = lo + lane * VEC;  // column of the next copy
      auto copy = [&](int stage) {
        if (next < whole) {
          verify_copy16(ring_at + stage * 1024, prow + next);
          if (both) verify_copy16(ring_at + stage * 1024 + 512, qrow + next);
          next += 32 * VEC;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll 1
      for (int i = 0; i < kVerifyAhead - 1; ++i) copy(i);
      int stage = 0;
#pragma unroll 1
      for (int j = lo + lane * VEC; j < whole; j += 32 * VEC) {
        copy(stage == 0 ? kVerifyAhead - 1 : stage - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kVerifyAhead - 1) : "memory");
        const V a = *reinterpret_cast<const V *>(ring + stage * 1024);
        V b{};
        if (both) b = *reinterpret_cast<const V *>(ring + stage * 1024 + 512);
        if (unsigned(one_at - j) < unsigned(VEC)) {
#pragma unroll
          for (int k = 0; k < VEC; ++k)
            if (j + k == one_at) b.v[k] = from_float<T>(1.f);
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) add(to_float(a.v[k]), to_float(b.v[k]));
        stage = stage + 1 == kVerifyAhead ? 0 : stage + 1;
      }
      if (whole + lane < hi) sum += weight_at(whole + lane);  // the row's last few
    } else {
#pragma unroll 4
      for (int j = lo + lane; j < hi; j += 32)
        add(to_float(load_cg(prow + j)), both ? to_float(load_cg(qrow + j)) : j == one_at ? 1.f : 0.f);
    }
    sum += double(rest);
    if (__any_sync(0xffffffffu, !(fabs(sum) <= 1.7976931348623157e308))) {
      sum = 0.0;
#pragma unroll 1
      for (int j = lo + lane; j < hi; j += 32) sum += weight_at(j);
    }
    sum = warp_sum(sum);
    if (lane == 0) own_sum[warp] = sum;
    __syncthreads();
    const uint32_t full = smem_u32(&s_full[round]);
    if (warp == 0) {
      for (int i = lane; i < C * kVerifyWarps; i += 32)
        send_to_cta(own_sum[i % kVerifyWarps], smem_u32(&all_sum[round][rank * kVerifyWarps + i % kVerifyWarps]), full,
                    i / kVerifyWarps);
    } else if (warp == 1 && rank == 0 && round == 0) {
      // the tokens around the new one, while it is looked for
      for (int i = lane; i <= p.drafts; i += 32)
        if (i != r) p.out[int64_t(seq) * (p.drafts + 1) + i] = i < r ? __ldcg(tokens + i) : -1;
      if (lane == 0) p.accepted[seq] = r;
    }
    // A wait that gives up meets the other CTAs at the cluster's barrier and waits once more.  Who comes
    // there has sent the sums of its round, and who has left has had all of them; a CTA of the first
    // round may meet one of the second there, which then comes once more.  So no CTA leaves before the
    // sums that are sent to it have arrived
    for (int late = 0;; ++late) {
      if (warp == 0) {
        int gave_up = 0;
        const bool here = __all_sync(0xffffffffu, mbar_wait(full, 0, &gave_up, nullptr, late ? max(p.wait_ns, 1000000ull) : p.wait_ns));
        SegmentAt found = {kSumsLate, 0.0, 0.0};
        if (here) found = find_segment(all_sum[round], segments, s_uniform, lane);
        if (lane == 0) {
          s_segment = found.segment;
          s_before = found.before;
          s_point = found.point;
        }
      }
      __syncthreads();
      if (s_segment != kSumsLate || late > round) break;
      cluster.sync();
    }
    const int seg = s_segment;
    if (seg == kSumsLate) {  // nothing that was computed holds
      for (int i = tid; i <= p.drafts; i += kVerifyThreads) p.out[int64_t(seq) * (p.drafts + 1) + i] = -1;
      if (tid == 0) p.accepted[seq] = -1;
      return;
    }
    if (seg >= 0 || !subtract) {
      int32_t *out = p.out + int64_t(seq) * (p.drafts + 1) + r;
      if (seg < 0) {
        if (rank == 0 && tid == 0) *out = -1;
        return;
      }
      if (seg / kVerifyWarps != rank) return;
      // four neighbouring columns a thread
      const int end = begin_of(seg + 1);
      const double point = s_point;
      double base = s_before;
      for (int j0 = begin_of(seg); j0 < end; j0 += 4 * kVerifyThreads) {
        const int j = j0 + 4 * tid;
        double w[4], c = 0.0;
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = j + k < end ? weight_at(j + k) : 0.0;
#pragma unroll
        for (int k = 0; k < 4; ++k) c += w[k];
        const double upto = warp_scan(c, lane);
        if (lane == 31) warp_total[warp] = upto;
        __syncthreads();
        double off = base;
        for (int k = 0; k < warp; ++k) off += warp_total[k];
        double run = off + (upto - c);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          run += w[k];
          if (w[k] > 0.0) {
            if (run > point) atomicMin(&s_found, j + k);
            atomicMax(&s_last, j + k);
          }
        }
        for (int k = warp; k < kVerifyWarps; ++k) off += warp_total[k];
        base = off;
        __syncthreads();
        if (s_found != 0x7fffffff) break;
      }
      // rounding may leave the scan a little short of the segment's sum: its last token then
      if (tid == 0) *out = s_found != 0x7fffffff ? s_found : s_last;
      return;
    }
    subtract = false;  // p <= q everywhere (rounded rows): draw from p itself
    __syncthreads();
  }
}

template <typename T, int VEC>
static cudaError_t launch_verify_vec(const VerifyParams &p, cudaStream_t stream) {
  constexpr int kRing = VEC > 1 ? kVerifyWarps * kVerifyAhead * 2 * 512 : 0;
  if (cudaError_t e = set_smem_once(reinterpret_cast<const void *>(verify_kernel<T, VEC>), kRing)) return e;
  int C = kVerifyMaxCluster;
  while (C > 1 && int64_t(p.batch) * C > 296) C /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.batch * C));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.dynamicSmemBytes = kRing;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(C);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T, VEC>, p);
}

template <typename T>
static cudaError_t launch_verify_typed(const VerifyParams &p, cudaStream_t stream) {
  constexpr int kVec = 16 / sizeof(T);
  const bool wide = reinterpret_cast<uintptr_t>(p.target) % 16 == 0 && reinterpret_cast<uintptr_t>(p.draft) % 16 == 0 &&
                    p.t_b % kVec == 0 && p.t_s % kVec == 0 && p.d_b % kVec == 0 && p.d_s % kVec == 0;
  return wide ? launch_verify_vec<T, kVec>(p, stream) : launch_verify_vec<T, 1>(p, stream);
}

cudaError_t launch_verify(const VerifyParams &p, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case MLA_DTYPE_BF16: return launch_verify_typed<__nv_bfloat16>(p, stream);
    case MLA_DTYPE_F16: return launch_verify_typed<__half>(p, stream);
    default: return launch_verify_typed<float>(p, stream);
  }
}

}  // namespace pagedmla
