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
#include <cooperative_groups.h>

#include "launch.h"
#include "rope.cuh"

namespace pagedmla {

constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32, kVerifyMaxCluster = 8;

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

// VEC: elements of an access (16 bytes when rows and strides allow it, else one).
template <typename T, int VEC>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const VerifyParams p) {
  namespace cg = cooperative_groups;
  using V = Pack<T, VEC>;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int seq = blockIdx.x / C, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  // the segments' sums, written by the whole cluster; a second set for the draw from p itself
  __shared__ double all_sum[2][kVerifyMaxCluster * kVerifyWarps];
  __shared__ double warp_total[kVerifyWarps];
  __shared__ double s_before, s_point;
  __shared__ int s_accepted, s_segment, s_found, s_last;
  cluster.barrier_arrive();  // waited for before the first write to another CTA's shared memory
  grid_launch_dependents();
  grid_dependency_wait();

  const int n = max(0, min(p.num_drafts ? __ldcg(p.num_drafts + seq) : p.drafts, p.drafts));
  const T *target = static_cast<const T *>(p.target) + seq * p.t_b;
  const T *draft = p.draft ? static_cast<const T *>(p.draft) + seq * p.d_b : nullptr;
  const int32_t *tokens = p.tokens + int64_t(seq) * p.drafts;
  if (warp == 0) {
    int r = 0;
    for (; r < n; r += 32) {
      const int i = r + lane;
      bool good = true;
      if (i < n) {
        const int tok = __ldcg(tokens + i);
        const double u = __ldcg(p.uniform + int64_t(seq) * p.drafts + i);
        good = false;
        if (tok >= 0 && tok < p.vocab) {
          const double pt = to_float(load_cg(target + i * p.t_s + tok));
          const double qt = draft ? double(to_float(load_cg(draft + i * p.d_s + tok))) : 1.0;
          good = u * qt < pt;
        }
      }
      const unsigned bad = __ballot_sync(0xffffffffu, !good);
      if (bad) {
        r += __ffs(bad) - 1;
        break;
      }
    }
    if (lane == 0) s_accepted = min(r, n);
  }
  __syncthreads();
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
    double sum = 0.0;
    const int whole = lo + (hi - lo) / VEC * VEC;
    if (subtract && qrow) {
#pragma unroll 4
      for (int j = lo + lane * VEC; j < whole; j += 32 * VEC) {
        const V a = load_cg(reinterpret_cast<const V *>(prow + j)), b = load_cg(reinterpret_cast<const V *>(qrow + j));
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum += verify_weight(to_float(a.v[k]), to_float(b.v[k]));
      }
    } else {
#pragma unroll 4
      for (int j = lo + lane * VEC; j < whole; j += 32 * VEC) {
        const V a = load_cg(reinterpret_cast<const V *>(prow + j));
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum += verify_weight(to_float(a.v[k]), subtract && j + k == sure ? 1.f : 0.f);
      }
    }
    auto weight_at = [&](int j) {
      const float q = !subtract ? 0.f : qrow ? to_float(load_cg(qrow + j)) : (j == sure ? 1.f : 0.f);
      return verify_weight(to_float(load_cg(prow + j)), q);
    };
    if (VEC > 1 && whole + lane < hi) sum += weight_at(whole + lane);  // the row's last few
    sum = warp_sum(sum);
    if (round == 0) cluster.barrier_wait();
    if (lane < C) *cluster.map_shared_rank(&all_sum[round][rank * kVerifyWarps + warp], lane) = sum;
    cluster.sync();
    if (warp == 0) {
      const double *sums = all_sum[round];
      const int per = (segments + 31) / 32, g0 = min(lane * per, segments), g1 = min(g0 + per, segments);
      double mine = 0.0;
      for (int g = g0; g < g1; ++g) mine += sums[g];
      const double upto = warp_scan(mine, lane);
      const double total = __shfl_sync(0xffffffffu, upto, 31);
      const double u = fmax(double(__ldcg(p.uniform_new + seq)), 0.0);
      const double point = u * total;
      // the first segment whose running sum exceeds the point; a point at or past the total
      // (u' of 1 or more) takes the last segment that holds anything
      int seg = 0x7fffffff, last = -1;
      double before = 0.0, run = upto - mine;
      for (int g = g0; g < g1; ++g) {
        const double next = run + sums[g];
        if (sums[g] > 0.0) {
          last = g;
          if (seg == 0x7fffffff && next > point) {
            seg = g;
            before = run;
          }
        }
        run = next;
      }
      const int first = __reduce_min_sync(0xffffffffu, seg), end = __reduce_max_sync(0xffffffffu, last);
      if (first != 0x7fffffff) {
        if (seg == first) {
          s_segment = first;
          s_before = before;
          s_point = point;
        }
      } else if (lane == 0) {
        s_segment = end;  // -1: nothing has weight
        s_before = 0.0;
        s_point = INFINITY;
      }
    }
    if (tid == 32) {
      s_found = 0x7fffffff;
      s_last = -1;
    }
    __syncthreads();
    if (s_segment >= 0 || !subtract) {
      const int seg = s_segment;
      if (seg >= 0 ? seg / kVerifyWarps != rank : rank != 0) return;
      int token = -1;
      if (seg >= 0) {
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
        token = s_found != 0x7fffffff ? s_found : s_last;
      }
      for (int i = tid; i <= p.drafts; i += kVerifyThreads)
        p.out[int64_t(seq) * (p.drafts + 1) + i] = i < r ? __ldcg(tokens + i) : i == r ? token : -1;
      if (tid == 0) p.accepted[seq] = r;
      return;
    }
    subtract = false;  // p <= q everywhere (rounded rows): draw from p itself
    __syncthreads();
  }
}

template <typename T, int VEC>
static cudaError_t launch_verify_vec(const VerifyParams &p, cudaStream_t stream) {
  int C = kVerifyMaxCluster;
  while (C > 1 && int64_t(p.batch) * C > 296) C /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.batch * C));
  cfg.blockDim = dim3(kVerifyThreads);
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
