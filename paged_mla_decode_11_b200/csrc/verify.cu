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
// sums are exchanged through distributed shared memory, every CTA finds the segment that holds
// the wanted point, and the CTA that owns it reads it again (from L2) and scans it.  Sums are
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

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int seq = blockIdx.x / C, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  __shared__ double seg_sum[kVerifyWarps];                       // read by the whole cluster
  __shared__ double all_sum[kVerifyMaxCluster * kVerifyWarps];
  __shared__ double warp_total[kVerifyWarps];
  __shared__ double s_before, s_point;
  __shared__ int s_accepted, s_segment, s_found, s_last;
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
        good = false;
        if (tok >= 0 && tok < p.vocab) {
          const double pt = to_float(load_cg(target + i * p.t_s + tok));
          const double qt = draft ? double(to_float(load_cg(draft + i * p.d_s + tok))) : 1.0;
          good = double(__ldcg(p.uniform + int64_t(seq) * p.drafts + i)) * qt < pt;
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
  const int len = (p.vocab + C * kVerifyWarps - 1) / (C * kVerifyWarps);
  bool subtract = r < n;
  for (;;) {
    const int64_t lo64 = int64_t(rank * kVerifyWarps + warp) * len;
    const int lo = int(min(lo64, int64_t(p.vocab))), hi = min(lo + len, p.vocab);
    double sum = 0.0;
    if (subtract && qrow) {
#pragma unroll 8
      for (int j = lo + lane; j < hi; j += 32) sum += verify_weight(to_float(load_cg(prow + j)), to_float(load_cg(qrow + j)));
    } else {
#pragma unroll 8
      for (int j = lo + lane; j < hi; j += 32)
        sum += verify_weight(to_float(load_cg(prow + j)), subtract && j == sure ? 1.f : 0.f);
    }
    sum = warp_sum(sum);
    if (lane == 0) seg_sum[warp] = sum;
    cluster.sync();
    for (int i = tid; i < C * kVerifyWarps; i += kVerifyThreads)
      all_sum[i] = *cluster.map_shared_rank(&seg_sum[i % kVerifyWarps], i / kVerifyWarps);
    cluster.sync();  // no CTA rewrites or leaves seg_sum while another reads it
    if (warp == 0) {
      // lane l takes C * 16 / 32 consecutive segments, an odd C leaves the last lanes without any
      const int per = (C * kVerifyWarps + 31) / 32, g0 = lane * per, g1 = min(g0 + per, C * kVerifyWarps);
      double mine = 0.0;
      for (int g = g0; g < g1; ++g) mine += all_sum[g];
      const double upto = warp_scan(mine, lane);
      const double total = __shfl_sync(0xffffffffu, upto, 31);
      const double u = fmax(double(__ldcg(p.uniform_new + seq)), 0.0);
      const double point = u * total;
      // the first segment whose running sum exceeds the point; a point at or past the total
      // (u' of 1 or more) takes the last segment that holds anything
      int seg = 0x7fffffff, last = -1;
      double before = 0.0, run = upto - mine;
      for (int g = g0; g < g1; ++g) {
        const double next = run + all_sum[g];
        if (all_sum[g] > 0.0) {
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
    __syncthreads();
    if (s_segment >= 0 || !subtract) break;
    subtract = false;  // p <= q everywhere (rounded rows): draw from p itself
    __syncthreads();
  }

  const int seg = s_segment;
  if (seg >= 0 ? seg / kVerifyWarps == rank : rank == 0) {
    int token = -1;
    if (seg >= 0) {
      const int lo = int(min(int64_t(seg) * len, int64_t(p.vocab))), hi = min(lo + len, p.vocab);
      const double point = s_point;
      double base = s_before;
      if (tid == 0) {
        s_found = 0x7fffffff;
        s_last = -1;
      }
      for (int j0 = lo; j0 < hi; j0 += kVerifyThreads) {
        const int j = j0 + tid;
        double w = 0.0;
        if (j < hi) {
          const float q = !subtract ? 0.f : qrow ? to_float(load_cg(qrow + j)) : (j == sure ? 1.f : 0.f);
          w = verify_weight(to_float(load_cg(prow + j)), q);
        }
        double c = warp_scan(w, lane);
        if (lane == 31) warp_total[warp] = c;
        __syncthreads();
        double off = base;
        for (int k = 0; k < warp; ++k) off += warp_total[k];
        c += off;
        if (w > 0.0) {
          if (c > point) atomicMin(&s_found, j);
          atomicMax(&s_last, j);
        }
        for (int k = warp; k < kVerifyWarps; ++k) off += warp_total[k];
        base = off;
        __syncthreads();
        if (s_found != 0x7fffffff) break;
      }
      __syncthreads();
      // rounding may leave the scan a little short of the segment's sum: its last token then
      token = s_found != 0x7fffffff ? s_found : s_last;
    }
    for (int i = tid; i <= p.drafts; i += kVerifyThreads)
      p.out[int64_t(seq) * (p.drafts + 1) + i] = i < r ? __ldcg(tokens + i) : i == r ? token : -1;
    if (tid == 0) p.accepted[seq] = r;
  }
}

template <typename T>
static cudaError_t launch_verify_typed(const VerifyParams &p, cudaStream_t stream) {
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
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, p);
}

cudaError_t launch_verify(const VerifyParams &p, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case MLA_DTYPE_BF16: return launch_verify_typed<__nv_bfloat16>(p, stream);
    case MLA_DTYPE_F16: return launch_verify_typed<__half>(p, stream);
    default: return launch_verify_typed<float>(p, stream);
  }
}

}  // namespace pagedmla
