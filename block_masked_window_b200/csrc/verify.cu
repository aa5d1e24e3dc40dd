// Verification of a window's drafted tokens against the target's probabilities, from given
// random numbers (la_pbd_verify). For sequence b with drafts x_0 .. x_{k-1}, target rows p_i, draft
// rows q_i and uniforms u_i, v:
//   draft i is accepted while u_i q_i(x_i) < p_i(x_i); n = number accepted before the first miss;
//   the next token is drawn from r = max(p_n - q_n, 0) (from p_n when n = k, or when r sums to 0):
//   the smallest j with r_0 + ... + r_j > v (r_0 + r_1 + ...).
// A token drawn this way has the target's distribution whatever the drafts' is. Without q the
// drafts are certain: accepted while u_i < p_i(x_i), and r is p_n without x_n.
//
// Everything is computed in 64 bits: the accept test is then exact (a product of two 24-bit
// numbers), and a border of the cumulative sum moves by 1e-16 of the total, not by the 1e-7 at which
// the neighbour's token comes out once in a thousand draws over 150,000 entries.
//
// Bound: memory, one row of p and one of q per sequence, read once. A cluster of C CTAs shares a
// sequence: each warp sums one contiguous range of the row (loads coalesced, 8 + 8 in flight
// a lane), the ranges' sums meet through distributed shared memory, and the CTA that owns the range
// in which the draw falls goes over that range alone again (1/(16 C) of the row, from L2).
#include <cooperative_groups.h>

#include "pbd_common.cuh"
#include "pbd_kernels.h"

namespace la {
namespace {

namespace cg = cooperative_groups;

constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVMaxCtas = 8;
constexpr int kVUnroll = 8;
constexpr int kVRun = 5;         // entries of a thread when the draw's range is gone over again

__device__ __forceinline__ double to_f64(float x) { return (double)x; }
__device__ __forceinline__ double to_f64(__nv_bfloat16 x) { return (double)__bfloat162float(x); }
__device__ __forceinline__ double to_f64(__half x) { return (double)__half2float(x); }
__device__ __forceinline__ double positive(double x) { return x > 0.0 ? x : 0.0; }   // (NaN: 0)

// Sum of f(j, x(j), y(j)) over j = j0, j0 + 32, ... < end: kVUnroll loads of each in flight, the
// last ones one by one only where the range is ragged.
template <typename X, typename Y, typename F>
__device__ __forceinline__ double sum_range(int j0, int end, X x, Y y, F f) {
  double even = 0.0, odd = 0.0;
  int j = j0;
  for (; j + 32 * (kVUnroll - 1) < end; j += 32 * kVUnroll) {
    decltype(x(0)) a[kVUnroll];
    decltype(y(0)) b[kVUnroll];
#pragma unroll
    for (int i = 0; i < kVUnroll; ++i) {
      a[i] = x(j + 32 * i);
      b[i] = y(j + 32 * i);
    }
#pragma unroll
    for (int i = 0; i < kVUnroll; i += 2) {
      even += f(j + 32 * i, a[i], b[i]);
      odd += f(j + 32 * (i + 1), a[i + 1], b[i + 1]);
    }
  }
  if (j < end) {
    decltype(x(0)) a[kVUnroll];
    decltype(y(0)) b[kVUnroll];
#pragma unroll
    for (int i = 0; i < kVUnroll; ++i) {   // (past the end: the last entry again, not counted)
      a[i] = x(min(j + 32 * i, end - 1));
      b[i] = y(min(j + 32 * i, end - 1));
    }
#pragma unroll
    for (int i = 0; i < kVUnroll; ++i)
      if (j + 32 * i < end) even += f(j + 32 * i, a[i], b[i]);
  }
  return even + odd;
}

template <typename E>
__global__ void __launch_bounds__(kVThreads, 2) verify_kernel(VerifyProblem a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  __shared__ double s_sum[2][kVWarps];     // ranges of this CTA (a buffer per attempt)
  __shared__ double s_scan[kVWarps];
  __shared__ double s_total, s_before;
  __shared__ int s_n, s_len, s_range, s_first, s_last;
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  const E* p = static_cast<const E*>(a.p) + (long long)b * a.p_batch;
  const E* q = a.q ? static_cast<const E*>(a.q) + (long long)b * a.q_batch : nullptr;
  const int* drafts = a.drafts + (long long)b * a.K;
  if (warp == 0) {
    const int len = a.draft_lens ? load_len(a.draft_lens + b) : a.K;
    bool ok = false;
    if (lane < a.K && lane < len) {
      const int x = load_len(drafts + lane);
      if (x >= 0 && x < a.V) {             // a token outside the vocabulary has probability 0
        const double px = to_f64(p[(long long)lane * a.p_row + x]);
        const double qx = q ? to_f64(q[(long long)lane * a.q_row + x]) : 1.0;
        ok = (double)load_f32(a.u + (long long)b * a.K + lane) * qx < px;
      }
    }
    const uint32_t miss = ~__ballot_sync(0xffffffffu, ok);
    if (lane == 0) {
      s_len = len;
      s_n = miss ? __ffs(miss) - 1 : 32;
      s_first = 0x7fffffff;
      s_last = -1;
    }
  }
  __syncthreads();
  const int n = s_n, len = s_len;
  const bool valid = len >= 0 && len <= a.K;
  int* tokens = a.tokens + (long long)b * (a.K + 1);
  if (rank == 0) {
    for (int i = tid; i <= a.K; i += kVThreads)
      if (!valid || i != n) tokens[i] = valid && i < n ? load_len(drafts + i) : -1;
    if (tid == 0) {
      a.accepted[b] = valid ? n : -1;
      if (a.seq_lens_out) a.seq_lens_out[b] = load_len(a.seq_lens + b) + (valid ? n + 1 : 0);
    }
  }
  if (!valid) return;                      // (the whole cluster)

  const E* pr = p + (long long)n * a.p_row;
  const bool rejected = n < len;
  const E* qr = rejected && q ? q + (long long)n * a.q_row : nullptr;
  const int skip = rejected && !q ? load_len(drafts + n) : -1;
  const int per = ((a.V + C * kVWarps - 1) / (C * kVWarps) + 31) & ~31;   // entries of a range
  const double v = (double)load_f32(a.sample_u + b);
  // First the residual, where a draft was rejected; then, if that is empty, p itself.
  bool rest = rejected;
  auto entry = [&](int j, E x, E less) {
    const double d = to_f64(x);
    return positive(!rest ? d : qr ? d - to_f64(less) : j == skip ? 0.0 : d);
  };
  for (int attempt = 0;; ++attempt) {
    const int w0 = (int)min((long long)(rank * kVWarps + warp) * per, (long long)a.V);
    const int w1 = min(w0 + per, a.V);
    double sum = 0.0;
    if (rest && qr) {
      sum = sum_range(w0 + lane, w1, [&](int j) { return pr[j]; }, [&](int j) { return qr[j]; },
                      [&](int, E x, E y) { return positive(to_f64(x) - to_f64(y)); });
    } else {
      const int without = rest ? skip : -1;
      sum = sum_range(w0 + lane, w1, [&](int j) { return pr[j]; }, [&](int) { return 0; },
                      [&](int j, E x, int) { return j == without ? 0.0 : positive(to_f64(x)); });
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[attempt][warp] = sum;
    cluster.sync();
    // Every CTA finds the draw's range among the C * kVWarps ranges (lane l of warp 0: `of_lane`).
    if (warp == 0) {
      constexpr int kPart = kVMaxCtas * kVWarps / 32;
      const int of_lane = (C * kVWarps + 31) / 32;
      double part[kPart], mine = 0.0;
#pragma unroll
      for (int i = 0; i < kPart; ++i) {
        const int r = lane * of_lane + i;
        part[i] = i < of_lane && r < C * kVWarps
                      ? *cluster.map_shared_rank(&s_sum[attempt][r % kVWarps], r / kVWarps) : 0.0;
      }
#pragma unroll
      for (int i = 0; i < kPart; ++i) mine += part[i];
      double incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const double total = __shfl_sync(0xffffffffu, incl, 31);
      const double goal = v * total;
      double run = incl - mine, before = 0.0, before_last = 0.0;
      int range = -1, range_last = -1;     // first range that passes the goal; last with any weight
#pragma unroll
      for (int i = 0; i < kPart; ++i) {
        if (part[i] > 0.0) {
          range_last = lane * of_lane + i;
          before_last = run;
          if (range < 0 && run + part[i] > goal) {
            range = lane * of_lane + i;
            before = run;
          }
          run += part[i];
        }
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, range >= 0);
      const uint32_t any = __ballot_sync(0xffffffffu, range_last >= 0);
      if (lane == 0) {
        s_total = total;
        if (!any) s_range = -1;
      }
      if (hit ? lane == __ffs(hit) - 1 : any && lane == 31 - __clz(any)) {
        s_range = hit ? range : range_last;
        s_before = hit ? before : before_last;
      }
    }
    __syncthreads();
    if (s_total > 0.0 || !rest) break;     // (the same in every CTA of the cluster)
    rest = false;
  }
  const int range = s_range;
  if (!(s_total > 0.0 && s_total < (double)INFINITY)) {
    if (rank == 0 && tid == 0) tokens[n] = -1;   // nothing can be drawn
  } else if (range / kVWarps == rank) {
    // The smallest entry of the range at which the cumulative sum passes the goal (its last
    // entry with any weight, where rounding lets none pass).
    const double goal = v * s_total;
    const long long w0 = (long long)range * per, w1 = min(w0 + per, (long long)a.V);
    const int m = min((per + kVThreads - 1) / kVThreads, kVRun);   // consecutive entries of a thread
    double run = s_before;
    for (long long c0 = w0; c0 < w1; c0 += (long long)kVThreads * m) {
      double e[kVRun], mine = 0.0;
#pragma unroll
      for (int i = 0; i < kVRun; ++i) {
        const long long j = c0 + (long long)tid * m + i;
        e[i] = 0.0;
        if (i < m && j < w1) e[i] = entry((int)j, pr[j], rest && qr ? qr[j] : pr[j]);
        mine += e[i];
      }
      double incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s_scan[warp] = incl;
      __syncthreads();
      double at = run + (incl - mine);
      for (int w = 0; w < kVWarps; ++w) {
        if (w < warp) at += s_scan[w];
        run += s_scan[w];
      }
#pragma unroll
      for (int i = 0; i < kVRun; ++i) {
        const long long j = c0 + (long long)tid * m + i;
        if (e[i] > 0.0) {
          atomicMax(&s_last, (int)j);
          if (at + e[i] > goal) atomicMin(&s_first, (int)j);
          at += e[i];
        }
      }
      __syncthreads();
      if (s_first != 0x7fffffff) break;
    }
    if (tid == 0) tokens[n] = s_first != 0x7fffffff ? s_first : s_last;
  }
  cluster.sync();   // no CTA leaves while another may read its sums
}

template <typename E>
cudaError_t launch_verify_t(const VerifyProblem& a, int sms, cudaStream_t s) {
  // CTAs per sequence: as many as keep two of them on every SM (the row is then read by the whole
  // GPU however few sequences there are), but at least 4096 entries each.
  int c = kVMaxCtas;
  while (c > 1 && ((long long)a.B * c > 2LL * sms || (long long)(c - 1) * 4096 >= a.V)) c /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * c));
  cfg.blockDim = dim3(kVThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<E>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyProblem& a, int dtype, int sms, cudaStream_t s) {
  switch (dtype) {
    case LA_DTYPE_F32: return launch_verify_t<float>(a, sms, s);
    case LA_DTYPE_BF16: return launch_verify_t<__nv_bfloat16>(a, sms, s);
    case LA_DTYPE_F16: return launch_verify_t<__half>(a, sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace la
