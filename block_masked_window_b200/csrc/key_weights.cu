// Attention weights of the keys, summed over the rows of a window and accumulated (the second
// half of la_pbd_attn_weights; the attention and merge kernels before it leave each row's
// log2-sum-exp in the workspace):
//   weights_out[b, h, j] = (j < P_b ? decay * weights_in[b, h, j] : 0)
//                        + sum_r 2^(scale_log2 <q_r, k_j> - lse2_r)        j in [0, P_b + W_b)
// over the R = W * G rows r that share KV head h.
//
// The scores are formed again rather than stored: S^T = K Q^T per 128-key tile (tcgen05,
// M = 128 keys, N = NQ rows, K = 128 channels), the same product as in the attention kernel.
// A key is a TMEM lane, so with the row statistics known each thread sums its own key's NQ
// probabilities in registers: no maximum, no exchange between threads, one store per key.
//
// Bound: the second reading of K from HBM (256 bytes per key against 4 to read and 4 to write of the
// weights): 8 sequences of 32768 keys add 29.5 us to the attention's 49 us, of which the copy is 20.5
// us at the measured rate. The exponentials (NQ per key, 16 per clock and SM) take a quarter of a
// tile's copy time at NQ = 48. Leaving a share of K in L2 for this reading (evict-last in the attention
// kernel, 40 to 134 MB of K) measured slower at every share (79.0 us without, 80.4 to 85.9 us with):
// the lines that stay push the streams and partials out.
//
// Plan: as the attention kernel's, without a fixed segment cost: every CTA gets the same
// number of whole key tiles, +-1, whatever the mix of lengths.
//
// Roles (320 threads, 1 CTA per SM): warp 0 TMA producer (Q per segment, double-buffered; K ring),
// warp 1 TMEM owner and MMA issuer, warps 2..5 and 6..9 sums of every other tile (one warp per
// scheduler took 1150 cycles for the 48 rows of a tile, more than its copy; two hide each other's
// latencies). Everything up to the first product only
// reads what was complete before the attention kernel started (the merge kernel starts after
// every attention CTA's wait), so it runs while the merge is still working; the sums wait for it.
// Every wait is bounded, as in the attention kernel.
#include "pbd_common.cuh"
#include "pbd_kernels.h"
#include "tc_util.cuh"
#include "tma_util.h"

namespace la {
namespace {

using namespace tc;

constexpr int kWThreads = 320;               // 2 + 8 warps
constexpr int kWMaxStages = 4;              // K ring: 128 KB in flight per SM (6 measured slower)
constexpr int kWSBufs = 4;                  // S^T buffers in TMEM
constexpr int kAhead = 4;                   // tiles by which the old weights are read ahead
constexpr int kWHalf = kTileKeys * 128;     // one 64-channel half of a K tile
constexpr int kWTile = 2 * kWHalf;

constexpr int kWBarKFull = 0;
constexpr int kWBarKEmpty = kWBarKFull + kWMaxStages;
constexpr int kWBarQFull = kWBarKEmpty + kWMaxStages;   // [2]
constexpr int kWBarQEmpty = kWBarQFull + 2;          // [2]
constexpr int kWBarSFull = kWBarQEmpty + 2;
constexpr int kWBarSEmpty = kWBarSFull + kWSBufs;
constexpr int kWBarDrain = kWBarSEmpty + kWSBufs;
constexpr int kWNumBars = kWBarDrain + 1;

struct WLayout {
  int k, q, bar, misc, lse, lim, old, pre, end;
};
__host__ __device__ inline WLayout w_layout(int nq, int stages, int B) {
  WLayout L;
  L.k = 0;
  L.q = stages * kWTile;
  L.bar = L.q + 2 * nq * 256;
  L.misc = L.bar + (kWNumBars + 1) / 2 * 16;
  L.lse = L.misc + 16;                      // [8 warps][nq] floats (16-byte multiples)
  L.lim = L.lse + 8 * nq * 4;               // [8][nq] ints
  L.old = L.lim + 8 * nq * 4;               // [2 groups][kAhead][128] floats
  L.pre = L.old + 2 * kAhead * 512;             // [B + 1] prefix sums, 32 ints
  L.end = L.pre + (round_up(B + 1, 4) + 32) * 4;
  return L;
}

__host__ __device__ constexpr int w_tmem_cols(int nq) {
  return nq <= 16 ? 64 : nq <= 32 ? 128 : nq <= 64 ? 256 : 512;
}

template <int NQ, bool LIMITS, bool PAGED>
__global__ void __launch_bounds__(kWThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmq,
                       Problem p, KeyWeights kw, int stages) {
  constexpr int kQHalf = NQ * 128;
  constexpr int kCols = w_tmem_cols(NQ);
  static_assert(kWSBufs * NQ <= kCols, "TMEM columns");
  constexpr uint32_t kIdesc = idesc_f16(128, NQ, 0, 0);

  extern __shared__ __align__(1024) char smem_raw[];
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const WLayout L = w_layout(NQ, stages, p.B);
  const uint32_t sb = smem_u32(base);
  auto bar = [&](int i) { return sb + (uint32_t)L.bar + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + L.misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + L.misc + 8);
  int* pre = reinterpret_cast<int*>(base + L.pre);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Ctl ctl{abort_flag, p.hdr, p.wait_limit_ns};

  pdl_trigger();
  // Rows R..NQ-1 of Q are zero in both buffers (TMA writes only rows < R).
  {
    const int per_half = (NQ - p.R) * 8;
    for (int i = tid; i < 4 * per_half; i += kWThreads) {
      const int half = i / per_half, c = i - half * per_half;
      reinterpret_cast<uint4*>(base + L.q + half * kQHalf + p.R * 128)[c] = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async_smem();
  }
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmk)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmq)) : "memory");
    for (int i = 0; i < kWNumBars; ++i) {
      const bool sums = i >= kWBarSEmpty && i < kWBarSEmpty + kWSBufs;
      mbar_init(bar(i), sums ? 128 : 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *abort_flag = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // seq_lens and window_lens were complete before the attention kernel's wait (see above).
  plan_prefix<true>(p, pre, pre + round_up(p.B + 1, 4));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long T = (long long)p.Hkv * pre[p.B];
  SegmentIter it = plan_begin(p, pre, blockIdx.x, T);
  Segment sg;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    // Lane 0 issues the copies. Of paged caches the whole warp looks up the pages of 16 tiles at once:
    // a look-up per tile would hold each copy back by its latency.
    const uint64_t policy = l2_policy_evict_first();   // read for the last time
    int g = 0, n = 0;
    bool ok = true;
    while (ok && it.next<true>(p, pre, blockIdx.x, sg)) {
      const int qs = n & 1;
      if (lane == 0) {
        if (n > 1 && !mbar_wait(bar(kWBarQEmpty + qs), ((n >> 1) - 1) & 1, ctl)) {
          ok = false;
        } else {
          const uint32_t dq = sb + L.q + qs * 2 * kQHalf;
          mbar_expect_tx(bar(kWBarQFull + qs), 2u * p.R * 128u);
          tma_load_3d(dq, &tmq, bar(kWBarQFull + qs), 0, sg.h * p.G, sg.b * p.W);
          tma_load_3d(dq + kQHalf, &tmq, bar(kWBarQFull + qs), 64, sg.h * p.G, sg.b * p.W);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      ++n;
      int rows = 0;   // lane l: the pool row of the l-th half tile of 16 tiles
      for (int jt = sg.j0; jt < sg.j1; jt += kTileKeys, ++g) {
        const int t = (jt - sg.j0) / kTileKeys;
        if (PAGED && (t & 15) == 0) {
          // A half tile past the segment reads the segment's last page again (its rows are not
          // used), so no table entry beyond the sequence is read.
          const int j = min(jt + 64 * lane, sg.j1 - 1);
          const int page = __ldcg(p.block_table + (size_t)sg.b * p.pages_per_seq + j / p.page_size);
          rows = (page * p.Hkv + sg.h) * p.page_size + j % p.page_size;
        }
        const int row0 = PAGED ? __shfl_sync(0xffffffffu, rows, 2 * (t & 15)) : (sg.b * p.Hkv + sg.h) * p.S + jt;
        const int row1 = PAGED ? __shfl_sync(0xffffffffu, rows, 2 * (t & 15) + 1) : 0;
        if (lane == 0) {
          const int ks = g % stages;
          if (g >= stages && !mbar_wait(bar(kWBarKEmpty + ks), (g / stages - 1) & 1, ctl)) {
            ok = false;
          } else {
            const uint32_t dk = sb + L.k + ks * kWTile, fb = bar(kWBarKFull + ks);
            mbar_expect_tx(fb, (uint32_t)kWTile);
            tma_load_2d_hint(dk, &tmk, fb, 0, row0, policy);
            tma_load_2d_hint(dk + kWHalf, &tmk, fb, 64, row0, policy);
            if (PAGED) {   // (64-row boxes)
              tma_load_2d_hint(dk + 8192, &tmk, fb, 0, row1, policy);
              tma_load_2d_hint(dk + kWHalf + 8192, &tmk, fb, 64, row1, policy);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
      }
    }
    // The copies issued last must have landed before shared memory is released.
    if (lane == 0) {
      for (int back = 1; back <= stages && g - back >= 0; ++back)
        mbar_drain(bar(kWBarKFull + (g - back) % stages), ((g - back) / stages) & 1, 100000000LL);
      for (int back = 1; back <= 2 && n - back >= 0; ++back)
        mbar_drain(bar(kWBarQFull + ((n - back) & 1)), ((n - back) >> 1) & 1, 100000000LL);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    int g = 0, n = 0;
    bool ok = true;
    while (ok && it.next<true>(p, pre, blockIdx.x, sg)) {
      const int qs = n & 1;
      if (lane == 0) ok = mbar_wait(bar(kWBarQFull + qs), (n >> 1) & 1, ctl);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      const uint32_t qb = sb + L.q + qs * 2 * kQHalf;
      if (LIMITS && sg.w < p.W) {
        // Padding rows of a shorter window may hold anything (a NaN): the warp makes them zeros, whose
        // scores of 0 add 2^(0 - inf) = 0.
        uint4* q0 = reinterpret_cast<uint4*>(base + L.q + qs * 2 * kQHalf);
        for (int i = sg.w * p.G * 8 + lane; i < p.R * 8; i += 32)
          q0[i] = q0[i + kQHalf / 16] = make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
        __syncwarp();
      }
      if (lane == 0) {
        for (int jt = sg.j0; jt < sg.j1; jt += kTileKeys, ++g) {
          const int ks = g % stages, s = g % kWSBufs;
          if (!mbar_wait(bar(kWBarKFull + ks), (g / stages) & 1, ctl) ||
              (g >= kWSBufs && !mbar_wait(bar(kWBarSEmpty + s), (g / kWSBufs - 1) & 1, ctl))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t kb = sb + L.k + ks * kWTile;
#pragma unroll
          for (int kk = 0; kk < kHeadDim / 16; ++kk) {
            const uint32_t ka = kb + (kk >> 2) * kWHalf + (kk & 3) * 32;
            const uint32_t qa = qb + (kk >> 2) * kQHalf + (kk & 3) * 32;
            umma(tmem + s * NQ, sdesc(ka, 16, 1024, 2), sdesc(qa, 16, 1024, 2), kIdesc, kk > 0);
          }
          umma_commit(bar(kWBarSFull + s));
          umma_commit(bar(kWBarKEmpty + ks));
        }
        if (ok) umma_commit(bar(kWBarQEmpty + qs));
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++n;
    }
    if (lane == 0) {
      umma_commit(bar(kWBarDrain));
      mbar_drain(bar(kWBarDrain), 0, 100000000LL);
    }
  } else {
    // ------------------------------------------------------------------ sums
    // Each warp keeps its own copy of a segment's row statistics: the warps share no barrier, so
    // one that gives up keeps no other waiting.
    const int sub = warp & 3, row = 32 * sub + lane, group = warp >= 6;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * sub) << 16);
    float* lse = reinterpret_cast<float*>(base + L.lse) + (warp - 2) * NQ;
    int* lim = reinterpret_cast<int*>(base + L.lim) + (warp - 2) * NQ;
    const uint32_t old_s = sb + (uint32_t)(L.old + group * kAhead * 512 + 4 * row);   // [kAhead][128]
    const float c2 = p.scale_log2;
    // The group's first tile is gone through once before the merge kernel (and with it the attention) is
    // complete, against statistics of +inf and to no effect: its instructions are then at hand when
    // the statistics are (one image, all three kernels: 14.4 us without this, 13.5 us with it).
    bool waited = false;
    int g = 0;
    bool ok = true;
    while (ok && it.next<true>(p, pre, blockIdx.x, sg)) {
      const long long head = (long long)sg.b * p.Hkv + sg.h;
      auto statistics = [&]() {
        __syncwarp();
#pragma unroll 1
        for (int q = lane; q < NQ; q += 32) {
          // A row that takes no part (operand padding, padding of a shorter window) adds 2^-inf.
          const bool live = q < p.R && (!LIMITS || q < sg.w * p.G);
          lse[q] = live && waited ? __ldcg(kw.lse2 + head * p.rows_pad + q) : INFINITY;
          if (LIMITS) lim[q] = live ? row_limit(p, sg.n, sg.w, q) : 0;
        }
        __syncwarp();
      };
      statistics();
      // Window rows start afresh: their slots may hold the weight of an earlier occupant. The old
      // weights are copied to shared memory kAhead tiles ahead, each lane its own (a tile takes less
      // time than a read, and a register with a read in flight cannot be passed on).
      const int old_end = kw.in ? min(sg.n - sg.w, sg.j1) : 0;
      auto read_ahead = [&](int key, int slot) {   // zero where there is no old weight
        const float* src = key < old_end ? kw.in + head * p.S + key : kw.out;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(old_s + (uint32_t)slot * 512u), "l"(src),
                     "r"(key < old_end ? 4 : 0)
                     : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      // This group's tiles of the segment: every other one of the CTA's.
      const int skip = (g ^ group) & 1, tiles = (sg.j1 - sg.j0 + kTileKeys - 1) / kTileKeys;
      const int g0 = g;
      g += tiles;
      // The copies that ran past the segment before (zeros) use the same slots, and a thread's copies land in
      // no order of their own: they are complete before the first ones of this segment.
      asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
      for (int i = 0; i < kAhead; ++i) read_ahead(sg.j0 + row + (skip + 2 * i) * kTileKeys, i);
#pragma unroll 1
      for (int t = skip, slot = 0; t < tiles;) {
        const int jt = sg.j0 + t * kTileKeys, gt = g0 + t;
        const int key = jt + row, s = gt % kWSBufs;
        const bool key_ok = key < sg.j1;
        const bool edge = p.mask_mode != 0 && jt + kTileKeys > sg.n - sg.w;   // rows differ in what they see
        ok = __all_sync(0xffffffffu, mbar_wait(bar(kWBarSFull + s), (gt / kWSBufs) & 1, ctl));
        if (!ok) break;
        tc_fence_after();
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        constexpr int kChunk = NQ <= 80 ? NQ : 64;   // columns held at once
        if (LIMITS && edge) {
          // The last tile or two of a sequence, in little code.
#pragma unroll 1
          for (int c = 0; c < NQ; c += 16) {
            float x[16];
            tmem_ld16(lane_addr + s * NQ + c, x);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              sum[i & 3] += key < lim[c + i] ? fast_exp2(fmaf(x[i], c2, -lse[c + i])) : 0.f;
          }
          tc_fence_before();
          if (waited) mbar_arrive(bar(kWBarSEmpty + s));
        } else {
#pragma unroll
          for (int c = 0; c < NQ; c += kChunk) {
            float x[kChunk];
#pragma unroll
            for (int e = 0; e < kChunk && c + e < NQ; e += 16) tmem_ld16(lane_addr + s * NQ + c + e, x + e);
            tc_wait_ld();
            if (c + kChunk >= NQ) {
              tc_fence_before();
              if (waited) mbar_arrive(bar(kWBarSEmpty + s));
            }
#pragma unroll
            for (int e = 0; e < kChunk && c + e < NQ; e += 4) {
              const float4 l = *reinterpret_cast<const float4*>(lse + c + e);
              sum[0] += fast_exp2(fmaf(x[e], c2, -l.x));
              sum[1] += fast_exp2(fmaf(x[e + 1], c2, -l.y));
              sum[2] += fast_exp2(fmaf(x[e + 2], c2, -l.z));
              sum[3] += fast_exp2(fmaf(x[e + 3], c2, -l.w));
            }
          }
        }
        float old;
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(old) : "r"(old_s + (uint32_t)slot * 512u) : "memory");
        if (key_ok && waited) kw.out[head * p.S + key] = fmaf(kw.decay, old, (sum[0] + sum[1]) + (sum[2] + sum[3]));
        if (!waited) {
          pdl_wait();
          waited = true;
          statistics();
          continue;
        }
        read_ahead(key + 2 * kAhead * kTileKeys, slot);
        t += 2;
        slot = (slot + 1) % kAhead;
      }
    }
    if (!waited) pdl_wait();   // (the kernel must not complete before its predecessors)
    asm volatile("cp.async.wait_all;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
  }
}

template <int NQ, bool LIMITS, bool PAGED>
cudaError_t launch_w(const Problem& p, const KeyWeights& kw, const CUtensorMap& k, const CUtensorMap& q,
                     cudaStream_t s) {
  // As deep a K ring as fits (a large batch's plan takes its share of shared memory).
  int stages = kWMaxStages;
  while (stages > 2 && 1024 + w_layout(NQ, stages, p.B).end > 227 * 1024) --stages;
  const size_t smem = (size_t)1024 + w_layout(NQ, stages, p.B).end;
  cudaError_t e = cudaFuncSetAttribute(key_weights_kernel<NQ, LIMITS, PAGED>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(key_weights_kernel<NQ, LIMITS, PAGED>, dim3(p.num_ctas), dim3(kWThreads), smem, s, k, q,
                    p, kw, stages);
}

}  // namespace

cudaError_t launch_key_weights(const Problem& p, const KeyWeights& kw, const void* tmap_k,
                               const void* tmap_q, cudaStream_t s) {
  const CUtensorMap& k = *static_cast<const CUtensorMap*>(tmap_k);
  const CUtensorMap& q = *static_cast<const CUtensorMap*>(tmap_q);
  const bool lim = row_limits(p), paged = p.block_table != nullptr;
#define LA_W_CASE(N)                                                          \
  case N:                                                                     \
    if (paged) return lim ? launch_w<N, true, true>(p, kw, k, q, s)           \
                          : launch_w<N, false, true>(p, kw, k, q, s);         \
    return lim ? launch_w<N, true, false>(p, kw, k, q, s)                     \
               : launch_w<N, false, false>(p, kw, k, q, s);
#define LA_W_CASE_WIDE(N)   /* more rows than the paged attention takes */    \
  case N:                                                                     \
    if (paged) return cudaErrorInvalidValue;                                  \
    return lim ? launch_w<N, true, false>(p, kw, k, q, s)                     \
               : launch_w<N, false, false>(p, kw, k, q, s);
  switch (round_up(p.R, 16)) {
    LA_W_CASE(16)
    LA_W_CASE(32)
    LA_W_CASE(48)
    LA_W_CASE(64)
    LA_W_CASE(80)
    LA_W_CASE_WIDE(96)
    LA_W_CASE_WIDE(112)
    LA_W_CASE_WIDE(128)
    default: return cudaErrorInvalidValue;
  }
#undef LA_W_CASE
#undef LA_W_CASE_WIDE
}

}  // namespace la
