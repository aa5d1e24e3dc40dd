// Eviction from the cache by accumulated attention weight (la_kv_evict): two kernels.
//
// Selection, per (sequence b, KV head h) with P_b keys and L = min(P_b, budget): the L keys of
// the highest rank stay. Rank: protected keys first (position < sink or >= next_pos - recent), then
// by weight (a NaN ranks as -inf), equal ranks by the lower slot. The weight becomes an unsigned
// key of the same order, and the L-th largest key is found by three histogram passes over its
// bits (11, 11, 10 from the top) instead of a sort. One cluster of up to 8 CTAs per (b, h): each CTA
// holds a contiguous part of the keys in shared memory, and the CTAs read one another's
// histograms through distributed shared memory. A last pass in slot order decides the ties,
// copies what stays where it is and lists the evicted slots below L (holes) and the kept slots from
// L on (movers).
//
// Moving: there are as many movers as holes, and mover k goes to hole k. Every hole lies below L
// and every mover at or above it, so no row that is read is ever written: the moves need no
// order among them, and the cost is the rows that change place, not the rows kept. (Closing the
// gaps in order would move almost the whole cache for a handful of evicted keys.)
//
// Bound: selection is latency (a few dependent passes over 4 bytes per key); moving is memory,
// 512 bytes read and 512 written per moved key and head.
#include <cooperative_groups.h>

#include "pbd_common.cuh"
#include "pbd_kernels.h"

namespace la {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kBins = 2048;                // of the widest pass
constexpr int kSelKeys = 8;                // keys of a thread in a tile
constexpr int kSelTile = kSelKeys * kSelThreads;

// Unsigned key of the same order as the weight; NaN as -inf, -0 as +0.
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Inclusive prefix sum over the block (kSelThreads threads). Two barriers.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* warp_tot, uint32_t* total) {
  constexpr int kWarps = kSelThreads / 32;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                         // warp_tot of the previous scan has been read
  if (lane == 31) warp_tot[wid] = x;
  __syncthreads();
  uint32_t t = lane < kWarps ? warp_tot[lane] : 0u;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += y;
  }
  *total = __shfl_sync(0xffffffffu, t, kWarps - 1);
  const uint32_t before = __shfl_sync(0xffffffffu, t, (wid + 31) & 31);
  return x + (wid ? before : 0u);
}

// Counts digit d of the lanes for which `in` holds. Where one digit prevails (equal weights, zeros)
// its lanes are counted with one addition; the rest add for themselves.
__device__ __forceinline__ void count_digit(uint32_t* hist, uint32_t d, bool in) {
  const uint32_t live = __ballot_sync(0xffffffffu, in);
  if (live == 0) return;
  const int first = __ffs(live) - 1;
  const uint32_t d0 = __shfl_sync(0xffffffffu, d, first);
  const uint32_t same = __ballot_sync(0xffffffffu, in && d == d0);
  if (in && d != d0) atomicAdd(hist + d, 1u);
  if ((threadIdx.x & 31) == first) atomicAdd(hist + d0, (uint32_t)__popc(same));
}

__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(EvictProblem p, int cap) {
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  __shared__ __align__(16) uint32_t hist[3][kBins];
  __shared__ uint32_t warp_tot[32];
  __shared__ uint32_t s_bin, s_above;      // digit of the wanted key, keys above that digit
  __shared__ uint32_t s_keep[kSelThreads]; // which keys of a tile stay, a byte of bits per thread
  extern __shared__ __align__(16) uint32_t s_key[];   // [cap] this CTA's keys (when they fit)
  const int tid = threadIdx.x;
  const int bh = blockIdx.x / C, b = bh / p.Hkv;
  for (int i = tid; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
  pdl_trigger();
  pdl_wait();
  const int P = __ldg(p.seq_lens + b);
  const bool valid = P >= 0 && P <= p.S;
  const int n = valid ? P : 0;
  const int Lk = min(n, p.budget);
  const long long next = p.next_pos ? (long long)__ldg(p.next_pos + b) : (long long)n;
  const float* w = p.weights + (size_t)bh * p.S;
  const int* pos = p.key_pos ? p.key_pos + (size_t)bh * p.S : nullptr;
  float* w_out = p.weights_out + (size_t)bh * p.S;
  int* pos_out = p.key_pos_out ? p.key_pos_out + (size_t)bh * p.S : nullptr;
  int* kept = p.kept_slots ? p.kept_slots + (size_t)bh * p.budget : nullptr;
  EvictList* list = p.lists + (size_t)bh * kMaxEvictCtas + rank;
  int* holes = p.slots + ((size_t)bh * C + rank) * 2 * p.part;
  int* movers = holes + p.part;

  // Slots without a key say so.
  if (kept)
    for (int j = Lk + rank * kSelThreads + tid; j < p.budget; j += C * kSelThreads) kept[j] = -1;
  if (rank == 0 && tid == 0 && !valid) atomicOr(&p.hdr->err, kErrSeqOverflow);

  // This CTA's keys [j0, j1).
  const int part = min(((n + C - 1) / C + 3) & ~3, p.part);
  const int j0 = min(rank * part, n), j1 = min(j0 + part, n);
  auto key_of = [&](int at, float weight) -> uint32_t {
    return at < p.sink || (long long)at >= next - p.recent ? 0xFFFFFFFFu : rank_of(weight);
  };
  // Keys t0 + tid + i * kSelThreads, all loads in flight together (0 past the end).
  auto load_tile = [&](int t0, uint32_t (&k)[kSelKeys]) {
    float x[kSelKeys];
    int at[kSelKeys];
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      const int j = t0 + tid + i * kSelThreads;
      x[i] = j < j1 ? w[j] : 0.f;
      at[i] = pos && j < j1 ? pos[j] : j;
    }
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) k[i] = key_of(at[i], x[i]);
  };

  uint32_t thr = 0, need_eq = 0, eq_before = 0;
  bool all_eq = true;                      // every key equal to the threshold stays
  const bool evicts = Lk < n;              // (uniform over the cluster)
  const bool held = part <= cap;
  if (evicts) {
    uint32_t want = (uint32_t)Lk;          // keys still wanted from the current prefix's keys
    __syncthreads();
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bits = pass == 2 ? 10 : 11;
      const uint32_t mask = (1u << bits) - 1;
      for (int t0 = j0; t0 < j1; t0 += kSelTile) {
        uint32_t k[kSelKeys];
        if (pass > 0 && held) {
#pragma unroll
          for (int i = 0; i < kSelKeys; ++i) {
            const int j = t0 + tid + i * kSelThreads;
            k[i] = j < j1 ? s_key[j - j0] : 0u;
          }
        } else {
          load_tile(t0, k);
          if (held) {
#pragma unroll
            for (int i = 0; i < kSelKeys; ++i) {
              const int j = t0 + tid + i * kSelThreads;
              if (j < j1) s_key[j - j0] = k[i];
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kSelKeys; ++i) {
          bool in = t0 + tid + i * kSelThreads < j1;
          if (pass > 0) in = in && (k[i] >> (shift + bits)) == (thr >> (shift + bits));
          count_digit(hist[pass], (k[i] >> shift) & mask, in);
        }
      }
      cluster.sync();
      // Sum over the cluster, then the digit at which the count from the top reaches `want`.
      // Thread t holds the four bins from top - 4t down.
      constexpr int kPer = kBins / kSelThreads;
      static_assert(kPer == 4, "bins of a thread");
      const int top = (int)mask - kPer * tid;
      uint32_t c[kPer] = {0, 0, 0, 0};     // c[0]: the highest bin
      if (top > 0) {
        uint4 v[kMaxEvictCtas];            // (all loads in flight together)
#pragma unroll
        for (int r = 0; r < kMaxEvictCtas; ++r)
          v[r] = r < C ? *reinterpret_cast<const uint4*>(cluster.map_shared_rank(&hist[pass][top - 3], r))
                       : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int r = 0; r < kMaxEvictCtas; ++r) {
          c[0] += v[r].w;
          c[1] += v[r].z;
          c[2] += v[r].y;
          c[3] += v[r].x;
        }
      }
      uint32_t total;
      const uint32_t sum = c[0] + c[1] + c[2] + c[3];
      const uint32_t incl = block_scan(sum, warp_tot, &total);
      uint32_t above = incl - sum;
      if (above < want && want <= incl) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (above < want && want <= above + c[i]) {
            s_bin = (uint32_t)(top - i);
            s_above = above;
          }
          above += c[i];
        }
      }
      __syncthreads();
      thr |= s_bin << shift;
      want -= s_above;
      if (pass == 2) {
        const uint32_t d = thr & mask;
        uint32_t all = 0;
        uint32_t x[kMaxEvictCtas];
#pragma unroll
        for (int r = 0; r < kMaxEvictCtas; ++r) x[r] = r < C ? *cluster.map_shared_rank(&hist[2][d], r) : 0u;
#pragma unroll
        for (int r = 0; r < kMaxEvictCtas; ++r) {
          if (r < rank) eq_before += x[r];
          all += x[r];
        }
        need_eq = want;
        all_eq = need_eq == all;
      }
    }
  }
  // In slot order: what stays, the holes and the movers of this CTA's part.
  const bool copy_w = p.weights_out != p.weights;
  const bool copy_pos = pos_out && p.key_pos_out != p.key_pos;
  uint32_t n_holes = 0, n_movers = 0;
  for (int t0 = j0; t0 < j1; t0 += kSelTile) {
    const int j = t0 + kSelKeys * tid;     // this thread's run of keys
    const int cnt = max(0, min(kSelKeys, j1 - j));
    uint32_t keep = (1u << cnt) - 1;       // bit e: key j + e stays
    if (evicts) {
      uint32_t above = 0, eq = 0;
#pragma unroll
      for (int e = 0; e < kSelKeys; ++e) {
        if (e < cnt) {
          const uint32_t k = held ? s_key[j + e - j0] : key_of(pos ? pos[j + e] : j + e, w[j + e]);
          above |= (uint32_t)(k > thr) << e;
          eq |= (uint32_t)(k == thr) << e;
        }
      }
      keep = above | eq;
      if (!all_eq) {                       // the lowest slots among equals
        uint32_t total;
        const uint32_t at = eq_before + block_scan(__popc(eq), warp_tot, &total) - __popc(eq);
        eq_before += total;
        uint32_t left = need_eq > at ? need_eq - at : 0u;
        keep = above;
#pragma unroll
        for (int e = 0; e < kSelKeys; ++e) {
          if ((eq >> e & 1) && left > 0) {
            keep |= 1u << e;
            --left;
          }
        }
      }
      const int low = max(0, min(kSelKeys, Lk - j));   // keys of the run below the new length
      const uint32_t below = (1u << low) - 1;
      uint32_t hole = ~keep & below & ((1u << cnt) - 1), mover = keep & ~below;
      uint32_t total;                      // two counts of at most kSelTile in one word
      const uint32_t both = __popc(hole) | __popc(mover) << 16;
      const uint32_t at = block_scan(both, warp_tot, &total) - both;
      int* hp = holes + n_holes + (at & 0xFFFFu);
      int* mp = movers + n_movers + (at >> 16);
      for (; hole; hole &= hole - 1) *hp++ = j + __ffs(hole) - 1;
      for (; mover; mover &= mover - 1) *mp++ = j + __ffs(mover) - 1;
      n_holes += total & 0xFFFFu;
      n_movers += total >> 16;
    }
    // What stays in place, consecutive threads on consecutive slots.
    s_keep[tid] = keep;
    __syncthreads();
    float wv[kSelKeys];
    int pv[kSelKeys];
    uint32_t in_place = 0;
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {   // (all loads in flight before the stores)
      const int x = tid + i * kSelThreads, s = t0 + x;
      if (s < min(j1, Lk) && (s_keep[x / kSelKeys] >> (x % kSelKeys) & 1)) {
        in_place |= 1u << i;
        if (copy_w) wv[i] = w[s];
        pv[i] = copy_pos && pos ? pos[s] : s;
      }
    }
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      const int s = t0 + tid + i * kSelThreads;
      if (in_place >> i & 1) {
        if (copy_w) w_out[s] = wv[i];
        if (copy_pos) pos_out[s] = pv[i];
        if (kept) kept[s] = s;
      }
    }
    __syncthreads();
  }
  if (tid == 0) {
    list->holes = (int)n_holes;
    list->movers = (int)n_movers;
    list->len = valid ? Lk : P;            // the sequence's new length
  }
  cluster.sync();   // no CTA leaves while another may read its histograms
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;               // keys a warp keeps in flight
constexpr int kMoveCtas = 6;               // blocks per SM

// Slot k of a list that is spread over the parts of C CTAs.
__device__ __forceinline__ int list_at(const int* slots, const int* ends, int C, int part, int which, int k) {
  int r = 0, before = 0;
  while (r + 1 < C && k >= ends[r]) {
    before = ends[r];
    ++r;
  }
  return slots[((size_t)r * 2 + which) * part + (k - before)];
}

__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) evict_move_kernel(EvictProblem p, int C) {
  __shared__ int s_holes[kMaxEvictCtas], s_movers[kMaxEvictCtas];
  const int bh = blockIdx.y, b = bh / p.Hkv, h = bh - b * p.Hkv;
  pdl_trigger();
  pdl_wait();
  const EvictList* list = p.lists + (size_t)bh * kMaxEvictCtas;
  if (threadIdx.x == 0) {
    int a = 0, m = 0;
    for (int r = 0; r < C; ++r) {
      s_holes[r] = a += list[r].holes;
      s_movers[r] = m += list[r].movers;
    }
    if (blockIdx.x == 0 && h == 0) p.new_lens[b] = list[0].len;
  }
  __syncthreads();
  const int moves = s_movers[C - 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int* slots = p.slots + (size_t)bh * C * 2 * p.part;
  float* w_out = p.weights_out + (size_t)bh * p.S;
  const float* w = p.weights + (size_t)bh * p.S;
  // Lanes 0..15 move a key's row of K, lanes 16..31 its row of V, 16 bytes each.
  uint4* cache = reinterpret_cast<uint4*>(lane < 16 ? p.kc : p.vc) + (lane & 15);
  auto row = [&](int slot) -> long long {   // -1: the table names no page of the pool
    if (!p.block_table) return ((long long)bh * p.S + slot) * (kHeadDim / 8);
    const int page = __ldg(p.block_table + (size_t)b * p.pages_per_seq + slot / p.page_size);
    if (page < 0 || page >= p.num_pages) return -1;
    return (((long long)page * p.Hkv + h) * p.page_size + slot % p.page_size) * (kHeadDim / 8);
  };
  const int stride = gridDim.x * (kMoveThreads / 32) * kMoveRows;
  // Lane l < kMoveRows looks up move k0 + l (one turn ahead of the rows' copies).
  auto look_up = [&](int k0, int& to, int& from) {
    to = from = -1;
    if (lane < kMoveRows && k0 + lane < moves) {
      to = list_at(slots, s_holes, C, p.part, 0, k0 + lane);
      from = list_at(slots, s_movers, C, p.part, 1, k0 + lane);
    }
  };
  int k0 = (blockIdx.x * (kMoveThreads / 32) + warp) * kMoveRows;
  int to, from, next_to, next_from;
  look_up(k0, to, from);
  for (; k0 < moves; k0 += stride) {
    const long long rt = to >= 0 ? row(to) : -1, rf = from >= 0 ? row(from) : -1;
    uint4 v[kMoveRows];
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i) {
      const long long f = __shfl_sync(0xffffffffu, rf, i);
      if (f >= 0) v[i] = __ldcs(cache + f);
    }
    look_up(k0 + stride, next_to, next_from);
    if (to >= 0) {                          // the lane's own move: weight and position
      w_out[to] = w[from];
      if (p.key_pos_out)
        p.key_pos_out[(size_t)bh * p.S + to] = p.key_pos ? p.key_pos[(size_t)bh * p.S + from] : from;
      if (p.kept_slots) p.kept_slots[(size_t)bh * p.budget + to] = from;
    }
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i) {
      const long long f = __shfl_sync(0xffffffffu, rf, i), t = __shfl_sync(0xffffffffu, rt, i);
      if (f >= 0 && t >= 0) cache[t] = v[i];
    }
    to = next_to;
    from = next_from;
  }
}

}  // namespace

int evict_ctas(int S) {
  // One CTA per 4096 keys of capacity (eight keys a thread), at most a portable cluster.
  int c = 1;
  while (c < kMaxEvictCtas && c * kSelTile < S) c *= 2;
  return c;
}

int evict_part(int S) { return ((S + evict_ctas(S) - 1) / evict_ctas(S) + 3) / 4 * 4; }

cudaError_t launch_evict(const EvictProblem& p, int sms, cudaStream_t s) {
  const int C = evict_ctas(p.S);
  constexpr int kMaxHeld = 40 * 1024;      // keys: 160 KB of shared memory
  const int cap = p.part <= kMaxHeld ? p.part : 0;
  const size_t smem = (size_t)cap * 4;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kMaxHeld * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * p.Hkv * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, cap);
  if (e != cudaSuccess) return e;
  // Blocks per (sequence, KV head): enough for every possible move, but together no more than
  // are resident at once (a block then takes several turns: one wave, evenly filled).
  const int heads = p.B * p.Hkv;
  const long long most = p.budget < p.S - p.budget ? p.budget : p.S - p.budget;
  const int per_block = kMoveThreads / 32 * kMoveRows;
  long long x = (most + per_block - 1) / per_block;
  const long long fill = (long long)kMoveCtas * sms / heads;
  if (x > fill) x = fill;
  if (x < 1) x = 1;
  return launch_pdl(evict_move_kernel, dim3((unsigned)x, (unsigned)heads), dim3(kMoveThreads), 0, s, p, C);
}

}  // namespace la
