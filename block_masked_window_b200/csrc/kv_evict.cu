// Eviction from the cache by accumulated attention weight (la_kv_evict): two kernels.
//
// Selection, per (sequence b, KV head h) with P_b keys and L = min(P_b, budget): the L keys of
// the highest rank stay. Rank: protected keys first (position < sink or >= next_pos - recent), then
// by weight (a NaN ranks as -inf), equal ranks by the lower slot. The weight becomes an unsigned
// number of the same order (its key), and the L-th largest is found by narrowing an interval of
// keys instead of sorting: a histogram of 512 bins over the interval tells in which bin it lies; when
// at most kCand keys are left, they are ranked against one another. The first interval is that of the
// weights at hand, at most 16 octaves below the largest, so that one histogram nearly always
// suffices whatever the weights' scale. One cluster of up to 8 CTAs per (b, h): each CTA
// holds a contiguous part of the keys in shared memory, and the CTAs read one another's
// histograms and candidates through distributed shared memory (which moves about 9 bytes a clock and
// SM: 512 bins, not the 2048 that would leave fewer candidates, keep its share below the barriers').
// A last pass in slot order lists the evicted slots below L (holes) and the kept slots from L on
// (movers).
//
// Moving: there are as many movers as holes, and mover k goes to hole k. Every hole lies below L
// and every mover at or above it, so no row that is read is ever written: the moves need no
// order among them, and the cost is the rows that change place, not the rows kept. (Closing the
// gaps in order would move almost the whole cache for a handful of evicted keys.) The second kernel
// also copies the weights and positions of what stays in place, where the outputs are separate.
//
// Bound: selection is latency, dependent passes over 4 bytes per key and two or three cluster barriers
// (8 us for 4096 keys of one sequence, 18 us for 8 x 2 heads of 32768 in clusters of 4: loads 3 us,
// histogram and its sum 3, candidates 4, lists 5; 1024 threads, 16 keys a thread and a listing by whole
// rows of bits measured within 0.5 us of it). Moving is memory, 512 bytes read and 512 written per
// moved key and head (131072 moves 28 us: 4.8 TB/s).
#include <cooperative_groups.h>

#include "pbd_common.cuh"
#include "pbd_kernels.h"

namespace la {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kBins = kSelThreads;         // one bin per thread
constexpr int kSelKeys = 8;                // keys of a thread in a tile
constexpr int kSelTile = kSelKeys * kSelThreads;
constexpr int kCand = kSelThreads / 2;     // candidates ranked directly, two threads each
constexpr uint32_t kSpan = (kBins - 2) << 18;   // keys of the first histogram: bins of 1/32 octave, 16 octaves

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

// What a CTA shows the others of its cluster.
struct SelShared {
  uint32_t hist[2][kBins];                 // (a buffer for every other histogram)
  unsigned long long cand[kCand];          // candidates: key in the high word, ~slot in the low
  uint32_t lowest, highest, guarded;       // of the unprotected keys; protected keys
  uint32_t n_cand;
  int holes, movers;
};

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(EvictProblem p, int cap) {
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  __shared__ __align__(16) SelShared sh;
  __shared__ __align__(16) unsigned long long s_all[kCand];   // the cluster's candidates
  __shared__ uint32_t warp_tot[32];
  __shared__ uint32_t s_bin, s_above, s_count, s_mine;   // wanted bin: keys above, in it, before this CTA's
  __shared__ unsigned long long s_last;    // the last candidate that stays
  extern __shared__ __align__(16) uint32_t s_key[];   // [cap] this CTA's keys (when they fit)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = blockIdx.x / C, b = bh / p.Hkv;
  sh.hist[0][tid] = 0;
  if (tid == 0) {
    sh.lowest = 0xFFFFFFFFu;
    sh.highest = sh.guarded = sh.n_cand = 0;
  }
  pdl_trigger();
  pdl_wait();
  const int P = load_len(p.seq_lens + b);
  const bool valid = P >= 0 && P <= p.S;
  const int n = valid ? P : 0;
  const int Lk = min(n, p.budget);
  const long long next = p.next_pos ? (long long)load_len(p.next_pos + b) : (long long)n;
  const float* w = p.weights + (size_t)bh * p.S;
  const int* pos = p.key_pos ? p.key_pos + (size_t)bh * p.S : nullptr;
  int* holes = p.slots + ((size_t)bh * C + rank) * 2 * p.part;
  int* movers = holes + p.part;
  uint32_t* hole_bits = p.hole_bits + (size_t)bh * p.bit_words;
  // A single CTA needs no barrier of the cluster.
  auto sync_all = [&]() {
    if (C == 1) __syncthreads();
    else cluster.sync();
  };

  if (rank == 0 && tid == 0 && !valid) atomicOr(&p.hdr->err, kErrSeqOverflow);

  // This CTA's keys [j0, j1).
  const int part = min(((n + C - 1) / C + 31) & ~31, p.part);   // (whole words of bits)
  const int j0 = min(rank * part, n), j1 = min(j0 + part, n);
  auto key_of = [&](int at, float weight) -> uint32_t {
    return at < p.sink || (long long)at >= next - p.recent ? 0xFFFFFFFFu : rank_of(weight);
  };
  // A warp's keys of a tile are consecutive, 32 to a row: lane l holds key l of each row, so that
  // ballots give the rows' order. All loads in flight together; a part of one tile keeps them in
  // registers.
  const int first = warp * 32 * kSelKeys + lane;
  float wv[kSelKeys];
  int pv[kSelKeys];
  auto load_tile = [&](int t0, int end) {
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      const int j = t0 + first + 32 * i;
      wv[i] = j < end ? w[j] : 0.f;
      pv[i] = pos && j < end ? pos[j] : j;
    }
  };
  const bool one_tile = part <= kSelTile;
  const bool evicts = Lk < n;              // (uniform over the cluster)
  const bool held = part <= cap;
  if (one_tile) load_tile(j0, j1);

  // Keys above `thr` stay, and of the keys equal to it those up to slot `thr_slot`, or the first
  // need_eq of the cluster in slot order where they are counted.
  uint32_t thr = 0, need_eq = 0, eq_before = 0;
  int thr_slot = 0x7fffffff;
  bool count_eq = false;
  if (evicts) {
    uint32_t low = 0xFFFFFFFFu, high = 0, guarded = 0;
#pragma unroll 1
    for (int t0 = j0; t0 < j1; t0 += kSelTile) {
      if (!one_tile) load_tile(t0, j1);
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i) {
        const int j = t0 + first + 32 * i;
        const uint32_t k = key_of(pv[i], wv[i]);
        if (j < j1) {
          if (held) s_key[j - j0] = k;
          const bool safe = k == 0xFFFFFFFFu;
          guarded += safe;
          low = min(low, safe ? 0xFFFFFFFFu : k);
          high = max(high, safe ? 0u : k);
        }
      }
    }
    __syncthreads();                       // s_key, and sh is initialised
    // f(key, slot) for this CTA's keys.
    auto for_keys = [&](auto f) {
#pragma unroll 4
      for (int j = j0 + tid; j < j1; j += kSelThreads)
        f(held ? s_key[j - j0] : key_of(pos ? pos[j] : j, w[j]), j);
    };
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    guarded = __reduce_add_sync(0xffffffffu, guarded);
    if (lane == 0) {
      atomicMin(&sh.lowest, low);
      atomicMax(&sh.highest, high);
      atomicAdd(&sh.guarded, guarded);
    }
    sync_all();
    {
      const SelShared* o = cluster.map_shared_rank(&sh, lane < C ? lane : 0);
      low = __reduce_min_sync(0xffffffffu, o->lowest);
      high = __reduce_max_sync(0xffffffffu, o->highest);
      guarded = __reduce_add_sync(0xffffffffu, lane < C ? o->guarded : 0u);
    }
    uint32_t want = (uint32_t)Lk;          // keys still wanted from [low, high]
    if (guarded >= want) {
      low = high = 0xFFFFFFFFu;            // protected keys alone: the lowest slots
    } else {
      want -= guarded;
    }
    for (int round = 0;; ++round) {
      // Bin 0: below `base`; bin i > 0: 2^shift keys from base + (i - 1) 2^shift on.
      const uint32_t base = round == 0 && high - low > kSpan ? high - kSpan : low;
      int shift = 0;
      while (((high - base) >> shift) > kBins - 2) ++shift;
      uint32_t* hist = sh.hist[round & 1];
      for_keys([&](uint32_t k, int) {
        if (k >= low && k <= high) atomicAdd(&hist[k < base ? 0u : 1u + ((k - base) >> shift)], 1u);
      });
      sync_all();
      sh.hist[(round + 1) & 1][tid] = 0;   // (read last before this barrier)
      // Thread t holds the t-th bin from the top, over the cluster.
      const int bin = kBins - 1 - tid;
      uint32_t v[kMaxEvictCtas], sum = 0, mine = 0;   // (all loads in flight together)
#pragma unroll
      for (int r = 0; r < kMaxEvictCtas; ++r)
        v[r] = r < C ? cluster.map_shared_rank(&sh, r)->hist[round & 1][bin] : 0u;
#pragma unroll
      for (int r = 0; r < kMaxEvictCtas; ++r) {
        if (r < rank) mine += v[r];
        sum += v[r];
      }
      uint32_t total;
      const uint32_t incl = block_scan(sum, warp_tot, &total);
      if (incl - sum < want && want <= incl) {
        s_bin = (uint32_t)bin;
        s_above = incl - sum;
        s_count = sum;
        s_mine = mine;
      }
      __syncthreads();
      const uint32_t in_bin = s_count;
      want -= s_above;
      if (s_bin == 0) {
        high = base - 1;
      } else {
        low = base + ((s_bin - 1) << shift);
        high = min(high, low + ((1u << shift) - 1));
      }
      if (low == high || in_bin == want) {
        // One key value, of which the first `want` in slot order stay, or a bin that stays whole.
        thr = low;
        count_eq = in_bin != want;
        need_eq = want;
        eq_before = s_mine;
        break;
      }
      if (in_bin <= kCand) {
        // The wanted key is the candidate with want - 1 candidates before it.
        for_keys([&](uint32_t k, int j) {
          if (k >= low && k <= high)
            sh.cand[atomicAdd(&sh.n_cand, 1u)] = (unsigned long long)k << 32 | (uint32_t)~j;
        });
        sync_all();
        uint32_t at = 0;                   // where CTA r's candidates go
#pragma unroll
        for (int r = 0; r < kMaxEvictCtas; ++r) {
          if (r < C) {
            const SelShared* o = cluster.map_shared_rank(&sh, r);
            const uint32_t have = o->n_cand;
            if ((uint32_t)tid < have) s_all[at + tid] = o->cand[tid];
            at += have;
          }
        }
        __syncthreads();
        const uint32_t c = tid >> 1;
        const unsigned long long own = c < in_bin ? s_all[c] : 0ull;
        uint32_t before = 0;
        for (uint32_t i = tid & 1; i < in_bin; i += 2) before += s_all[i] > own;
        before += __shfl_xor_sync(0xffffffffu, before, 1);
        if (c < in_bin && before == want - 1) s_last = own;
        __syncthreads();
        thr = (uint32_t)(s_last >> 32);
        thr_slot = (int)~(uint32_t)s_last;
        break;
      }
    }
  }
  // In slot order: the holes and the movers of this CTA's part.
  const uint32_t before = (1u << lane) - 1;
  // Sum of a warp's x over the warps before it, and over all of them.
  auto warps_before = [&](uint32_t x, uint32_t* total) {
    __syncthreads();                       // warp_tot has been read
    if (lane == 0) warp_tot[warp] = x;
    __syncthreads();
    uint32_t t = lane < kSelThreads / 32 ? warp_tot[lane] : 0u;
    *total = __reduce_add_sync(0xffffffffu, t);
    return __reduce_add_sync(0xffffffffu, lane < warp ? t : 0u);
  };
  uint32_t n_holes = 0, n_movers = 0;
#pragma unroll 1
  for (int t0 = j0; t0 < j1 && evicts; t0 += kSelTile) {
    uint32_t keep[kSelKeys], eq[kSelKeys]; // a bit for each key of a row
    if (!held) load_tile(t0, j1);
    uint32_t n_eq = 0;
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      const int j = t0 + first + 32 * i;
      const uint32_t k = j >= j1 ? 0u : held ? s_key[j - j0] : key_of(pv[i], wv[i]);
      // (A bin that stays whole: thr is its lowest key.)
      const bool same = k == thr && j <= thr_slot;
      keep[i] = __ballot_sync(0xffffffffu, j < j1 && (k > thr || (same && !count_eq)));
      eq[i] = __ballot_sync(0xffffffffu, j < j1 && same);
      n_eq += __popc(eq[i]);
    }
    if (count_eq) {                        // the lowest slots among equals
      uint32_t total;
      uint32_t at = eq_before + warps_before(n_eq, &total);
      eq_before += total;
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i) {
        keep[i] |= __ballot_sync(0xffffffffu, (eq[i] >> lane & 1) && at + __popc(eq[i] & before) < need_eq);
        at += __popc(eq[i]);
      }
    }
    uint32_t both = 0, total;              // holes, and movers in the high half (at most kSelTile)
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      const int j = t0 + first + 32 * i;
      const bool stays = keep[i] >> lane & 1;
      const uint32_t hm = __ballot_sync(0xffffffffu, j < j1 && j < Lk && !stays);
      const uint32_t mm = __ballot_sync(0xffffffffu, j >= Lk && stays);
      if (lane == 0 && j < j1 && j < Lk) hole_bits[j >> 5] = hm;
      eq[i] = hm;                          // (equals are settled)
      keep[i] = mm;
      both += __popc(hm) + (__popc(mm) << 16);
    }
    const uint32_t at = warps_before(both, &total);
    int* hp = holes + n_holes + (at & 0xFFFFu);
    int* mp = movers + n_movers + (at >> 16);
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      const int j = t0 + first + 32 * i;
      if (eq[i] >> lane & 1) hp[__popc(eq[i] & before)] = j;
      if (keep[i] >> lane & 1) mp[__popc(keep[i] & before)] = j;
      hp += __popc(eq[i]);
      mp += __popc(keep[i]);
    }
    n_holes += total & 0xFFFFu;
    n_movers += total >> 16;
  }
  if (tid == 0) {
    sh.holes = (int)n_holes;
    sh.movers = (int)n_movers;
  }
  sync_all();
  // The first CTA writes where each CTA's holes and movers end in the head's order.
  if (rank == 0 && tid < 32) {
    int h = 0, m = 0;
    if (lane < C) {
      const SelShared* o = cluster.map_shared_rank(&sh, lane);
      h = o->holes;
      m = o->movers;
    }
#pragma unroll
    for (int o = 1; o < kMaxEvictCtas; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, h, o), c = __shfl_up_sync(0xffffffffu, m, o);
      if (lane >= o) {
        h += a;
        m += c;
      }
    }
    EvictList* list = p.lists + bh;
    if (lane < kMaxEvictCtas) {
      list->holes[lane] = h;
      list->movers[lane] = m;
    }
    const int moves = __shfl_sync(0xffffffffu, m, kMaxEvictCtas - 1);
    if (lane == 0) {
      p.moves[bh] = moves;
      p.kept_lens[bh] = Lk;
      if (bh == b * p.Hkv) p.lens[b] = valid ? Lk : P;   // the sequence's new length
    }
  }
  if (C > 1) cluster.sync();   // no CTA leaves while another may read its shared memory
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 8;               // keys a warp keeps in flight
constexpr int kMoveCtas = 4;               // blocks per SM
constexpr int kCopySlots = 4 * kMoveThreads;
constexpr int kMoveHeads = 1024;           // heads whose moves a block of blocks shares out

// Slot k of a list that is spread over the parts of C CTAs, which end at ends[0 .. C - 1].
__device__ __forceinline__ int list_at(const int* slots, const int* ends, int C, int part, int which, int k) {
  int r = 0, before = 0;
  if (C > 1) {
    int e[kMaxEvictCtas - 1];
#pragma unroll
    for (int i = 0; i < kMaxEvictCtas - 1; ++i) e[i] = ends[i];
#pragma unroll
    for (int i = 0; i < kMaxEvictCtas - 1; ++i) {
      if (k >= e[i]) {
        r = i + 1;
        before = e[i];
      }
    }
  }
  return slots[((size_t)r * 2 + which) * part + (k - before)];
}

// blockIdx.y: a group of kMoveHeads heads. Its moves are laid end to end and cut into one run for
// each warp of the group's blocks, equal to +-1, so heads with many moves and heads with none share
// the GPU evenly. The 32 lanes look up 32 moves of the run at once (head, slots, rows), and the warp
// then copies their rows, kMoveRows at a time.
__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) evict_move_kernel(EvictProblem p, int C) {
  __shared__ int s_end[kMoveHeads];        // moves up to and including a head
  __shared__ int s_warp[kMoveThreads / 32];
  constexpr int kPer = kMoveHeads / kMoveThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h0 = blockIdx.y * kMoveHeads, heads = min(kMoveHeads, p.B * p.Hkv - h0);
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = tid; b < p.B; b += kMoveThreads) p.new_lens[b] = p.lens[b];
  int cnt[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int h = tid * kPer + i;
    cnt[i] = h < heads ? p.moves[h0 + h] : 0;
    sum += cnt[i];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int at = incl - sum, total = 0;
#pragma unroll
  for (int i = 0; i < kMoveThreads / 32; ++i) {
    if (i < warp) at += s_warp[i];
    total += s_warp[i];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) s_end[tid * kPer + i] = at += cnt[i];
  __syncthreads();

  // What stays in place: the weight, position and origin of slots without a hole. Chunks of
  // kCopySlots slots of a head, from the last block on (the moves start at the first).
  const bool copy_w = p.weights_out != p.weights;
  const bool copy_pos = p.key_pos_out && p.key_pos_out != p.key_pos;
  if (copy_w || copy_pos || p.kept_slots) {
    const int per_head = (p.budget + kCopySlots - 1) / kCopySlots;
    for (long long c = gridDim.x - 1 - blockIdx.x; c < (long long)heads * per_head; c += gridDim.x) {
      const int bh = h0 + (int)(c / per_head), s0 = (int)(c % per_head) * kCopySlots;
      const int len = p.kept_lens[bh];       // slots that hold a key afterwards
      const bool any = p.moves[bh] > 0;
      const size_t row = (size_t)bh * p.S;
      float x[kCopySlots / kMoveThreads];
      int t[kCopySlots / kMoveThreads];
      uint32_t stays = 0;
#pragma unroll
      for (int i = 0; i < kCopySlots / kMoveThreads; ++i) {
        const int j = s0 + tid + i * kMoveThreads;
        const uint32_t holes = any && j < len ? p.hole_bits[(size_t)bh * p.bit_words + (j >> 5)] : 0u;
        if (j < len && copy_w) x[i] = p.weights[row + j];
        t[i] = j < len && copy_pos && p.key_pos ? p.key_pos[row + j] : j;
        stays |= (uint32_t)(j < len && !(holes >> (j & 31) & 1)) << i;
      }
#pragma unroll
      for (int i = 0; i < kCopySlots / kMoveThreads; ++i) {
        const int j = s0 + tid + i * kMoveThreads;
        if (stays >> i & 1) {
          if (copy_w) p.weights_out[row + j] = x[i];
          if (copy_pos) p.key_pos_out[row + j] = t[i];
          if (p.kept_slots) p.kept_slots[(size_t)bh * p.budget + j] = j;
        } else if (p.kept_slots && j >= len && j < p.budget) {
          p.kept_slots[(size_t)bh * p.budget + j] = -1;
        }
      }
    }
  }

  // Lanes 0..15 move a key's row of K, lanes 16..31 its row of V, 16 bytes each.
  uint4* cache = reinterpret_cast<uint4*>(lane < 16 ? p.kc : p.vc) + (lane & 15);
  auto row = [&](int bh, int slot) -> long long {   // -1: the table names no page of the pool
    if (!p.block_table) return ((long long)bh * p.S + slot) * (kHeadDim / 8);
    const int b = bh / p.Hkv, h = bh - b * p.Hkv;
    const int page = load_len(p.block_table + (size_t)b * p.pages_per_seq + slot / p.page_size);
    if (page < 0 || page >= p.num_pages) return -1;
    return (((long long)page * p.Hkv + h) * p.page_size + slot % p.page_size) * (kHeadDim / 8);
  };
  const int warps = gridDim.x * (kMoveThreads / 32), w = blockIdx.x * (kMoveThreads / 32) + warp;
  const int end = (int)((w + 1LL) * total / warps);
  for (int m0 = (int)((long long)w * total / warps); m0 < end; m0 += 32) {
    const int cnt = min(32, end - m0);
    long long rt = -1, rf = -1;
    if (lane < cnt) {
      const int m = m0 + lane;
      int lo = 0, hi = heads - 1;          // the first head whose end lies beyond the move
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_end[mid] > m) hi = mid;
        else lo = mid + 1;
      }
      const int bh = h0 + lo, k = m - (lo ? s_end[lo - 1] : 0);
      const EvictList* list = p.lists + bh;
      const int* slots = p.slots + (size_t)bh * C * 2 * p.part;
      const int to = list_at(slots, list->holes, C, p.part, 0, k);
      const int from = list_at(slots, list->movers, C, p.part, 1, k);
      rt = row(bh, to);
      rf = row(bh, from);
      const size_t at = (size_t)bh * p.S;  // the lane's own move: weight and position
      p.weights_out[at + to] = p.weights[at + from];
      if (p.key_pos_out) p.key_pos_out[at + to] = p.key_pos ? p.key_pos[at + from] : from;
      if (p.kept_slots) p.kept_slots[(size_t)bh * p.budget + to] = from;
    }
    for (int i0 = 0; i0 < cnt; i0 += kMoveRows) {
      uint4 v[kMoveRows];
#pragma unroll
      for (int i = 0; i < kMoveRows; ++i) {
        const long long f = __shfl_sync(0xffffffffu, rf, i0 + i);
        if (f >= 0) v[i] = __ldcs(cache + f);
      }
#pragma unroll
      for (int i = 0; i < kMoveRows; ++i) {
        const long long f = __shfl_sync(0xffffffffu, rf, i0 + i), t = __shfl_sync(0xffffffffu, rt, i0 + i);
        if (f >= 0 && t >= 0) cache[t] = v[i];
      }
    }
  }
}

}  // namespace

int evict_ctas(int S, int heads) {
  // One CTA up to 8192 keys of capacity (16 a thread), then one per 4096, at most a portable cluster,
  // and no more than are resident together: a CTA takes an SM, and clusters of 8 leave up to a
  // quarter of the SMs out (16 heads of 32768 keys: 8 CTAs each 28 us in two waves, 4 each 18 us).
  if (S <= 2 * kSelTile) return 1;
  int c = 2;
  while (c < kMaxEvictCtas && c * kSelTile < S && 2 * c * heads <= 112) c *= 2;
  return c;
}

int evict_part(int S, int heads) {
  const int c = evict_ctas(S, heads);
  return ((S + c - 1) / c + 31) / 32 * 32;
}

cudaError_t launch_evict(const EvictProblem& p, int sms, cudaStream_t s) {
  const int C = evict_ctas(p.S, p.B * p.Hkv);
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
  // Blocks that are resident at once, in equal shares of the groups of heads; no more than for the
  // most moves there can be and the chunks of what stays.
  const int heads = p.B * p.Hkv, groups = (heads + kMoveHeads - 1) / kMoveHeads;
  const long long most = p.budget < p.S - p.budget ? p.budget : p.S - p.budget;
  const int per_block = kMoveThreads / 32 * kMoveRows;
  const long long full = (most + per_block - 1) / per_block * (heads < kMoveHeads ? heads : kMoveHeads);
  long long x = (long long)kMoveCtas * sms / groups;
  const long long chunks = (long long)(p.budget + kCopySlots - 1) / kCopySlots * heads;
  if (x > full + chunks) x = full + chunks;
  if (x < 1) x = 1;
  return launch_pdl(evict_move_kernel, dim3((unsigned)x, (unsigned)groups), dim3(kMoveThreads), 0, s, p, C);
}

}  // namespace la
