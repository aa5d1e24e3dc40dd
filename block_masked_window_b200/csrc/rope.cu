// Rotary positions: rotation alone (la_rope) and fused with the append of the rotated keys
// and the values into the cache (la_rope_append).
//
// Pair i of a head at position t turns by a = 2 pi t f_i (f_i = turns per position, made by
// la_rope_plan_init):
//   y1 = s (x1 cos a - x2 sin a),   y2 = s (x2 cos a + x1 sin a)
// with (x1, x2) = channels (i, i + Rd/2) in the half layout and (2i, 2i + 1) in the
// interleaved one; channels from Rd on are copied. The inverse turns by -a.
//
// Angles: t f_i is formed and reduced to a fraction of a turn in 64 bits (error below 2^-22
// turns at t = 2^31), then sine and cosine are taken in 32 bits. A block computes the
// cosines and sines of its tokens once into shared memory; every head of those tokens uses
// them, so the transcendental work is 1/(heads) of the elements.
//
// Bound: memory. One item is 32 bytes of input (two 16-byte chunks, the two halves of 8 pairs in
// the half layout) and 32 bytes of output, and a thread's loads are issued before the angles are
// computed, so that the two overlap.
#include "pbd_common.cuh"
#include "pbd_kernels.h"

namespace la {
namespace {

constexpr int kRopeThreads = 256;
// Items whose loads a thread keeps in flight: 128 bytes, with registers for four blocks an SM.
template <typename E> constexpr int kItemsOf = sizeof(E) == 4 ? 2 : 4;

template <typename E> struct Vec8;
template <> struct Vec8<float> {
  uint4 r[2];
  __device__ void load(const float* p) {
    r[0] = *reinterpret_cast<const uint4*>(p);
    r[1] = *reinterpret_cast<const uint4*>(p + 4);
  }
  __device__ void store(float* p) const {
    *reinterpret_cast<uint4*>(p) = r[0];
    *reinterpret_cast<uint4*>(p + 4) = r[1];
  }
  __device__ void get(float* f) const {
    const float* s = reinterpret_cast<const float*>(r);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = s[e];
  }
  __device__ void set(const float* f) {
    float* d = reinterpret_cast<float*>(r);
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = f[e];
  }
};
template <> struct Vec8<__nv_bfloat16> {
  uint4 r;
  __device__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = r; }
  __device__ void get(float* f) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 t = __bfloat1622float2(h[e]);
      f[2 * e] = t.x;
      f[2 * e + 1] = t.y;
    }
  }
  __device__ void set(const float* f) {   // one rounding to the cache's type, to nearest even
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
  }
};
template <> struct Vec8<__half> {
  uint4 r;
  __device__ void load(const __half* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ void store(__half* p) const { *reinterpret_cast<uint4*>(p) = r; }
  __device__ void get(float* f) const {
    const __half2* h = reinterpret_cast<const __half2*>(&r);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 t = __half22float2(h[e]);
      f[2 * e] = t.x;
      f[2 * e + 1] = t.y;
    }
  }
  __device__ void set(const float* f) {
    __half2* h = reinterpret_cast<__half2*>(&r);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __floats2half2_rn(f[2 * e], f[2 * e + 1]);
  }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(float* d, float x) { *d = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* d, float x) { *d = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(__half* d, float x) { *d = __float2half_rn(x); }

// (scaled cosine, scaled sine) of pair i at position t.
__device__ __forceinline__ float2 turn_of(const la_rope_plan& pl, int i, long long t, float sign) {
  const double turns = (double)t * pl.turns[i];
  const float x = (float)(2.0 * (turns - rint(turns)));   // half turns in [-1, 1]
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(c * pl.out_scale, s * pl.out_scale * sign);
}

// Rotates the 16 channels of one item. cs: the token's (cos, sin) pairs. Half layout: a and b
// hold the first and second halves of pairs i0 .. i0 + 7. Interleaved: a and b hold pairs
// i0 .. i0 + 3 and i0 + 4 .. i0 + 7; pairs from `pairs` on are copied.
template <bool HALF, typename E>
__device__ __forceinline__ void rotate_item(Vec8<E>& a, Vec8<E>& b, const float2* cs, int i0, int pairs) {
  float x[8], y[8];
  a.get(x);
  b.get(y);
  if (HALF) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 c = cs[i0 + e];
      const float u = x[e], w = y[e];
      x[e] = fmaf(u, c.x, -(w * c.y));
      y[e] = fmaf(w, c.x, u * c.y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i0 + e < pairs) {
        const float2 c = cs[i0 + e];
        const float u = x[2 * e], w = x[2 * e + 1];
        x[2 * e] = fmaf(u, c.x, -(w * c.y));
        x[2 * e + 1] = fmaf(w, c.x, u * c.y);
      }
      if (i0 + 4 + e < pairs) {
        const float2 c = cs[i0 + 4 + e];
        const float u = y[2 * e], w = y[2 * e + 1];
        y[2 * e] = fmaf(u, c.x, -(w * c.y));
        y[2 * e + 1] = fmaf(w, c.x, u * c.y);
      }
    }
  }
  a.set(x);
  b.set(y);
}

// Channel offsets of item s of a head: its two 8-channel chunks and whether they are rotated.
template <bool HALF>
__device__ __forceinline__ bool item_chunks(int s, int pairs, int* ca, int* cb) {
  if (HALF) {
    const int rot = pairs >> 3;          // items that hold pairs (pairs % 8 == 0)
    if (s < rot) {
      *ca = 8 * s;
      *cb = 8 * s + pairs;
      return true;
    }
    *ca = 2 * pairs + 16 * (s - rot);
    *cb = *ca + 8;
    return false;
  }
  *ca = 16 * s;
  *cb = *ca + 8;
  return 8 * s < pairs;
}

// ---- Rotation alone: `tok` tokens per block.
template <typename E, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 4)
    rope_kernel(const __grid_constant__ la_rope_plan pl, RopeProblem p, int tok) {
  extern __shared__ float2 s_cs[];      // [tok][pairs]
  constexpr int kItems = kItemsOf<E>;
  pdl_trigger();
  pdl_wait();
  const int pairs = pl.rotary_dim >> 1;
  const long long t0 = (long long)blockIdx.x * tok;
  const int nt = (int)min((long long)tok, p.tokens - t0);
  const int ns = p.head_dim >> 4;
  const int per_tok = p.heads * ns;
  const int total = nt * per_tok;
  const E* x = static_cast<const E*>(p.x);
  E* y = static_cast<E*>(p.out);
  for (int base = threadIdx.x; base < total || base == threadIdx.x; base += kRopeThreads * kItems) {
    Vec8<E> a[kItems], b[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int it = base + k * kRopeThreads;
      if (it < total) {
        const int t = it / per_tok, rem = it - t * per_tok, h = rem / ns, s = rem - h * ns;
        int ca, cb;
        item_chunks<HALF>(s, pairs, &ca, &cb);
        const E* src = x + (t0 + t) * p.x_tok + h * p.x_head;
        a[k].load(src + ca);
        b[k].load(src + cb);
      }
    }
    if (base == threadIdx.x) {          // (first pass, every thread)
      for (int i = threadIdx.x; i < nt * pairs; i += kRopeThreads) {
        const int t = i / pairs;
        s_cs[i] = turn_of(pl, i - t * pairs, __ldg(p.positions + t0 + t), p.sign);
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int it = base + k * kRopeThreads;
      if (it < total) {
        const int t = it / per_tok, rem = it - t * per_tok, h = rem / ns, s = rem - h * ns;
        int ca, cb;
        if (item_chunks<HALF>(s, pairs, &ca, &cb))
          rotate_item<HALF>(a[k], b[k], s_cs + t * pairs, 8 * s, pairs);
        E* dst = y + (t0 + t) * p.y_tok + h * p.y_head;
        a[k].store(dst + ca);
        b[k].store(dst + cb);
      }
    }
  }
}

// The same for shapes and strides without 16-byte chunks: one thread per channel pair.
template <typename E, bool HALF>
__global__ void __launch_bounds__(kRopeThreads)
    rope_scalar_kernel(const __grid_constant__ la_rope_plan pl, RopeProblem p, int tok) {
  extern __shared__ float2 s_cs[];
  pdl_trigger();
  pdl_wait();
  const int pairs = pl.rotary_dim >> 1;
  const long long t0 = (long long)blockIdx.x * tok;
  const int nt = (int)min((long long)tok, p.tokens - t0);
  for (int i = threadIdx.x; i < nt * pairs; i += kRopeThreads) {
    const int t = i / pairs;
    s_cs[i] = turn_of(pl, i - t * pairs, __ldg(p.positions + t0 + t), p.sign);
  }
  __syncthreads();
  const int half = p.head_dim >> 1;
  const int per_tok = p.heads * half;
  for (int it = threadIdx.x; it < nt * per_tok; it += kRopeThreads) {
    const int t = it / per_tok, rem = it - t * per_tok, h = rem / half, i = rem - h * half;
    const E* src = static_cast<const E*>(p.x) + (t0 + t) * p.x_tok + h * p.x_head;
    E* dst = static_cast<E*>(p.out) + (t0 + t) * p.y_tok + h * p.y_head;
    const bool rot = i < pairs;
    const int ca = (HALF && rot) ? i : 2 * i, cb = (HALF && rot) ? i + pairs : 2 * i + 1;
    const E xa = src[ca], xb = src[cb];
    if (rot) {
      const float2 c = s_cs[t * pairs + i];
      const float u = to_f32(xa), w = to_f32(xb);
      from_f32(dst + ca, fmaf(u, c.x, -(w * c.y)));
      from_f32(dst + cb, fmaf(w, c.x, u * c.y));
    } else {
      dst[ca] = xa;
      dst[cb] = xb;
    }
  }
}

// ---- Rotation and append. Row (b, i) of a padded batch of T rows a sequence: q rotated into
// q_out, k rotated into the cache slot P_b + i, v copied there, its position into key_pos.
constexpr int kAppendTok = 16;          // most tokens per block

struct TokenAt {
  long long row;                        // cache row of KV head 0, or -1: nothing is appended
  long long tok;                        // row of q, k_new, v_new and q_out, or -1: padding
  long long pos;
  int b, slot;
};

template <bool HALF, bool SCALAR>
__global__ void __launch_bounds__(kRopeThreads, 4)
    rope_append_kernel(const __grid_constant__ la_rope_plan pl, RopeAppendProblem p, int tok) {
  using E = __nv_bfloat16;
  constexpr int kItems = kItemsOf<E>;
  __shared__ float2 s_cs[kAppendTok * kHeadDim / 2];
  __shared__ TokenAt s_at[kAppendTok];
  pdl_trigger();
  pdl_wait();
  const int pairs = pl.rotary_dim >> 1;
  const long long t0 = (long long)blockIdx.x * tok;
  const int nt = (int)min((long long)tok, (long long)p.B * p.T - t0);
  const int heads = p.Hq + 2 * p.Hkv;
  if (threadIdx.x < nt) {
    const long long t = t0 + threadIdx.x;
    const int b = (int)(t / p.T), i = (int)(t - (long long)b * p.T);
    const int P = p.seq_lens ? __ldg(p.seq_lens + b) : 0;
    const int w = p.row_lens ? __ldg(p.row_lens + b) : p.T;
    const int at = p.pos0 ? __ldg(p.pos0 + b) : P;
    TokenAt a;
    a.b = b;
    a.pos = (long long)at + i;
    a.slot = P + i;
    a.tok = t;
    a.row = -1;
    if (P < 0 || w < 0 || w > p.T || (long long)P + w > p.S || i >= w) {
      a.tok = -1;                       // padding, or a sequence whose lengths are invalid
    } else if (p.block_table) {
      const int page = __ldg(p.block_table + (size_t)b * p.pages_per_seq + a.slot / p.page_size);
      if (page >= 0 && page < p.num_pages)
        a.row = (long long)page * p.Hkv * p.page_size + a.slot % p.page_size;
    } else {
      a.row = (long long)b * p.Hkv * p.S + a.slot;
    }
    s_at[threadIdx.x] = a;
  }
  // Row r of the block: (token r / heads, head r % heads; q heads, then k, then v).
  auto source = [&](int t, int h) -> const E* {
    const long long row = t0 + t;
    if (h < p.Hq) return p.q + row * p.q_tok + (long long)h * kHeadDim;
    h -= p.Hq;
    if (h < p.Hkv) return p.k_new + row * p.k_tok + (long long)h * kHeadDim;
    return p.v_new + row * p.v_tok + (long long)(h - p.Hkv) * kHeadDim;
  };
  auto target = [&](const TokenAt& a, int h) -> E* {   // null: not written
    if (a.tok < 0) return nullptr;
    if (h < p.Hq) return p.q_out + (a.tok * p.Hq + h) * kHeadDim;
    if (a.row < 0) return nullptr;
    h -= p.Hq;
    const int hk = h < p.Hkv ? h : h - p.Hkv;
    const long long row = a.row + (long long)hk * (p.block_table ? p.page_size : p.S);
    return (h < p.Hkv ? p.kc : p.vc) + row * kHeadDim;
  };
  auto angles = [&]() {
    __syncthreads();                    // s_at
    for (int i = threadIdx.x; i < nt * pairs; i += kRopeThreads) {
      const int t = i / pairs;
      if (s_at[t].tok >= 0) s_cs[i] = turn_of(pl, i - t * pairs, s_at[t].pos, 1.f);
    }
    if (p.key_pos) {
      for (int i = threadIdx.x; i < nt * p.Hkv; i += kRopeThreads) {
        const TokenAt a = s_at[i / p.Hkv];
        if (a.row >= 0)
          p.key_pos[((size_t)a.b * p.Hkv + i % p.Hkv) * p.S + a.slot] = (int)a.pos;
      }
    }
    __syncthreads();
  };
  if (SCALAR) {
    angles();
    const int total = nt * heads * (kHeadDim / 2);
    for (int it = threadIdx.x; it < total; it += kRopeThreads) {
      const int i = it % (kHeadDim / 2), r = it / (kHeadDim / 2), t = r / heads, h = r - t * heads;
      E* dst = target(s_at[t], h);
      if (!dst) continue;
      const E* src = source(t, h);
      const bool rot = i < pairs && h < p.Hq + p.Hkv;
      const int ca = (HALF && i < pairs) ? i : 2 * i, cb = (HALF && i < pairs) ? i + pairs : 2 * i + 1;
      const E xa = src[ca], xb = src[cb];
      if (rot) {
        const float2 c = s_cs[t * pairs + i];
        const float u = to_f32(xa), w = to_f32(xb);
        dst[ca] = __float2bfloat16_rn(fmaf(u, c.x, -(w * c.y)));
        dst[cb] = __float2bfloat16_rn(fmaf(w, c.x, u * c.y));
      } else {
        dst[ca] = xa;
        dst[cb] = xb;
      }
    }
    return;
  }
  constexpr int kNs = kHeadDim / 16;    // items of a head
  const int s = threadIdx.x % kNs;
  int ca, cb;
  const bool rot = item_chunks<HALF>(s, pairs, &ca, &cb);
  const int rows = nt * heads;
  bool first = true;
  for (int r0 = threadIdx.x / kNs; first || r0 < rows; r0 += kRopeThreads / kNs * kItems) {
    Vec8<E> a[kItems], b[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int r = r0 + k * (kRopeThreads / kNs);
      if (r < rows) {
        const int t = r / heads, h = r - t * heads;
        const E* src = source(t, h);
        a[k].load(src + ca);
        b[k].load(src + cb);
      }
    }
    if (first) angles();
    first = false;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int r = r0 + k * (kRopeThreads / kNs);
      if (r < rows) {
        const int t = r / heads, h = r - t * heads;
        E* dst = target(s_at[t], h);
        if (dst) {
          if (rot && h < p.Hq + p.Hkv) rotate_item<HALF>(a[k], b[k], s_cs + t * pairs, 8 * s, pairs);
          a[k].store(dst + ca);
          b[k].store(dst + cb);
        }
      }
    }
  }
}

template <typename E>
cudaError_t launch_rope_t(const la_rope_plan& pl, const RopeProblem& p, bool vec, cudaStream_t s) {
  const bool half = pl.layout == LA_ROPE_HALF;
  const int pairs = pl.rotary_dim / 2;
  // Tokens per block: a full set of loads for every thread, at most 32 KB of cosines and sines, and
  // (few tokens) no more than spreads them over two blocks per SM.
  const int per_tok = p.heads * (vec ? p.head_dim / 16 : p.head_dim / 2);
  long long tok = (long long)kRopeThreads * kItemsOf<E> / per_tok;
  if (tok > 4096 / pairs) tok = 4096 / pairs;
  if (tok > p.tokens / 296) tok = p.tokens / 296;
  if (tok < 1) tok = 1;
  const dim3 grid((unsigned)((p.tokens + tok - 1) / tok));
  const size_t smem = (size_t)tok * pairs * sizeof(float2);
  if (vec)
    return half ? launch_pdl(rope_kernel<E, true>, grid, dim3(kRopeThreads), smem, s, pl, p, (int)tok)
                : launch_pdl(rope_kernel<E, false>, grid, dim3(kRopeThreads), smem, s, pl, p, (int)tok);
  return half ? launch_pdl(rope_scalar_kernel<E, true>, grid, dim3(kRopeThreads), smem, s, pl, p, (int)tok)
              : launch_pdl(rope_scalar_kernel<E, false>, grid, dim3(kRopeThreads), smem, s, pl, p, (int)tok);
}

}  // namespace

cudaError_t launch_rope(const la_rope_plan& pl, const RopeProblem& p, int dtype, cudaStream_t s) {
  const int es = dtype == LA_DTYPE_F32 ? 4 : 2;
  auto al = [&](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  auto st = [&](long long n) { return n * es % 16 == 0; };
  // 16-byte chunks need aligned rows, and in the half layout both halves of a pair chunk-aligned.
  const bool vec = p.head_dim % 16 == 0 && (pl.layout == LA_ROPE_INTERLEAVED || pl.rotary_dim % 16 == 0) &&
                   al(p.x) && al(p.out) && st(p.x_tok) && st(p.x_head) && st(p.y_tok) && st(p.y_head);
  switch (dtype) {
    case LA_DTYPE_F32: return launch_rope_t<float>(pl, p, vec, s);
    case LA_DTYPE_BF16: return launch_rope_t<__nv_bfloat16>(pl, p, vec, s);
    case LA_DTYPE_F16: return launch_rope_t<__half>(pl, p, vec, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_rope_append(const la_rope_plan& pl, const RopeAppendProblem& p, cudaStream_t s) {
  const long long tokens = (long long)p.B * p.T;
  // Tokens per block: one full set of loads for every thread (6 at 16 + 2 + 2 heads), and few tokens
  // spread over two blocks per SM.
  long long tok = kRopeThreads * kItemsOf<__nv_bfloat16> / ((p.Hq + 2LL * p.Hkv) * (kHeadDim / 16));
  if (tok > kAppendTok) tok = kAppendTok;
  if (tok > tokens / 296) tok = tokens / 296;
  if (tok < 1) tok = 1;
  const dim3 grid((unsigned)((tokens + tok - 1) / tok));
  const bool half = pl.layout == LA_ROPE_HALF;
  if (half && pl.rotary_dim % 16 != 0)
    return launch_pdl(rope_append_kernel<true, true>, grid, dim3(kRopeThreads), 0, s, pl, p, (int)tok);
  return half ? launch_pdl(rope_append_kernel<true, false>, grid, dim3(kRopeThreads), 0, s, pl, p, (int)tok)
              : launch_pdl(rope_append_kernel<false, false>, grid, dim3(kRopeThreads), 0, s, pl, p, (int)tok);
}

}  // namespace la
