// Rotary positions: rotation alone (la_rope) and fused with the append of the rotated keys
// and the values into the cache (la_rope_append).
//
// Pair i of a head at position t turns by a = 2 pi t f_i (f_i = turns per position, made by
// la_rope_plan_init):
//   y1 = s (x1 cos a - x2 sin a),   y2 = s (x2 cos a + x1 sin a)
// with (x1, x2) = channels (i, i + Rd/2) in the half layout and (2i, 2i + 1) in the
// interleaved one; channels from Rd on are copied. The inverse turns by -a.
//
// Angles: f_i is handed to the kernels as a 64-bit fraction of a turn, so that t f_i modulo a turn is
// one wrapping integer product (in 64-bit floating point the product, its reduction and the
// conversions took a third of the kernel's instructions). The product and its reduction add less than
// 2^-31 turns; the plan's frequencies, doubles, are off by up to 2^-56 a position, 2^-24 turns (4e-7 of
// an angle in radians) at 2^31 positions and 2^-38 at 2^17. Sine and cosine
// are taken of it in 32 bits: for fp32 results of what is left of it after whole quarter turns, with an
// error near a rounding's, and for 16-bit ones, whose rounding is 2^-12 of the value at best, of its
// upper 32 bits with the fast functions (2^-21 absolute).
//
// Bound: memory. An item is 16-byte chunks holding both channels of 8 pairs (4 in fp32). In la_rope a
// thread keeps its pairs over all its tokens and heads, so a token's cosines are taken once for the
// heads that the thread turns; in la_rope_append a warp owns a token and shares its cosines over all
// heads through a table of its own in shared memory.
#include <cmath>

#include "pbd_common.cuh"
#include "pbd_kernels.h"

namespace la {
namespace {

constexpr int kMaxPairs = 128;
constexpr int kRopeThreads = 128;
// Blocks per SM: as many as keep the kernel's registers.
constexpr int rope_ctas(bool half) { return half ? 7 : 6; }
// Items whose loads a thread keeps in flight: 64 bytes.
template <typename E> constexpr int kItemsOf = sizeof(E) == 4 ? 1 : 2;

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

// A plan as the kernels take it.
struct Turns {
  int pairs;
  float scale, sign;                       // sign: -1 turns back
  unsigned long long f[kMaxPairs];         // fraction of a turn per position, times 2^64
};
Turns turns_of(const la_rope_plan& pl, bool inverse) {
  Turns t;
  t.pairs = pl.rotary_dim / 2;
  t.scale = pl.out_scale;
  t.sign = inverse ? -1.f : 1.f;
  for (int i = 0; i < t.pairs; ++i) {
    const double f = pl.turns[i] - std::floor(pl.turns[i]);          // (exact; a NaN stays one)
    t.f[i] = f >= 0.0 && f < 1.0 ? (unsigned long long)(f * 18446744073709551616.0) : 0ull;
  }
  return t;
}

// Sine and cosine of x half turns, |x| <= 1/4 and a little: the Taylor series in x to degrees 9 and 10
// (cut off below 2^-28), with pi in two parts because its first factor stands alone in the sine. Errors
// against exact values over all x: sine 1.4e-8 rms, cosine 1.9e-8, where a correct rounding has 1.1e-8 and
// 1.7e-8. (sincospif reduces its argument first, which has been done here: 37.3 us for 12291 x 16 x 128
// fp32 with it, 33.1 so.)
__device__ __forceinline__ void sincos_quarter(float x, float* s, float* c) {
  const float z = x * x;
  float p = fmaf(z, 0.0821458866f, -0.599264529f);   // pi^9 / 9!, -pi^7 / 7!, pi^5 / 5!, -pi^3 / 3!
  p = fmaf(z, p, 2.55016404f);
  p = fmaf(z, p, -5.16771278f);
  p = fmaf(z, p, -8.74227766e-8f);                   // pi less its fp32 value
  *s = fmaf(x, 3.14159274f, x * p);
  float q = fmaf(z, -0.0258068914f, 0.235330631f);   // -pi^10 / 10!, pi^8 / 8!, -pi^6 / 6!, pi^4 / 4!
  q = fmaf(z, q, -1.33526277f);
  q = fmaf(z, q, 4.05871213f);
  q = fmaf(z, q, -4.93480220f);                      // -pi^2 / 2!
  *c = fmaf(z, q, 1.f);
}

// (scaled cosine, scaled sine) at position t of a pair that turns by the fraction f per position.
template <bool EXACT>
__device__ __forceinline__ float2 turn_at(unsigned long long f, float scale, float sign, long long t) {
  const int half = (int)((f * (unsigned long long)t) >> 32);         // of a turn, times 2^32
  float s, c;
  if (EXACT) {
    // Less the nearest quarter turn, so that the argument's 24 bits are of an eighth of a turn at most: of half
    // a turn, their rounding alone made the cosine's error 3.3e-8 rms.
    const int q = (int)((unsigned)half + (1u << 29)) >> 30;
    float s0, c0;
    sincos_quarter((float)(int)((unsigned)half - ((unsigned)q << 30)) * 4.656612873077393e-10f, &s0, &c0);   // 2^-31
    s = (q & 1) ? c0 : s0;
    c = (q & 1) ? s0 : c0;
    s = __uint_as_float(__float_as_uint(s) ^ (unsigned)(q & 2) << 30);
    c = __uint_as_float(__float_as_uint(c) ^ (unsigned)((q + 1) & 2) << 30);
  } else {
    const float x = (float)half * 1.4629180792671596e-9f;            // 2^-31 pi: in [-pi, pi]
    s = __sinf(x);
    c = __cosf(x);
  }
  return make_float2(c * scale, s * scale * sign);
}

// What a thread handles at a time: item s of a head, two chunks of 8 channels, so that neighbouring lanes
// move neighbouring chunks (16 channels in one piece would leave every memory instruction with half of
// each sector). Half layout: pairs 8s .. 8s + 7, their first and second channels (items past the pairs
// hold channels that are copied). Interleaved: channels 8s on and head_dim / 2 + 8s on, that is pairs 4s
// .. 4s + 3 and head_dim / 4 + 4s .. + 3.
template <bool HALF>
__device__ __forceinline__ int pair_of(int s, int e, int head_dim) {
  return HALF ? 8 * s + e : e < 4 ? 4 * s + e : (head_dim >> 2) + 4 * s + e - 4;
}
// The item's chunks, and whether any of its pairs turns.
template <bool HALF>
__device__ __forceinline__ bool item_chunks(int s, int pairs, int head_dim, int* ca, int* cb) {
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
  *ca = 8 * s;
  *cb = *ca + (head_dim >> 1);
  return 4 * s < pairs;
}

// Cosines and sines of an item's eight pairs, two pairs to a float4 (cos, cos, sin, sin), so that two are
// turned by one packed instruction. In a table of a token (items of 128 channels) the float4 of pairs
// 2e and 2e + 1 of item s lies at [e][s]: neighbouring lanes read neighbouring words.
constexpr int kItemsOfHead = kHeadDim / 16;
struct Turn8 {
  float4 cs[4];
  __device__ __forceinline__ void load(const float* table, int s) {
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = reinterpret_cast<const float4*>(table)[e * kItemsOfHead + s];
  }
  __device__ __forceinline__ float cos_of(int e) const { return (e & 1) ? cs[e >> 1].y : cs[e >> 1].x; }
  __device__ __forceinline__ float sin_of(int e) const { return (e & 1) ? cs[e >> 1].w : cs[e >> 1].z; }
};

// Two fp32 products, or products and sums, in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}

// Rotates the 16 channels of item `s`; pairs from `pairs` on are copied.
template <bool HALF, typename E>
__device__ __forceinline__ void rotate_item(Vec8<E>& a, Vec8<E>& b, const Turn8& t, int s, int pairs,
                                            int head_dim) {
  float x[8], y[8];
  a.get(x);
  b.get(y);
  if (HALF) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 c = make_float2(t.cs[e].x, t.cs[e].y), s = make_float2(t.cs[e].z, t.cs[e].w);
      const float2 u = make_float2(x[2 * e], x[2 * e + 1]), w = make_float2(y[2 * e], y[2 * e + 1]);
      const float2 p = fma2(u, c, mul2(w, make_float2(-s.x, -s.y))), q = fma2(w, c, mul2(u, s));
      x[2 * e] = p.x;
      x[2 * e + 1] = p.y;
      y[2 * e] = q.x;
      y[2 * e + 1] = q.y;
    }
  } else {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float* z = half ? y : x;
      const int n = pairs - pair_of<false>(s, 4 * half, head_dim);   // of the chunk's pairs that turn
      if (n >= 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float c = t.cos_of(4 * half + e), d = t.sin_of(4 * half + e), u = z[2 * e], w = z[2 * e + 1];
          z[2 * e] = fmaf(u, c, -(w * d));
          z[2 * e + 1] = fmaf(w, c, u * d);
        }
      } else if (n > 0) {
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          const float c = t.cos_of(4 * half + e), d = t.sin_of(4 * half + e), u = z[2 * e], w = z[2 * e + 1];
          z[2 * e] = e < n ? fmaf(u, c, -(w * d)) : u;
          z[2 * e + 1] = e < n ? fmaf(w, c, u * d) : w;
        }
      }
    }
  }
  a.set(x);
  b.set(y);
}

// ---- Rotation alone. A unit of work is `tok` tokens by `hb` heads, one set of items for every
// thread; blocks stride over the units. What an item is (its token, head, chunks and pairs) is the
// same in every unit, so its offsets and its 8 fractions stay in registers, and each thread computes
// its own cosines and sines: 8 of each per 16 channels are within the issue slots that the memory
// leaves free (about 180 instructions per item against 350), where a table shared by the heads costs a
// barrier per unit and, with one or two heads, more than it saves (one head of 128, 400000
// tokens: 204 us with a table).
template <typename E, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, rope_ctas(HALF))
    rope_kernel(const __grid_constant__ Turns pl, RopeProblem p, int tok, int hb) {
  __shared__ unsigned long long s_f[kMaxPairs];
  constexpr int kItems = kItemsOf<E>;
  const int pairs = pl.pairs;
  pdl_trigger();
  for (int i = threadIdx.x; i < kMaxPairs; i += kRopeThreads) s_f[i] = i < pairs ? pl.f[i] : 0;
  __syncthreads();
  const int ns = p.head_dim >> 4;
  const int nhb = (p.heads + hb - 1) / hb;
  const long long units = (p.tokens + tok - 1) / tok * nhb;
  // (The threads past the last whole head of a pass stay idle, so that a thread's items are alike.)
  const int item = threadIdx.x % ns, pass = kRopeThreads / ns * ns;
  int ca = 0, cb = 0;
  const bool turns = item_chunks<HALF>(item, pairs, p.head_dim, &ca, &cb);
  const int gap = cb - ca;              // distance of the second chunk
  unsigned long long f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = s_f[min(pair_of<HALF>(item, e, p.head_dim), kMaxPairs - 1)];
  long long from[kItems], to[kItems];   // offsets of the item's first chunk in x and out
  int at[kItems], head[kItems];         // its token (or none) and head in the unit
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int i = threadIdx.x + k * pass;
    const int t = i / (hb * ns), h = (i - t * hb * ns) / ns;
    at[k] = threadIdx.x < pass && t < tok ? t : 1 << 30;
    head[k] = h;
    from[k] = t * p.x_tok + h * p.x_head + ca;
    to[k] = t * p.y_tok + h * p.y_head + ca;
  }
  pdl_wait();
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long t0 = u / nhb * tok;
    const int h0 = (int)(u % nhb) * hb;
    const int nt = (int)min((long long)tok, p.tokens - t0);
    const E* x = static_cast<const E*>(p.x) + t0 * p.x_tok + (long long)h0 * p.x_head;
    E* y = static_cast<E*>(p.out) + t0 * p.y_tok + (long long)h0 * p.y_head;
    Vec8<E> a[kItems], b[kItems];
    int pos[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if (at[k] < nt && h0 + head[k] < p.heads) {
        a[k].load(x + from[k]);
        b[k].load(x + from[k] + gap);
        pos[k] = load_len(p.positions + t0 + at[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if (at[k] < nt && h0 + head[k] < p.heads) {
        if (turns) {
          Turn8 turn;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 c0 = turn_at<sizeof(E) == 4>(f[2 * e], pl.scale, pl.sign, pos[k]);
            const float2 c1 = turn_at<sizeof(E) == 4>(f[2 * e + 1], pl.scale, pl.sign, pos[k]);
            turn.cs[e] = make_float4(c0.x, c1.x, c0.y, c1.y);
          }
          rotate_item<HALF>(a[k], b[k], turn, item, pairs, p.head_dim);
        }
        a[k].store(y + to[k]);
        b[k].store(y + to[k] + gap);
      }
    }
  }
}

// The same for shapes and strides without 16-byte chunks: one thread per channel pair.
template <typename E, bool HALF>
__global__ void __launch_bounds__(kRopeThreads)
    rope_scalar_kernel(const __grid_constant__ Turns pl, RopeProblem p, int tok) {
  extern __shared__ float2 s_cs[];
  pdl_trigger();
  pdl_wait();
  const int pairs = pl.pairs;
  const long long t0 = (long long)blockIdx.x * tok;
  const int nt = (int)min((long long)tok, p.tokens - t0);
  for (int i = threadIdx.x; i < nt * pairs; i += kRopeThreads) {
    const int t = i / pairs;
    s_cs[i] = turn_at<true>(pl.f[i - t * pairs], pl.scale, pl.sign, load_len(p.positions + t0 + t));
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
//
// One warp per token (warps stride over the tokens): lane l holds channels of item l % 8 of heads
// l / 8, l / 8 + 4, ... of q, and of k and v, so that the 8 pairs it turns are the same for all of them. The lanes
// compute two pairs' cosines and sines each, exchange them through the warp's shared memory, and
// keep their eight in registers. No barrier of the block, no division per item.
constexpr int kAppendWarps = 1;         // per block
constexpr int kAppendCtas = 16;         // blocks per SM (24 warps, with spills: 32.5 us for 16384 tokens, 16: 29.9)
constexpr int kAppendQ = 4;             // q heads a lane keeps in flight, besides one of k or v

// kWhole: the whole head turns. kPart: part of it. kScalar: no 16-byte chunks (half layout, rotary_dim
// not a multiple of 16). The first is a form of its own because it needs no test per lane and pair.
enum AppendForm { kWhole, kPart, kScalar };

template <bool HALF, AppendForm FORM>
__global__ void __launch_bounds__(32 * kAppendWarps, kAppendCtas)
    rope_append_kernel(const __grid_constant__ Turns pl, RopeAppendProblem p) {
  using E = __nv_bfloat16;
  __shared__ __align__(16) float s_table[kAppendWarps][kHeadDim];
  constexpr bool SCALAR = FORM == kScalar;
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* table = s_table[warp];
  const int pairs = FORM == kWhole ? kHeadDim / 2 : pl.pairs;
  const int heads = p.Hq + 2 * p.Hkv;
  const int s = lane & 7, g = lane >> 3;
  // The lane's two pairs of the table: the float4 at [g][s] (see Turn8).
  const int own = pair_of<HALF>(s, 2 * g, kHeadDim);
  const unsigned long long f0 = own < pairs ? pl.f[own] : 0, f1 = own + 1 < pairs ? pl.f[own + 1] : 0;
  int ca, cb;
  const bool turns = item_chunks<HALF>(s, pairs, kHeadDim, &ca, &cb) || FORM == kWhole;
  pdl_wait();
  const int tokens = p.B * p.T, step = gridDim.x * kAppendWarps;
  const bool whole_q = (p.Hq & 3) == 0;
  for (int tok = blockIdx.x * kAppendWarps + warp; tok < tokens; tok += step) {
    // Heads g, g + 4, ... of q: where there are fewer, a lane repeats the last one (the same values to
    // the same place), so that the loops are the warp's, not the lane's. Heads of k and v: e < Hkv is
    // k's, then v's.
    const E* qs = p.q + (long long)tok * p.q_tok;
    const E* ks = p.k_new + (long long)tok * p.k_tok;
    const E* vs = p.v_new + (long long)tok * p.v_tok;
    auto kv_source = [&](int e) { return e < p.Hkv ? ks + e * kHeadDim : vs + (e - p.Hkv) * kHeadDim; };
    auto q_head = [&](int h) { return whole_q ? h + g : min(h + g, p.Hq - 1); };
    Vec8<E> a[kAppendQ], b[kAppendQ], ka, kb;
    auto load_q = [&](int h0) {
#pragma unroll
      for (int k = 0; k < kAppendQ; ++k) {
        if (h0 + 4 * k < p.Hq) {
          const E* src = qs + q_head(h0 + 4 * k) * kHeadDim;
          a[k].load(src + ca);
          b[k].load(src + cb);
        }
      }
    };
    auto load_kv = [&](int e) {
      if (e < 2 * p.Hkv) {
        const E* src = kv_source(e);
        ka.load(src + ca);
        kb.load(src + cb);
      }
    };
    if (!SCALAR) {                      // in flight while the slot and the angles are worked out
      load_q(0);
      load_kv(g);
    }
    const int sq = tok / p.T, i = tok - sq * p.T;
    const int P = p.seq_lens ? load_len(p.seq_lens + sq) : 0;
    const int w = p.row_lens ? load_len(p.row_lens + sq) : p.T;
    const long long pos = (long long)(p.pos0 ? load_len(p.pos0 + sq) : P) + i;
    // Padding, or a sequence whose lengths are invalid: nothing is written.
    if (P < 0 || w < 0 || w > p.T || (long long)P + w > p.S || i >= w) continue;
    const int slot = P + i;
    long long row, head_rows;           // cache row of KV head 0 (-1: none), rows between heads
    if (p.block_table) {
      const int page = load_len(p.block_table + (size_t)sq * p.pages_per_seq + slot / p.page_size);
      row = page >= 0 && page < p.num_pages ? (long long)page * p.Hkv * p.page_size + slot % p.page_size : -1;
      head_rows = p.page_size;
    } else {
      row = (long long)sq * p.Hkv * p.S + slot;
      head_rows = p.S;
    }
    if (p.key_pos && row >= 0)
      for (int h = lane; h < p.Hkv; h += 32) p.key_pos[((size_t)sq * p.Hkv + h) * p.S + slot] = (int)pos;
    E* qd = p.q_out + (long long)tok * p.Hq * kHeadDim;
    auto kv_target = [&](int e) {
      return (e < p.Hkv ? p.kc + (row + e * head_rows) * kHeadDim
                        : p.vc + (row + (e - p.Hkv) * head_rows) * kHeadDim);
    };
    __syncwarp();                       // the previous token's table has been read
    if (own < pairs) {
      const float2 c0 = turn_at<false>(f0, pl.scale, pl.sign, pos), c1 = turn_at<false>(f1, pl.scale, pl.sign, pos);
      reinterpret_cast<float4*>(table)[g * kItemsOfHead + s] = make_float4(c0.x, c1.x, c0.y, c1.y);
    }
    __syncwarp();
    if (SCALAR) {
      for (int it = lane; it < heads * (kHeadDim / 2); it += 32) {
        const int h = it / (kHeadDim / 2), j = it % (kHeadDim / 2);
        if (h >= p.Hq && row < 0) continue;
        E* dst = h < p.Hq ? p.q_out + ((long long)tok * p.Hq + h) * kHeadDim : kv_target(h - p.Hq);
        const E* src = h < p.Hq ? p.q + (long long)tok * p.q_tok + h * kHeadDim : kv_source(h - p.Hq);
        const int xa = (HALF && j < pairs) ? j : 2 * j, xb = (HALF && j < pairs) ? j + pairs : 2 * j + 1;
        const E ea = src[xa], eb = src[xb];
        if (j < pairs && h < p.Hq + p.Hkv) {
          const float* at = table + 4 * (((j & 7) >> 1) * kItemsOfHead + (j >> 3)) + (j & 1);
          const float2 c = make_float2(at[0], at[2]);
          const float u = to_f32(ea), v = to_f32(eb);
          dst[xa] = __float2bfloat16_rn(fmaf(u, c.x, -(v * c.y)));
          dst[xb] = __float2bfloat16_rn(fmaf(v, c.x, u * c.y));
        } else {
          dst[xa] = ea;
          dst[xb] = eb;
        }
      }
      continue;
    }
    Turn8 turn;
    if (turns) turn.load(table, s);
    for (int h0 = 0;;) {
#pragma unroll
      for (int k = 0; k < kAppendQ; ++k) {
        if (h0 + 4 * k < p.Hq) {
          if (turns) rotate_item<HALF>(a[k], b[k], turn, s, pairs, kHeadDim);
          E* dst = qd + q_head(h0 + 4 * k) * kHeadDim;
          a[k].store(dst + ca);
          b[k].store(dst + cb);
        }
      }
      h0 += 4 * kAppendQ;
      if (h0 >= p.Hq) break;
      load_q(h0);
      if (!whole_q) __syncwarp();       // in place, a repeated head is read by every lane before one writes it
    }
    if (row < 0) continue;
    for (int e = g; e < 2 * p.Hkv;) {
      if (turns && e < p.Hkv) rotate_item<HALF>(ka, kb, turn, s, pairs, kHeadDim);
      E* dst = kv_target(e);
      ka.store(dst + ca);
      kb.store(dst + cb);
      e += 4;
      load_kv(e);
    }
  }
}

template <typename E>
cudaError_t launch_rope_t(const la_rope_plan& plan, const RopeProblem& p, bool vec, int sms, cudaStream_t s) {
  const Turns pl = turns_of(plan, p.inverse);
  const bool half = plan.layout == LA_ROPE_HALF;
  const int pairs = pl.pairs;
  if (vec) {
    // One set of items for every thread: whole tokens, or a block of one token's heads.
    const int ns = p.head_dim / 16, heads = kRopeThreads / ns * kItemsOf<E>;   // of a unit, over its tokens
    const int hb = p.heads < heads ? p.heads : heads;
    long long tok = heads / hb;
    if (tok > p.tokens / (2 * sms)) tok = p.tokens / (2 * sms);   // few tokens: spread over the SMs
    if (tok < 1) tok = 1;
    const long long units = (p.tokens + tok - 1) / tok * ((p.heads + hb - 1) / hb);
    const long long full = (long long)rope_ctas(half) * sms;
    const dim3 grid((unsigned)(units < full ? units : full));
    return launch_pdl(half ? rope_kernel<E, true> : rope_kernel<E, false>, grid, dim3(kRopeThreads), 0, s, pl, p,
                      (int)tok, hb);
  }
  // Tokens per block: a few pairs for every thread, at most 32 KB of cosines and sines, and (few
  // tokens) no more than spreads them over the SMs.
  long long tok = 4LL * kRopeThreads / (p.heads * (p.head_dim / 2));
  if (tok > 4096 / pairs) tok = 4096 / pairs;
  if (tok > p.tokens / (2 * sms)) tok = p.tokens / (2 * sms);
  if (tok < 1) tok = 1;
  const dim3 grid((unsigned)((p.tokens + tok - 1) / tok));
  return launch_pdl(half ? rope_scalar_kernel<E, true> : rope_scalar_kernel<E, false>, grid, dim3(kRopeThreads),
                    (size_t)tok * pairs * sizeof(float2), s, pl, p, (int)tok);
}

}  // namespace

cudaError_t launch_rope(const la_rope_plan& pl, const RopeProblem& p, int dtype, int sms, cudaStream_t s) {
  const int es = dtype == LA_DTYPE_F32 ? 4 : 2;
  auto al = [&](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  auto st = [&](long long n) { return n * es % 16 == 0; };
  // 16-byte chunks need aligned rows, and in the half layout both halves of a pair chunk-aligned.
  const bool vec = p.head_dim % 16 == 0 && (pl.layout == LA_ROPE_INTERLEAVED || pl.rotary_dim % 16 == 0) &&
                   al(p.x) && al(p.out) && st(p.x_tok) && st(p.x_head) && st(p.y_tok) && st(p.y_head);
  switch (dtype) {
    case LA_DTYPE_F32: return launch_rope_t<float>(pl, p, vec, sms, s);
    case LA_DTYPE_BF16: return launch_rope_t<__nv_bfloat16>(pl, p, vec, sms, s);
    case LA_DTYPE_F16: return launch_rope_t<__half>(pl, p, vec, sms, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_rope_append(const la_rope_plan& plan, const RopeAppendProblem& p, int sms, cudaStream_t s) {
  // One warp per token while they fit on the GPU at once, else as many tokens in turn.
  const int tokens = p.B * p.T;
  const int full = kAppendCtas * sms, blocks = (tokens + kAppendWarps - 1) / kAppendWarps;
  const dim3 grid((unsigned)(blocks < full ? blocks : full)), block(32 * kAppendWarps);
  const Turns pl = turns_of(plan, false);
  const bool half = plan.layout == LA_ROPE_HALF;
#define LA_APPEND(HALF, FORM) launch_pdl(rope_append_kernel<HALF, FORM>, grid, block, 0, s, pl, p)
  if (plan.rotary_dim == kHeadDim) return half ? LA_APPEND(true, kWhole) : LA_APPEND(false, kWhole);
  if (half && plan.rotary_dim % 16 != 0) return LA_APPEND(true, kScalar);
  return half ? LA_APPEND(true, kPart) : LA_APPEND(false, kPart);
#undef LA_APPEND
}

}  // namespace la
