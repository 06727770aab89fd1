// The indexer's inputs from a projection's rows: E4M3 queries with one scale a
// head, NVFP4 keys written into the index-K pages.
//
// A row x of 128 elements is normed (r = 1 / sqrt(mean x^2 + eps)) and turned
// as in idx_norm_rope_append, y = r u with u = x cw + x_p sw.  A query's codes
// are those of 448 u / max|u|: r cancels, and only the scale has it.  A key's
// blocks of 16 take s = e4m3(max|y| / 6) ("vllm ... gather_nvfp4_index_k": no
// global scale) and codes e2m1(y / s).
//
// The codes are those of 64-bit arithmetic.  Sines and cosines are formed to
// 2^-44, once a token, by their Taylor series.  In units of 2^-24 of M = |x cw| +
// |x_p sw|, u comes in fp32 with an error of at most 4, the sines' 1, their products
// with weights 1, and 1 each of |x_p sw| and of |u| for product and sum; or of 5
// where the sum of weight and offset is rounded.  M of the pair of the largest element
// is at most sqrt 2 times that, so its own error is at most 3 sqrt 2 + 1 (4 sqrt 2 +
// 1); the scaling adds 5, the ends' rounding 1: 15.3 M for 448 u / max|u| (17.7;
// kSlack is 15.6, kSlackSums 17.9 units).  A norm's r is off by 9, a key's y / s by 18
// M in all (kSlackKey 20.1).  So each element is converted at both ends
// of kSlack (kSlackKey) times M around it; where the two codes differ (0.5% of
// the rows) the element is formed again as a pair of fp32 numbers (exact products,
// 2^-44) and compared with the middle between the codes.  A key whose codes or
// scales may differ is formed again as a whole, in 64 bits.
//
// Bound by the instructions of a row (about 220 a warp for two heads) and by their
// latency: the issue slots are 63% full with 16 warps an SM.  8,191 tokens of 64
// heads take 90 us, 0.34 of HBM (fp32 87, 0.59); without the look for borders 68,
// with 64-bit floating point for the elements near one 91, for the angles about
// 20 more; 4 and 6 CTAs of 128 threads an SM 91 and 95.  512 tokens of 4 heads take
// 8 us.  A query's row is 16 lanes', both elements of a pair in one (passed between
// lanes they took as long); cosines, sines and weights are folded into a lane's
// factors once a token; a lane forms the scale of one row in 16.  Every warp takes
// as many batches of heads as the others, whichever tokens they are of (whole parts
// of tokens left SMs idle: 105).  Rows near a border put off to the end of a CTA and
// shared among its warps took 97.  A key's row keeps 8 elements in a row a lane: two
// lanes have a block.
#include "idx_internal.h"
#include "idx_rope.cuh"

namespace idx {
namespace {

constexpr int kThreadsI = 128;
constexpr int kCtasI = 5;    // of an SM
constexpr int kBatchI = 2;  // rows in flight a lane
constexpr int kLanesI = 16;  // of a row
constexpr int kLookI = 4;    // rows in flight a lane of k_index_small
constexpr float kSlack = 9.3e-7f, kSlackSums = 1.07e-6f, kSlackKey = 1.2e-6f;
constexpr float kSmallI = 0x1p-96f;  // a mean of squares with eps below it is formed again: fp32 holds the squares with fewer bits, or none

struct IndexArgs {
  const void *q, *k;
  int64_t q_ts, q_hs, k_ts;
  int32_t heads, num_tokens, rotary_dim;
  const void *q_w, *k_w;
  float eps, offset, mscale, scale;
  const int32_t* positions;
  const double* inv_freq;
  uint8_t* q_out;
  float* q_scale;
  const float* head_weights;
  const int32_t* cu;
  int32_t num_reqs, req_slots;
  const int64_t* slots;
  uint8_t* index_k;
  int64_t num_slots;
  int32_t page;
  int32_t* status;
};

// Two fp32 values to E2M1, to nearest even, at most 6 in magnitude; `lo` in bits 0-3.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight elements of a row as words.
template <typename T>
struct Eight {
  static constexpr int kN = 2 * (int)sizeof(T);
  uint32_t w[kN];
};
template <typename T, bool kWide>
__device__ __forceinline__ Eight<T> load8(const T* p) {
  Eight<T> x;
  if (kWide) {
#pragma unroll
    for (int i = 0; i < Eight<T>::kN / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      x.w[4 * i] = v.x, x.w[4 * i + 1] = v.y, x.w[4 * i + 2] = v.z, x.w[4 * i + 3] = v.w;
    }
  } else if (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < Eight<T>::kN; ++i) x.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < Eight<T>::kN; ++i)
      x.w[i] = (uint32_t) reinterpret_cast<const uint16_t*>(p)[2 * i] | (uint32_t) reinterpret_cast<const uint16_t*>(p)[2 * i + 1] << 16;
  }
  return x;
}

// The same as two fours, from p and q on.
template <typename T, bool kWide>
__device__ __forceinline__ Eight<T> load4x2(const T* p, const T* q) {
  Eight<T> x;
  constexpr int kN = Eight<T>::kN / 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const T* from = i == 0 ? p : q;
    if (kWide && sizeof(T) == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(from);
      x.w[kN * i] = v.x, x.w[kN * i + 1] = v.y, x.w[kN * i + kN - 2] = v.z, x.w[kN * i + kN - 1] = v.w;
    } else if (kWide) {
      const uint2 v = *reinterpret_cast<const uint2*>(from);
      x.w[kN * i] = v.x, x.w[kN * i + 1] = v.y;
    } else if (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < kN; ++e) x.w[kN * i + e] = reinterpret_cast<const uint32_t*>(from)[e];
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e)
        x.w[kN * i + e] = (uint32_t) reinterpret_cast<const uint16_t*>(from)[2 * e] | (uint32_t) reinterpret_cast<const uint16_t*>(from)[2 * e + 1] << 16;
    }
  }
  return x;
}

// A number as hi + lo, hi the nearest fp32 to it.  Sums are Dekker's (two_sum) and Knuth's (exact_sum, plus), products take
// their error from a fused multiply-add.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {  // |a| >= |b| or a = 0
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two exact_sum(float a, float b) {  // of any magnitudes
  const float s = __fadd_rn(a, b), from_b = __fsub_rn(s, a), lo = __fadd_rn(__fsub_rn(a, __fsub_rn(s, from_b)), __fsub_rn(b, from_b));
  return {s, lo == lo ? lo : 0.f};  // (of an infinity nothing is left out)
}
__device__ __forceinline__ Two times(Two a, Two b) {
  const float p = __fmul_rn(a.hi, b.hi);
  return two_sum(p, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.hi, -p))));
}
__device__ __forceinline__ Two plus(Two a, Two b) {  // of any magnitudes, to 2^-46 of the larger one
  const float s = __fadd_rn(a.hi, b.hi), from_b = __fsub_rn(s, a.hi);
  const float lo = __fadd_rn(__fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, from_b)), __fsub_rn(b.hi, from_b)), __fadd_rn(a.lo, b.lo));
  const float t = __fadd_rn(s, lo), from_lo = __fsub_rn(t, s);
  return {t, __fadd_rn(__fsub_rn(s, __fsub_rn(t, from_lo)), __fsub_rn(lo, from_lo))};
}
__device__ __forceinline__ Two negative(Two a) { return {-a.hi, -a.lo}; }
__device__ __forceinline__ Two magnitude(Two a) { return a.hi < 0.f || (a.hi == 0.f && a.lo < 0.f) ? negative(a) : a; }
__device__ __forceinline__ bool above(Two a, Two b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
// c + a b, where |c| is larger than |a b|
__device__ __forceinline__ Two plus_times(Two c, Two a, Two b) {
  const Two p = times(a, b), s = two_sum(c.hi, p.hi);
  return two_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(c.lo, p.lo)));
}
__host__ __device__ constexpr Two two_of(double x) { return Two{(float)x, (float)(x - (double)(float)x)}; }

// cos and sin of 2 pi phase / 2^64, to about 2^-44: the phase less its nearest quarter turn, then the Taylor series in pairs
// of fp32 numbers (its later terms in one), |y| <= pi / 4.  (64-bit floating point gives two results a clock and SM here; a
// token's angles took 12 us of 8,191 tokens.)
__device__ __forceinline__ void turn_of_two(unsigned long long phase, Two* cosine, Two* sine) {
  const unsigned long long quarter = (phase + (1ull << 61)) >> 62;
  const long long rest = (long long)(phase - (quarter << 62));  // |rest| <= 2^61
  const long long top = (rest + (1ll << 37)) >> 38;             // 24 bits, then the 38 below
  constexpr Two kStep = two_of(6.283185307179586 / 67108864.0);  // 2 pi / 2^26: a unit of top
  const Two y = times(Two{(float)(int)top, (float)(rest - (top << 38)) * 3.637978807091713e-12f}, kStep);  // 2^-38
  const Two z = times(y, y);
  constexpr Two s3 = two_of(-1.0 / 6.0), s5 = two_of(1.0 / 120.0), s7 = two_of(-1.0 / 5040.0);
  constexpr Two c4 = two_of(1.0 / 24.0), c6 = two_of(-1.0 / 720.0), c8 = two_of(1.0 / 40320.0);
  float s = fmaf(z.hi, (float)(1.0 / 6227020800.0), (float)(-1.0 / 39916800.0));
  s = fmaf(z.hi, s, (float)(1.0 / 362880.0));
  float c = fmaf(z.hi, (float)(-1.0 / 87178291200.0), (float)(1.0 / 479001600.0));
  c = fmaf(z.hi, c, (float)(-1.0 / 3628800.0));
  Two sp = plus_times(s7, z, Two{s, 0.f});
  sp = plus_times(s3, z, plus_times(s5, z, sp));
  Two cp = plus_times(c8, z, Two{c, 0.f});
  cp = plus_times(Two{-0.5f, 0.f}, z, plus_times(c4, z, plus_times(c6, z, cp)));
  const Two sn = plus_times(y, times(y, z), sp), cn = plus_times(Two{1.f, 0.f}, z, cp);
  const Two a = quarter & 1ull ? Two{-sn.hi, -sn.lo} : cn, b = quarter & 1ull ? cn : sn;
  *cosine = quarter & 2ull ? Two{-a.hi, -a.lo} : a, *sine = quarter & 2ull ? Two{-b.hi, -b.lo} : b;
}

// A weight, with the offset, as the CTA keeps it.
__device__ __forceinline__ Two weight_of(const float* w, int e) { return {w[e], w[kHeadDim + e]}; }

// A row as its elements are formed in 64 bits.
template <typename T>
struct Row64 {
  const T* x;
  const float* w;
  const float4* turns;  // of the token's pairs: cosines (hi, lo), then sines
  int rd;
  __device__ __forceinline__ double weight(int e) const { return (double)w[e] + (double)w[kHeadDim + e]; }
  template <bool kInter>
  __device__ __forceinline__ double u(int e) const {
    const double n = (double)to_f(x[e]) * weight(e);
    if (e >= rd) return n;
    const int half = rd / 2, pair = kInter ? e / 2 : e < half ? e : e - half;
    const int mate = kInter ? e ^ 1 : e < half ? e + half : e - half;
    const bool second = kInter ? e & 1 : e >= half;
    const float4 t = turns[pair];
    const double2 cs = make_double2((double)t.x + (double)t.y, (double)t.z + (double)t.w);
    const double o = (double)to_f(x[mate]) * weight(mate);
    return second ? fma(n, cs.x, o * cs.y) : fma(n, cs.x, -(o * cs.y));
  }
};

// The same as pairs of fp32 numbers: products of elements and weights to 2^-46, turned ones to 2^-44.
template <typename T, bool kInter>
__device__ __forceinline__ Two element_of(const T* x, const float* w, const float4* turns, int rd, int e) {
  const Two n = times(Two{to_f(x[e]), 0.f}, weight_of(w, e));
  if (e >= rd) return n;
  const int half = rd / 2, pair = kInter ? e / 2 : e < half ? e : e - half;
  const int mate = kInter ? e ^ 1 : e < half ? e + half : e - half;
  const bool second = kInter ? e & 1 : e >= half;
  const float4 t = turns[pair];
  const Two o = times(times(Two{to_f(x[mate]), 0.f}, weight_of(w, mate)), Two{t.z, t.w});
  return plus(times(n, Two{t.x, t.y}), second ? o : negative(o));
}

__device__ __forceinline__ double shfl_xor_64(double x, int o) {
  return __hiloint2double(__shfl_xor_sync(0xFFFFFFFFu, __double2hiint(x), o), __shfl_xor_sync(0xFFFFFFFFu, __double2loint(x), o));
}

// A key's lane again: scale (in y) and codes (in x) of its 8 elements.  All lanes together.
template <typename T, bool kInter>
__device__ __noinline__ uint2 key_64(const Row64<T> row, int at, bool normed, float eps) {
  double u[8], ss = 0.0, top = 0.0;
  for (int e = 0; e < 8; ++e) {
    const double x = (double)to_f(row.x[at + e]);
    ss = fma(x, x, ss), u[e] = row.template u<kInter>(at + e), top = fmax(top, fabs(u[e]));
  }
#pragma unroll
  for (int o = 1; o < kLanesI; o <<= 1) ss += shfl_xor_64(ss, o);
  top = fmax(top, shfl_xor_64(top, 1));
  const double r = normed ? 1.0 / sqrt(ss * (1.0 / kHeadDim) + (double)eps) : 1.0;
  const double six = top * r / 6.0;
  if (!(six >= 0.0)) return make_uint2(0u, 0x7Fu);  // (zeros without eps)
  uint32_t scale = f32x2_to_e4m3x2(__double2float_rz(six) * (1.f - kSlackKey), 0.f) & 0x7Fu;
  if (scale > 0) --scale;
  for (; scale < 0x7Eu; ++scale) {
    const double edge = 0.5 * ((double)e4m3_to_f32(scale) + (double)e4m3_to_f32(scale + 1));
    if (!(six > edge || (six == edge && (scale & 1u)))) break;
  }
  uint32_t codes = 0;
  const double s = (double)e4m3_to_f32(scale);
  for (int e = 0; e < 8 && scale != 0; ++e) {
    const double z = fabs(u[e]) * r / s;
    // borders between the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6, halves to the even code
    const uint32_t code = (z > 0.25) + (z >= 0.75) + (z > 1.25) + (z >= 1.75) + (z > 2.5) + (z >= 3.5) + (z > 5.0);
    codes |= (code | (u[e] < 0.0 ? 8u : 0u)) << (4 * e);
  }
  return make_uint2(codes, scale);
}

// What a lane knows of its piece of a row: factors, u = x c + x_p s, and where x_p is.
struct Piece8 {
  float2 c[4], s[4];
};
struct Place {
  int at, angle, mate, partner;  // first element, pair and partner's first element; the lane that has it
  bool turns, upper;
};
template <bool kInter>
__device__ __forceinline__ Place place_of(int lane, int rd) {
  Place p;
  p.at = lane % kLanesI * 8;
  // a pair's other half lies a whole number of pieces away (rotary_dim a multiple of 16, or of 8 with neighbours paired)
  p.turns = p.at < rd, p.upper = !kInter && p.at >= rd / 2;
  const int hop = p.turns && !kInter ? (p.upper ? -(rd / 16) : rd / 16) : 0;
  p.partner = lane + hop, p.mate = p.at + 8 * hop, p.angle = kInter ? p.at / 2 : p.upper ? p.at - rd / 2 : p.at;
  return p;
}
template <bool kInter>
__device__ __forceinline__ Piece8 factors_of(const Place& p, const float* w, const float4* turns) {
  Piece8 f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float w0 = w[p.at + 2 * e], w1 = w[p.at + 2 * e + 1];
    if (p.turns && kInter) {
      const float x = turns[p.angle + e].x, y = turns[p.angle + e].z;
      f.c[e] = make_float2(x * w0, x * w1), f.s[e] = make_float2(-y * w1, y * w0);
    } else if (p.turns) {
      const float4 t0 = turns[p.angle + 2 * e], t1 = turns[p.angle + 2 * e + 1];
      const float y0 = t0.z * w[p.mate + 2 * e], y1 = t1.z * w[p.mate + 2 * e + 1];
      f.c[e] = make_float2(t0.x * w0, t1.x * w1);
      f.s[e] = p.upper ? make_float2(y0, y1) : make_float2(-y0, -y1);
    } else {
      f.c[e] = make_float2(w0, w1), f.s[e] = make_float2(0.f, 0.f);
    }
  }
  return f;
}
// u of a lane's elements and M, which their errors go by; returns the sum of squares of the elements.
template <typename T, bool kInter>
__device__ __forceinline__ float turn8(const Eight<T>& x, const Place& p, const Piece8& f, float2 (&u)[4], float2 (&mag)[4]) {
  Eight<T> y;
  if (!kInter) {
#pragma unroll
    for (int e = 0; e < Eight<T>::kN; ++e) y.w[e] = __shfl_sync(0xFFFFFFFFu, x.w[e], p.partner);
  }
  float2 ss = make_float2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 one = Words<T>::get(x.w, e), two = kInter ? make_float2(one.y, one.x) : Words<T>::get(y.w, e);
    const float2 part = mul2(two, f.s[e]);
    u[e] = fma2(one, f.c[e], part);
    const float2 own = fma2(part, make_float2(-1.f, -1.f), u[e]);  // x cw, but for a rounding of u
    mag[e] = make_float2(fabsf(own.x) + fabsf(part.x), fabsf(own.y) + fabsf(part.y));
    ss = fma2(one, one, ss);
  }
  return ss.x + ss.y;
}
// A query's lane has both elements of its pairs: fours of elements from a0 and from a1 on.
struct Fours {
  int a0, a1;
  bool turns;
};
template <bool kInter>
__device__ __forceinline__ Fours fours_of(int lane, int rd) {
  const int piece = lane % kLanesI;
  if (!kInter && 8 * piece < rd) return {4 * piece, rd / 2 + 4 * piece, true};
  return {8 * piece, 8 * piece + 4, 8 * piece < rd};
}
template <bool kInter>
__device__ __forceinline__ Piece8 factors_of(const Fours& p, const float* w, const float4* turns) {
  Piece8 f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = (e < 2 ? p.a0 : p.a1) + 2 * (e & 1), mate = (e < 2 ? p.a1 : p.a0) + 2 * (e & 1);
    const float w0 = w[i], w1 = w[i + 1];
    if (p.turns && kInter) {
      const float x = turns[i / 2].x, y = turns[i / 2].z;
      f.c[e] = make_float2(x * w0, x * w1), f.s[e] = make_float2(-y * w1, y * w0);
    } else if (p.turns) {
      const float4 t0 = turns[p.a0 + 2 * (e & 1)], t1 = turns[p.a0 + 2 * (e & 1) + 1];
      const float y0 = t0.z * w[mate], y1 = t1.z * w[mate + 1];
      f.c[e] = make_float2(t0.x * w0, t1.x * w1);
      f.s[e] = e < 2 ? make_float2(-y0, -y1) : make_float2(y0, y1);
    } else {
      f.c[e] = make_float2(w0, w1), f.s[e] = make_float2(0.f, 0.f);
    }
  }
  return f;
}
template <typename T, bool kInter>
__device__ __forceinline__ float turn4x2(const Eight<T>& x, const Piece8& f, float2 (&u)[4], float2 (&mag)[4]) {
  float2 one[4], ss = make_float2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 4; ++e) one[e] = Words<T>::get(x.w, e);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 part = mul2(kInter ? make_float2(one[e].y, one[e].x) : one[e ^ 2], f.s[e]);
    u[e] = fma2(one[e], f.c[e], part);
    const float2 own = fma2(part, make_float2(-1.f, -1.f), u[e]);  // x cw, but for a rounding of u
    mag[e] = make_float2(fabsf(own.x) + fabsf(part.x), fabsf(own.y) + fabsf(part.y));
    ss = fma2(one[e], one[e], ss);
  }
  return ss.x + ss.y;
}
__device__ __forceinline__ float largest8(const float2 (&u)[4]) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) m = fmaxf(m, fmaxf(fabsf(u[e].x), fabsf(u[e].y)));
  return m;
}
// Codes of both ends of where 448 u / top may lie: pairs of elements in 16 bits.
__device__ __forceinline__ float inverse_of(float top) { return top > 7.9e-31f ? __fdividef(448.f, top) : 0.f; }
__device__ __forceinline__ void both_ends(const float2 (&u)[4], const float2 (&mag)[4], float inv, float slack, uint32_t (&low)[4], uint32_t (&high)[4]) {
  slack *= inv;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 v = mul2(u[e], make_float2(inv, inv));
    const float2 l = fma2(mag[e], make_float2(-slack, -slack), v), t = fma2(mag[e], make_float2(slack, slack), v);
    low[e] = f32x2_to_e4m3x2(l.x, l.y), high[e] = f32x2_to_e4m3x2(t.x, t.y);
  }
}

// A query's row again, whose codes may not all be right: those that lie near a border in pairs of fp32 numbers
// (in 64-bit floating point, which is slow here, it took 15 us of 8,191 tokens).  Each half of the warp has
// a row of its own; all lanes together.
template <typename T, bool kInter, bool kWide>
__device__ __noinline__ void again(const T* x, const float* w, const float4* turns, int rd, uint8_t* out, bool live) {
  const Place p = place_of<kInter>(threadIdx.x & 31, rd);
  float2 u[4], mag[4];
  float ss = turn8<T, kInter>(load8<T, kWide>(x + p.at), p, factors_of<kInter>(p, w, turns), u, mag), most = largest8(u);
#pragma unroll
  for (int o = 1; o < kLanesI; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o), most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
  uint32_t low[4], high[4], near = 0, tops = 0;
  both_ends(u, mag, inverse_of(most), kSlackSums, low, high);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if ((low[e / 2] ^ high[e / 2]) >> (8 * (e % 2)) & 0xFFu) near |= 1u << e;
    if (fabsf(e % 2 ? u[e / 2].y : u[e / 2].x) >= most * (1.f - 4.f * kSlackSums)) tops |= 1u << e;
  }
  uint32_t codes[2] = {__byte_perm(low[0], low[1], 0x5410), __byte_perm(low[2], low[3], 0x5410)};
  if (!(ss <= 3.4e38f) || inverse_of(most) == 0.f) live = false, near = tops = 0;  // (its codes stand)
  Two top{0.f, 0.f};  // the largest magnitude
  for (uint32_t m = tops; m != 0; m &= m - 1) {
    const Two y = magnitude(element_of<T, kInter>(x, w, turns, rd, p.at + __ffs(m) - 1));
    if (above(y, top)) top = y;
  }
#pragma unroll
  for (int o = 1; o < kLanesI; o <<= 1) {
    const Two y{__shfl_xor_sync(0xFFFFFFFFu, top.hi, o), __shfl_xor_sync(0xFFFFFFFFu, top.lo, o)};
    if (above(y, top)) top = y;
  }
  const float unit = top.hi > 1.f ? 0x1p-9f : 1.f;  // (448 times the largest may pass fp32's range)
  for (; near != 0; near &= near - 1) {
    const int e = __ffs(near) - 1;
    const Two y = element_of<T, kInter>(x, w, turns, rd, p.at + e), v = times(Two{448.f * unit, 0.f}, magnitude(y));
    // from the lower end's code up while the middle to the next one is (halves to even)
    const uint32_t l = low[e / 2] >> (8 * (e % 2)) & 0xFFu, h = high[e / 2] >> (8 * (e % 2)) & 0xFFu;
    uint32_t code = (l ^ h) & 0x80u ? 0u : min(l, h) & 0x7Fu;
    for (; code < 0x7Eu; ++code) {
      const Two edge = times(Two{0.5f * unit * (e4m3_to_f32(code) + e4m3_to_f32(code + 1)), 0.f}, top);
      if (!(above(v, edge) || (!above(edge, v) && (code & 1u)))) break;
    }
    code |= above(Two{0.f, 0.f}, y) ? 0x80u : 0u;
    codes[e / 4] = (codes[e / 4] & ~(0xFFu << (8 * (e & 3)))) | code << (8 * (e & 3));
  }
  if (live) *reinterpret_cast<uint2*>(out + p.at) = make_uint2(codes[0], codes[1]);
}

// The largest magnitude of a row after its norm, where the mean of its squares, with eps, is small: from the squares of 2^100
// times the elements, which are below 2^56 then.  -1 for other rows.  Each half of the warp has a row of its own.
template <typename T, bool kInter, bool kWide>
__device__ __forceinline__ float small_top(const T* x, const float* w, const float4* turns, int rd, float eps) {
  const Place p = place_of<kInter>(threadIdx.x & 31, rd);
  float2 u[4], mag[4];
  const Eight<T> row = load8<T, kWide>(x + p.at);
  float ss = turn8<T, kInter>(row, p, factors_of<kInter>(p, w, turns), u, mag), most = largest8(u), scaled = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 y = mul2(Words<T>::get(row.w, e), make_float2(0x1p100f, 0x1p100f));
    scaled = fmaf(y.x, y.x, fmaf(y.y, y.y, scaled));
  }
#pragma unroll
  for (int o = 1; o < kLanesI; o <<= 1) {
    ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o), scaled += __shfl_xor_sync(0xFFFFFFFFu, scaled, o);
    most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
  }
  const bool small = fmaf(ss, 1.f / kHeadDim, eps) < kSmallI;
  return small ? most * 0x1p100f * rsqrtf(fmaf(scaled, 1.f / kHeadDim, eps * 0x1p100f * 0x1p100f)) : -1.f;
}

// The request of token t: greatest r with cu[r] <= t, all lanes together.
__device__ __forceinline__ int request_of(const int32_t* cu, int num_reqs, int t, int lane) {
  int lo = 0, hi = num_reqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + step * lane;
    const uint32_t below = __ballot_sync(0xFFFFFFFFu, at < hi && cu[min(at, num_reqs)] <= t);
    lo += step * max(0, __popc(below) - 1);
    hi = min(hi, lo + step);
  }
  return lo;
}

// Frequencies and weights of a CTA; whether a sum of a query's weight and the offset is rounded.
template <typename T>
__device__ __forceinline__ bool prepare(const IndexArgs& a, unsigned long long* steps, float (*weights)[2 * kHeadDim]) {
  for (int i = threadIdx.x; i < a.rotary_dim / 2; i += kThreadsI) steps[i] = step_of(a.inv_freq[i]);
  bool rounded = false;
  for (int i = threadIdx.x; i < kHeadDim; i += kThreadsI) {
    const Two q = a.q_w != nullptr ? exact_sum(a.offset, to_f(static_cast<const T*>(a.q_w)[i])) : Two{1.f, 0.f};
    const Two k = a.k_w != nullptr ? exact_sum(a.offset, to_f(static_cast<const T*>(a.k_w)[i])) : Two{1.f, 0.f};
    weights[0][i] = q.hi, weights[0][kHeadDim + i] = q.lo, weights[1][i] = k.hi, weights[1][kHeadDim + i] = k.lo;
    rounded |= q.lo != 0.f;
  }
  return rounded;
}

// Cosines and sines of a token's pairs, a warp together.
__device__ __forceinline__ void turn_token(const IndexArgs& a, int position, const unsigned long long* steps, float4* turns) {
  for (int i = threadIdx.x & 31; i < a.rotary_dim / 2; i += 32) {
    Two c, s;
    turn_of_two(steps[i] * (unsigned long long)(long long)position, &c, &s);
    c = times(c, Two{a.mscale, 0.f}), s = times(s, Two{a.mscale, 0.f});
    turns[i] = make_float4(c.hi, c.lo, s.hi, s.lo);
  }
}

// The scales of queries whose mean of squares, with eps, is below kSmallI, again: launched after k_index_append where eps is
// below it.  A token's rows are read for their squares first and turned only where one is small: with eps 0 and ordinary rows
// 8,191 tokens of 64 heads take 122 us, 92 with an eps (209 where each row was turned).  In k_index_append, whose registers are
// all taken, it cost 3 to 5 us of calls that need none of it.
template <typename T, bool kInter, bool kWide>
__global__ void __launch_bounds__(kThreadsI) k_index_small(const __grid_constant__ IndexArgs a) {
  pdl_enter();
  __shared__ float4 turns_[kThreadsI / 32][kHeadDim / 2];
  __shared__ unsigned long long steps[kHeadDim / 2];
  __shared__ float weights[2][2 * kHeadDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  prepare<T>(a, steps, weights);
  __syncthreads();
  float4* mine = turns_[warp];
  for (int64_t t = (int64_t)blockIdx.x * (kThreadsI / 32) + warp; t < a.num_tokens; t += (int64_t)gridDim.x * (kThreadsI / 32)) {
    int64_t out = t * a.heads;
    if (a.cu != nullptr) {
      const int r = request_of(a.cu, a.num_reqs, (int)t, lane);
      const int begin = a.cu[r], end = a.cu[r + 1], slot = a.req_slots - end + (int)t;
      if (t < begin || t >= end || slot < 0) continue;
      out = ((int64_t)r * a.req_slots + slot) * a.heads;
    }
    auto row_of = [&](int h) { return static_cast<const T*>(a.q) + t * a.q_ts + (int64_t)min(h, a.heads - 1) * a.q_hs; };
    bool small = false;
    for (int h0 = 0; h0 < a.heads; h0 += 2 * kLookI) {
      Eight<T> x[kLookI];
#pragma unroll
      for (int u = 0; u < kLookI; ++u) x[u] = load8<T, kWide>(row_of(h0 + lane / kLanesI + 2 * u) + lane % kLanesI * 8);
#pragma unroll
      for (int u = 0; u < kLookI; ++u) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 y = Words<T>::get(x[u].w, e);
          ss = fma2(y, y, ss);
        }
        float sum = ss.x + ss.y;
#pragma unroll
        for (int o = 1; o < kLanesI; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        small |= fmaf(sum, 1.f / kHeadDim, a.eps) < kSmallI;
      }
    }
    if (!__any_sync(0xFFFFFFFFu, small)) continue;
    __syncwarp();
    turn_token(a, a.positions[t], steps, mine);
    __syncwarp();
    for (int h0 = 0; h0 < a.heads; h0 += 2) {
      const int h = h0 + lane / kLanesI;
      const float top = small_top<T, kInter, kWide>(row_of(h), weights[0], mine, a.rotary_dim, a.eps);
      if (lane % kLanesI == 0 && h < a.heads && top >= 0.f)
        a.q_scale[out + h] = top * (1.f / 448.f) * a.scale * (a.head_weights != nullptr ? a.head_weights[t * a.heads + h] : 1.f);
    }
  }
}

template <typename T, bool kInter, bool kWide>
__global__ void __launch_bounds__(kThreadsI, kCtasI) k_index_append(const __grid_constant__ IndexArgs a, int64_t warps) {
  pdl_enter();
  __shared__ float4 turns_[kThreadsI / 32][kHeadDim / 2];  // cosines and sines of a warp's token, each in two numbers
  __shared__ unsigned long long steps[kHeadDim / 2];
  __shared__ float weights[2][2 * kHeadDim];  // offset + w of queries and keys, 1 without, then what its rounding left out
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rd = a.rotary_dim, sub = lane / kLanesI, piece = lane % kLanesI;
  const Place p = place_of<kInter>(lane, rd);
  const Fours fours = fours_of<kInter>(lane, rd);
  const int at = p.at;
  const float slack = __syncthreads_or(prepare<T>(a, steps, weights)) ? kSlackSums : kSlack;
  float4* mine = turns_[warp];
  // A token's units: batches of steps of two heads, then its key.  Every warp takes as many units, one after another.
  const int rows = (a.heads + 1) / 2, batches = (rows + kBatchI - 1) / kBatchI, units = batches + (a.k != nullptr ? 1 : 0);
  const int64_t all = (int64_t)a.num_tokens * units, number = (int64_t)blockIdx.x * (kThreadsI / 32) + warp;
  const int64_t last = number < warps ? all * (number + 1) / warps : 0;
  for (int64_t unit = number < warps ? all * number / warps : 0; unit < last;) {
    const int t = (int)(unit / units), first = (int)(unit - (int64_t)t * units), past = (int)min((int64_t)units, first + (last - unit));
    unit += past - first;
    const int position = a.positions[t];
    __syncwarp();  // the angles of the token before are used up
    turn_token(a, position, steps, mine);
    __syncwarp();
    if (first < batches) {
      const Piece8 f = factors_of<kInter>(fours, weights[0], mine);
      int64_t out = (int64_t)t * a.heads;  // the token's first row
      bool stored = true;
      if (a.cu != nullptr) {
        const int r = request_of(a.cu, a.num_reqs, t, lane);
        const int begin = a.cu[r], end = a.cu[r + 1], slot = a.req_slots - end + t;
        stored = t >= begin && t < end && slot >= 0;
        if (t >= begin && t < end && slot < 0 && lane == 0 && first == 0) report(a.status, IDX_ST_BAD_OUTPUT);
        out = ((int64_t)r * a.req_slots + slot) * a.heads;
      }
      const int r0 = first * kBatchI, r1 = min(rows, past * kBatchI);
      const T* row0 = static_cast<const T*>(a.q) + (int64_t)t * a.q_ts;
      if (stored) {
        uint64_t open = 0;  // steps whose codes lie near a border (at most 64 heads' worth: kMtpMaxHeads / 2)
        Eight<T> ahead[kBatchI];
        const T* src = row0 + (int64_t)(2 * r0 + sub) * a.q_hs + fours.a0;
        uint8_t* dst = a.q_out + (out + 2 * r0 + sub) * kHeadDim + fours.a0;
        const int apart = fours.a1 - fours.a0, mine_to = min(r1, (a.heads - sub + 1) / 2);  // this half's steps
        float kept_sq = 0.f, kept_top = 0.f;  // of the step that this lane forms the scale of
        const int64_t step = 2 * a.q_hs;
        auto ask = [&](int g) {
#pragma unroll
          for (int b = 0; b < kBatchI; ++b) {
            if (g + b < mine_to) ahead[b] = load4x2<T, kWide>(src + b * step, src + b * step + apart);
            else ahead[b] = Eight<T>{};
          }
        };
        ask(r0);
        for (int g = r0; g < r1; g += kBatchI) {
          Eight<T> x[kBatchI];
#pragma unroll
          for (int b = 0; b < kBatchI; ++b) x[b] = ahead[b];
          src += kBatchI * step;
          if (g + kBatchI < r1) ask(g + kBatchI);
          float2 u[kBatchI][4], mag[kBatchI][4];
          float ss[kBatchI], top[kBatchI];
#pragma unroll
          for (int b = 0; b < kBatchI; ++b) ss[b] = turn4x2<T, kInter>(x[b], f, u[b], mag[b]), top[b] = largest8(u[b]);
#pragma unroll
          for (int o = 1; o < kLanesI; o <<= 1) {
#pragma unroll
            for (int b = 0; b < kBatchI; ++b) {
              ss[b] += __shfl_xor_sync(0xFFFFFFFFu, ss[b], o);
              top[b] = fmaxf(top[b], __shfl_xor_sync(0xFFFFFFFFu, top[b], o));
            }
          }
#pragma unroll
          for (int b = 0; b < kBatchI; ++b) {
            const float inv = inverse_of(top[b]);
            uint32_t low[4], high[4];
            both_ends(u[b], mag[b], inv, slack, low, high);
            const uint32_t differ = (low[0] ^ high[0]) | (low[1] ^ high[1]) | (low[2] ^ high[2]) | (low[3] ^ high[3]);
            if (differ != 0) open |= 1ull << (g + b - r0);
            uint2 codes = make_uint2(__byte_perm(low[0], low[1], 0x5410), __byte_perm(low[2], low[3], 0x5410));
            if (inv == 0.f || !(ss[b] <= 3.4e38f)) codes = ss[b] <= 3.4e38f ? make_uint2(0u, 0u) : make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
            if (g + b < mine_to) {
              *reinterpret_cast<uint32_t*>(dst + b * 2 * kHeadDim) = codes.x;
              *reinterpret_cast<uint32_t*>(dst + b * 2 * kHeadDim + apart) = codes.y;
            }
            if (piece == ((g + b - r0) & (kLanesI - 1))) kept_sq = ss[b], kept_top = top[b];
          }
          dst += kBatchI * 2 * kHeadDim;
          const int done = g + kBatchI - r0;
          if (done % kLanesI == 0 || g + kBatchI >= r1) {
            // the scales of the last steps, a lane each
            const int step_of_lane = r0 + (done - 1) / kLanesI * kLanesI + piece, h = 2 * step_of_lane + sub;
            if (step_of_lane < mine_to) {
              const float r = a.q_w != nullptr ? rsqrtf(fmaf(kept_sq, 1.f / kHeadDim, a.eps)) : 1.f;
              float scale = kept_top * r * (1.f / 448.f) * a.scale;
              if (a.head_weights != nullptr) scale *= a.head_weights[(int64_t)t * a.heads + h];
              a.q_scale[out + h] = kept_sq <= 3.4e38f ? scale : __int_as_float(0x7FC00000);
            }
          }
        }
        // (a vote for each step took 11 us)
        open = __reduce_or_sync(0xFFFFFFFFu, (uint32_t)open) | (uint64_t)__reduce_or_sync(0xFFFFFFFFu, (uint32_t)(open >> 32)) << 32;
        if (open != 0) __syncwarp();  // the codes are stored, by other lanes than those that store them now
        for (; open != 0; open &= open - 1) {
          const int h = 2 * (r0 + __ffsll(open) - 1) + sub;
          again<T, kInter, kWide>(row0 + (int64_t)min(h, a.heads - 1) * a.q_hs, weights[0], mine, rd, a.q_out + (out + h) * kHeadDim, h < a.heads);
        }
      }
    }
    if (a.k != nullptr && past == units) {
      const int64_t slot = a.slots != nullptr ? a.slots[t] : t;
      if (slot >= a.num_slots && lane == 0) report(a.status, IDX_ST_BLOCK_OOR);
      if (slot >= 0 && slot < a.num_slots) {
        const Piece8 f = factors_of<kInter>(p, weights[1], mine);
        const T* src = static_cast<const T*>(a.k) + (int64_t)t * a.k_ts;
        float2 u[4], mag[4];
        float ss = turn8<T, kInter>(load8<T, kWide>(src + at), p, f, u, mag);  // the same row in both halves
#pragma unroll
        for (int o = 1; o < kLanesI; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        float top = largest8(u), most = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) most = fmaxf(most, fmaxf(mag[e].x, mag[e].y));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1)), most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        const float mean = fmaf(ss, 1.f / kHeadDim, a.eps), r = a.k_w != nullptr ? rsqrtf(mean) : 1.f;
        const bool bad = !(ss <= 3.4e38f);
        const float six = top * r * (1.f / 6.f), off = most * r * (kSlackKey / 6.f);
        const uint32_t both = f32x2_to_e4m3x2(six - off, six + off);
        uint32_t scale = both & 0xFFu, codes = 0;
        const float sv = e4m3_to_f32(scale), inv = scale == 0x7Fu || scale == 0u ? 0.f : r / sv;
        bool open = (both & 0xFFu) != both >> 8 || (a.k_w != nullptr && mean < kSmallI);
        if (inv != 0.f) {
          uint32_t high = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = mul2(u[e], make_float2(inv, inv)), d = mul2(mag[e], make_float2(inv * kSlackKey, inv * kSlackKey));
            codes |= f32x2_to_e2m1x2(v.x - d.x, v.y - d.y) << (8 * e), high |= f32x2_to_e2m1x2(v.x + d.x, v.y + d.y) << (8 * e);
          }
          open |= codes != high;
        }
        if (__any_sync(0xFFFFFFFFu, open && !bad)) {
          const uint2 again = key_64<T, kInter>(Row64<T>{src, weights[1], mine, rd}, at, a.k_w != nullptr, a.eps);
          codes = again.x, scale = again.y;
        }
        if (bad) codes = 0, scale = 0x7Fu;
        if (sub == 0) {
          const int64_t block = slot / a.page;
          const int place = (int)(slot - block * a.page);
          uint8_t* page = a.index_k + block * (a.page * 72);
          *reinterpret_cast<uint32_t*>(page + place * 64 + piece * 4) = codes;
          if (piece % 2 == 0) page[a.page * 64 + place * 8 + piece / 2] = (uint8_t)scale;
        }
      }
    }
  }
}

template <typename T, bool kInter, bool kWide>
void launch_index(const IndexArgs& a, cudaStream_t s) {
  const int rows = (a.heads + 1) / 2, sms = max(device_sms(), 1);
  const int64_t all = (int64_t)a.num_tokens * ((rows + kBatchI - 1) / kBatchI + (a.k != nullptr ? 1 : 0));
  // a unit a warp, or an equal number of them a warp of those that run at once
  const int64_t warps = min(all, (int64_t)sms * kCtasI * (kThreadsI / 32));
  launch_pdl(k_index_append<T, kInter, kWide>, dim3((unsigned)((warps + kThreadsI / 32 - 1) / (kThreadsI / 32))), dim3(kThreadsI), 0, s, a, warps);
  if (a.heads > 0 && a.q_w != nullptr && a.eps < kSmallI) {
    const unsigned grid = (unsigned)min(((int64_t)a.num_tokens + kThreadsI / 32 - 1) / (kThreadsI / 32), (int64_t)sms * kCtasI);
    launch_pdl(k_index_small<T, kInter, kWide>, dim3(grid), dim3(kThreadsI), 0, s, a);
  }
}
template <typename T>
void launch_index(const IndexArgs& a, bool inter, bool wide, cudaStream_t s) {
  if (inter) wide ? launch_index<T, true, true>(a, s) : launch_index<T, true, false>(a, s);
  else wide ? launch_index<T, false, true>(a, s) : launch_index<T, false, false>(a, s);
}

}  // namespace
}  // namespace idx

extern "C" int idx_index_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, int32_t heads, const void* k, int64_t k_token_stride,
                                int32_t num_tokens, int32_t rotary_dim, const void* q_weight, const void* k_weight, float eps, float offset,
                                const int32_t* positions, const double* inv_freq, float mscale, const float* head_weights, float scale,
                                const int32_t* cu_tokens, int32_t num_reqs, int32_t req_slots, uint8_t* q_out, float* q_scale,
                                const int64_t* slots, uint8_t* index_k, int64_t num_blocks, int32_t page_tokens, int32_t dtype, int32_t flags,
                                int32_t* status, void* stream) {
  using namespace idx;
  const bool inter = (flags & IDX_ROPE_INTERLEAVED) != 0;
  if (num_tokens < 0 || heads < 0 || rotary_dim < 0 || rotary_dim > kHeadDim || rotary_dim % (inter ? 8 : 16) != 0 || num_blocks < 0 ||
      (page_tokens != 128 && page_tokens != 256) || (flags & ~IDX_ROPE_INTERLEAVED) != 0 || dtype < IDX_BF16 || dtype > IDX_F32 || !(eps >= 0.f) ||
      q_token_stride < 0 || q_head_stride < 0 || k_token_stride < 0 || num_reqs < 0 || (cu_tokens != nullptr && req_slots < 1))
    return IDX_E_BAD_SHAPE;
  if (heads > kMtpMaxHeads || num_reqs > 65535) return IDX_E_TOO_LARGE;
  if (num_tokens == 0 || (heads == 0 && k == nullptr)) return IDX_OK;
  if (heads > 0 && (!q || !q_out || !q_scale)) return IDX_E_NULL_PTR;
  if ((k == nullptr) != (index_k == nullptr) || !positions || (rotary_dim > 0 && !inv_freq)) return IDX_E_NULL_PTR;
  const int size = dtype == IDX_F32 ? 4 : 2;
  for (const void* p : {q, k, q_weight, k_weight})
    if (!aligned(p, size)) return IDX_E_MISALIGNED;
  for (const void* p : {(const void*)positions, (const void*)head_weights, (const void*)cu_tokens, (const void*)q_scale, (const void*)status})
    if (!aligned(p, 4)) return IDX_E_MISALIGNED;
  if (!aligned(inv_freq, 8) || !aligned(slots, 8) || !aligned(q_out, 16) || !aligned(index_k, 16)) return IDX_E_MISALIGNED;
  int rc;
  if ((rc = check_device()) != IDX_OK) return rc;
  IndexArgs a{};
  a.heads = cu_tokens != nullptr && num_reqs == 0 ? 0 : heads;  // no request, no slot for a query
  if (a.heads == 0 && k == nullptr) return IDX_OK;
  a.num_tokens = num_tokens, a.rotary_dim = rotary_dim, a.eps = eps, a.offset = offset, a.mscale = mscale, a.scale = scale;
  a.positions = positions, a.inv_freq = inv_freq, a.status = status;
  bool wide = true;
  auto fit = [&](const void* p, int64_t stride) { wide = wide && aligned(p, 16) && stride * size % 16 == 0; };
  if (a.heads > 0) {
    a.q = q, a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.q_w = q_weight, a.q_out = q_out, a.q_scale = q_scale;
    a.head_weights = head_weights, a.cu = cu_tokens, a.num_reqs = num_reqs, a.req_slots = req_slots;
    fit(q, q_token_stride), fit(q, q_head_stride);
  }
  if (k != nullptr) {
    a.k = k, a.k_ts = k_token_stride, a.k_w = k_weight, a.slots = slots, a.index_k = index_k, a.page = page_tokens;
    a.num_slots = num_blocks * page_tokens;
    fit(k, k_token_stride);
  }
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == IDX_BF16) launch_index<__nv_bfloat16>(a, inter, wide, s);
  else if (dtype == IDX_F16) launch_index<__half>(a, inter, wide, s);
  else launch_index<float>(a, inter, wide, s);
  return launch_result();
}
