// Rotary positions of queries and keys, keys and values appended to the
// paged cache.
//
// Each pair (x1, x2) of a head turns by a = position * inv_freq: y1 = m (x1
// cos a - x2 sin a), y2 = m (x2 cos a + x1 sin a).  inv_freq / 2 pi becomes a
// 64-bit fraction of a turn (to the nearest 2^-64: a product rounded to one
// double is off by up to 2^-55.7, 2^-24.7 turns at a position of 2^31), and
// position * fraction in 64-bit integer arithmetic drops the whole turns by
// itself; what remains is a signed fraction in [-1/2, 1/2)
// turns whose sine and cosine CUDA's sincospif gives.  A position of 2^31
// leaves an error of 2^-34 turns and fp32's rounding of the fraction, where a
// product in fp32 would be off by whole turns; no table of positions is read
// (one of fp32 pairs would add 8 bytes a pair and token to the traffic).
//
// The kernels are bound by HBM: every element is read once and written once.
// k_rope_rows, for heads of at most 32 pieces (of up to 16 bytes, as the
// alignment of pointers and strides allows): a warp takes a token, or with few
// tokens a part of its heads, by itself.  Its lanes form the sines and cosines,
// a lane keeps those of its own piece, and the warp goes through the heads'
// rows in order, whole rows at a time, kBatchR in flight; halves of a pair meet
// by a shuffle.  k_rope_append, for the other heads: a CTA takes a token, its
// threads the pieces that turn, then those that pass, then the values.  The
// second order reads each row twice over, half of it each time, and took 211 us
// where the first takes 180, 0.91 of HBM (30,011 tokens of 64 + 4 heads of 128
// in bf16; batches of 1, 2, 4, 8 rows: 236, 178, 180, 194, and on 512 tokens
// 7.4, 7.4, 5.3, 5.9 us).
#include <cmath>

#include "idx_internal.h"
#include "idx_rope.cuh"

namespace idx {
namespace {

constexpr int kThreadsR = 256;
constexpr int kMaxDimR = 512;
constexpr int kTokR = 4;     // tokens of a CTA's turn (k_rope_append)
constexpr int kBatchR = 4;   // rows in flight a lane (k_rope_rows)

struct RopeArgs {
  const void* q;
  void* q_out;
  const void *k, *v;
  void *kc, *vc;
  int64_t q_ts, q_hs, o_ts, o_hs, k_ts, k_hs, v_ts, v_hs, c_bs, c_ts, c_hs;
  int32_t q_heads, kv_heads, num_tokens, head_dim, rotary_dim;
  const int32_t* positions;
  const double* inv_freq;
  float mscale;
  const int64_t* slots;
  int64_t num_slots;
  int32_t page;
  int32_t* status;
  int32_t turn;  // tokens of a turn
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Piece {
  T e[V];
};

// Elements e and e + 1 of a piece, and their rounding back.
template <int V>
__device__ __forceinline__ float2 get2(const Piece<float, V>& x, int e) { return make_float2(x.e[e], x.e[e + 1]); }
template <int V>
__device__ __forceinline__ float2 get2(const Piece<__half, V>& x, int e) { return __half22float2(__halves2half2(x.e[e], x.e[e + 1])); }
template <int V>
__device__ __forceinline__ float2 get2(const Piece<__nv_bfloat16, V>& x, int e) {
  return make_float2(__bfloat162float(x.e[e]), __bfloat162float(x.e[e + 1]));
}
template <int V>
__device__ __forceinline__ void put2(Piece<float, V>& x, int e, float2 y) { x.e[e] = y.x, x.e[e + 1] = y.y; }
template <int V>
__device__ __forceinline__ void put2(Piece<__half, V>& x, int e, float2 y) {
  const __half2 h = __floats2half2_rn(y.x, y.y);
  x.e[e] = __low2half(h), x.e[e + 1] = __high2half(h);
}
template <int V>
__device__ __forceinline__ void put2(Piece<__nv_bfloat16, V>& x, int e, float2 y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(y.x, y.y);
  x.e[e] = __low2bfloat16(h), x.e[e + 1] = __high2bfloat16(h);
}

// Turns the pairs of one piece (V / 2 side by side) or of two (V, one of each).
template <typename T, int V, bool kInter>
__device__ __forceinline__ void rotate(Piece<T, V>& one, Piece<T, V>& two, const float* c, const float* s) {
  if (V == 1) {
    const float x1 = to_f(one.e[0]), x2 = to_f(two.e[0]);
    one.e[0] = from_f<T>(x1 * c[0] - x2 * s[0]);
    two.e[0] = from_f<T>(x2 * c[0] + x1 * s[0]);
  } else if (kInter) {
#pragma unroll
    for (int e = 0; e + 1 < V; e += 2) {
      const float2 x = get2(one, e);
      const float cc = c[e / 2], ss = s[e / 2];
      put2(one, e, fma2(x, make_float2(cc, cc), mul2(make_float2(x.y, x.x), make_float2(-ss, ss))));
    }
  } else {
#pragma unroll
    for (int e = 0; e + 1 < V; e += 2) {
      const float2 x1 = get2(one, e), x2 = get2(two, e);
      const float2 cc = make_float2(c[e], c[e + 1]), ss = make_float2(s[e], s[e + 1]);
      put2(one, e, fma2(x1, cc, mul2(x2, make_float2(-ss.x, -ss.y))));
      put2(two, e, fma2(x2, cc, mul2(x1, ss)));
    }
  }
}

template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreadsR) k_rope_append(const __grid_constant__ RopeArgs a) {
  pdl_enter();
  // [turn][token][cosines, sines][pair], two turns in turn
  __shared__ __align__(16) float angles[2][kTokR][2][kMaxDimR / 2];
  __shared__ unsigned long long steps[kMaxDimR / 2];
  __shared__ int64_t places[2][kTokR];  // of the tokens in the cache, in elements; -1: none
  using P = Piece<T, V>;
  constexpr bool kSide = kInter && V > 1;  // a pair's elements lie in one piece
  constexpr int kAngles = kSide ? V / 2 : V;
  const int rd = a.rotary_dim, half = rd / 2;
  const int pair_pieces = kSide ? rd / V : half / V, rest_pieces = (a.head_dim - rd) / V, all_pieces = a.head_dim / V;
  const T* q = static_cast<const T*>(a.q);
  const T* k = static_cast<const T*>(a.k);
  const T* v = static_cast<const T*>(a.v);
  T* qo = static_cast<T*>(a.q_out);
  T* kc = static_cast<T*>(a.kc);
  T* vc = static_cast<T*>(a.vc);
  const int heads = a.q_heads + a.kv_heads;
  for (int i = threadIdx.x; i < half; i += kThreadsR) steps[i] = step_of(a.inv_freq[i]);
  __syncthreads();
  int buf = 0;
  for (int64_t base = (int64_t)blockIdx.x * a.turn; base < a.num_tokens; base += (int64_t)gridDim.x * a.turn, buf ^= 1) {
    const int count = (int)min((int64_t)a.turn, a.num_tokens - base);
    for (int i = threadIdx.x; i < half * count; i += kThreadsR) {
      const int tk = i / half, pr = i - tk * half;
      const float2 w = turn_of(a.positions[base + tk], steps[pr], a.mscale);
      angles[buf][tk][0][pr] = w.x, angles[buf][tk][1][pr] = w.y;
    }
    if (threadIdx.x >= kThreadsR - kTokR && a.kv_heads > 0) {
      // one thread a token: 64-bit divisions
      const int tk = kThreadsR - 1 - threadIdx.x;
      if (tk < count) {
        const int64_t slot = a.slots != nullptr ? a.slots[base + tk] : base + tk;
        const bool keep = slot >= 0 && slot < a.num_slots;
        if (slot >= a.num_slots && blockIdx.y == 0) report(a.status, IDX_ST_BLOCK_OOR);
        places[buf][tk] = keep ? slot / a.page * a.c_bs + slot % a.page * a.c_ts : -1;
      }
    }
    __syncthreads();  // (the buffer of the turn before last is free: every thread has passed the sync between)

    // Goes through `pieces` pieces of each of the turn's `n` heads a token:
    // this thread's piece is the same in all of its heads (but for heads of
    // more pieces than the CTA has threads).
    auto each = [&](int pieces, int n, auto&& body) {
      if (pieces == 0 || n == 0) return;
      const int lanes = max(1, kThreadsR / pieces), first = threadIdx.x / pieces;
      if (first >= lanes) return;
      for (int p = threadIdx.x % pieces; p < pieces; p += kThreadsR)
        for (int i = blockIdx.y * lanes + first; i < n * count; i += lanes * (int)gridDim.y) {
          int tk = 0, h = i;  // a turn has few tokens
#pragma unroll
          for (int x = 1; x < kTokR; ++x)
            if (h >= n) h -= n, ++tk;
          body(p, tk, h);
        }
    };
    // source and destination of a rotated head; false: it goes nowhere
    auto head_at = [&](int tk, int h, const T*& src, T*& dst) {
      const int64_t t = base + tk;
      if (h < a.q_heads) {
        src = q + t * a.q_ts + h * a.q_hs, dst = qo + t * a.o_ts + h * a.o_hs;
        return true;
      }
      const int64_t place = places[buf][tk];
      src = k + t * a.k_ts + (h - a.q_heads) * a.k_hs, dst = kc + place + (h - a.q_heads) * a.c_hs;
      return place >= 0;
    };
    each(pair_pieces, heads, [&](int p, int tk, int h) {
      const int at = kInter && V == 1 ? 2 * p : p * V, far = kSide ? at : kInter ? at + 1 : at + half;
      const T* src;
      T* dst;
      if (!head_at(tk, h, src, dst)) return;
      P one = *reinterpret_cast<const P*>(src + at), two{};
      if (!kSide) two = *reinterpret_cast<const P*>(src + far);
      float c[kAngles], s[kAngles];
#pragma unroll
      for (int e = 0; e < kAngles; ++e) c[e] = angles[buf][tk][0][p * kAngles + e], s[e] = angles[buf][tk][1][p * kAngles + e];
      rotate<T, V, kInter>(one, two, c, s);
      *reinterpret_cast<P*>(dst + at) = one;
      if (!kSide) *reinterpret_cast<P*>(dst + far) = two;
    });
    each(rest_pieces, heads, [&](int p, int tk, int h) {
      const T* src;
      T* dst;
      if (head_at(tk, h, src, dst)) *reinterpret_cast<P*>(dst + rd + p * V) = *reinterpret_cast<const P*>(src + rd + p * V);
    });
    each(all_pieces, v != nullptr ? a.kv_heads : 0, [&](int p, int tk, int h) {
      if (places[buf][tk] >= 0)
        *reinterpret_cast<P*>(vc + places[buf][tk] + h * a.c_hs + p * V) =
            *reinterpret_cast<const P*>(v + (base + tk) * a.v_ts + h * a.v_hs + p * V);
    });
  }
}

// Rows g0 .. g1 - 1 of `heads` heads, per_warp a row: from src to dst (this
// lane's piece of row g0), a batch of loads in flight.
template <typename T, int V, bool kInter, bool kTurn>
__device__ __forceinline__ void walk_rows(const T* src, int64_t src_step, T* dst, int64_t dst_step, int left, int rows, int per_warp,
                                          bool turns, int partner, const float2* c, const float2* s) {
  constexpr int kN = (int)sizeof(T) * V / 4;
  using R = Row<kN>;
  for (int g = 0; g < rows; g += kBatchR) {
    R x[kBatchR];
#pragma unroll
    for (int u = 0; u < kBatchR; ++u) {
      if (g + u < rows && left > u * per_warp) x[u] = *reinterpret_cast<const R*>(src + u * src_step);
      else x[u] = R{};
    }
#pragma unroll
    for (int u = 0; u < kBatchR; ++u) {
      if (kTurn) {
        R y;
        if (!kInter) {
#pragma unroll
          for (int e = 0; e < kN; ++e) y.w[e] = __shfl_sync(0xFFFFFFFFu, x[u].w[e], partner);
        }
        float2 z[V / 2];
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          const float2 one = Words<T>::get(x[u].w, e), two = kInter ? make_float2(one.y, one.x) : Words<T>::get(y.w, e);
          z[e] = fma2(one, c[e], mul2(two, s[e]));
        }
#pragma unroll
        for (int e = 0; e < V / 2; ++e) Words<T>::put(x[u].w, e, z[e], turns);
      }
      if (g + u < rows && left > u * per_warp) *reinterpret_cast<R*>(dst + u * dst_step) = x[u];
    }
    src += kBatchR * src_step, dst += kBatchR * dst_step, left -= kBatchR * per_warp;
  }
}

// A warp a token (or a part of its heads), heads of at most 32 pieces.
template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreadsR, 4) k_rope_rows(const __grid_constant__ RopeArgs a, int parts) {
  pdl_enter();
  __shared__ float angles[kThreadsR / 32][2][kMaxDimR / 2];
  __shared__ unsigned long long steps[kMaxDimR / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rd = a.rotary_dim, half = rd / 2, pieces = a.head_dim / V, per_warp = 32 / pieces;
  const int sub = lane / pieces, at = lane % pieces * V;  // the lane's head of the warp's row, its piece
  const bool turns = at < rd, upper = !kInter && at >= half;
  const int partner = !turns || kInter ? lane : upper ? lane - half / V : lane + half / V;
  const int angle = kInter ? at / 2 : upper ? at - half : at;
  const int q_rows = (a.q_heads + per_warp - 1) / per_warp, kv_rows = (a.kv_heads + per_warp - 1) / per_warp;
  for (int i = threadIdx.x; i < half; i += kThreadsR) steps[i] = step_of(a.inv_freq[i]);
  __syncthreads();
  float(*mine)[kMaxDimR / 2] = angles[warp];
  const int64_t tasks = (int64_t)a.num_tokens * parts;
  for (int64_t task = (int64_t)blockIdx.x * (kThreadsR / 32) + warp; task < tasks; task += (int64_t)gridDim.x * (kThreadsR / 32)) {
    const int t = (int)(task / parts), part = (int)(task - (int64_t)t * parts);
    const int r0 = q_rows * part / parts, r1 = q_rows * (part + 1) / parts;
    const int position = a.positions[t];
    __syncwarp();  // the angles of the task before are used up
    for (int i = lane; i < half; i += 32) {
      const float2 w = turn_of(position, steps[i], a.mscale);
      mine[0][i] = w.x, mine[1][i] = w.y;
    }
    __syncwarp();
    float2 c[V / 2], s[V / 2];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      c[e] = s[e] = make_float2(0.f, 0.f);
      if (turns && kInter) {
        const float x = mine[0][angle + e], y = mine[1][angle + e];
        c[e] = make_float2(x, x), s[e] = make_float2(-y, y);
      } else if (turns) {
        const float y0 = mine[1][angle + 2 * e], y1 = mine[1][angle + 2 * e + 1];
        c[e] = make_float2(mine[0][angle + 2 * e], mine[0][angle + 2 * e + 1]);
        s[e] = upper ? make_float2(y0, y1) : make_float2(-y0, -y1);
      }
    }
    // a lane without a head has none left
    if (a.q_heads > 0) {
      const int h = r0 * per_warp + sub;
      walk_rows<T, V, kInter, true>(static_cast<const T*>(a.q) + (int64_t)t * a.q_ts + h * a.q_hs + at, per_warp * a.q_hs,
                                    static_cast<T*>(a.q_out) + (int64_t)t * a.o_ts + h * a.o_hs + at, per_warp * a.o_hs,
                                    sub < per_warp ? a.q_heads - h : 0, r1 - r0, per_warp, turns, partner, c, s);
    }
    if (a.kv_heads > 0 && part == parts - 1) {
      const int64_t slot = a.slots != nullptr ? a.slots[t] : t;
      if (slot >= a.num_slots && lane == 0) report(a.status, IDX_ST_BLOCK_OOR);
      if (slot >= 0 && slot < a.num_slots) {
        const int64_t place = slot / a.page * a.c_bs + slot % a.page * a.c_ts + sub * a.c_hs + at;
        const int left = sub < per_warp ? a.kv_heads - sub : 0;
        walk_rows<T, V, kInter, true>(static_cast<const T*>(a.k) + (int64_t)t * a.k_ts + sub * a.k_hs + at, per_warp * a.k_hs,
                                      static_cast<T*>(a.kc) + place, per_warp * a.c_hs, left, kv_rows, per_warp, turns, partner, c, s);
        if (a.v != nullptr)
          walk_rows<T, V, kInter, false>(static_cast<const T*>(a.v) + (int64_t)t * a.v_ts + sub * a.v_hs + at, per_warp * a.v_hs,
                                         static_cast<T*>(a.vc) + place, per_warp * a.c_hs, left, kv_rows, per_warp, false, lane, c, s);
      }
    }
  }
}

template <typename T, int V>
void launch_v(RopeArgs a, bool inter, cudaStream_t s) {
  const int sms = max(device_sms(), 1);
  const int pieces = a.head_dim / V;
  if constexpr (V > 1) {
    if (pieces <= 32) {
      // parts of a token's heads while they keep a batch of rows and the SMs
      // have room for their warps
      const int per_warp = 32 / pieces, rows = (a.q_heads + per_warp - 1) / per_warp;
      const int most = max(1, (rows + kBatchR - 1) / kBatchR);
      const int parts = (int)min((int64_t)most, max((int64_t)1, ((int64_t)sms * 32 + a.num_tokens - 1) / a.num_tokens));
      const int64_t ctas = ((int64_t)a.num_tokens * parts + kThreadsR / 32 - 1) / (kThreadsR / 32);
      const unsigned grid = (unsigned)min(ctas, (int64_t)sms * 8);
      if (inter) launch_pdl(k_rope_rows<T, V, true>, dim3(grid), dim3(kThreadsR), 0, s, a, parts);
      else launch_pdl(k_rope_rows<T, V, false>, dim3(grid), dim3(kThreadsR), 0, s, a, parts);
      return;
    }
  }
  // several tokens a turn where every SM gets some turns all the same
  a.turn = a.num_tokens >= 8 * kTokR * sms ? kTokR : 1;
  const int64_t turns = ((int64_t)a.num_tokens + a.turn - 1) / a.turn;
  const int64_t per_token = ((int64_t)(a.q_heads + 2 * a.kv_heads) * (a.head_dim / V) + kThreadsR - 1) / kThreadsR;
  const int x = (int)min(turns, (int64_t)sms * 8);
  const int y = (int)max((int64_t)1, min(per_token, (int64_t)(sms * 8 / x)));
  if (inter) launch_pdl(k_rope_append<T, V, true>, dim3(x, y), dim3(kThreadsR), 0, s, a);
  else launch_pdl(k_rope_append<T, V, false>, dim3(x, y), dim3(kThreadsR), 0, s, a);
}

template <typename T>
void launch_t(const RopeArgs& a, int v, bool inter, cudaStream_t s) {
  if (sizeof(T) == 2 && v == 8) launch_v<T, sizeof(T) == 2 ? 8 : 4>(a, inter, s);
  else if (v >= 4) launch_v<T, 4>(a, inter, s);
  else if (v == 2) launch_v<T, 2>(a, inter, s);
  else launch_v<T, 1>(a, inter, s);
}

}  // namespace
}  // namespace idx

extern "C" int idx_rope_frequencies(int32_t rotary_dim, double base, int32_t kind, double factor, double orig_len,
                                    double beta_fast, double beta_slow, double* inv_freq, double* mscale) {
  if (rotary_dim < 0 || rotary_dim % 2 != 0 || !(base > 1.0) || kind < IDX_ROPE_PLAIN || kind > IDX_ROPE_RAMP)
    return IDX_E_BAD_SHAPE;
  if (kind != IDX_ROPE_PLAIN && !(factor > 0.0)) return IDX_E_BAD_SHAPE;
  if (kind == IDX_ROPE_RAMP && (!(orig_len > 0.0) || !(beta_fast > 0.0) || !(beta_slow > 0.0))) return IDX_E_BAD_SHAPE;
  if ((rotary_dim > 0 && !inv_freq) || !mscale) return IDX_E_NULL_PTR;
  const double two_pi = 6.283185307179586;
  double lo = 0.0, hi = 0.0;
  if (kind == IDX_ROPE_RAMP) {
    const double per = rotary_dim / (2.0 * std::log(base));
    lo = std::fmax(0.0, std::floor(per * std::log(orig_len / (two_pi * beta_fast))));
    hi = std::fmin(rotary_dim - 1.0, std::ceil(per * std::log(orig_len / (two_pi * beta_slow))));
  }
  for (int32_t i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rotary_dim);
    if (kind == IDX_ROPE_PLAIN) {
      inv_freq[i] = f;
    } else if (kind == IDX_ROPE_LINEAR) {
      inv_freq[i] = f / factor;
    } else {
      const double w = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 1e-3)));
      inv_freq[i] = f * (1.0 - w) + f / factor * w;
    }
  }
  *mscale = kind == IDX_ROPE_RAMP && factor > 1.0 ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return IDX_OK;
}

extern "C" int idx_rope_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                               int64_t qo_token_stride, int64_t qo_head_stride, int32_t q_heads, const void* k,
                               int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                               int64_t v_head_stride, int32_t kv_heads, int32_t num_tokens, int32_t head_dim,
                               int32_t rotary_dim, const int32_t* positions, const double* inv_freq, float mscale,
                               const int64_t* slots, void* k_cache, void* v_cache, int64_t num_blocks,
                               int32_t page_tokens, int64_t c_block_stride, int64_t c_token_stride,
                               int64_t c_head_stride, int32_t dtype, int32_t flags, int32_t* status, void* stream) {
  using namespace idx;
  if (num_tokens < 0 || q_heads < 0 || kv_heads < 0 || head_dim < 1 || rotary_dim < 0 || rotary_dim % 2 != 0 ||
      rotary_dim > head_dim || num_blocks < 0 || page_tokens < 1 || (flags & ~IDX_ROPE_INTERLEAVED) != 0 || dtype < IDX_BF16 ||
      dtype > IDX_F32)
    return IDX_E_BAD_SHAPE;
  for (int64_t s : {q_token_stride, q_head_stride, qo_token_stride, qo_head_stride, k_token_stride, k_head_stride,
                    v_token_stride, v_head_stride, c_block_stride, c_token_stride, c_head_stride})
    if (s < 0) return IDX_E_BAD_SHAPE;
  if (head_dim > kMaxDimR || q_heads > 65535 || kv_heads > 65535) return IDX_E_TOO_LARGE;
  if (num_tokens == 0 || q_heads + kv_heads == 0) return IDX_OK;
  if (q_heads > 0 && (!q || !q_out)) return IDX_E_NULL_PTR;
  if (kv_heads > 0 && (!k || !k_cache || (v == nullptr) != (v_cache == nullptr))) return IDX_E_NULL_PTR;
  if (!positions || (rotary_dim > 0 && !inv_freq)) return IDX_E_NULL_PTR;
  // different tokens and heads must not share outputs
  if (q_heads > 0 && ((q_heads > 1 && qo_head_stride < head_dim) || (num_tokens > 1 && qo_token_stride < head_dim)))
    return IDX_E_BAD_SHAPE;
  if (kv_heads > 0 && ((kv_heads > 1 && c_head_stride < head_dim) || (page_tokens > 1 && c_token_stride < head_dim) ||
                       (num_blocks > 1 && c_block_stride < head_dim)))
    return IDX_E_BAD_SHAPE;
  const int size = dtype == IDX_F32 ? 4 : 2;
  for (const void* p : {q, (const void*)q_out, k, v, (const void*)k_cache, (const void*)v_cache})
    if (!aligned(p, size)) return IDX_E_MISALIGNED;
  if (!aligned(positions, 4) || !aligned(inv_freq, 8) || !aligned(slots, 8) || !aligned(status, 4)) return IDX_E_MISALIGNED;
  int rc;
  if ((rc = check_device()) != IDX_OK) return rc;
  RopeArgs a{};
  a.head_dim = head_dim, a.rotary_dim = rotary_dim, a.num_tokens = num_tokens;
  a.positions = positions, a.inv_freq = inv_freq, a.mscale = mscale, a.status = status;
  a.page = page_tokens, a.num_slots = num_blocks * page_tokens;
  // the widest piece that every address, stride and part of the head allows
  int vmax = 16 / size;
  auto fit = [&](int64_t x) {
    while (x % vmax != 0) vmax /= 2;
  };
  fit((flags & IDX_ROPE_INTERLEAVED) ? rotary_dim : rotary_dim / 2);
  fit(head_dim);
  if (q_heads > 0) {
    a.q = q, a.q_out = q_out, a.q_heads = q_heads;
    a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.o_ts = qo_token_stride, a.o_hs = qo_head_stride;
    for (int64_t x : {q_token_stride, q_head_stride, qo_token_stride, qo_head_stride}) fit(x);
    fit(reinterpret_cast<uintptr_t>(q) / size);
    fit(reinterpret_cast<uintptr_t>(q_out) / size);
  }
  if (kv_heads > 0) {
    a.k = k, a.v = v, a.kc = k_cache, a.vc = v_cache, a.kv_heads = kv_heads, a.slots = slots;
    a.k_ts = k_token_stride, a.k_hs = k_head_stride, a.v_ts = v_token_stride, a.v_hs = v_head_stride;
    a.c_bs = c_block_stride, a.c_ts = c_token_stride, a.c_hs = c_head_stride;
    for (int64_t x : {k_token_stride, k_head_stride, c_block_stride, c_token_stride, c_head_stride}) fit(x);
    fit(reinterpret_cast<uintptr_t>(k) / size);
    fit(reinterpret_cast<uintptr_t>(k_cache) / size);
    if (v != nullptr) {
      fit(v_token_stride), fit(v_head_stride);
      fit(reinterpret_cast<uintptr_t>(v) / size);
      fit(reinterpret_cast<uintptr_t>(v_cache) / size);
    }
  }
  const bool inter = (flags & IDX_ROPE_INTERLEAVED) != 0;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == IDX_BF16) launch_t<__nv_bfloat16>(a, vmax, inter, s);
  else if (dtype == IDX_F16) launch_t<__half>(a, vmax, inter, s);
  else launch_t<float>(a, vmax, inter, s);
  return launch_result();
}
