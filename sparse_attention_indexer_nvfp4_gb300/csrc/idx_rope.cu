// Rotary positions of queries and keys, keys and values appended to the
// paged cache.
//
// Each pair (x1, x2) of a head turns by a = position * inv_freq: y1 = m (x1
// cos a - x2 sin a), y2 = m (x2 cos a + x1 sin a).  The angle is reduced
// exactly: inv_freq / 2 pi becomes a 64-bit fraction of a turn (a multiple of
// 2^-63), and position * fraction in 64-bit integer arithmetic drops the
// whole turns by itself; what remains is a signed fraction in [-1/2, 1/2)
// turns whose sine and cosine CUDA's sincospif gives.  A position of 2^31
// leaves an error of 2^-33 turns, where a product in fp32 would be off by
// whole turns; no table of positions is read (one of fp32 pairs would add 8
// bytes a pair and token to the traffic).
//
// The kernel is bound by HBM: every element is read once and written once.  A
// CTA takes kTokR tokens; it forms each (token, pair)'s sine and cosine once
// in shared memory, then its threads take the tokens' heads in pieces of V
// elements (up to 16 bytes), which the alignment of pointers and strides
// sets.  With few tokens their heads are spread over gridDim.y CTAs.
#include <cuda_bf16.h>

#include <cmath>

#include "idx_common.cuh"
#include "idx_internal.h"

namespace idx {
namespace {

constexpr int kThreadsR = 256;
constexpr int kMaxDimR = 512;

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
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Piece {
  T e[V];
};

// The sine and cosine of position * freq, times m.
__device__ __forceinline__ float2 turn_of(int position, double freq, float m) {
  // turns a position, modulo 1, as a multiple of 2^-63
  double turns = freq * 0.15915494309189535;  // 1 / (2 pi)
  turns -= rint(turns);
  const unsigned long long step = (unsigned long long)__double2ll_rn(turns * 9223372036854775808.0) << 1;
  const unsigned long long phase = step * (unsigned long long)(long long)position;
  const float half_turns = (float)(long long)phase * 1.0842021724855044e-19f;  // 2^-63: signed, in half turns
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * m, s * m);
}

// One piece of a head's row: the first pair_pieces hold pairs, the others pass.
template <typename T, int V, bool kInter>
__device__ __forceinline__ void rotate_piece(const T* src, T* dst, const float2* cs, int piece, int pair_pieces, int rd) {
  using P = Piece<T, V>;
  if (piece < pair_pieces) {
    if (kInter && V == 1) {
      // two elements that do not share an aligned load
      const float2 w = cs[piece];
      const float x1 = to_f(src[2 * piece]), x2 = to_f(src[2 * piece + 1]);
      dst[2 * piece] = from_f<T>(x1 * w.x - x2 * w.y);
      dst[2 * piece + 1] = from_f<T>(x2 * w.x + x1 * w.y);
    } else if (kInter) {
      const P x = *reinterpret_cast<const P*>(src + piece * V);
      P y;
#pragma unroll
      for (int e = 0; e + 1 < V; e += 2) {
        const float2 w = cs[(piece * V + e) >> 1];
        const float x1 = to_f(x.e[e]), x2 = to_f(x.e[e + 1]);
        y.e[e] = from_f<T>(x1 * w.x - x2 * w.y);
        y.e[e + 1] = from_f<T>(x2 * w.x + x1 * w.y);
      }
      *reinterpret_cast<P*>(dst + piece * V) = y;
    } else {
      const int at = piece * V, far = at + rd / 2;
      const P a = *reinterpret_cast<const P*>(src + at), b = *reinterpret_cast<const P*>(src + far);
      P ya, yb;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 w = cs[at + e];
        const float x1 = to_f(a.e[e]), x2 = to_f(b.e[e]);
        ya.e[e] = from_f<T>(x1 * w.x - x2 * w.y);
        yb.e[e] = from_f<T>(x2 * w.x + x1 * w.y);
      }
      *reinterpret_cast<P*>(dst + at) = ya;
      *reinterpret_cast<P*>(dst + far) = yb;
    }
  } else {
    const int at = rd + (piece - pair_pieces) * V;
    *reinterpret_cast<P*>(dst + at) = *reinterpret_cast<const P*>(src + at);
  }
}

template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreadsR) k_rope_append(const __grid_constant__ RopeArgs a) {
  pdl_enter();
  __shared__ float2 cs[kMaxDimR / 2];
  const int rd = a.rotary_dim, half = rd / 2;
  const int pair_pieces = kInter && V > 1 ? rd / V : half / V;
  const int pieces = pair_pieces + (a.head_dim - rd) / V;  // of a rotated head
  const int copy_pieces = a.head_dim / V;                  // of a value head
  const T* q = static_cast<const T*>(a.q);
  const T* k = static_cast<const T*>(a.k);
  const T* v = static_cast<const T*>(a.v);
  T* qo = static_cast<T*>(a.q_out);
  T* kc = static_cast<T*>(a.kc);
  T* vc = static_cast<T*>(a.vc);
  const int nq = a.q_heads * pieces, nk = a.kv_heads * pieces, nv = v != nullptr ? a.kv_heads * copy_pieces : 0;
  const int total = nq + nk + nv;
  for (int64_t t = blockIdx.x; t < a.num_tokens; t += gridDim.x) {
    __syncthreads();
    const int position = a.positions[t];
    for (int i = threadIdx.x; i < half; i += kThreadsR) cs[i] = turn_of(position, a.inv_freq[i], a.mscale);
    __syncthreads();
    const int64_t slot = a.kv_heads > 0 ? (a.slots != nullptr ? a.slots[t] : t) : -1;
    const bool keep = slot >= 0 && slot < a.num_slots;
    if (slot >= a.num_slots && threadIdx.x == 0 && blockIdx.y == 0) report(a.status, IDX_ST_BLOCK_OOR);
    const int64_t place = keep ? slot / a.page * a.c_bs + slot % a.page * a.c_ts : 0;
    for (int w = blockIdx.y * kThreadsR + threadIdx.x; w < total; w += gridDim.y * kThreadsR) {
      if (w < nq) {
        const int h = w / pieces, p = w - h * pieces;
        rotate_piece<T, V, kInter>(q + t * a.q_ts + h * a.q_hs, qo + t * a.o_ts + h * a.o_hs, cs, p, pair_pieces, rd);
      } else if (!keep) {
        break;  // only the cache's pieces are left
      } else if (w < nq + nk) {
        const int h = (w - nq) / pieces, p = w - nq - h * pieces;
        rotate_piece<T, V, kInter>(k + t * a.k_ts + h * a.k_hs, kc + place + h * a.c_hs, cs, p, pair_pieces, rd);
      } else {
        const int h = (w - nq - nk) / copy_pieces, p = w - nq - nk - h * copy_pieces;
        using P = Piece<T, V>;
        *reinterpret_cast<P*>(vc + place + h * a.c_hs + p * V) =
            *reinterpret_cast<const P*>(v + t * a.v_ts + h * a.v_hs + p * V);
      }
    }
  }
}

template <typename T, int V>
void launch_v(const RopeArgs& a, bool inter, cudaStream_t s) {
  const int sms = max(device_sms(), 1);
  const int64_t per_token = ((int64_t)(a.q_heads + 2 * a.kv_heads) * (a.head_dim / V) + kThreadsR - 1) / kThreadsR;
  const int x = (int)min((int64_t)a.num_tokens, (int64_t)sms * 8);
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
