// Norms of each head of queries and keys, rotary positions in the same pass,
// keys and values appended to the paged cache.
//
// A head's row x with weights w: n = r (offset + w) x, r = 1 / sqrt(mean x^2 +
// eps), then the pairs of its first rotary_dim elements turn as in
// idx_rope_append.  r is one number a row, so it is multiplied in last: a lane
// keeps, for its piece of a head, cw = (offset + w) cos and sw = (offset + w_p)
// (-)sin of the partner's weight, and an element is r (x cw + x_p sw).  Sums
// are fp32; each element is rounded once.
//
// Bound by HBM, as k_rope_rows is: every element is read once and written once.
// 30,011 tokens of 64 + 4 heads of 128 in bf16 take 191 us, 0.85 of HBM (180
// without a norm), with the next rows asked for while these are worked on (two a
// batch, 6 CTAs of 128 threads an SM: 191 to 193; four a batch, 2 of 256: 193;
// without asking ahead 208 to 225); one token 4.8 us.
//
// k_norm_rows, for heads of at most 32 pieces: a warp takes a token (with few
// tokens a part of its heads), a group of lanes a head's row, a piece a lane; the
// sum of squares is a butterfly over the group, which is the pieces' number rounded
// up to a power of two (lanes past the pieces add 0).  A side without weights is
// turned as idx_rope_append does it; where neither has any that call is the faster.
//
// k_norm_any, for other heads (single elements by alignment, heads of more than 32
// pieces): a warp takes a row through shared memory, element by element, and forms
// its angles for each head again.  It is bound by those instructions: 7,500 tokens
// of 64 + 4 heads of 512 take 387 us with 64 elements turned, 909 with all, where
// HBM would take 163.
#include "idx_internal.h"
#include "idx_rope.cuh"

namespace idx {
namespace {

constexpr int kThreadsN = 128;
constexpr int kMaxDimN = 512;
constexpr int kBatchN = 2;  // rows in flight a lane
constexpr int kCtasN = 6;   // of an SM

struct NormArgs {
  const void* q;
  void* q_out;
  const void *k, *v;
  void *kc, *vc;
  const void *q_w, *k_w;
  int64_t q_ts, q_hs, o_ts, o_hs, k_ts, k_hs, v_ts, v_hs, c_bs, c_ts, c_hs;
  int32_t q_heads, kv_heads, num_tokens, head_dim, rotary_dim;
  const int32_t* positions;
  const double* inv_freq;
  float mscale, eps, offset, inv_dim;
  const int64_t* slots;
  int64_t num_slots;
  int32_t page;
  int32_t* status;
};

// A lane's factors of a piece: out = r (x c + x_p s).
template <int V>
struct Factors {
  float2 c[V / 2], s[V / 2];
};

// Rows g0 .. of `left` heads, per_warp a row of the warp: normed (kNorm),
// turned and stored, a batch of loads in flight.
template <typename T, int V, bool kInter, bool kNorm>
__device__ __forceinline__ void norm_rows(const T* src, int64_t src_step, T* dst, int64_t dst_step, int left, int rows, int per_warp, int group,
                                          int partner, bool turns, const NormArgs& a, const Factors<V>& f) {
  constexpr int kN = (int)sizeof(T) * V / 4;
  using R = Row<kN>;
  R ahead[kBatchN];
  auto ask = [&](int g) {  // the batch from row g on; src and left are at it
#pragma unroll
    for (int u = 0; u < kBatchN; ++u) {
      if (g + u < rows && left > u * per_warp) ahead[u] = *reinterpret_cast<const R*>(src + u * src_step);
      else ahead[u] = R{};
    }
  };
  ask(0);
  for (int g = 0; g < rows; g += kBatchN) {
    R x[kBatchN];
#pragma unroll
    for (int u = 0; u < kBatchN; ++u) x[u] = ahead[u];
    const int here = left;
    src += kBatchN * src_step, left -= kBatchN * per_warp;
    if (g + kBatchN < rows) ask(g + kBatchN);
    float r[kBatchN];
#pragma unroll
    for (int u = 0; u < kBatchN; ++u) r[u] = 1.f;
    if (kNorm) {
#pragma unroll
      for (int u = 0; u < kBatchN; ++u) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          const float2 one = Words<T>::get(x[u].w, e);
          ss = fma2(one, one, ss);
        }
        r[u] = ss.x + ss.y;
      }
      for (int o = 1; o < group; o <<= 1) {
#pragma unroll
        for (int u = 0; u < kBatchN; ++u) r[u] += __shfl_xor_sync(0xFFFFFFFFu, r[u], o);
      }
#pragma unroll
      for (int u = 0; u < kBatchN; ++u) r[u] = rsqrtf(fmaf(r[u], a.inv_dim, a.eps));
    }
    float least = r[0];
#pragma unroll
    for (int u = 1; u < kBatchN; ++u) least = fminf(least, r[u]);
    if (kNorm && __any_sync(0xFFFFFFFFu, least == 0.f)) {
      // a squares' sum passed fp32's range, and the row's turn may: 0 for each of its elements, NaN for an infinity (a test
      // of each row took 201 us where this takes what none takes)
#pragma unroll
      for (int u = 0; u < kBatchN; ++u) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) Words<T>::put(x[u].w, e, mul2(Words<T>::get(x[u].w, e), make_float2(0.f, 0.f)), r[u] == 0.f);
      }
    }
#pragma unroll
    for (int u = 0; u < kBatchN; ++u) {
      R y;
      if (!kInter) {
#pragma unroll
        for (int e = 0; e < kN; ++e) y.w[e] = __shfl_sync(0xFFFFFFFFu, x[u].w[e], partner);
      }
      float2 z[V / 2];
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const float2 one = Words<T>::get(x[u].w, e), two = kInter ? make_float2(one.y, one.x) : Words<T>::get(y.w, e);
        z[e] = fma2(one, f.c[e], mul2(two, f.s[e]));
        if (kNorm) z[e] = mul2(z[e], make_float2(r[u], r[u]));
      }
#pragma unroll
      for (int e = 0; e < V / 2; ++e) Words<T>::put(x[u].w, e, z[e], kNorm || turns);  // without a norm the other elements pass as they are
      if (g + u < rows && here > u * per_warp) *reinterpret_cast<R*>(dst + u * dst_step) = x[u];
    }
    dst += kBatchN * dst_step;
  }
}

// Values, which pass as they are.
template <typename T, int V>
__device__ __forceinline__ void copy_rows(const T* src, int64_t src_step, T* dst, int64_t dst_step, int left, int rows, int per_warp) {
  using R = Row<(int)sizeof(T) * V / 4>;
  for (int g = 0; g < rows; g += kBatchN) {
    R x[kBatchN];
#pragma unroll
    for (int u = 0; u < kBatchN; ++u)
      if (g + u < rows && left > u * per_warp) x[u] = *reinterpret_cast<const R*>(src + u * src_step);
#pragma unroll
    for (int u = 0; u < kBatchN; ++u)
      if (g + u < rows && left > u * per_warp) *reinterpret_cast<R*>(dst + u * dst_step) = x[u];
    src += kBatchN * src_step, dst += kBatchN * dst_step, left -= kBatchN * per_warp;
  }
}

template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreadsN, kCtasN) k_norm_rows(const __grid_constant__ NormArgs a, int parts, int group) {
  pdl_enter();
  __shared__ float angles[kThreadsN / 32][2][kMaxDimN / 2];
  __shared__ unsigned long long steps[kMaxDimN / 2];
  __shared__ float weights[2][kMaxDimN];  // offset + w of queries and keys, 1 without
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rd = a.rotary_dim, half = rd / 2, pieces = a.head_dim / V, per_warp = 32 / group;
  const int sub = lane / group, piece = lane % group, at = min(piece, pieces - 1) * V;  // the lane's head of the warp's row, its piece
  const bool live = piece < pieces, turns = at < rd, upper = !kInter && at >= half;
  const int hop = turns && !kInter && live ? (upper ? -(half / V) : half / V) : 0, partner = lane + hop;
  const int angle = kInter ? at / 2 : upper ? at - half : at, mate = at + hop * V;
  const int q_rows = (a.q_heads + per_warp - 1) / per_warp, kv_rows = (a.kv_heads + per_warp - 1) / per_warp;
  for (int i = threadIdx.x; i < half; i += kThreadsN) steps[i] = step_of(a.inv_freq[i]);
  for (int i = threadIdx.x; i < a.head_dim; i += kThreadsN) {
    weights[0][i] = a.q_w != nullptr ? a.offset + to_f(static_cast<const T*>(a.q_w)[i]) : 1.f;
    weights[1][i] = a.k_w != nullptr ? a.offset + to_f(static_cast<const T*>(a.k_w)[i]) : 1.f;
  }
  __syncthreads();
  float(*mine)[kMaxDimN / 2] = angles[warp];
  const int64_t tasks = (int64_t)a.num_tokens * parts;
  for (int64_t task = (int64_t)blockIdx.x * (kThreadsN / 32) + warp; task < tasks; task += (int64_t)gridDim.x * (kThreadsN / 32)) {
    const int t = (int)(task / parts), part = (int)(task - (int64_t)t * parts);
    const int r0 = q_rows * part / parts, r1 = q_rows * (part + 1) / parts;
    const int position = a.positions[t];
    __syncwarp();  // the angles of the task before are used up
    for (int i = lane; i < half; i += 32) {
      const float2 w = turn_of(position, steps[i], a.mscale);
      mine[0][i] = w.x, mine[1][i] = w.y;
    }
    __syncwarp();
    auto factors = [&](const float* w) {
      Factors<V> f;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const float w0 = w[at + 2 * e], w1 = w[at + 2 * e + 1];
        if (turns && kInter) {
          const float x = mine[0][angle + e], y = mine[1][angle + e];
          f.c[e] = make_float2(x * w0, x * w1), f.s[e] = make_float2(-y * w1, y * w0);
        } else if (turns) {
          const float y0 = mine[1][angle + 2 * e] * w[mate + 2 * e], y1 = mine[1][angle + 2 * e + 1] * w[mate + 2 * e + 1];
          f.c[e] = make_float2(mine[0][angle + 2 * e] * w0, mine[0][angle + 2 * e + 1] * w1);
          f.s[e] = upper ? make_float2(y0, y1) : make_float2(-y0, -y1);
        } else {
          f.c[e] = make_float2(w0, w1), f.s[e] = make_float2(0.f, 0.f);
        }
      }
      return f;
    };
    // a lane without a head or a piece has none left
    if (a.q_heads > 0 && r1 > r0) {
      const int h = r0 * per_warp + sub;
      const T* src = static_cast<const T*>(a.q) + (int64_t)t * a.q_ts + h * a.q_hs + at;
      T* dst = static_cast<T*>(a.q_out) + (int64_t)t * a.o_ts + h * a.o_hs + at;
      const Factors<V> f = factors(weights[0]);
      if (a.q_w != nullptr)
        norm_rows<T, V, kInter, true>(src, per_warp * a.q_hs, dst, per_warp * a.o_hs, live ? a.q_heads - h : 0, r1 - r0, per_warp, group, partner, turns, a, f);
      else
        norm_rows<T, V, kInter, false>(src, per_warp * a.q_hs, dst, per_warp * a.o_hs, live ? a.q_heads - h : 0, r1 - r0, per_warp, group, partner, turns, a, f);
    }
    if (a.kv_heads > 0 && part == parts - 1) {
      const int64_t slot = a.slots != nullptr ? a.slots[t] : t;
      if (slot >= a.num_slots && lane == 0) report(a.status, IDX_ST_BLOCK_OOR);
      if (slot >= 0 && slot < a.num_slots) {
        const int64_t place = slot / a.page * a.c_bs + slot % a.page * a.c_ts + sub * a.c_hs + at;
        const int left = live ? a.kv_heads - sub : 0;
        const T* src = static_cast<const T*>(a.k) + (int64_t)t * a.k_ts + sub * a.k_hs + at;
        const Factors<V> f = factors(weights[1]);
        if (a.k_w != nullptr)
          norm_rows<T, V, kInter, true>(src, per_warp * a.k_hs, static_cast<T*>(a.kc) + place, per_warp * a.c_hs, left, kv_rows, per_warp, group, partner, turns, a, f);
        else
          norm_rows<T, V, kInter, false>(src, per_warp * a.k_hs, static_cast<T*>(a.kc) + place, per_warp * a.c_hs, left, kv_rows, per_warp, group, partner, turns, a, f);
        if (a.v != nullptr)
          copy_rows<T, V>(static_cast<const T*>(a.v) + (int64_t)t * a.v_ts + sub * a.v_hs + at, per_warp * a.v_hs,
                          static_cast<T*>(a.vc) + place, per_warp * a.c_hs, left, kv_rows, per_warp);
      }
    }
  }
}

// A warp a row of any size up to kMaxDimN, element by element.
template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreadsN) k_norm_any(const __grid_constant__ NormArgs a) {
  pdl_enter();
  __shared__ float rows_[kThreadsN / 32][kMaxDimN];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dim = a.head_dim, rd = a.rotary_dim, half = rd / 2;
  float* row = rows_[warp];
  const int heads = a.q_heads + a.kv_heads;
  const int64_t tasks = (int64_t)a.num_tokens * heads;
  for (int64_t task = (int64_t)blockIdx.x * (kThreadsN / 32) + warp; task < tasks; task += (int64_t)gridDim.x * (kThreadsN / 32)) {
    const int64_t t = task / heads;
    const int h = (int)(task - t * heads);
    const bool is_q = h < a.q_heads;
    const T* src;
    T* dst;
    const void* w;
    if (is_q) {
      src = static_cast<const T*>(a.q) + t * a.q_ts + h * a.q_hs, dst = static_cast<T*>(a.q_out) + t * a.o_ts + h * a.o_hs, w = a.q_w;
    } else {
      const int kh = h - a.q_heads;
      const int64_t slot = a.slots != nullptr ? a.slots[t] : t;
      if (slot >= a.num_slots && lane == 0) report(a.status, IDX_ST_BLOCK_OOR);
      if (slot < 0 || slot >= a.num_slots) continue;
      const int64_t place = slot / a.page * a.c_bs + slot % a.page * a.c_ts + kh * a.c_hs;
      src = static_cast<const T*>(a.k) + t * a.k_ts + kh * a.k_hs, dst = static_cast<T*>(a.kc) + place, w = a.k_w;
      if (a.v != nullptr)
        for (int e = lane; e < dim; e += 32) static_cast<T*>(a.vc)[place + e] = static_cast<const T*>(a.v)[t * a.v_ts + kh * a.v_hs + e];
    }
    __syncwarp();
    float ss = 0.f;
    for (int e = lane; e < dim; e += 32) {
      const float x = to_f(src[e]);
      ss = fmaf(x, x, ss);
      row[e] = w != nullptr ? x * (a.offset + to_f(static_cast<const T*>(w)[e])) : x;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    const float r = w != nullptr ? rsqrtf(fmaf(ss, a.inv_dim, a.eps)) : 1.f;
    if (r == 0.f) {  // (as in norm_rows; unrolled, it took 60 us of 7,500 tokens with heads of 512)
#pragma unroll 1
      for (int e = lane; e < dim; e += 32) row[e] = __fmul_rn(to_f(src[e]), 0.f);
    }
    __syncwarp();
    const int position = a.positions[t];
    for (int p = lane; p < half; p += 32) {
      const float2 cs = turn_of(position, step_of(a.inv_freq[p]), a.mscale);
      const int e1 = kInter ? 2 * p : p, e2 = kInter ? e1 + 1 : p + half;
      const float x1 = row[e1], x2 = row[e2];
      dst[e1] = from_f<T>(r * (x1 * cs.x - x2 * cs.y)), dst[e2] = from_f<T>(r * (x2 * cs.x + x1 * cs.y));
    }
    for (int e = rd + lane; e < dim; e += 32) dst[e] = from_f<T>(r * row[e]);
  }
}

template <typename T, int V>
void launch_rows(const NormArgs& a, bool inter, cudaStream_t s) {
  const int sms = max(device_sms(), 1), pieces = a.head_dim / V;
  int group = 1;
  while (group < pieces) group *= 2;
  // parts of a token's heads while they keep a batch of rows and the SMs have room for their warps
  const int per_warp = 32 / group, rows = (a.q_heads + per_warp - 1) / per_warp;
  const int most = max(1, (rows + kBatchN - 1) / kBatchN);
  const int parts = (int)min((int64_t)most, max((int64_t)1, ((int64_t)sms * kCtasN * (kThreadsN / 32) + a.num_tokens - 1) / a.num_tokens));
  const int64_t ctas = ((int64_t)a.num_tokens * parts + kThreadsN / 32 - 1) / (kThreadsN / 32);
  const unsigned grid = (unsigned)min(ctas, (int64_t)sms * kCtasN);
  if (inter) launch_pdl(k_norm_rows<T, V, true>, dim3(grid), dim3(kThreadsN), 0, s, a, parts, group);
  else launch_pdl(k_norm_rows<T, V, false>, dim3(grid), dim3(kThreadsN), 0, s, a, parts, group);
}

template <typename T>
void launch_norm(const NormArgs& a, int v, bool inter, cudaStream_t s) {
  constexpr int kWide = 16 / (int)sizeof(T);
  if (v >= 2 && a.head_dim / v <= 32) {
    if (v == 8) launch_rows<T, kWide == 8 ? 8 : 4>(a, inter, s);
    else if (v == 4) launch_rows<T, 4>(a, inter, s);
    else launch_rows<T, 2>(a, inter, s);
    return;
  }
  const int64_t ctas = ((int64_t)a.num_tokens * (a.q_heads + a.kv_heads) + kThreadsN / 32 - 1) / (kThreadsN / 32);
  const unsigned grid = (unsigned)min(ctas, (int64_t)max(device_sms(), 1) * 16);
  if (inter) launch_pdl(k_norm_any<T, true>, dim3(grid), dim3(kThreadsN), 0, s, a);
  else launch_pdl(k_norm_any<T, false>, dim3(grid), dim3(kThreadsN), 0, s, a);
}

}  // namespace
}  // namespace idx

extern "C" int idx_norm_rope_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out, int64_t qo_token_stride,
                                    int64_t qo_head_stride, int32_t q_heads, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                                    const void* v, int64_t v_token_stride, int64_t v_head_stride, int32_t kv_heads, int32_t num_tokens,
                                    int32_t head_dim, int32_t rotary_dim, const void* q_weight, const void* k_weight, float eps, float offset,
                                    const int32_t* positions, const double* inv_freq, float mscale, const int64_t* slots, void* k_cache,
                                    void* v_cache, int64_t num_blocks, int32_t page_tokens, int64_t c_block_stride, int64_t c_token_stride,
                                    int64_t c_head_stride, int32_t dtype, int32_t flags, int32_t* status, void* stream) {
  using namespace idx;
  if (num_tokens < 0 || q_heads < 0 || kv_heads < 0 || head_dim < 1 || rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > head_dim ||
      num_blocks < 0 || page_tokens < 1 || (flags & ~IDX_ROPE_INTERLEAVED) != 0 || dtype < IDX_BF16 || dtype > IDX_F32 || !(eps >= 0.f))
    return IDX_E_BAD_SHAPE;
  for (int64_t s : {q_token_stride, q_head_stride, qo_token_stride, qo_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                    c_block_stride, c_token_stride, c_head_stride})
    if (s < 0) return IDX_E_BAD_SHAPE;
  if (head_dim > kMaxDimN || q_heads > 65535 || kv_heads > 65535) return IDX_E_TOO_LARGE;
  if (num_tokens == 0 || q_heads + kv_heads == 0) return IDX_OK;
  if (q_heads > 0 && (!q || !q_out)) return IDX_E_NULL_PTR;
  if (kv_heads > 0 && (!k || !k_cache || (v == nullptr) != (v_cache == nullptr))) return IDX_E_NULL_PTR;
  if (!positions || (rotary_dim > 0 && !inv_freq)) return IDX_E_NULL_PTR;
  // different tokens and heads must not share outputs
  if (q_heads > 0 && ((q_heads > 1 && qo_head_stride < head_dim) || (num_tokens > 1 && qo_token_stride < head_dim))) return IDX_E_BAD_SHAPE;
  if (kv_heads > 0 && ((kv_heads > 1 && c_head_stride < head_dim) || (page_tokens > 1 && c_token_stride < head_dim) ||
                       (num_blocks > 1 && c_block_stride < head_dim)))
    return IDX_E_BAD_SHAPE;
  const int size = dtype == IDX_F32 ? 4 : 2;
  for (const void* p : {q, (const void*)q_out, k, v, (const void*)k_cache, (const void*)v_cache, q_weight, k_weight})
    if (!aligned(p, size)) return IDX_E_MISALIGNED;
  if (!aligned(positions, 4) || !aligned(inv_freq, 8) || !aligned(slots, 8) || !aligned(status, 4)) return IDX_E_MISALIGNED;
  int rc;
  if ((rc = check_device()) != IDX_OK) return rc;
  NormArgs a{};
  a.head_dim = head_dim, a.rotary_dim = rotary_dim, a.num_tokens = num_tokens;
  a.positions = positions, a.inv_freq = inv_freq, a.mscale = mscale, a.eps = eps, a.offset = offset, a.inv_dim = 1.f / (float)head_dim, a.status = status;
  a.page = page_tokens, a.num_slots = num_blocks * page_tokens;
  // the widest piece that every address, stride and part of the head allows
  int vmax = 16 / size;
  auto fit = [&](int64_t x) {
    while (x % vmax != 0) vmax /= 2;
  };
  fit((flags & IDX_ROPE_INTERLEAVED) ? rotary_dim : rotary_dim / 2);
  fit(head_dim);
  if (q_heads > 0) {
    a.q = q, a.q_out = q_out, a.q_heads = q_heads, a.q_w = q_weight;
    a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.o_ts = qo_token_stride, a.o_hs = qo_head_stride;
    for (int64_t x : {q_token_stride, q_head_stride, qo_token_stride, qo_head_stride}) fit(x);
    fit(reinterpret_cast<uintptr_t>(q) / size);
    fit(reinterpret_cast<uintptr_t>(q_out) / size);
  }
  if (kv_heads > 0) {
    a.k = k, a.v = v, a.kc = k_cache, a.vc = v_cache, a.kv_heads = kv_heads, a.slots = slots, a.k_w = k_weight;
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
  if (dtype == IDX_BF16) launch_norm<__nv_bfloat16>(a, vmax, inter, s);
  else if (dtype == IDX_F16) launch_norm<__half>(a, vmax, inter, s);
  else launch_norm<float>(a, vmax, inter, s);
  return launch_result();
}
