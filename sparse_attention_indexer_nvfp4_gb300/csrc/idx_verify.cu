// Verification of drafted tokens against the target's probabilities from
// given random numbers.
//
// A node's children are tried in turn against the residual of its target row
// p after the siblings refused before.  The usual recursion r <- max(r - q,
// 0) / mass needs the whole residual row each time; unnormalised it has a
// closed form.  With s_k the residual times the masses divided out so far,
// s_k = max(s_{k-1} - W_{k-1} q, 0), and max(max(a, 0) - b, 0) = max(a - b, 0)
// for b >= 0, so
//     s_k = max(p - c_k q, 0),  c_k = c_{k-1} + W_{k-1},  W_k = sum s_k,
// c_0 = 0, W_0 = 1: a refusal changes one number, and one pass over p and q
// gives the next mass.  No residual row is stored.
//
// A drawn token must be that of the definition in 64 bits: fp32 sums over
// 200,000 terms would move about one draw in 200.  fp64 would do, but at 2 adds
// a clock and SM it, not HBM, would set the pace.  So a thread adds its terms
// in pairs of fp32 numbers (each difference and each addition with its exact
// error, about 2^-45 of the sum), 12 instructions a term where 64-bit integers
// took 54 and the call on 64 rows 49 us; the threads' sums become integer
// multiples of 2^-60, which add up the same in any order.  Sums of p alone are
// formed of such integers from the start, since refused tokens are taken off
// them exactly.
//
// One cluster of CTAs a request.  Each CTA gathers the nodes' probabilities
// and walks the tree by itself (the same numbers in each); a mass is summed
// over the cluster, each warp over its own stretch of the vocabulary, and the
// totals go to every CTA through distributed shared memory.  The draw finds
// CTA and warp from the totals, and the owning CTA reads that one stretch again.
//
// The floor is the HBM read of one target row and, where a token was refused,
// one draft row a request.  What bounds it is the chain of passes: a fixed ~8
// us of latency (launch, gather of the nodes' probabilities, walk, one pass, the
// draw's second look), then a refused token's pass or two a request.  64 chains
// of 8 over 200,003 entries: 28.8 us with clusters of 8 CTAs of 256 threads (of
// 16, 4 and 2 CTAs: 42.7, 33.5 and 48.9; of 512 and 128 threads: 43 and 40; with
// each pass' entries asked into L2 at its start: 33.4); 48 trees of 24 over
// 128,000: 32.6 us, up to 39 as the inputs go (clusters of 16: 36.6; asked into
// L2: 33.0); a chain of 4 over 32,000: 8.6 us.
#include "idx_common.cuh"
#include "idx_internal.h"

namespace idx {
namespace {

constexpr int kThreadsV = 256;
constexpr int kWarpsV = kThreadsV / 32;
constexpr int kMaxNodes = IDX_VERIFY_MAX_NODES;
constexpr int kCluster = 8;
constexpr int kUnrollV = 4;  // loads of four entries in flight a thread and row
constexpr double kUnit = 1152921504606846976.0;  // 2^60
constexpr double kUnitC = 4503599627370496.0;    // 2^52
constexpr double kMostC = 4095.0;

using u64 = unsigned long long;

struct VerifyArgs {
  const float* target;
  int64_t target_stride;
  const float* draft;
  int64_t draft_stride;
  int32_t vocab;
  const int32_t *tokens, *parents, *cu;
  int32_t num_reqs, num_tokens;
  const float *accept_u, *sample_u;
  int32_t *out_tokens, *out_nodes;
  int32_t max_out;
  int32_t* num_accepted;
  int32_t* status;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Store to the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster(u64* p, uint32_t rank, u64 v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.u64 [a], %2;\n\t}" ::"r"(smem_u32(p)),
      "r"(rank), "l"(v)
      : "memory");
}

// Two values at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.f, -1.f), a); }

// A probability: negative and NaN count as 0.
__device__ __forceinline__ float clean(float x) { return fmaxf(x, 0.f); }

// floor(x * 2^60) for 0 <= x < 8, from the bits of x: 24 bits of mantissa
// times 2^(e - 150), so shifted by e - 90 (a right shift of mantissa << 40).
__device__ __forceinline__ u64 fixed_of(float x) {
  const uint32_t bits = __float_as_uint(fminf(x, 7.99f));
  const uint32_t e = bits >> 23;
  const u64 m = (u64)((bits & 0x7FFFFFu) | 0x800000u) << 40;
  const uint32_t sh = 130u - e;
  return e == 0u || sh > 63u ? 0ull : m >> sh;
}

// The term of one vocabulary entry, max(p - c q, 0), in multiples of 2^-60; c
// in multiples of 2^-52 (`one`: c is 1, the first refusal of nearly all walks).
__device__ __forceinline__ u64 term(float p, float q, u64 c52, bool one) {
  const u64 f = fixed_of(clean(q));
  u64 cq = f;
  if (!one) {
    const u64 hi = __umul64hi(f, c52);
    cq = hi >> 52 ? ~0ull : hi << 12 | (f * c52) >> 52;
  }
  const u64 fp = fixed_of(clean(p));
  return fp > cq ? fp - cq : 0ull;
}

// Entries v .. v + 3 of a row, 0 outside it; `vec`: v is at an aligned address.
__device__ __forceinline__ float4 quad_of(const float* row, int v, int vocab, bool vec) {
  if (vec && v >= 0 && v + 4 <= vocab) return *reinterpret_cast<const float4*>(row + v);
  float4 x;
  x.x = v >= 0 && v < vocab ? row[v] : 0.f;
  x.y = v + 1 >= 0 && v + 1 < vocab ? row[v + 1] : 0.f;
  x.z = v + 2 >= 0 && v + 2 < vocab ? row[v + 2] : 0.f;
  x.w = v + 3 < vocab ? row[v + 3] : 0.f;
  return x;
}

// A sum of non-negative numbers as hi + lo, two sums side by side.
struct Sum2 {
  float2 hi = make_float2(0.f, 0.f), lo = make_float2(0.f, 0.f);
  // x and an error term that comes with it
  __device__ __forceinline__ void add(float2 x, float2 err) {
    // two numbers' sum and its exact error, whichever is larger
    const float2 t = add2(hi, x), b = sub2(t, hi);
    const float2 e = add2(sub2(hi, sub2(t, b)), sub2(x, b));
    hi = t;
    lo = add2(lo, add2(e, err));
  }
  __device__ __forceinline__ u64 fixed() const {
    const double v = ((double)hi.x + (double)lo.x) + ((double)hi.y + (double)lo.y);
    return v > 0.0 ? __double2ull_rn(fmin(v, 15.0) * kUnit) : 0ull;
  }
};

// Adds max(p - c q, 0) of two entries, c = ch + cl (kOne: c = 1).  Where p > c q
// the error of the difference is (p - d) - c q exactly.
template <bool kOne>
__device__ __forceinline__ void add_terms(Sum2& s, float2 p, float2 q, float2 ch, float2 cl) {
  p = make_float2(clean(p.x), clean(p.y)), q = make_float2(clean(q.x), clean(q.y));
  float2 cq = q, low = make_float2(0.f, 0.f);
  if (!kOne) {
    cq = mul2(ch, q);
    low = fma2(cl, q, fma2(ch, q, neg2(cq)));  // the product's error and the small part of c
  }
  const float2 d = sub2(p, cq);
  float2 e = sub2(sub2(p, d), cq);
  if (!kOne) e = sub2(e, low);
  s.add(make_float2(fmaxf(d.x, 0.f), fmaxf(d.y, 0.f)), make_float2(d.x > 0.f ? e.x : 0.f, d.y > 0.f ? e.y : 0.f));
}

struct Shared {
  int tok[kMaxNodes], par[kMaxNodes];
  float u[kMaxNodes], p[kMaxNodes], q[kMaxNodes];
  int path[kMaxNodes];
  int refused[kMaxNodes];
  u64 warp_sum[kWarpsV];
  u64 cta_sum[2][kCluster];
  u64 scan[kWarpsV];
  int at, next, taken, num_refused, more;
  double c, w;
};

__global__ void __launch_bounds__(kThreadsV) k_verify(const __grid_constant__ VerifyArgs a) {
  pdl_enter();
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), cs = cluster_size();
  const int r = blockIdx.x / cs;
  const int t0 = max(0, min(a.cu[r], a.num_tokens));
  const int all = max(0, min(a.cu[r + 1], a.num_tokens) - t0);
  const int n = min(all, kMaxNodes);
  int32_t* out_tokens = a.out_tokens + (int64_t)r * a.max_out;
  int32_t* out_nodes = a.out_nodes + (int64_t)r * a.max_out;
  if (rank == 0 && tid == 0 && all > n) report(a.status, IDX_ST_BAD_TREE);
  if (n == 0) {
    if (rank == 0) {
      if (tid == 0) a.num_accepted[r] = 0;
      for (int i = tid; i < a.max_out; i += kThreadsV) out_tokens[i] = out_nodes[i] = -1;
    }
    return;
  }
  for (int i = tid; i < n; i += kThreadsV) {
    const int x = a.tokens[t0 + i];
    int par = a.parents != nullptr ? a.parents[t0 + i] : i - 1;
    if (par < 0 || par >= i || x < 0 || x >= a.vocab) par = -1;
    s.tok[i] = x, s.par[i] = par;
    if (par >= 0) {
      s.u[i] = a.accept_u[t0 + i];
      s.p[i] = clean(a.target[(int64_t)(t0 + par) * a.target_stride + x]);
      s.q[i] = a.draft != nullptr ? clean(a.draft[(int64_t)(t0 + par) * a.draft_stride + x]) : 0.f;
    }
  }
  if (tid == 0) s.at = 0, s.next = 1, s.taken = 0, s.num_refused = 0, s.c = 0.0, s.w = 1.0;
  __syncthreads();

  // The vocabulary in quads of four entries that share an aligned 16-byte load
  // of the target's row (the first and the last quad may be cut); this CTA's
  // quads, and the warp's stretch of them.  `shift` entries lie before the row
  // in its first quad.
  struct Span {
    int shift, lo, hi;  // quads [lo, hi) are this CTA's
  };
  auto span_of = [&](int at) {
    Span w;
    const float* p = a.target + (int64_t)(t0 + at) * a.target_stride;
    w.shift = (int)((reinterpret_cast<uintptr_t>(p) >> 2) & 3);
    const int64_t quads = ((int64_t)a.vocab + w.shift + 3) / 4;
    w.lo = (int)(quads * rank / cs), w.hi = (int)(quads * (rank + 1) / cs);
    return w;
  };
  auto stretch = [&](const Span& w, int k) { return w.lo + (int)((int64_t)(w.hi - w.lo) * k / kWarpsV); };
  int parity = 0;
  bool summed = false;  // a pass has run; with c != 0 it was the state's
  u64 total = 0;

  // Sums of max(p - c q, 0) (q NULL: p without the refused tokens) of node `at`.
  auto pass = [&](int at, double c, bool subtract) {
    const float* p = a.target + (int64_t)(t0 + at) * a.target_stride;
    const float* q = a.draft + (int64_t)(t0 + at) * a.draft_stride;
    const bool with_q = a.draft != nullptr && c != 0.0, one = c == 1.0;
    const bool both = with_q && ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    const float ch1 = (float)c, cl1 = (float)(c - (double)ch1);
    const float2 ch = make_float2(ch1, ch1), cl = make_float2(cl1, cl1);
    Sum2 pair;
    const Span w = span_of(at);
    const int w_lo = stretch(w, warp), w_hi = stretch(w, warp + 1);
    u64 sum = 0;
    for (int k = w_lo + lane; k < w_hi; k += 32 * kUnrollV) {
      float4 pv[kUnrollV], qv[kUnrollV];
#pragma unroll
      for (int e = 0; e < kUnrollV; ++e) {
        pv[e] = qv[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k + 32 * e < w_hi) {
          const int v = 4 * (k + 32 * e) - w.shift;
          pv[e] = quad_of(p, v, a.vocab, true);
          if (with_q) qv[e] = quad_of(q, v, a.vocab, both);
        }
      }
      if (with_q) {
#pragma unroll
        for (int e = 0; e < kUnrollV; ++e) {
          const float2 p0 = make_float2(pv[e].x, pv[e].y), p1 = make_float2(pv[e].z, pv[e].w);
          const float2 q0 = make_float2(qv[e].x, qv[e].y), q1 = make_float2(qv[e].z, qv[e].w);
          if (one) add_terms<true>(pair, p0, q0, ch, cl), add_terms<true>(pair, p1, q1, ch, cl);
          else add_terms<false>(pair, p0, q0, ch, cl), add_terms<false>(pair, p1, q1, ch, cl);
        }
      } else {
#pragma unroll
        for (int e = 0; e < kUnrollV; ++e)
          sum += (fixed_of(clean(pv[e].x)) + fixed_of(clean(pv[e].y))) + (fixed_of(clean(pv[e].z)) + fixed_of(clean(pv[e].w)));
      }
    }
    if (with_q) sum = pair.fixed();
    sum = warp_sum_u64(sum);
    if (subtract)  // the refused tokens of the warp's stretch (each listed once)
      for (int k = 0; k < s.num_refused; ++k) {
        const int x = s.refused[k];
        if ((x + w.shift) / 4 >= w_lo && (x + w.shift) / 4 < w_hi) sum -= fixed_of(clean(p[x]));
      }
    if (lane == 0) s.warp_sum[warp] = sum;
    __syncthreads();
    parity ^= 1;
    if (warp == 0) {
      const u64 mine = warp_sum_u64(lane < kWarpsV ? s.warp_sum[lane] : 0ull);
      if (lane < (int)cs) st_cluster(&s.cta_sum[parity][rank], (uint32_t)lane, mine);
    }
    cluster_sync();
    u64 all_sum = 0;
    for (uint32_t k = 0; k < cs; ++k) all_sum += s.cta_sum[parity][k];
    return all_sum;
  };

  double last_c = 0.0;  // of the last pass
  bool last_excl = false;
  cluster_sync();  // every CTA of the cluster runs: its shared memory may be written
  for (;;) {
    if (warp == 0) {
      int at = s.at, next = s.next, taken = s.taken, nref = s.num_refused, more = 0;
      double c = s.c, w = s.w;
      while (taken < a.max_out - 1) {
        int j = -1;
        for (int b = next; b < n; b += 32) {
          const uint32_t m = __ballot_sync(0xFFFFFFFFu, b + lane < n && s.par[b + lane] == at);
          if (m) {
            j = b + __ffs(m) - 1;
            break;
          }
        }
        if (j < 0) break;
        const double u = s.u[j], q = s.q[j];
        double p = s.p[j];
        bool stands;
        if (a.draft != nullptr) {
          stands = __dmul_rn(u * q, w) < fmax(__dsub_rn(p, __dmul_rn(c, q)), 0.0);
        } else {
          bool again = false;
          for (int k = lane; k < nref; k += 32) again |= s.refused[k] == s.tok[j];
          if (__any_sync(0xFFFFFFFFu, again)) p = 0.0;
          stands = __dmul_rn(u, w) < p;
        }
        next = j + 1;
        if (stands) {
          if (lane == 0) s.path[taken] = j;
          ++taken;
          at = j, c = 0.0, w = 1.0, nref = 0;
        } else if (a.draft != nullptr) {
          c += w;
          more = 1;
          break;
        } else if (p > 0.0) {
          w -= p;
          if (lane == 0) s.refused[nref] = s.tok[j];
          ++nref;
          __syncwarp();
        }
      }
      __syncwarp();
      if (lane == 0) s.at = at, s.next = next, s.taken = taken, s.num_refused = nref, s.more = more, s.c = c;
    }
    __syncthreads();
    const int at = s.at, more = s.more;
    const double c = s.c;
    if (!more) {
      last_excl = a.draft == nullptr;
      if (!summed || c == 0.0) total = pass(at, c, last_excl), last_c = c;  // else the pass of the last refusal holds
      if (total == 0) total = pass(at, 0.0, false), last_c = 0.0, last_excl = false;  // no residual: the row itself
      break;
    }
    total = pass(at, c, false), last_c = c;
    summed = true;
    if (tid == 0) s.w = (double)total / kUnit;
    __syncthreads();
  }

  const int taken = s.taken, at = s.at;
  if (rank == 0) {
    if (tid == 0) a.num_accepted[r] = taken;
    for (int i = tid; i < a.max_out; i += kThreadsV) {
      out_nodes[i] = i < taken ? s.path[i] : -1;
      if (i != taken) out_tokens[i] = i < taken ? s.tok[s.path[i]] : -1;
      else if (total == 0) out_tokens[i] = a.vocab - 1;
    }
  }
  if (total == 0) return;
  // the draw: the first entry whose cumulative sum is above u * total
  u64 thr = __double2ull_rz(fmin(fmax((double)a.sample_u[r], 0.0), 1.0) * (double)total);
  if (thr >= total) thr = total - 1;
  u64 before = 0;
  for (uint32_t k = 0; k < rank; ++k) before += s.cta_sum[parity][k];
  if (thr < before || thr - before >= s.cta_sum[parity][rank]) return;  // another CTA's
  int seg = 0;
  while (seg < kWarpsV - 1 && thr - before >= s.warp_sum[seg]) before += s.warp_sum[seg++];
  const Span span = span_of(at);
  const int lo = stretch(span, seg), hi = stretch(span, seg + 1);
  const float* p = a.target + (int64_t)(t0 + at) * a.target_stride;
  const float* q = a.draft + (int64_t)(t0 + at) * a.draft_stride;
  const bool with_q = a.draft != nullptr && last_c != 0.0, one = last_c == 1.0;
  const u64 c52 = (u64)(fmin(last_c, kMostC) * kUnitC);
  int last = -1;  // this thread's last entry with a term
  if (tid == 0) s.next = -1;
  for (int base = lo; base < hi; base += kThreadsV) {
    const int v0 = 4 * (base + tid) - span.shift;
    const bool in = base + tid < hi;
    const float4 pv = in ? quad_of(p, v0, a.vocab, true) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 qv = in && with_q ? quad_of(q, v0, a.vocab, false) : make_float4(0.f, 0.f, 0.f, 0.f);
    u64 f[4] = {term(pv.x, qv.x, c52, one), term(pv.y, qv.y, c52, one), term(pv.z, qv.z, c52, one), term(pv.w, qv.w, c52, one)};
    if (last_excl)
      for (int k = 0; k < s.num_refused; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (s.refused[k] == v0 + e) f[e] = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (f[e] > 0) last = v0 + e;
    const u64 mine = (f[0] + f[1]) + (f[2] + f[3]);
    u64 incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s.scan[warp] = incl;
    __syncthreads();
    u64 at_warp = before, whole = 0;
#pragma unroll
    for (int w = 0; w < kWarpsV; ++w) {
      if (w < warp) at_warp += s.scan[w];
      whole += s.scan[w];
    }
    u64 sum = at_warp + incl - mine;
    if (mine > 0 && thr >= sum && thr - sum < mine) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (thr >= sum && thr - sum < f[e]) out_tokens[taken] = v0 + e;
        sum += f[e];
      }
    }
    if (thr - before < whole) return;
    before += whole;
    __syncthreads();
  }
  // the sum above was larger by a rounding than these terms: the last of them
  if (last >= 0) atomicMax(&s.next, last);
  __syncthreads();
  if (tid == 0) out_tokens[taken] = s.next >= 0 ? s.next : a.vocab - 1;
}

}  // namespace
}  // namespace idx

extern "C" int idx_verify_drafts(const float* target, int64_t target_stride, const float* draft, int64_t draft_stride,
                                 int32_t vocab, const int32_t* tokens, const int32_t* parents,
                                 const int32_t* cu_tokens, int32_t num_reqs, int32_t num_tokens,
                                 const float* accept_u, const float* sample_u, int32_t* out_tokens,
                                 int32_t* out_nodes, int32_t max_out, int32_t* num_accepted, int32_t* status,
                                 void* stream) {
  using namespace idx;
  if (num_reqs < 0 || num_tokens < 0 || vocab < 1 || max_out < 1) return IDX_E_BAD_SHAPE;
  if (num_tokens > 1 && (target_stride < vocab || (draft && draft_stride < vocab))) return IDX_E_BAD_SHAPE;
  if (num_reqs > 65535 || vocab > (1 << 30)) return IDX_E_TOO_LARGE;
  if (num_reqs == 0) return IDX_OK;
  if (!cu_tokens || !sample_u || !out_tokens || !out_nodes || !num_accepted) return IDX_E_NULL_PTR;
  if (num_tokens > 0 && (!target || !tokens || !accept_u)) return IDX_E_NULL_PTR;
  for (const void* p : {(const void*)target, (const void*)draft, (const void*)tokens, (const void*)parents,
                        (const void*)cu_tokens, (const void*)accept_u, (const void*)sample_u, (const void*)out_tokens,
                        (const void*)out_nodes, (const void*)num_accepted, (const void*)status})
    if (!aligned(p, 4)) return IDX_E_MISALIGNED;
  int rc;
  if ((rc = check_device()) != IDX_OK) return rc;
  const VerifyArgs a{target,  target_stride, draft,    draft_stride, vocab,      tokens,    parents, cu_tokens,   num_reqs,
                     num_tokens, accept_u,   sample_u, out_tokens,   out_nodes,  max_out,   num_accepted, status};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_reqs * kCluster);
  cfg.blockDim = dim3(kThreadsV);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, k_verify, a);
  return launch_result();
}
