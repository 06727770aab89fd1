// Probabilities from logits, with penalties for repeated tokens, biases and a
// grammar's mask.
//
// A row's entries are x_v = logit, changed where the request has the token
// already (counts, and the drafted tokens on the node's path), biased, -inf
// where the mask has no bit; p_v = e^((x_v - m) / T) / sum.  The entries that
// are changed are few (a request's distinct tokens), so a pass over the row
// knows them by one bit an entry: it takes all others as they are, and a
// second, short pass forms the changed ones one by one, rounded at each step
// as the formula is written.
//
// Bound by HBM: a row is read once and written once.  A cluster of CTAs takes a
// row, each a stretch of the vocabulary, whose x stay in shared memory as fp32
// between the pass that finds maximum and sum (a running maximum and a sum
// rescaled when it grows, a thread) and the one that writes; the CTAs exchange
// both through distributed shared memory.  A cluster takes rows that follow one
// another, so a request's bits are formed from its counts once for its rows.
#include "idx_internal.h"
#include "idx_rope.cuh"

namespace idx {
namespace {

constexpr int kThreadsP = 512;
constexpr int kWarpsP = kThreadsP / 32;
constexpr int kClusterP = 8;
constexpr int kPathP = IDX_VERIFY_MAX_NODES;
constexpr int kFixP = 8;  // words of bits a warp looks at together
constexpr float kNegInf = -INFINITY;

struct ProbArgs {
  const void* logits;
  int64_t l_stride;
  float* probs;
  int64_t p_stride;
  int32_t vocab, num_tokens, num_reqs;
  const int32_t* cu;
  const float *temperature, *repetition, *presence, *frequency;
  const int32_t* counts;
  int64_t c_stride;
  const int32_t* tokens;
  const uint64_t* mask;
  const int32_t *bias_cu, *bias_tokens;
  const float* bias_values;
  int32_t num_bias;
  const int32_t* allowed;
  int64_t a_stride;
  float* lse;
  int32_t* status;
  int32_t slice;  // entries of a CTA, a multiple of 32
};

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cta_count() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void sync_cluster() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void put_cluster(void* p, uint32_t rank, unsigned long long v) {
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.u64 [a], %2;\n\t}" ::"r"(smem_u32(p)), "r"(rank), "l"(v)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A running maximum and the sum of 2^((x - m) k) below it.
struct Mass {
  float m = kNegInf, s = 0.f;
  __device__ __forceinline__ float base() const { return m == kNegInf ? 0.f : m; }
  __device__ __forceinline__ void raise(float to, float k) {
    if (to > m) {
      s *= ex2((m - to) * k);
      m = to;
    }
  }
  __device__ __forceinline__ void add(float x, float k) {
    raise(x, k);
    s += ex2((x - base()) * k);
  }
  __device__ __forceinline__ void join(float om, float os, float k) {
    const float top = fmaxf(m, om), b = top == kNegInf ? 0.f : top;
    s = s * ex2((m - b) * k) + os * ex2((om - b) * k);
    m = top;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreadsP, 2) k_logit_probs(const __grid_constant__ ProbArgs a) {
  pdl_enter();
  constexpr int kV = 16 / (int)sizeof(T);
  constexpr int kUnroll = 4;
  extern __shared__ __align__(16) float xs[];  // slice + 16 entries, then three rows of bits
  const int words = a.slice / 32;
  uint32_t* seen = reinterpret_cast<uint32_t*>(xs + a.slice + 16);  // tokens with counts
  uint32_t* listed = seen + words;                                  // tokens on the path or in the biases
  uint32_t* skip = listed + words;                                  // entries that the main pass leaves out
  __shared__ int path[kPathP];
  __shared__ float2 warp_mass[kWarpsP];
  __shared__ unsigned long long cta_mass[2][kClusterP];
  __shared__ unsigned long long cta_first[2][kClusterP];
  __shared__ int first_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cta_rank(), cs = (int)cta_count();
  const int cluster = blockIdx.x / cs, clusters = gridDim.x / cs;
  const int lo = min(a.vocab, rank * a.slice), hi = min(a.vocab, lo + a.slice), n_here = hi - lo;
  const int t_lo = (int)((int64_t)a.num_tokens * cluster / clusters), t_hi = (int)((int64_t)a.num_tokens * (cluster + 1) / clusters);
  int r_at = -1, parity = 0;
  bool bad_tree = false;
  sync_cluster();  // every CTA of the cluster runs: its shared memory may be written

  for (int t = t_lo; t < t_hi; ++t) {
    // the row's request
    int r = 0;
    {
      int top = a.num_reqs;
      while (top - r > 1) {
        const int step = (top - r + 31) / 32, at = r + step * lane;
        const uint32_t below = __ballot_sync(0xFFFFFFFFu, at < top && a.cu[min(at, a.num_reqs)] <= t);
        r += step * max(0, __popc(below) - 1);
        top = min(top, r + step);
      }
    }
    const int begin = a.num_reqs > 0 ? max(a.cu[r], 0) : 0, end = a.num_reqs > 0 ? min(a.cu[r + 1], a.num_tokens) : 0;
    float* out = a.probs + (int64_t)t * a.p_stride + lo;
    if (t < begin || t >= end) {  // a padded batch
      for (int i = tid; i < n_here; i += kThreadsP) out[i] = 0.f;
      if (rank == 0 && tid == 0 && a.lse != nullptr) a.lse[t] = kNegInf;
      continue;
    }
    const float heat = a.temperature != nullptr ? a.temperature[r] : 1.f;
    const bool greedy = !(heat > 8.7e-19f);  // 2^-60
    const float k = greedy ? 1.44269504f : 1.44269504f / heat;
    const T* row = static_cast<const T*>(a.logits) + (int64_t)t * a.l_stride + lo;
    const int32_t* counts = a.counts != nullptr ? a.counts + (int64_t)r * a.c_stride + lo : nullptr;
    const uint32_t* allowed = a.allowed != nullptr ? reinterpret_cast<const uint32_t*>(a.allowed) + (int64_t)t * a.a_stride + lo / 32 : nullptr;

    // which entries are changed
    const bool any = counts != nullptr || a.tokens != nullptr || a.bias_cu != nullptr, some = any || allowed != nullptr;
    const int here = (n_here + 31) / 32;
    if (counts != nullptr && r != r_at) {
      for (int w = warp; w < here; w += kWarpsP) {
        const int i = 32 * w + lane;
        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, i < n_here && counts[i] != 0);
        if (lane == 0) seen[w] = bits;
      }
    }
    r_at = r;
    int n_path = 0, b0 = 0, b1 = 0;
    if (any) {
      for (int w = tid; w < here; w += kThreadsP) listed[w] = 0;
      if (a.tokens != nullptr) {
        const int node = t - begin;
        if (a.mask != nullptr) {
          uint64_t m = a.mask[t] & ~1ull;
          if (end - begin < 64) m &= (1ull << (end - begin)) - 1ull;
          n_path = __popcll(m);
          if (tid < 64 && (m >> tid & 1)) path[__popcll(m & ((1ull << tid) - 1ull))] = a.tokens[begin + tid];
        } else {
          n_path = min(node, kPathP);
          bad_tree |= node > kPathP;
          for (int j = tid; j < n_path; j += kThreadsP) path[j] = a.tokens[begin + 1 + j];
        }
      }
      if (a.bias_cu != nullptr) b0 = max(0, a.bias_cu[r]), b1 = min(a.num_bias, a.bias_cu[r + 1]);
      __syncthreads();
      for (int j = tid; j < n_path; j += kThreadsP) {
        const int v = path[j];
        if (v >= lo && v < hi) atomicOr(&listed[(v - lo) >> 5], 1u << ((v - lo) & 31));
      }
      for (int b = b0 + tid; b < b1; b += kThreadsP) {
        const int v = a.bias_tokens[b];
        if (v >= lo && v < hi) atomicOr(&listed[(v - lo) >> 5], 1u << ((v - lo) & 31));
      }
      __syncthreads();
    }
    if (some) {
      for (int w = tid; w < here; w += kThreadsP) {
        uint32_t bits = 0;
        if (any) bits = listed[w] | (counts != nullptr ? seen[w] : 0u);
        if (allowed != nullptr) bits |= ~allowed[w];
        skip[w] = bits;
      }
      __syncthreads();
    }

    // the row into shared memory, as vectors at their aligned addresses
    const int shift = (int)(reinterpret_cast<uintptr_t>(row) / sizeof(T) % kV);
    const int vectors = n_here > 0 ? (n_here + shift + kV - 1) / kV : 0;
    Mass mass;
    for (int j0 = tid; j0 < vectors; j0 += kThreadsP * kUnroll) {
      uint4 raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int j = j0 + u * kThreadsP, i = j * kV - shift;
        if (j < vectors && i >= 0 && i + kV <= n_here) raw[u] = ld_stream_u4(row + i);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int j = j0 + u * kThreadsP, i = j * kV - shift;
        if (j >= vectors) continue;
        float x[kV];
        uint32_t bits = 0;
        if (i >= 0 && i + kV <= n_here) {
          const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
          for (int e = 0; e < kV / 2; ++e) {
            const float2 p = Words<T>::get(w, e);
            x[2 * e] = p.x, x[2 * e + 1] = p.y;
          }
          if (some) bits = __funnelshift_r(skip[i >> 5], (i & 31) + kV > 32 ? skip[(i >> 5) + 1] : 0u, i & 31);
        } else {
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            const bool in = i + e >= 0 && i + e < n_here;
            x[e] = in ? to_f(row[i + e]) : 0.f;
            if (!in || (some && (skip[(i + e) >> 5] >> ((i + e) & 31) & 1u))) bits |= 1u << e;
          }
        }
        if (some || bits) {
#pragma unroll
          for (int e = 0; e < kV; ++e) x[e] = bits >> e & 1u ? kNegInf : x[e];
        }
        float top = x[0];
#pragma unroll
        for (int e = 1; e < kV; ++e) top = fmaxf(top, x[e]);
        mass.raise(top, k);
        const float b = mass.base();
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int e = 0; e < kV; e += 2) s0 += ex2((x[e] - b) * k), s1 += ex2((x[e + 1] - b) * k);
        mass.s += s0 + s1;
#pragma unroll
        for (int e = 0; e < kV; e += 4) *reinterpret_cast<float4*>(xs + j * kV + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
      }
    }
    if (any) {
      // the changed entries: a warp looks at kFixP words of bits, a lane has a bit of each
      const float rep = a.repetition != nullptr ? a.repetition[r] : 1.f, pres = a.presence != nullptr ? a.presence[r] : 0.f,
                  freq = a.frequency != nullptr ? a.frequency[r] : 0.f;
      __syncthreads();
      for (int w0 = warp * kFixP; w0 < here; w0 += kWarpsP * kFixP) {
        float x[kFixP];
        int c[kFixP];
        uint32_t on = 0;
#pragma unroll
        for (int u = 0; u < kFixP; ++u) {
          const int w = w0 + u, i = 32 * w + lane;
          if (w >= here) continue;
          uint32_t bits = listed[w] | (counts != nullptr ? seen[w] : 0u);
          if (allowed != nullptr && bits != 0) bits &= allowed[w];
          if (bits >> lane & 1u) {
            on |= 1u << u;
            x[u] = to_f(row[i]);
            c[u] = counts != nullptr ? counts[i] : 0;
          }
        }
#pragma unroll
        for (int u = 0; u < kFixP; ++u) {
          if (!(on >> u & 1u)) continue;
          const int w = w0 + u, i = 32 * w + lane;
          const bool in_list = listed[w] >> lane & 1u, prompt = c[u] < 0;
          int times = c[u] & 0x7FFFFFFF;
          if (in_list)
            for (int j = 0; j < n_path; ++j) times += path[j] == lo + i;
          float y = x[u];
          if (prompt || times > 0) y = y > 0.f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
          if (times > 0) y = __fsub_rn(y, __fadd_rn(__fmul_rn(freq, (float)times), pres));
          if (in_list)
            for (int b = b0; b < b1; ++b)
              if (a.bias_tokens[b] == lo + i) y = __fadd_rn(y, a.bias_values[b]);
          xs[i + shift] = y;
          mass.add(y, k);
        }
      }
    }

    // maximum and sum over the cluster
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) mass.join(__shfl_xor_sync(0xFFFFFFFFu, mass.m, o), __shfl_xor_sync(0xFFFFFFFFu, mass.s, o), k);
    if (lane == 0) warp_mass[warp] = make_float2(mass.m, mass.s);
    __syncthreads();
    parity ^= 1;
    if (warp == 0) {
      const float2 w = lane < kWarpsP ? warp_mass[lane] : make_float2(kNegInf, 0.f);
      mass.m = w.x, mass.s = w.y;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) mass.join(__shfl_xor_sync(0xFFFFFFFFu, mass.m, o), __shfl_xor_sync(0xFFFFFFFFu, mass.s, o), k);
      if (lane < cs)
        put_cluster(&cta_mass[parity][rank], (uint32_t)lane,
                    (unsigned long long)__float_as_uint(mass.m) << 32 | (unsigned long long)__float_as_uint(mass.s));
    }
    if (tid == 0) first_s = 0x7FFFFFFF;
    __syncwarp();
    sync_cluster();
    Mass all;
    for (int c = 0; c < cs; ++c) {
      const unsigned long long v = cta_mass[parity][c];
      all.join(__uint_as_float((uint32_t)(v >> 32)), __uint_as_float((uint32_t)v), k);
    }
    const bool none = all.m == kNegInf && all.s == 0.f, broken = !(all.s <= 3.4e38f);
    float value = 0.f;
    if (greedy && !none && !broken) {
      // the lowest entry of the largest
      int first = 0x7FFFFFFF;
      for (int i = tid; i < n_here; i += kThreadsP)
        if (xs[i + shift] == all.m) {
          first = i;
          break;
        }
      first = __reduce_min_sync(0xFFFFFFFFu, first);
      if (lane == 0 && first != 0x7FFFFFFF) atomicMin(&first_s, first);
      __syncthreads();
      if (tid < cs)
        put_cluster(&cta_first[parity][rank], (uint32_t)tid, first_s == 0x7FFFFFFF ? ~0ull : (unsigned long long)(lo + first_s));
      __syncwarp();
      sync_cluster();
      unsigned long long at = ~0ull;
      for (int c = 0; c < cs; ++c) at = min(at, cta_first[parity][c]);
      for (int i = tid; i < n_here; i += kThreadsP) out[i] = (unsigned long long)(lo + i) == at ? 1.f : 0.f;
      value = all.m;
    } else {
      const float inv = none ? 0.f : 1.f / all.s, b = all.base();
#pragma unroll 4
      for (int i = tid; i < n_here; i += kThreadsP) out[i] = ex2((xs[i + shift] - b) * k) * inv;
      value = none ? kNegInf : broken ? __int_as_float(0x7FC00000) : all.m / heat + logf(all.s);
    }
    if (rank == 0 && tid == 0 && a.lse != nullptr) a.lse[t] = value;
    __syncthreads();  // the entries are used up
  }
  if (bad_tree && tid == 0) report(a.status, IDX_ST_BAD_TREE);
}

template <typename T>
void launch_probs(ProbArgs a, cudaStream_t s) {
  const int sms = max(device_sms(), 1);
  // CTAs a row: stretches of at most 8,192 entries, shorter ones where a few rows leave SMs without any
  int cs = 1;
  auto slice_of = [&](int c) { return ((a.vocab + c - 1) / c + 31) / 32 * 32; };
  while (cs < kClusterP && (slice_of(cs) > 8192 || ((int64_t)a.num_tokens * cs < 2 * sms && slice_of(cs) > 2048))) cs *= 2;
  a.slice = slice_of(cs);
  const size_t smem = (size_t)(a.slice + 16) * 4 + (size_t)a.slice / 32 * 12;
  const int per_sm = max(1, min(4, (int)(220 * 1024 / (smem + 8192))));
  const int clusters = (int)min((int64_t)a.num_tokens, max((int64_t)1, (int64_t)sms * per_sm / cs));
  cudaFuncSetAttribute(k_logit_probs<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * cs));
  cfg.blockDim = dim3(kThreadsP);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cs, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, k_logit_probs<T>, a);
}

}  // namespace
}  // namespace idx

extern "C" int idx_logit_probs(const void* logits, int64_t logits_stride, int32_t dtype, int32_t vocab, int32_t num_tokens,
                               const int32_t* cu_tokens, int32_t num_reqs, const float* temperature, const float* repetition,
                               const float* presence, const float* frequency, const int32_t* counts, int64_t counts_stride,
                               const int32_t* tokens, const uint64_t* tree_mask, const int32_t* bias_cu, const int32_t* bias_tokens,
                               const float* bias_values, int32_t num_bias, const int32_t* allowed, int64_t allowed_stride, float* probs,
                               int64_t probs_stride, float* lse, int32_t* status, void* stream) {
  using namespace idx;
  if (vocab < 1 || num_tokens < 0 || num_reqs < 0 || num_bias < 0 || dtype < IDX_BF16 || dtype > IDX_F32) return IDX_E_BAD_SHAPE;
  if (num_tokens > 1 && (logits_stride < vocab || probs_stride < vocab)) return IDX_E_BAD_SHAPE;
  if (counts && num_reqs > 1 && counts_stride < vocab) return IDX_E_BAD_SHAPE;
  if (allowed && num_tokens > 1 && allowed_stride < (vocab + 31) / 32) return IDX_E_BAD_SHAPE;
  if (vocab > IDX_PROBS_MAX_VOCAB || num_reqs > 65535) return IDX_E_TOO_LARGE;
  if (num_tokens == 0) return IDX_OK;
  if (!logits || !probs || !cu_tokens || (tree_mask && !tokens)) return IDX_E_NULL_PTR;
  if (bias_cu && num_bias > 0 && (!bias_tokens || !bias_values)) return IDX_E_NULL_PTR;
  if (!aligned(logits, dtype == IDX_F32 ? 4 : 2) || !aligned(tree_mask, 8)) return IDX_E_MISALIGNED;
  for (const void* p : {(const void*)cu_tokens, (const void*)temperature, (const void*)repetition, (const void*)presence, (const void*)frequency,
                        (const void*)counts, (const void*)tokens, (const void*)bias_cu, (const void*)bias_tokens, (const void*)bias_values,
                        (const void*)allowed, (const void*)probs, (const void*)lse, (const void*)status})
    if (!aligned(p, 4)) return IDX_E_MISALIGNED;
  int rc;
  if ((rc = check_device()) != IDX_OK) return rc;
  ProbArgs a{};
  a.logits = logits, a.l_stride = logits_stride, a.probs = probs, a.p_stride = probs_stride;
  a.vocab = vocab, a.num_tokens = num_tokens, a.num_reqs = num_reqs, a.cu = cu_tokens, a.temperature = temperature;
  if (repetition || presence || frequency) {  // without a penalty no count is looked at
    a.repetition = repetition, a.presence = presence, a.frequency = frequency;
    a.counts = counts, a.c_stride = counts_stride, a.tokens = tokens, a.mask = tree_mask;
  }
  if (num_bias > 0) a.bias_cu = bias_cu, a.bias_tokens = bias_tokens, a.bias_values = bias_values, a.num_bias = num_bias;
  a.allowed = allowed, a.a_stride = allowed_stride, a.lse = lse, a.status = status;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == IDX_BF16) launch_probs<__nv_bfloat16>(a, s);
  else if (dtype == IDX_F16) launch_probs<__half>(a, s);
  else launch_probs<float>(a, s);
  return launch_result();
}
