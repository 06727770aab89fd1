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
// A cluster of CTAs takes a row, each a stretch of the vocabulary, which stays in
// shared memory as it was read (entries that are left out as -inf) between the
// pass that finds maximum and sum and the one that writes.  Every warp sends its
// two numbers to all CTAs through distributed shared memory and puts the
// cluster's together by itself.  The next row is copied into a second buffer
// meanwhile, where two CTAs an SM have room for one (16-bit logits, up to 200,000
// entries).  A cluster takes rows that follow one another, so a request's special
// entries are found in its counts once for its rows, and there are no more
// clusters than run at once.
//
// HBM bounds it, and the stages of a row: 512 rows of 200,003 bf16 logits with
// counts, 16 biases a request and masks take 192 us where HBM would take 100 for
// their 679 MB.  A row's stages follow one another (in cycles of a CTA, traced
// when it took 200: left out and summed 3,300, changed entries 2,300, the exchange
// 5,000, written 4,000, between them 2,500), and two CTAs an SM do not cover all
// of it.  512 threads a CTA took 272 us, 3 CTAs of 256 with one buffer 219, 128
// threads 257; entries kept in fp32, one CTA an SM, 833.  Past 200,192 16-bit
// entries there is one buffer: 202,048 take 197 us, without counts, biases and masks
// 155 (138 of 200,003).  More than 256 biases a request, or a token with two, are
// searched for by a warp an entry: 388 us with 300 (192 with 250).  One row of
// 32,000: 9.4 us, all latency.
#include <algorithm>
#include <atomic>

#include "idx_internal.h"
#include "idx_rope.cuh"

namespace idx {
namespace {

constexpr int kThreadsP = 256;
constexpr int kWarpsP = kThreadsP / 32;
constexpr int kClusterP = 8;
constexpr int kPathP = IDX_VERIFY_MAX_NODES;
constexpr int kTreeP = 64;    // bits of a tree's mask
constexpr int kMaskP = IDX_PROBS_MAX_VOCAB / kClusterP / 32 / kThreadsP;  // words of bits a thread
constexpr int kCountP = 16;   // words of counts in flight a warp
constexpr int kFixP = 4;      // changed entries a thread takes at a time
constexpr int kListP = kFixP * kThreadsP;
constexpr int kBitsP = IDX_PROBS_MAX_VOCAB / kClusterP / 32;  // words of a stretch
constexpr int kWordP = 4;      // words of special entries a warp takes at a time
constexpr int kStretchP = 8192;  // entries of a CTA with counts, unless a row has 4 CTAs
constexpr size_t kRoomP = 104 * 1024;  // dynamic shared memory of each of two CTAs an SM (which has 228 KB)
// The most that a call takes: that, or one fp32 buffer of the longest stretch with its bits.
constexpr size_t kMostP = std::max(kRoomP, (IDX_PROBS_MAX_VOCAB / kClusterP + 16) * sizeof(float) + (kBitsP + 2) * 8);
constexpr int kBiased = 0x8000;  // an entry of the list that has a bias
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
  int32_t buffers;  // rows in shared memory: the next one comes while one is worked on, or after it
  uint32_t polls;
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
__device__ __forceinline__ void put_cluster_32(void* p, uint32_t rank, uint32_t v) {
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.u32 [a], %2;\n\t}" ::"r"(smem_u32(p)), "r"(rank), "r"(v)
               : "memory");
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
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
};

// Four entries of a row in shared memory from element e on.
__device__ __forceinline__ float4 four_of(const float* xs, int e) { return make_float4(xs[e], xs[e + 1], xs[e + 2], xs[e + 3]); }
template <typename T>
__device__ __forceinline__ float4 four_of(const T* xs, int e) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(xs) + (e >> 1);
  uint32_t y[2] = {w[0], w[1]};
  if (e & 1) y[0] = __funnelshift_r(y[0], y[1], 16), y[1] = __funnelshift_r(y[1], w[2], 16);
  const float2 a = Words<T>::get(y, 0), b = Words<T>::get(y, 1);
  return make_float4(a.x, a.y, b.x, b.y);
}

// What depends on the type of a row's words: -inf, the larger of two words' entries, masked entries.
template <typename T>
struct Packed;
template <>
struct Packed<__nv_bfloat16> {
  static constexpr uint32_t kNeg = 0xFF80FF80u;
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    const __nv_bfloat162 c = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&c);
  }
};
template <>
struct Packed<__half> {
  static constexpr uint32_t kNeg = 0xFC00FC00u;
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    const __half2 c = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&c);
  }
};
template <>
struct Packed<float> {
  static constexpr uint32_t kNeg = 0xFF800000u;
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b))); }
};
// Bytes of the sign bits of x's bytes, as the selector's nibbles (8 + byte) say.
__device__ __forceinline__ uint32_t signs_of(uint32_t x, uint32_t selector) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(r) : "r"(x), "r"(selector));
  return r;
}
// Entries whose bit is set become -inf.
template <typename T>
__device__ __forceinline__ void take_out(uint32_t (&w)[4], uint32_t bits) {
  // bit i to the sign of byte i
  const uint32_t low = (bits & 15u) * 0x10204080u, high = (bits >> 4 & 15u) * 0x10204080u;
  const uint32_t m[4] = {signs_of(low, sizeof(T) == 2 ? 0x9988u : 0x8888u), signs_of(low, sizeof(T) == 2 ? 0xBBAAu : 0x9999u),
                         signs_of(sizeof(T) == 2 ? high : low, sizeof(T) == 2 ? 0x9988u : 0xAAAAu),
                         signs_of(sizeof(T) == 2 ? high : low, sizeof(T) == 2 ? 0xBBAAu : 0xBBBBu)};
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = (w[e] & ~m[e]) | (Packed<T>::kNeg & m[e]);
}

template <typename T>
__global__ void __launch_bounds__(kThreadsP, 2) k_logit_probs(const __grid_constant__ ProbArgs a) {
  pdl_enter();
  constexpr int kV = 16 / (int)sizeof(T);
  // buffers of slice + 16 entries, then two rows of bits, a word before and behind each
  extern __shared__ __align__(16) unsigned char store[];
  const int stretch = a.slice + 16;
  uint32_t* special = reinterpret_cast<uint32_t*>(reinterpret_cast<T*>(store) + (size_t)a.buffers * stretch) + 1;  // entries that the request's counts or biases change
  uint32_t* skip = special + a.slice / 32 + 2;  // entries that the main pass leaves out, those around the stretch among them
  __shared__ uint64_t full[2];
  __shared__ int tokens[kTreeP];       // of the request's first nodes
  __shared__ int bias_at[kThreadsP];     // its biases, where they are no more than this; with `placed`, bias_of as the list has them
  __shared__ float bias_of[kThreadsP];
  __shared__ uint64_t masks[kTreeP];   // of its first nodes
  __shared__ int path_of_tree[kTreeP];
  // The special entries (kBiased: some bias is theirs); where they are more than that, the bits of those that have a bias.
  __shared__ uint32_t list_or_bits[kBitsP];
  uint16_t* list = reinterpret_cast<uint16_t*>(list_or_bits);
  __shared__ uint32_t warp_count[kWarpsP];
  __shared__ int warp_biases[kWarpsP];
  __shared__ unsigned long long parts[2][kClusterP * kWarpsP];  // maximum and sum of each warp of the cluster
  __shared__ int part_at[2][kClusterP * kWarpsP];  // the lowest entry of that maximum (rows of temperature 0)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cta_rank(), cs = (int)cta_count();
  const int lo = min(a.vocab, rank * a.slice), n_here = min(a.vocab, lo + a.slice) - lo, here = (n_here + 31) / 32;
  const int clusters = gridDim.x / cs, cluster = blockIdx.x / cs;
  const int t_lo = (int)((int64_t)a.num_tokens * cluster / clusters), t_hi = (int)((int64_t)a.num_tokens * (cluster + 1) / clusters);
  const T* logits = static_cast<const T*>(a.logits);
  const T* logits_end = logits + (int64_t)(a.num_tokens - 1) * a.l_stride + a.vocab;
  const bool any = a.counts != nullptr || a.bias_cu != nullptr;
  bool bad_tree = false;

  auto row_of = [&](int t) { return logits + (int64_t)t * a.l_stride + lo; };
  auto shift_of = [&](const T* row) { return (int)(reinterpret_cast<uintptr_t>(row) / sizeof(T) % kV); };
  auto vectors_of = [&](int shift) { return n_here > 0 ? (n_here + shift + kV - 1) / kV : 0; };
  int asked = t_lo - 1;  // thread 0's last; after a wait that ran out it asks for none, so a buffer has one copy at most
  auto buffer_of = [&](int t) { return a.buffers == 2 ? (t - t_lo) & 1 : 0; };
  // Thread 0 asks for a row, as whole vectors at their aligned addresses, whatever else is in them; the tensor's first and last
  // vectors may not be whole and are left out.
  auto ask = [&](int t) {
    const T* row = row_of(t);
    const int shift = shift_of(row), vectors = vectors_of(shift);
    const int first = vectors > 0 && row - shift < logits ? 1 : 0, last = vectors > 0 && row - shift + vectors * kV > logits_end ? vectors - 1 : vectors;
    uint64_t* bar = &full[buffer_of(t)];
    const uint32_t bytes = (uint32_t)max(0, last - first) * 16u;
    asked = t;
    mbar_arrive_expect_tx(bar, bytes);
    if (bytes > 0) bulk_g2s(reinterpret_cast<T*>(store) + (size_t)buffer_of(t) * stretch + first * kV, row - shift + first * kV, bytes, bar);
  };
  const uint32_t behind = n_here % 32 != 0 ? ~0u << (n_here % 32) : 0u;  // bits past the stretch in its last word
  auto mask_row = [&](int t) { return reinterpret_cast<const uint32_t*>(a.allowed) + (int64_t)t * a.a_stride + lo / 32; };
  if (tid == 0) {
    skip[-1] = skip[here] = ~0u;
    mbar_init(&full[0], 1), mbar_init(&full[1], 1);
    fence_mbar_init();
    fence_proxy_async_smem();
    if (t_lo < t_hi) ask(t_lo);
  }
  sync_cluster();  // every CTA of the cluster runs: its shared memory may be written

  // the request that the rows are of, and counts and biases of this thread's special entries
  int r = 0, begin = 0, end = 0, changed = 0, unbiased = 0, mine_at = 0, b0 = 0, b1 = 0;
  bool placed = true;  // the list ends with the biased entries, in the biases' order; not where a token has several
  float heat = 1.f, repetition = 1.f, presence = 0.f, frequency = 0.f;
  const int32_t* counts = nullptr;
  const int* path = path_of_tree;  // the drafted tokens on the node's path
  int fix_c[kFixP];
  float fix_b[kFixP], fix[kFixP];
  uint32_t mask_words[kMaskP], fix_mask[kFixP];
  bool timed_out = false;
  bool known = false, many = false, ready = false;  // of the request; more special entries than the list holds; bits and path of the row are there
  int parity = 0, n_path = 0;

  // The special entries into the list: those without a bias (`flags`: the others), or all.
  auto fill = [&](const uint32_t* flags) {
    int at = mine_at;
    for (int w = tid; w < here; w += kThreadsP)
      for (uint32_t bits = special[w] & (flags != nullptr ? ~flags[w] : ~0u); bits != 0; bits &= bits - 1, ++at)
        list[at] = (uint16_t)((32 * w + __ffs(bits) - 1) | (flags != nullptr ? 0 : kBiased));
  };
  // The bias of entry i of lane `of`, a warp together: NaN for several.
  auto find_bias = [&](int i, int of) {
    const bool near = b1 - b0 <= kThreadsP;
    const int* tokens_of = near ? bias_at : a.bias_tokens + b0;
    const int v = lo + __shfl_sync(0xFFFFFFFFu, i, of);
    int found = 0, where = 0;
    for (int b = 0; b < b1 - b0; b += 32) {
      const uint32_t hits = __ballot_sync(0xFFFFFFFFu, b + lane < b1 - b0 && tokens_of[b + lane] == v);
      if (found == 0 && hits != 0) where = b + __ffs(hits) - 1;
      found += __popc(hits);
    }
    return found == 0 ? 0.f : found > 1 ? __int_as_float(0x7FC00000) : near ? bias_of[where] : a.bias_values[b0 + where];
  };
  // counts and biases of this thread's entries of the list
  auto look_up = [&] {
#pragma unroll
    for (int u = 0; u < kFixP; ++u) {
      const int at = tid + u * kThreadsP, e = at < changed ? list[at] : 0;
      fix_c[u] = at < changed && counts != nullptr ? counts[e & ~kBiased] : 0, fix_b[u] = 0.f;
      if (placed) {
        if (e & kBiased) fix_b[u] = bias_of[at - unbiased];
        continue;
      }
      for (uint32_t left = __ballot_sync(0xFFFFFFFFu, (e & kBiased) != 0 && b1 > b0); left != 0; left &= left - 1) {
        const float bias = find_bias(e & ~kBiased, __ffs(left) - 1);
        if (lane == __ffs(left) - 1) fix_b[u] = bias;
      }
    }
  };
  // an entry as it becomes, which the request has `times` times
  auto value_of = [&](int i, float y, int c, int times, bool biased, float bias) {
    if (c < 0 || times > 0) y = y > 0.f ? __fdiv_rn(y, repetition) : __fmul_rn(y, repetition);
    if (times > 0) y = __fsub_rn(y, __fadd_rn(__fmul_rn(frequency, (float)times), presence));
    if (biased) {
      if (bias == bias) {
        y = __fadd_rn(y, bias);
      } else {  // several
        for (int b = b0; b < b1; ++b)
          if (a.bias_tokens[b] == lo + i) y = __fadd_rn(y, a.bias_values[b]);
      }
    }
    return y;
  };
  auto changed_value = [&](int i, float y, int c, bool biased, float bias) {
    int times = c & 0x7FFFFFFF;
    for (int j = 0; j < n_path; ++j) times += path[j] == lo + i;
    return value_of(i, y, c, times, biased, bias);
  };

  for (int t = t_lo; t < t_hi; ++t) {
    float* out = a.probs + (int64_t)t * a.p_stride + lo;
    const T* row = row_of(t);
    const int shift = shift_of(row), vectors = vectors_of(shift);
    T* xs = reinterpret_cast<T*>(store) + (size_t)buffer_of(t) * stretch;
    const bool next = t + 1 < t_hi;
    // (the row before, which was in the other buffer, is used up)
    if (next && a.buffers == 2 && tid == 0 && !timed_out) ask(t + 1);
    auto arrived = [&] {
      const uint32_t phase = (uint32_t)(a.buffers == 2 ? (t - t_lo) >> 1 : t - t_lo) & 1u;
      uint64_t* bar = &full[buffer_of(t)];
      if (!mbar_try_wait_nosuspend(bar, phase) && !mbar_wait(bar, phase, nullptr, timed_out ? 0u : a.polls)) timed_out = true;
    };
    // with one buffer, the next row is asked for when all are done with this one
    auto used_up = [&] {
      fence_proxy_async_smem();
      __syncthreads();
      if (next && a.buffers == 1 && tid == 0 && !timed_out) ask(t + 1);
    };
    if (!known || t < begin || t >= end) {
      // the row's request
      r = 0;
      int top = a.num_reqs;
      while (top - r > 1) {
        const int step = (top - r + 31) / 32, at = r + step * lane;
        const uint32_t below = __ballot_sync(0xFFFFFFFFu, at < top && a.cu[min(at, a.num_reqs)] <= t);
        r += step * max(0, __popc(below) - 1);
        top = min(top, r + step);
      }
      begin = a.num_reqs > 0 ? max(a.cu[r], 0) : 0, end = a.num_reqs > 0 ? min(a.cu[r + 1], a.num_tokens) : 0;
      known = t >= begin && t < end, ready = false;
      if (!known) {  // a padded batch
        for (int i = tid; i < n_here; i += kThreadsP) out[i] = 0.f;
        if (rank == 0 && tid == 0 && a.lse != nullptr) a.lse[t] = kNegInf;
        arrived();
        used_up();
        continue;
      }
      heat = a.temperature != nullptr ? a.temperature[r] : 1.f;
      repetition = a.repetition != nullptr ? a.repetition[r] : 1.f;
      presence = a.presence != nullptr ? a.presence[r] : 0.f, frequency = a.frequency != nullptr ? a.frequency[r] : 0.f;
      if (a.tokens != nullptr) {
        if (a.mask == nullptr) path = a.tokens + begin + 1;  // (a chain's stay where they are)
        else if (tid < min(end - begin, kTreeP)) tokens[tid] = a.tokens[begin + tid];
        if (a.mask != nullptr && tid < min(end - begin, kTreeP)) masks[tid] = a.mask[begin + tid];
        if (a.mask != nullptr) __syncthreads();  // put_path reads other threads' masks
      }
      changed = 0;
      if (any) {
        counts = a.counts != nullptr ? a.counts + (int64_t)r * a.c_stride + lo : nullptr;
        if (a.bias_cu != nullptr) b0 = max(0, a.bias_cu[r]), b1 = min(a.num_bias, a.bias_cu[r + 1]);
        if (counts == nullptr)
          for (int w = tid; w < here; w += kThreadsP) special[w] = 0, skip[w] = 0;
        // words of bits from 32 counts each, kCountP of them in flight a warp (fours a thread, put together by shuffles, took twice the time)
        for (int w0 = counts != nullptr ? warp : here; w0 < here; w0 += kWarpsP * kCountP) {
          int c[kCountP];
#pragma unroll
          for (int u = 0; u < kCountP; ++u) {
            const int i = 32 * (w0 + u * kWarpsP) + lane;
            c[u] = i < n_here ? counts[i] : 0;
          }
#pragma unroll
          for (int u = 0; u < kCountP; ++u) {
            const uint32_t bits = __ballot_sync(0xFFFFFFFFu, c[u] != 0);
            if (lane == 0 && w0 + u * kWarpsP < here) special[w0 + u * kWarpsP] = bits, skip[w0 + u * kWarpsP] = 0;
          }
        }
        __syncthreads();
        bool mine = false, twice = false;  // this thread's bias (the first kThreadsP) is in the stretch; a token has two
        int mine_i = 0;
        float mine_b = 0.f;
        for (int b = b0 + tid; b < b1; b += kThreadsP) {
          const int v = a.bias_tokens[b], i = v - lo;
          const float y = a.bias_values[b];
          if (b1 - b0 <= kThreadsP) bias_at[tid] = v, bias_of[tid] = y, mine_b = y;
          if (v >= lo && i < n_here) {
            atomicOr(&special[i >> 5], 1u << (i & 31));
            twice |= (atomicOr(&skip[i >> 5], 1u << (i & 31)) >> (i & 31) & 1u) != 0;
            mine = true, mine_i = i;
          }
        }
        placed = !__syncthreads_or(twice) && b1 - b0 <= kThreadsP;
        // numbers of special entries: of those without a bias, and (above 16 bits) of all
        uint32_t number = 0;
        for (int w = tid; w < here; w += kThreadsP) number += (uint32_t)__popc(special[w] & ~skip[w]) + ((uint32_t)__popc(special[w]) << 16);
        uint32_t incl = number;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (lane >= o) incl += y;
        }
        const uint32_t with_bias = __ballot_sync(0xFFFFFFFFu, mine);
        if (lane == 31) warp_count[warp] = incl;
        if (lane == 0) warp_biases[warp] = __popc(with_bias);
        __syncthreads();
        uint32_t before = incl - number, all_of = 0;
        int biases = 0, rank_b = __popc(with_bias & ((1u << lane) - 1u));
#pragma unroll
        for (int w = 0; w < kWarpsP; ++w) {
          before += w < warp ? warp_count[w] : 0u, all_of += warp_count[w];
          rank_b += w < warp ? warp_biases[w] : 0, biases += warp_biases[w];
        }
        unbiased = (int)(all_of & 0xFFFFu), mine_at = (int)(before & 0xFFFFu), changed = unbiased + biases;
        placed = placed && changed <= kListP;
        if (!placed) changed = (int)(all_of >> 16), mine_at = (int)(before >> 16);
        many = changed > kListP;
        if (many) {
          for (int w = tid; w < here; w += kThreadsP) list_or_bits[w] = skip[w];
          changed = 0;
        } else if (changed > 0) {
          fill(placed ? skip : nullptr);
        }
        if (placed && mine) list[unbiased + rank_b] = (uint16_t)(mine_i | kBiased), bias_of[rank_b] = mine_b;
        __syncthreads();
        if (changed > 0) look_up();
      }
    }
    if (tid == 0 && counts != nullptr && t + 2 >= end && end < t_hi && r + 1 < a.num_reqs && n_here > 0) {
      // soon the next request's: its counts into L2 (whole 16 bytes inside them)
      const uintptr_t from = (reinterpret_cast<uintptr_t>(counts + a.c_stride) + 15) & ~(uintptr_t)15;
      const uintptr_t to = reinterpret_cast<uintptr_t>(counts + a.c_stride + n_here) & ~(uintptr_t)15;
      if (to > from) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"((uint32_t)(to - from)) : "memory");
    }
    const bool greedy = !(heat > 8.7e-19f);  // 2^-60
    // (not 0 where T is infinite: an entry at -inf, left out ones among them, times 0 would be NaN)
    const float k = greedy ? 1.44269504f : fmaxf(1.44269504f / heat, 0x1p-149f);

    // The path of row t among its request's tokens; then its bits.
    auto put_path = [&](int t) {
      if (a.tokens == nullptr) return;
      const int node = t - begin;
      if (a.mask != nullptr) {
        uint64_t m = (node < kTreeP ? masks[node] : a.mask[begin + node]) & ~1ull;
        if (end - begin < kTreeP) m &= (1ull << (end - begin)) - 1ull;
        n_path = __popcll(m);
        if (tid < kTreeP && (m >> tid & 1)) path_of_tree[__popcll(m & ((1ull << tid) - 1ull))] = tokens[tid];
      } else {
        bad_tree |= node > kPathP;
        n_path = min(node, kPathP);
      }
    };
    auto mark_path = [&] {
      for (int j = tid; j < n_path; j += kThreadsP) {
        const int v = path[j];
        if (v >= lo && v < lo + n_here) atomicOr(&skip[(v - lo) >> 5], 1u << ((v - lo) & 31));
      }
    };
    // bits of this thread's words of row t's mask, and of its special entries (asked for before they are needed)
    auto ask_mask = [&](int t) {
#pragma unroll
      for (int u = 0; u < kMaskP; ++u) {
        mask_words[u] = ~0u;
        if (a.allowed != nullptr && tid + u * kThreadsP < here) mask_words[u] = mask_row(t)[tid + u * kThreadsP];
      }
#pragma unroll
      for (int u = 0; u < kFixP; ++u) {
        fix_mask[u] = ~0u;
        if (a.allowed != nullptr && tid + u * kThreadsP < changed) fix_mask[u] = mask_row(t)[(list[tid + u * kThreadsP] & ~kBiased) >> 5];
      }
    };
    auto put_skip = [&] {
#pragma unroll
      for (int u = 0; u < kMaskP; ++u) {
        const int w = tid + u * kThreadsP;
        if (w < here) skip[w] = (any ? special[w] : 0u) | ~mask_words[u] | (w == here - 1 ? behind : 0u);
      }
    };
    if (!ready) {
      ask_mask(t);
      put_skip();
      put_path(t);
      __syncthreads();
      mark_path();
    }
    const uint32_t* mask = a.allowed != nullptr ? mask_row(t) : nullptr;
    const bool slow = many || n_path > kThreadsP;  // more special entries, or tokens of a path, than one for each thread
    const bool same = next && t + 1 < end && !slow && n_path < kThreadsP;  // the next row is the request's too

    // The row is there.  This thread's special entries as they are, and a token of the path that is none and comes first there.
    arrived();
    if (vectors > 0 && (row - shift < logits || row - shift + vectors * kV > logits_end)) {  // the tensor's first or last vector
      if (tid < 2) {
        const int j = tid == 0 ? 0 : vectors - 1, i = j * kV - shift;
        if (row + i < logits || row + i + kV > logits_end)
          for (int e = 0; e < kV; ++e)
            if (i + e >= 0 && i + e < n_here) xs[j * kV + e] = row[i + e];
      }
      __syncthreads();
    }
    auto stray = [&](int j) {  // entry of the path's token j where it is in this stretch and not special; -1
      const int v = path[j], i = v - lo;
      return v >= lo && i < n_here && (!any || !(special[i >> 5] >> (i & 31) & 1u)) ? i : -1;
    };
    auto comes_first = [&](int j, int i) {
      bool again = false;
      for (int l = 0; l < j; ++l) again |= path[l] == lo + i;
      return !again;
    };
    uint32_t on = 0, extra_mask = ~0u;
    int extra = tid < n_path ? stray(tid) : -1;
    float extra_y = 0.f;
#pragma unroll
    for (int u = 0; u < kFixP; ++u)
      if (tid + u * kThreadsP < changed) fix[u] = to_f(xs[(list[tid + u * kThreadsP] & ~kBiased) + shift]);
    if (extra >= 0) {
      if (mask != nullptr) extra_mask = mask[extra >> 5];
      extra_y = to_f(xs[extra + shift]);
    }
    __syncthreads();
    // Where they are many: body(entry, value) for each, a lane a bit of a word, from the tensor.
    auto each_word = [&](auto&& body) {
      for (int w0 = warp; w0 < here; w0 += kWarpsP * kWordP) {
        float x[kWordP];
        int c[kWordP];
        uint32_t own = 0;
#pragma unroll
        for (int u = 0; u < kWordP; ++u) {
          const int w = w0 + u * kWarpsP, i = 32 * w + lane;
          if (w >= here) continue;
          const uint32_t bits = special[w] & (mask != nullptr ? mask[w] : ~0u);
          x[u] = 0.f, c[u] = 0;
          if (bits >> lane & 1u) own |= 1u << u, x[u] = to_f(row[i]), c[u] = counts != nullptr ? counts[i] : 0;
        }
#pragma unroll
        for (int u = 0; u < kWordP; ++u) {
          const int w = w0 + u * kWarpsP, i = 32 * w + lane;
          if (w >= here) continue;
          const bool mine = own >> u & 1u, biased = mine && (list_or_bits[w] >> lane & 1u);
          float bias = 0.f;
          for (uint32_t left = __ballot_sync(0xFFFFFFFFu, biased); left != 0; left &= left - 1) {
            const float b = find_bias(i, __ffs(left) - 1);
            if (lane == __ffs(left) - 1) bias = b;
          }
          if (mine) body(i, changed_value(i, x[u], c[u], biased, bias));
        }
      }
    };

    // the row: entries that are left out become -inf, then maximum and sum of the others
    Mass mass;
    uint32_t top2 = Packed<T>::kNeg;
#pragma unroll 2
    for (int j = tid; j < vectors; j += kThreadsP) {
      const int i = j * kV - shift, at = i >> 5;  // rounded down: -1 in the first vector
      uint4* here4 = reinterpret_cast<uint4*>(xs + j * kV);
      const uint4 v = *here4;
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
      take_out<T>(w, __funnelshift_r(skip[at], skip[at + 1], i & 31));
      *here4 = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) top2 = Packed<T>::larger(top2, w[e]);
    }
    if (sizeof(T) == 2) {
      const float2 two = Words<T>::get(&top2, 0);
      mass.raise(fmaxf(two.x, two.y), k);
    } else {
      mass.raise(__uint_as_float(top2), k);
    }
    {
      const float b = mass.base();
      const float2 nb = make_float2(-b, -b), kk = make_float2(k, k);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int j = tid; j < vectors; j += kThreadsP) {
        const uint4 v = *reinterpret_cast<const uint4*>(xs + j * kV);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < kV / 2; ++e) {
          const float2 y = mul2(add2(Words<T>::get(w, e), nb), kk);
          sum = add2(sum, make_float2(ex2(y.x), ex2(y.y)));
        }
      }
      mass.s = sum.x + sum.y;
    }
    // the changed entries, all of a thread's together
    {
      int times[kFixP], entry[kFixP];
      float top = kNegInf;
#pragma unroll
      for (int u = 0; u < kFixP; ++u) {
        const int at = tid + u * kThreadsP;
        entry[u] = at < changed ? list[at] : 0, times[u] = fix_c[u] & 0x7FFFFFFF;
        if (at < changed && (fix_mask[u] >> (entry[u] & 31) & 1u)) on |= 1u << u;
      }
      for (int j = 0; j < n_path; ++j) {
        const int i = path[j] - lo;
#pragma unroll
        for (int u = 0; u < kFixP; ++u) times[u] += i == (entry[u] & ~kBiased);
      }
#pragma unroll
      for (int u = 0; u < kFixP; ++u) {
        if (!(on >> u & 1u)) continue;
        fix[u] = value_of(entry[u] & ~kBiased, fix[u], fix_c[u], times[u], (entry[u] & kBiased) && b1 > b0, fix_b[u]);
        top = fmaxf(top, fix[u]);
      }
      mass.raise(top, k);
#pragma unroll
      for (int u = 0; u < kFixP; ++u)
        if (on >> u & 1u) mass.s += ex2((fix[u] - mass.base()) * k);
    }
    if (many) each_word([&](int, float y) { mass.add(y, k); });
    if (extra >= 0 && (!(extra_mask >> (extra & 31) & 1u) || !comes_first(tid, extra))) extra = -1;
    if (extra >= 0) extra_y = changed_value(extra, extra_y, 0, false, 0.f), mass.add(extra_y, k);
    // (of a long chain a thread has more; their values are formed again for each use)
    auto each_later = [&](auto&& body) {
      for (int j = tid + kThreadsP; j < n_path; j += kThreadsP) {
        const int i = stray(j);
        if (i >= 0 && (mask == nullptr || (mask[i >> 5] >> (i & 31) & 1u)) && comes_first(j, i)) body(i, changed_value(i, to_f(row[i]), 0, false, 0.f));
      }
    };
    each_later([&](int, float y) { mass.add(y, k); });

    // body(entry, value) for each of this thread's changed entries; all threads together
    auto each_changed = [&](auto&& body) {
#pragma unroll
      for (int u = 0; u < kFixP; ++u)
        if (on >> u & 1u) body(list[tid + u * kThreadsP] & ~kBiased, fix[u]);
      if (many) each_word(body);
      if (extra >= 0) body(extra, extra_y);
      each_later(body);
    };
    // maximum and sum over the cluster
    auto join = [&] {
      float top = mass.m;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      const float b = top == kNegInf ? 0.f : top;
      mass.s *= ex2((mass.m - b) * k), mass.m = top;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) mass.s += __shfl_xor_sync(0xFFFFFFFFu, mass.s, o);
    };
    const float top_here = mass.m;  // of this thread
    join();
    parity ^= 1;
    if (greedy) {
      int first = 0x7FFFFFFF;
      if (top_here == mass.m && top_here > kNegInf) {  // a thread or few
        for (int j = tid; j < vectors && first == 0x7FFFFFFF; j += kThreadsP) {
          const uint4 v = *reinterpret_cast<const uint4*>(xs + j * kV);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = kV / 2 - 1; e >= 0; --e) {
            const float2 x = Words<T>::get(w, e);
            first = x.x == mass.m ? j * kV - shift + 2 * e : x.y == mass.m ? j * kV - shift + 2 * e + 1 : first;
          }
        }
      }
      __syncwarp();
      each_changed([&](int i, float y) { first = y == mass.m ? min(first, i) : first; });
      const int lowest = __reduce_min_sync(0xFFFFFFFFu, first);
      if (lane < cs) put_cluster_32(&part_at[parity][rank * kWarpsP + warp], (uint32_t)lane, (uint32_t)(lowest == 0x7FFFFFFF ? lowest : lo + lowest));
    }
    if (lane < cs)
      put_cluster(&parts[parity][rank * kWarpsP + warp], (uint32_t)lane,
                  (unsigned long long)__float_as_uint(mass.m) << 32 | (unsigned long long)__float_as_uint(mass.s));
    ready = same;
    if (same) ask_mask(t + 1);
    __syncwarp();
    sync_cluster();
    if (same) put_skip(), put_path(t + 1);
    // each warp puts the cluster's parts together by itself
    float part_m[kClusterP * kWarpsP / 32], part_s[kClusterP * kWarpsP / 32];
    mass.m = kNegInf;
#pragma unroll
    for (int q = 0; q < kClusterP * kWarpsP / 32; ++q) {
      const unsigned long long v = lane + 32 * q < cs * kWarpsP ? parts[parity][lane + 32 * q] : (unsigned long long)__float_as_uint(kNegInf) << 32;
      part_m[q] = __uint_as_float((uint32_t)(v >> 32)), part_s[q] = __uint_as_float((uint32_t)v);
      mass.m = fmaxf(mass.m, part_m[q]);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) mass.m = fmaxf(mass.m, __shfl_xor_sync(0xFFFFFFFFu, mass.m, o));
    mass.s = 0.f;
#pragma unroll
    for (int q = 0; q < kClusterP * kWarpsP / 32; ++q) mass.s += part_s[q] * ex2((part_m[q] - mass.base()) * k);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) mass.s += __shfl_xor_sync(0xFFFFFFFFu, mass.s, o);
    const Mass all = mass;
    const bool none = all.m == kNegInf && all.s == 0.f, broken = !(all.s <= 3.4e38f);
    const float inv = none ? 0.f : 1.f / all.s, b = all.base();
    const float2 nb = make_float2(-b, -b), kk = make_float2(k, k), ii = make_float2(inv, inv);
    auto chance = [&](float2 x) {
      const float2 y = mul2(add2(x, nb), kk);
      return mul2(make_float2(ex2(y.x), ex2(y.y)), ii);
    };
    float value = none ? kNegInf : broken ? __int_as_float(0x7FC00000) : all.m / heat + logf(all.s);
    const bool one = greedy && !none && !broken;
    int chosen = -1;
    if (one) {
      // the lowest entry of the largest
      int at = 0x7FFFFFFF;
#pragma unroll
      for (int q = 0; q < kClusterP * kWarpsP / 32; ++q)
        if (lane + 32 * q < cs * kWarpsP && part_m[q] == all.m) at = min(at, part_at[parity][lane + 32 * q]);
      at = __reduce_min_sync(0xFFFFFFFFu, at);
      chosen = at >= lo && at < lo + n_here ? at - lo : -1;
      value = all.m;
    }
    // fours at the output's aligned addresses
    const int head = min(n_here, (int)(-(reinterpret_cast<uintptr_t>(out) >> 2) & 3)), fours = (n_here - head) / 4, tail = head + 4 * fours;
    const int edge = tid < 4 ? tid : tail + tid - 4;
    const bool at_edge = (tid < 4 && tid < head) || (tid >= 4 && tid < 8 && edge < n_here);
    if (one) {
      for (int f = tid; f < fours; f += kThreadsP) *reinterpret_cast<float4*>(out + head + 4 * f) = make_float4(0.f, 0.f, 0.f, 0.f);
      if (at_edge) out[edge] = 0.f;
    } else if (slow) {
      // changed entries are left as they are (probs may be logits) until each is formed again
      for (int i = tid; i < n_here; i += kThreadsP)
        if (!(skip[i >> 5] >> (i & 31) & 1u) || !(mask == nullptr || (mask[i >> 5] >> (i & 31) & 1u)))
          out[i] = chance(make_float2(to_f(xs[i + shift]), 0.f)).x;
      each_changed([&](int i, float y) { out[i] = chance(make_float2(y, 0.f)).x; });
    } else {
#pragma unroll 4
      for (int f = tid; f < fours; f += kThreadsP) {
        const int i = head + 4 * f;
        const float4 x = four_of(xs, i + shift);
        const float2 p = chance(make_float2(x.x, x.y)), q = chance(make_float2(x.z, x.w));
        *reinterpret_cast<float4*>(out + i) = make_float4(p.x, p.y, q.x, q.y);
      }
      if (at_edge) out[edge] = chance(make_float2(to_f(xs[edge + shift]), 0.f)).x;
    }
    if (rank == 0 && tid == 0 && a.lse != nullptr) a.lse[t] = value;
    used_up();
    if (one) {
      if (tid == 0 && chosen >= 0) out[chosen] = 1.f;
    } else if (!slow) {
      each_changed([&](int i, float y) { out[i] = chance(make_float2(y, 0.f)).x; });
    }
    if (same) mark_path();
  }
  if (timed_out) {
    report(a.status, IDX_ST_TIMEOUT);
    // no copy may come after the CTA is gone
    if (tid == 0)
      for (int t = max(t_lo, asked + 1 - a.buffers); t <= asked; ++t)
        mbar_wait(&full[buffer_of(t)], (uint32_t)(a.buffers == 2 ? (t - t_lo) >> 1 : t - t_lo) & 1u, nullptr);
  }
  if (bad_tree && tid == 0) report(a.status, IDX_ST_BAD_TREE);
}

template <typename T>
int launch_probs(ProbArgs a, cudaStream_t s) {
  const int sms = max(device_sms(), 1);
  // CTAs a row: as few as hold two of its stretches in shared memory, two CTAs an SM (3,200 rows of 32,000 bf16: 2 a row, 152
  // us, where 4 took 213); with counts 4 of them, between which some thousand tokens of a long prompt fit the lists (220 rows
  // of 17,427: 29 us, where 1 took 152; 264 rows of 79,678: 57, where 8 took 71); and more where a few rows leave SMs without any
  auto slice_of = [&](int c) { return ((a.vocab + c - 1) / c + 31) / 32 * 32; };
  auto row_of = [&](int c) { return ((size_t)slice_of(c) + 16) * sizeof(T); };
  auto bits_of = [&](int c) { return ((size_t)slice_of(c) / 32 + 2) * 8; };
  int cs = 1;
  while (cs < kClusterP && (2 * row_of(cs) + bits_of(cs) > kRoomP || (a.counts != nullptr && cs < 4 && slice_of(cs) > kStretchP) || ((int64_t)a.num_tokens * cs < 2 * sms && slice_of(cs) > 2048))) cs *= 2;
  a.slice = slice_of(cs);
  const size_t row = row_of(cs), bits = bits_of(cs);
  a.buffers = 2 * row + bits <= kRoomP ? 2 : 1;
  a.polls = wait_polls();
  const size_t smem = a.buffers * row + bits;
  // The limit belongs to the kernel, not to a call: it is set once a device to what the largest call takes.  (Set by each call
  // to its own size, one host thread lowered it between another's and its launch.)
  static std::atomic<bool> ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return IDX_E_CUDA;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(k_logit_probs<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostP) != cudaSuccess) return IDX_E_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreadsP);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // as many clusters as run at once, and no more than rows
  int clusters = a.num_tokens;
  if ((int64_t)a.num_tokens * cs > sms) {
    cfg.gridDim = dim3((unsigned)(cs * sms));
    int most = 0;
    if (cudaOccupancyMaxActiveClusters(&most, k_logit_probs<T>, &cfg) != cudaSuccess || most < 1) return IDX_E_CUDA;
    clusters = min(clusters, most);
  }
  cfg.gridDim = dim3((unsigned)(clusters * cs));
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, k_logit_probs<T>, a);
  return launch_result();
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
  if (dtype == IDX_BF16) return launch_probs<__nv_bfloat16>(a, s);
  if (dtype == IDX_F16) return launch_probs<__half>(a, s);
  return launch_probs<float>(a, s);
}
