// Attention of a step's tokens over the paged cache (tcgen05 + TMA, sm_103a).
//
//     out = sum_p e^(s_p - L) v_p,  L = ln sum_p e^s_p,  s_p = scale (q . k_p)
//
// over the places p that a token sees, in one pass over the keys: with M a
// reference maximum of the scores met so far, l = sum e^(s - M) and O = sum
// e^(s - M) v are carried along, and a larger score only rescales them.
//
// A segment is (request, block of tokens, KV head): the block's tokens times
// the query heads of one KV head are the 128 rows of an MMA, so each key and
// value tile is read once for all of them.  Its keys come in tiles of 128
// places, gathered by TMA from the pages (several boxes a tile for pages
// below 128 places).  All tiles of all segments form one line of units; each
// of the persistent CTAs, one an SM, takes an equal stretch of it.  A segment cut
// by a stretch's end leaves partial (O, M, l) in the workspace, which
// k_tree_combine joins.
//
// Roles of a CTA (six warps):
//   warps 0-3  one thread a row: scores from TMEM, softmax, weights back to
//              TMEM, and at a segment's end the rows' results;
//   warp 4     TMA: the queries, then key and value tiles through a ring of
//              kStages, and a record of each tile (its places, what is masked);
//   warp 5     one thread issues the MMAs: S = Q K^T (both from shared
//              memory), O += P V (P in TMEM, V as it lies, places along K);
//              S is doubled, so tile i+1's scores form during tile i's softmax.
// With at most 64 (32) live rows the queries stand two (four) times in the
// 128 rows, and copy c of a row takes the softmax of the c-th part of each
// tile's places, its weights for the others being zero: four warps share the
// work that otherwise one would do, and the copies' (O, M, l) join at the end.
//
// The bound is HBM for up to ~128 rows a KV head (4 D flops a row and key
// against 4 D bytes a key: 128 flops a byte, below the ridge of ~280).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "idx_common.cuh"
#include "idx_internal.h"
#include "idx_tc.cuh"

namespace idx {
namespace {

constexpr int kRowsA = 128;         // rows of an MMA
constexpr int kTile = 128;          // places of a tile
constexpr int kMaxCtas = 160;       // persistent CTAs at most (workspace sizes depend on it)
constexpr int kStagesA = 5;         // key and value tiles in flight
constexpr int kSoftWarps = 4;
constexpr int kTmaWarp = 4, kMmaWarpA = 5;
constexpr int kThreadsA = 6 * 32;
constexpr int kRecs = 8;            // tile records (the producer leads by at most 3 tiles)
constexpr int kRecWords = 32;
constexpr int kGroup = 16;          // places of a record's group
constexpr int kMaxListTokens = 32;  // tokens of a block with page lists (bits of a mask)
constexpr float kRescale = 8.f;     // powers of two that a weight may exceed 1 before O is rescaled
constexpr float kLog2e = 1.4426950408889634f;

// TMEM columns
constexpr uint32_t kColS = 0, kColO = 256, kColP = 384, kTmemColsA = 512;

enum RecWord { kRFlags, kRTok0, kRTokens, kRHead, kRCtx, kRNew, kRNode0, kRLen, kRPos, kRMask = kRPos + 8, kROut = kRMask + 8,
               kRReq, kRFirst, kREnd, kRList };
static_assert(kRList < kRecWords, "a record fits");
constexpr int kFlagFirst = 1, kFlagLast = 2, kKindShift = 2, kFoldShift = 4;
enum Kind { kFull = 0, kRowMask = 1, kGeneral = 2 };  // every row sees every place / whole rows do or do not / place by place

struct ListEntry {
  int32_t block, page;
  uint32_t tokens;  // bit i: token i of the block lists the page
  int32_t pad;
};

struct TreeArgs {
  const void* q;
  int64_t q_ts, q_hs;
  const void *kc, *vc;
  int64_t num_blocks;
  int32_t page;
  int64_t c_bs, c_ts, c_hs;
  const int32_t* bt;
  int64_t bt_stride;
  int32_t max_blocks;
  const int32_t *seq_lens, *cu;
  int32_t num_reqs, num_tokens, q_heads, kv_heads, group;
  const uint64_t* mask;
  const int32_t* pages;
  int32_t lists, per;
  float scale;
  void* out;
  int64_t o_ts, o_hs;
  float* lse;
  int32_t* status;
  // workspace
  int32_t* cuts;       // [kMaxCtas][8]: the segment that each CTA's stretch begins inside
  float* part_ml;      // [2 * kMaxCtas][128][2]
  float* part_o;       // [2 * kMaxCtas][128][D]
  int32_t* counts;     // [num_tokens * lists], at a block's first token
  ListEntry* entries;  // [num_tokens * lists * per]
  int32_t block_tokens;
  uint32_t polls;
};

// The cut of all requests into segments and tiles.
struct Plan {
  const TreeArgs& a;
  __device__ explicit Plan(const TreeArgs& args) : a(args) {}
  __device__ int tok0(int r) const { return max(0, min(a.cu[r], a.num_tokens)); }
  __device__ int ntok(int r) const { return max(0, min(a.cu[r + 1], a.num_tokens) - tok0(r)); }
  __device__ int seq(int r) const { return max(0, a.seq_lens[r]); }
  __device__ int len(int s) const { return (int)min((int64_t)s, (int64_t)a.max_blocks * a.page); }
  __device__ int blocks(int n) const { return (n + a.block_tokens - 1) / a.block_tokens; }
  // tiles of block b of a request with n tokens from t0 on, list lh
  __device__ int tiles(int s, int n, int t0, int b, int lh) const {
    if (a.pages != nullptr) {
      // (cut to what a block can list, so that bad cu_tokens cannot make the line of units endless)
      const int64_t c = max(0, min(a.counts[(int64_t)(t0 + b * a.block_tokens) * a.lists + lh], a.block_tokens * a.per));
      return max(1, (int)((c * a.page + kTile - 1) / kTile));
    }
    int lim = len(s);
    // a chain's block sees nothing past its last token
    if (a.mask == nullptr) lim = min(lim, max(0, s - n + min(n, (b + 1) * a.block_tokens)));
    return max(1, (int)(((int64_t)lim + kTile - 1) / kTile));
  }
  __device__ unsigned long long units(int r) const {
    const int n = ntok(r), t0 = tok0(r), s = seq(r), nl = a.pages != nullptr ? a.lists : 1;
    unsigned long long sum = 0;
    for (int b = 0; b < blocks(n); ++b)
      for (int l = 0; l < nl; ++l) sum += (unsigned long long)tiles(s, n, t0, b, l);
    return sum * (unsigned)(a.kv_heads / nl);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 consecutive 32-bit columns of this thread's TMEM lane from registers.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// tcgen05 instruction descriptor, kind::f16: D f32, A and B both f16 (0) or
// bf16 (1), A K-major, B K-major or (tb) N-major.
__host__ __device__ constexpr uint32_t idesc_16(bool bf16, int m, int n, bool tb) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((tb ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Shared-memory descriptor of an N-major operand, 128-byte swizzle: rows of 64
// elements along N (128 bytes), 8 of them along K an atom of 1,024 bytes; the
// next 8 along K 1,024 bytes on (stride offset), the next 64 along N
// kTile * 128 bytes on (leading offset).
__device__ __forceinline__ uint64_t sw128_desc_nmajor(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((kTile * 128) >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void mma_16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}

// 4-D TMA box into shared memory.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

template <typename T>
struct Num;
template <>
struct Num<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static constexpr CUtensorMapDataType kMap = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  // two values rounded to nearest: the weights of the product with v
  static __device__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ float2 unpack(uint32_t x) { return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)); }
};
template <>
struct Num<__half> {
  static constexpr bool kBf16 = false;
  static constexpr CUtensorMapDataType kMap = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  static __device__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ float2 unpack(uint32_t x) {
    return make_float2(__half2float(__ushort_as_half((unsigned short)(x & 0xFFFFu))),
                       __half2float(__ushort_as_half((unsigned short)(x >> 16))));
  }
};

// Shared memory
template <int D>
struct Smem {
  static constexpr int kQ = kRowsA * D * 2, kKv = kTile * D * 2;
  static constexpr int kScratchRow = 33;  // floats: 32 columns and one of padding
  static constexpr int kOffQ = 0;
  static constexpr int kOffKv = kOffQ + kQ;
  static constexpr int kOffScratch = kOffKv + kStagesA * kKv;
  static constexpr int kOffStats = kOffScratch + kRowsA * kScratchRow * 4;
  static constexpr int kOffRec = kOffStats + kRowsA * 8;
  static constexpr int kOffBar = kOffRec + kRecs * kRecWords * 4;
  static constexpr int kOffMisc = kOffBar + 64 * 8;
  static constexpr int kBytes = kOffMisc + 64 + 1024;
};
enum BarsA { kKvFull = 0, kKvEmpty = kKvFull + kStagesA, kQFullA = kKvEmpty + kStagesA, kQEmptyA, kSFull, kPFull = kSFull + 2,
             kPvDone, kOEmpty, kMerge, kRecFull, kDrainA = kRecFull + kRecs, kNumBarsA };
static_assert(kNumBarsA <= 64, "barriers fit");

struct MiscA {
  uint32_t tmem_base;
  int abort_flag;
  unsigned long long total;
  unsigned long long rem0;
  int r0;
};

// What a row's softmax needs of its segment.
struct RowState {
  uint64_t tree;  // drafted tokens that the row's token sees
  int ctx, len, chain_end;  // cached places; places that exist; places that a chain's token sees
  int token;                // of the block
};

// Bits of a record's group (places pos .. pos + 15) that the row sees.
__device__ __forceinline__ uint32_t group_bits(int pos, uint32_t tokens, const RowState& s, bool tree, bool lists) {
  if (pos < 0 || (lists && !((tokens >> s.token) & 1u))) return 0u;
  auto below = [](int n) { return n >= kGroup ? 0xFFFFu : n <= 0 ? 0u : (1u << n) - 1u; };
  const uint32_t exist = below(s.len - pos);
  if (!tree) return exist & below(s.chain_end - pos);
  const int j = pos - s.ctx;  // the drafted token at the first place
  const uint32_t drafted = j >= 64 || j <= -kGroup ? 0u : j >= 0 ? (uint32_t)(s.tree >> j) : (uint32_t)(s.tree << -j);
  const uint32_t cached = below(-j);
  return exist & (cached | (drafted & ~cached)) & 0xFFFFu;
}

// One tile's softmax for copies of 128 / F rows: scores in, weights out.
// Returns through m, l the row's reference maximum (of raw scores) and sum.
template <typename T, int D, int F>
__device__ __forceinline__ bool soft_tile(uint32_t tmem_row, uint32_t s_col, const volatile uint32_t* rec, const RowState& st,
                                          bool tree, bool lists, float c, bool negate, int part, bool first, float& m, float& l,
                                          uint64_t* pv_done, int prev, volatile int* abort_flag, int32_t* status, uint32_t polls) {
  constexpr int kCols = kTile / F;
  const uint32_t flags = rec[kRFlags];
  const int kind = (flags >> kKindShift) & 3;
  uint32_t v[kCols / 32][32];
#pragma unroll
  for (int k = 0; k < kCols / 32; ++k) tmem_ld32(tmem_row + s_col + (uint32_t)(part * kCols + 32 * k), v[k]);
  tmem_wait_ld();
  if (negate) {
#pragma unroll
    for (int k = 0; k < kCols / 32; ++k)
#pragma unroll
      for (int e = 0; e < 32; ++e) v[k][e] ^= 0x80000000u;
  }
  if (kind == kRowMask) {
    if (!((rec[kRMask] >> st.token) & 1u)) {
#pragma unroll
      for (int k = 0; k < kCols / 32; ++k)
#pragma unroll
        for (int e = 0; e < 32; ++e) v[k][e] = 0xFF800000u;
    }
  } else if (kind == kGeneral) {
#pragma unroll
    for (int k = 0; k < kCols / 32; ++k) {
      const int g = part * (kCols / kGroup) + 2 * k;
      const uint32_t bits = group_bits((int)rec[kRPos + g], rec[kRMask + g], st, tree, lists) |
                            group_bits((int)rec[kRPos + g + 1], rec[kRMask + g + 1], st, tree, lists) << 16;
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (!((bits >> e) & 1u)) v[k][e] = 0xFF800000u;
    }
  }
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int k = 0; k < kCols / 32; ++k)
#pragma unroll
    for (int e = 0; e < 32; ++e) top[e & 3] = fmaxf(top[e & 3], __uint_as_float(v[k][e]));
  const float big = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));

  // O is complete up to the tile before, and its weights are free
  bool ok = true;
  if (prev >= 0) ok = timed_wait_flag(pv_done, (uint32_t)prev & 1u, abort_flag, status, polls);
  if (!__all_sync(0xFFFFFFFFu, ok)) return false;
  tc_fence_after();
  float scale = 1.f;
  if (big > m && (m == -INFINITY || (big - m) * c > kRescale)) {
    scale = m == -INFINITY ? 1.f : ex2((m - big) * c);  // with no score so far O and l are zero
    m = big;
  }
  l *= scale;
  if (!first && __any_sync(0xFFFFFFFFu, scale != 1.f)) {
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      uint32_t o[32];
      tmem_ld32(tmem_row + kColO + 32 * k, o);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scale);
      tmem_st32(tmem_row + kColO + 32 * k, o);
    }
  }
  if (F > 1 && first) {
    // the other copies' parts of the weights are zero throughout the segment
    const uint32_t zero[16] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) tmem_st16(tmem_row + kColP + 16 * k, zero);
  }
  const float mc = m == -INFINITY ? 0.f : m * c;
  float sum[4] = {};
#pragma unroll
  for (int k = 0; k < kCols / 32; ++k) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float x = ex2(fmaf(__uint_as_float(v[k][e]), c, -mc)), y = ex2(fmaf(__uint_as_float(v[k][e + 1]), c, -mc));
      sum[(e >> 1) & 3] += x + y;
      w[e >> 1] = Num<T>::pack(x, y);
    }
    tmem_st16(tmem_row + kColP + (uint32_t)(part * (kCols / 2) + 16 * k), w);
  }
  l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  return true;
}

// A row whose O is not finite although its scores are: some value that it
// does not see (or whose weight is zero) is an infinity or NaN.  The warp
// forms the row's O again, place by place, from what the row sees alone.
template <typename T, int D>
__device__ __noinline__ void row_again(const TreeArgs& a, const volatile uint32_t* rec, int row, const RowState st, float m, float c,
                                       int col0, int col1, float* dst) {
  const int lane = (int)lane_id();
  constexpr int kE = D / 32;
  const int t = (int)rec[kRTok0] + st.token, kvh = (int)rec[kRHead], r = (int)rec[kRReq];
  const int h = kvh * a.group + row % a.group;
  const bool tree = a.mask != nullptr, lists = a.pages != nullptr;
  const float cs = a.scale < 0.f ? -c : c;
  float q[kE], o[kE];
  const T* qp = static_cast<const T*>(a.q) + (int64_t)t * a.q_ts + (int64_t)h * a.q_hs + lane * kE;
#pragma unroll
  for (int e = 0; e < kE; ++e) q[e] = (float)qp[e], o[e] = 0.f;
  const int64_t list = (int64_t)rec[kRList];
  const int lh = lists ? kvh / (a.kv_heads / a.lists) : 0;
  const int count = lists ? min(a.counts[(int64_t)rec[kRTok0] * a.lists + lh], (int)rec[kRTokens] * a.per) : 0;
  for (int tile = (int)rec[kRFirst]; tile < (int)rec[kREnd]; ++tile)
    for (int col = col0; col < col1; ++col) {
      int64_t place = (int64_t)tile * kTile + col, blk = -1;
      uint32_t tokens = 0xFFFFFFFFu;
      if (lists) {
        const int64_t e = place / a.page;
        if (e >= count) continue;
        const ListEntry en = a.entries[list + e];
        blk = en.block, tokens = en.tokens;
        place = (int64_t)en.page * a.page + place % a.page;
      } else if (place < st.len) {
        blk = a.bt[r * a.bt_stride + place / a.page];
      }
      if (blk < 0 || blk >= a.num_blocks || place >= st.len) continue;
      const int pos = (int)(place / kGroup * kGroup);
      if (!((group_bits(pos, tokens, st, tree, lists) >> (int)(place - pos)) & 1u)) continue;
      const int64_t at = blk * a.c_bs + place % a.page * a.c_ts + (int64_t)kvh * a.c_hs + lane * kE;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) s = fmaf(q[e], (float)static_cast<const T*>(a.kc)[at + e], s);
#pragma unroll
      for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
      const float p = ex2(s * cs - m * c);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float vv = (float)static_cast<const T*>(a.vc)[at + e];
        // a weight below the smallest number still carries an infinity's sign
        o[e] = fmaf(p == 0.f && isinf(vv) ? 1.f : p, vv, o[e]);
      }
    }
#pragma unroll
  for (int e = 0; e < kE; ++e) dst[lane * kE + e] = o[e];
  __syncwarp();
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsA, 1)
    k_tree_attention(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeArgs a) {
  using S = Smem<D>;
  pdl_enter();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  MiscA* misc = reinterpret_cast<MiscA*>(smem + S::kOffMisc);
  uint32_t* recs = reinterpret_cast<uint32_t*>(smem + S::kOffRec);
  volatile int* abort_flag = &misc->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Plan plan(a);
  const bool lists = a.pages != nullptr, tree = a.mask != nullptr;

  if (tid == 0) {
    misc->total = 0;
    misc->abort_flag = 0;
    for (int s = 0; s < kStagesA; ++s) {
      mbar_init(&bars[kKvFull + s], 1);
      mbar_init(&bars[kKvEmpty + s], 1);
    }
    mbar_init(&bars[kQFullA], 1);
    mbar_init(&bars[kQEmptyA], 1);
    mbar_init(&bars[kSFull], 1);
    mbar_init(&bars[kSFull + 1], 1);
    mbar_init(&bars[kPFull], kSoftWarps);
    mbar_init(&bars[kPvDone], 1);
    mbar_init(&bars[kOEmpty], kSoftWarps);
    mbar_init(&bars[kMerge], kSoftWarps);
    for (int s = 0; s < kRecs; ++s) mbar_init(&bars[kRecFull + s], 1);
    mbar_init(&bars[kDrainA], 1);
    fence_mbar_init();
  }
  __syncthreads();
  {
    unsigned long long local = 0;
    for (int r = tid; r < a.num_reqs; r += kThreadsA) local += plan.units(r);
    local = warp_sum_u64(local);
    if (lane == 0 && local) atomicAdd(&misc->total, local);
  }
  if (warp == 0) tmem_alloc(&misc->tmem_base, kTmemColsA);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem_base;
  const unsigned long long W = misc->total;
  const unsigned long long w0 = W * blockIdx.x / gridDim.x, w1 = W * (blockIdx.x + 1) / gridDim.x;
  const int count = (int)(w1 - w0);

  if (warp == kTmaWarp && count > 0) {
    // the request of the stretch's first unit
    unsigned long long acc = 0;
    int r = 0;
    unsigned long long rem = 0;
    for (int base = 0; base < a.num_reqs; base += 32) {
      const unsigned long long n = base + lane < a.num_reqs ? plan.units(base + lane) : 0ull;
      unsigned long long incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned long long excl = acc + incl - n;
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, n > 0 && excl <= w0 && w0 < excl + n);
      if (hit) {
        const int who = __ffs(hit) - 1;
        r = base + who;
        rem = w0 - __shfl_sync(0xFFFFFFFFu, excl, who);
        break;
      }
      acc += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    // and its block, head and tile; all lanes hold the same cursor
    int n = plan.ntok(r), t0 = plan.tok0(r), s = plan.seq(r), b = 0, kvh = 0;
    const int per_list = lists ? a.kv_heads / a.lists : a.kv_heads;
    int tiles = plan.tiles(s, n, t0, 0, 0);
    while (rem >= (unsigned)tiles) {
      rem -= (unsigned)tiles;
      if (++kvh == a.kv_heads) kvh = 0, ++b;
      tiles = plan.tiles(s, n, t0, b, kvh / per_list);
    }
    int tile = (int)rem;
    if (lane == 0) {
      // where this stretch begins inside a segment, the segment's units
      int32_t* cut = a.cuts + 8 * blockIdx.x;
      const unsigned long long u0 = w0 - rem, u1 = u0 + tiles;
      cut[0] = rem > 0 ? 1 : 0;
      cut[1] = t0 + b * a.block_tokens;
      cut[2] = min(a.block_tokens, n - b * a.block_tokens);
      cut[3] = kvh;
      reinterpret_cast<unsigned long long*>(cut)[2] = u0;
      reinterpret_cast<unsigned long long*>(cut)[3] = u1;
    }

    const int bs = min(a.page, kTile), boxes = kTile / bs;  // places of a box, boxes of a tile
    const uint32_t tile_bytes = (uint32_t)S::kKv;
    int i = 0, seg = 0, piece_first = tile, items = 0, queries = 0;  // items, queries: copies issued
    bool ok = true, bad_block = false;
    bool fresh = true;  // the queries of the segment are still to load
    // Block ids of the next 32 boxes, loaded together by the lanes.
    int box_base = 0, ids = -1, id_page = 0;
    uint32_t id_tokens = 0;
    while (i < count) {
      const int len = plan.len(s), ctx = s - n;
      const int m = min(a.block_tokens, n - b * a.block_tokens), tok = t0 + b * a.block_tokens;
      const int rows = m * a.group;
      const int fold = rows <= kRowsA / 4 ? 4 : rows <= kRowsA / 2 ? 2 : 1;
      const int lh = lists ? kvh / per_list : 0;
      const int64_t list = ((int64_t)tok * a.lists + (int64_t)lh * m) * a.per;
      const int entries = lists ? min(a.counts[(int64_t)tok * a.lists + lh], m * a.per) : 0;
      const int piece_end = min(tiles, tile + (count - i));
      if (fresh) {
        if (seg > 0) ok = timed_wait_flag(&bars[kQEmptyA], (uint32_t)(seg - 1) & 1u, abort_flag, a.status, a.polls);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        const int loads = m * fold * (D / 64);
        if (lane == 0) mbar_arrive_expect_tx(&bars[kQFullA], (uint32_t)(loads * a.group * 128));
        ++queries;
        __syncwarp();
        for (int k = lane; k < loads; k += 32) {
          const int sub = k % (D / 64), tk = k / (D / 64) % m, copy = k / (D / 64) / m;
          tma_load_3d(smem + S::kOffQ + sub * (kRowsA * 128) + (copy * (kRowsA / fold) + tk * a.group) * 128, &qmap, sub * 64,
                      kvh * a.group, tok + tk, &bars[kQFullA]);
        }
        fresh = false;
        piece_first = tile;
        box_base = -1;
      }
      const int first_box = tile * boxes;
      if (box_base < 0 || first_box >= box_base + 32) {
        box_base = first_box;
        const int64_t p = (int64_t)(box_base + lane) * bs;  // in the order of the list's or the table's places
        ids = -1;
        if (lists) {
          const int64_t e = p / a.page;
          if (e < entries) {
            const ListEntry en = a.entries[list + e];
            ids = en.block, id_page = en.page, id_tokens = en.tokens;
          }
        } else if (p < len) {
          id_page = (int)(p / a.page);
          const int blk = a.bt[r * a.bt_stride + id_page];
          if (blk >= 0 && blk < a.num_blocks) ids = blk;
          else bad_block = true;
        }
      }
      // this lane's box and group of the tile
      const int my_box = first_box - box_base + lane % boxes, my_grp_box = first_box - box_base + (lane % 8) * kGroup / bs;
      const int box_id = __shfl_sync(0xFFFFFFFFu, ids, my_box);
      const int grp_id = __shfl_sync(0xFFFFFFFFu, ids, my_grp_box), grp_page = __shfl_sync(0xFFFFFFFFu, id_page, my_grp_box);
      const uint32_t grp_tokens = lists ? __shfl_sync(0xFFFFFFFFu, id_tokens, my_grp_box) : 0xFFFFFFFFu;
      const int in_order = (int)(((int64_t)tile * kTile) % a.page);  // offset of a whole-page tile within its page
      const int off = bs < kTile ? ((lane % 8) * kGroup) % bs : in_order + (lane % 8) * kGroup;
      const int pos = grp_id < 0 ? -1 : grp_page * a.page + off;
      const uint32_t every = m >= 32 ? 0xFFFFFFFFu : (1u << m) - 1u;
      const bool cached = pos >= 0 && pos + kGroup <= ctx && pos + kGroup <= len;
      const bool all_cached = __all_sync(0xFFFFFFFFu, cached);
      const bool all_tokens = !lists || __all_sync(0xFFFFFFFFu, (grp_tokens & every) == every);
      const int kind = all_cached && all_tokens ? kFull : all_cached && boxes == 1 ? kRowMask : kGeneral;
      const bool last = tile + 1 == piece_end;
      uint32_t word = 0;
      const int fold_code = fold == 4 ? 2 : fold == 2 ? 1 : 0;
      // partial results: slot 2x for the first segment of stretch x, 2x + 1 for the last; -1: the whole segment is here
      const bool whole = piece_first == 0 && piece_end == tiles;
      switch (lane) {
        case kRFlags:
          word = (uint32_t)((tile == piece_first ? kFlagFirst : 0) | (last ? kFlagLast : 0) | (kind << kKindShift) |
                            (fold_code << kFoldShift));
          break;
        case kRTok0: word = (uint32_t)tok; break;
        case kRTokens: word = (uint32_t)m; break;
        case kRHead: word = (uint32_t)kvh; break;
        case kRCtx: word = (uint32_t)ctx; break;
        case kRNew: word = (uint32_t)n; break;
        case kRNode0: word = (uint32_t)(b * a.block_tokens); break;
        case kRLen: word = (uint32_t)len; break;
        case kROut: word = whole ? 0xFFFFFFFFu : (uint32_t)(2 * blockIdx.x + (seg > 0 ? 1 : 0)); break;
        case kRReq: word = (uint32_t)r; break;
        case kRFirst: word = (uint32_t)piece_first; break;
        case kREnd: word = (uint32_t)piece_end; break;
        case kRList: word = (uint32_t)list; break;
        default: break;
      }
      {
        const int g = lane >= kRMask ? lane - kRMask : lane - kRPos;
        const uint32_t p = __shfl_sync(0xFFFFFFFFu, (uint32_t)pos, g & 7), k = __shfl_sync(0xFFFFFFFFu, grp_tokens, g & 7);
        if (lane >= kRPos && lane < kRMask) word = p;
        if (lane >= kRMask && lane < kROut) word = k;
      }
      // the record's slot was read at tile i - kRecs, whose value stage is free since tile i - 3
      for (int half = 0; half < 2; ++half) {
        const int item = 2 * i + half, stage = item % kStagesA;
        if (ok) ok = timed_wait_flag(&bars[kKvEmpty + stage], ((uint32_t)(item / kStagesA) & 1u) ^ 1u, abort_flag, a.status, a.polls);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ok = false;
          break;
        }
        if (half == 0) {
          recs[(i % kRecs) * kRecWords + lane] = word;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kRecFull + i % kRecs]);
        }
        if (lane == 0) mbar_arrive_expect_tx(&bars[kKvFull + stage], tile_bytes);
        items = item + 1;
        __syncwarp();
        if (lane < boxes * (D / 64)) {
          const int bx = lane % boxes, sub = lane / boxes;
          const int c2 = boxes == 1 ? in_order : 0;
          // a block outside the pool reads as zeros
          tma_load_4d(smem + S::kOffKv + stage * S::kKv + sub * (kTile * 128) + bx * bs * 128, half == 0 ? &kmap : &vmap, sub * 64,
                      kvh, c2, box_id < 0 ? (int)a.num_blocks : box_id, &bars[kKvFull + stage]);
        }
      }
      if (!ok) break;
      ++i;
      if (++tile == tiles) {
        // next segment
        tile = 0;
        ++seg;
        fresh = true;
        if (++kvh == a.kv_heads) {
          kvh = 0;
          if (++b >= plan.blocks(n)) {
            b = 0;
            do {
              ++r;
              n = r < a.num_reqs ? plan.ntok(r) : 0;
            } while (r < a.num_reqs && n == 0);
            if (r < a.num_reqs) t0 = plan.tok0(r), s = plan.seq(r);
          }
        }
        if (i < count) tiles = plan.tiles(s, n, t0, b, kvh / per_list);
      }
    }
    if (bad_block) report(a.status, IDX_ST_BLOCK_OOR);
    // never leave with a copy in flight
    if (lane == 0) {
      for (int k = max(0, items - kStagesA); k < items; ++k)
        mbar_wait(&bars[kKvFull + k % kStagesA], (uint32_t)(k / kStagesA) & 1u, nullptr);
      if (queries > 0) mbar_wait(&bars[kQFullA], (uint32_t)(queries - 1) & 1u, nullptr);
    }
  } else if (warp == kMmaWarpA && count > 0) {
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_16(Num<T>::kBf16, kRowsA, kTile, false);
      constexpr uint32_t kIdO = idesc_16(Num<T>::kBf16, kRowsA, D, true);
      int seg = 0, done_seg = 0;
      bool ok = true, issued = false;
      uint32_t prev_flags = 0;
      for (int i = 0; i <= count && ok; ++i) {
        uint32_t flags = 0;
        if (i < count) {
          const int item = 2 * i, stage = item % kStagesA;
          ok = spin_wait_flag(&bars[kKvFull + stage], (uint32_t)(item / kStagesA) & 1u, abort_flag, a.status, a.polls);
          if (!ok) break;
          flags = *reinterpret_cast<volatile uint32_t*>(recs + (i % kRecs) * kRecWords);
          if (flags & kFlagFirst) {
            ok = spin_wait_flag(&bars[kQFullA], (uint32_t)seg & 1u, abort_flag, a.status, a.polls);
            if (!ok) break;
          }
          tc_fence_after();
          const uint64_t qd = sw128_desc(sbase + S::kOffQ), kd = sw128_desc(sbase + S::kOffKv + stage * S::kKv);
          const uint32_t d = tmem + kColS + (uint32_t)(i & 1) * kTile;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t step = (uint64_t)((k / 4) * (kRowsA * 128 / 16) + (k % 4) * 2);
            mma_16(d, qd + step, kd + step, kIdS, k > 0 ? 1u : 0u);
          }
          mma_commit(&bars[kSFull + (i & 1)]);
          mma_commit(&bars[kKvEmpty + stage]);
          if (flags & kFlagLast) {
            mma_commit(&bars[kQEmptyA]);
            ++seg;
          }
          issued = true;
        }
        if (i > 0) {
          const int item = 2 * (i - 1) + 1, stage = item % kStagesA;
          ok = spin_wait_flag(&bars[kKvFull + stage], (uint32_t)(item / kStagesA) & 1u, abort_flag, a.status, a.polls) &&
               spin_wait_flag(&bars[kPFull], (uint32_t)(i - 1) & 1u, abort_flag, a.status, a.polls);
          if (!ok) break;
          if ((prev_flags & kFlagFirst) && done_seg > 0) {
            ok = spin_wait_flag(&bars[kOEmpty], (uint32_t)(done_seg - 1) & 1u, abort_flag, a.status, a.polls);
            if (!ok) break;
          }
          tc_fence_after();
          const uint64_t vd = sw128_desc_nmajor(sbase + S::kOffKv + stage * S::kKv);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_16_ta(tmem + kColO, tmem + kColP + 8 * k, vd + (uint64_t)(k * (2048 / 16)), kIdO,
                      k > 0 || !(prev_flags & kFlagFirst) ? 1u : 0u);
          mma_commit(&bars[kPvDone]);
          mma_commit(&bars[kKvEmpty + stage]);
          if (prev_flags & kFlagLast) ++done_seg;
        }
        prev_flags = flags;
      }
      if (issued) {
        mma_commit(&bars[kDrainA]);
        mbar_wait(&bars[kDrainA], 0, nullptr);
      }
    }
  } else if (warp < kSoftWarps) {
    const uint32_t tmem_row = tmem + ((uint32_t)(warp * 32) << 16);
    float* scratch = reinterpret_cast<float*>(smem + S::kOffScratch);
    float2* stats = reinterpret_cast<float2*>(smem + S::kOffStats);
    const bool negate = a.scale < 0.f;
    // scores in powers of two; a scale of 0 becomes one that still hides masked places
    const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
    float m = -INFINITY, l = 0.f;
    RowState st{};
    uint32_t merges = 0;
    int row = 0, part = 0, fold = 1;
    auto meet = [&]() {  // the four warps
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kMerge]);
      const bool ok = timed_wait_flag(&bars[kMerge], merges & 1u, abort_flag, a.status, a.polls);
      ++merges;
      return __all_sync(0xFFFFFFFFu, ok) != 0;
    };
    for (int i = 0; i < count; ++i) {
      bool ok_r, ok_s;
      mbar_test2(&bars[kRecFull + i % kRecs], (uint32_t)(i / kRecs) & 1u, &bars[kSFull + (i & 1)], (uint32_t)(i >> 1) & 1u, ok_r, ok_s);
      if (!ok_r) ok_r = timed_wait_flag(&bars[kRecFull + i % kRecs], (uint32_t)(i / kRecs) & 1u, abort_flag, a.status, a.polls);
      if (!__all_sync(0xFFFFFFFFu, ok_r)) break;
      const volatile uint32_t* rec = recs + (i % kRecs) * kRecWords;
      const uint32_t flags = rec[kRFlags];
      const bool first = (flags & kFlagFirst) != 0;
      if (first) {
        fold = 1 << ((flags >> kFoldShift) & 3);
        row = tid & (kRowsA / fold - 1), part = tid / (kRowsA / fold);
        m = -INFINITY, l = 0.f;
        st.token = min(row / a.group, (int)rec[kRTokens] - 1);  // rows past the block's compute on the last token's mask
        st.ctx = (int)rec[kRCtx], st.len = (int)rec[kRLen];
        const int n = (int)rec[kRNew];
        st.chain_end = st.ctx + (int)rec[kRNode0] + st.token + 1;
        st.tree = tree ? a.mask[(int)rec[kRTok0] + st.token] & (n >= 64 ? ~0ull : (1ull << n) - 1ull) : 0ull;
      }
      if (!ok_s) ok_s = timed_wait_flag(&bars[kSFull + (i & 1)], (uint32_t)(i >> 1) & 1u, abort_flag, a.status, a.polls);
      if (!__all_sync(0xFFFFFFFFu, ok_s)) break;
      tc_fence_after();
      const uint32_t s_col = kColS + (uint32_t)(i & 1) * kTile;
      bool ok;
      if (fold == 4)
        ok = soft_tile<T, D, 4>(tmem_row, s_col, rec, st, tree, lists, c, negate, part, first, m, l, &bars[kPvDone], i - 1, abort_flag,
                                a.status, a.polls);
      else if (fold == 2)
        ok = soft_tile<T, D, 2>(tmem_row, s_col, rec, st, tree, lists, c, negate, part, first, m, l, &bars[kPvDone], i - 1, abort_flag,
                                a.status, a.polls);
      else
        ok = soft_tile<T, D, 1>(tmem_row, s_col, rec, st, tree, lists, c, negate, part, first, m, l, &bars[kPvDone], i - 1, abort_flag,
                                a.status, a.polls);
      if (!ok) break;
      if (((flags >> kKindShift) & 3) == kGeneral) {
        // values at places that do not exist may be anything: zeros in their stead
        const int pos = (int)rec[kRPos + tid / kGroup];
        if (pos >= 0 && pos + tid % kGroup >= st.len) {
          const int item = 2 * i + 1, stage = item % kStagesA;
          ok = timed_wait_flag(&bars[kKvFull + stage], (uint32_t)(item / kStagesA) & 1u, abort_flag, a.status, a.polls);
          if (ok) {
            uint4* vrow = reinterpret_cast<uint4*>(smem + S::kOffKv + stage * S::kKv + tid * 128);
#pragma unroll
            for (int sub = 0; sub < D / 64; ++sub)
#pragma unroll
              for (int e = 0; e < 8; ++e) vrow[sub * (kTile * 128 / 16) + e] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kPFull]);
      if (!(flags & kFlagLast)) continue;

      // the segment's rows
      ok = timed_wait_flag(&bars[kPvDone], (uint32_t)i & 1u, abort_flag, a.status, a.polls);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc_fence_after();
      const int rows = (int)rec[kRTokens] * a.group;
      const bool live = row < rows;
      {
        float probe = 0.f;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[32];
          tmem_ld32(tmem_row + kColO + 32 * k, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) probe = fmaf(__uint_as_float(o[e]), 0.f, probe);
        }
        uint32_t again = __ballot_sync(0xFFFFFFFFu, live && l > 0.f && l < INFINITY && probe != 0.f);
        while (again) {
          const int who = __ffs(again) - 1;
          again &= again - 1;
          RowState w;
          w.tree = __shfl_sync(0xFFFFFFFFu, st.tree, who);
          w.ctx = st.ctx, w.len = st.len;
          w.chain_end = __shfl_sync(0xFFFFFFFFu, st.chain_end, who);
          w.token = __shfl_sync(0xFFFFFFFFu, st.token, who);
          float* dst = scratch + warp * 32 * S::kScratchRow;
          row_again<T, D>(a, rec, __shfl_sync(0xFFFFFFFFu, row, who), w, __shfl_sync(0xFFFFFFFFu, m, who), c,
                          __shfl_sync(0xFFFFFFFFu, part, who) * (kTile / fold),
                          (__shfl_sync(0xFFFFFFFFu, part, who) + 1) * (kTile / fold), dst);
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            uint32_t o[32];
            tmem_ld32(tmem_row + kColO + 32 * k, o);
            tmem_wait_ld();
            if (lane == who)
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(dst[32 * k + e]);
            tmem_st32(tmem_row + kColO + 32 * k, o);
            tmem_wait_st();
          }
          __syncwarp();
        }
      }
      float big = m, factor = 1.f, whole_l = l;
      if (fold > 1) {
        stats[tid] = make_float2(m, l);
        if (!meet()) break;
        whole_l = 0.f;
        for (int p = 0; p < fold; ++p) big = fmaxf(big, stats[p * (kRowsA / fold) + row].x);
        for (int p = 0; p < fold; ++p) {
          const float2 x = stats[p * (kRowsA / fold) + row];
          if (x.x != -INFINITY) whole_l += x.y * ex2((x.x - big) * c);
        }
        factor = m == -INFINITY ? 0.f : ex2((m - big) * c);
      }
      const uint32_t slot = rec[kROut];
      const int t = (int)rec[kRTok0] + st.token, h = (int)rec[kRHead] * a.group + row % a.group;
      const bool direct = slot == 0xFFFFFFFFu;
      const bool empty = whole_l == 0.f;
      const float inv = direct ? (empty ? 0.f : 1.f / whole_l) : 1.f;
      if (live && part == 0) {
        if (direct) {
          if (a.lse != nullptr) a.lse[(int64_t)t * a.q_heads + h] = empty ? -INFINITY : (big * c + log2f(whole_l)) * 0.6931471805599453f;
        } else {
          reinterpret_cast<float2*>(a.part_ml)[(int64_t)slot * kRowsA + row] = make_float2(empty ? -INFINITY : big * c, whole_l);
        }
      }
      T* out = static_cast<T*>(a.out) + (int64_t)t * a.o_ts + (int64_t)h * a.o_hs;
      float* part_o = a.part_o + ((int64_t)(direct ? 0 : slot) * kRowsA + row) * D;
      bool alive = true;
#pragma unroll 1
      for (int k = 0; k < D / 32; ++k) {
        uint32_t o[32];
        tmem_ld32(tmem_row + kColO + 32 * k, o);
        tmem_wait_ld();
        const int width = 32 / fold;  // columns that this thread writes
        float f[32];
        if (fold == 1) {
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = empty ? 0.f : __uint_as_float(o[e]) * inv;
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) scratch[tid * S::kScratchRow + e] = factor == 0.f ? 0.f : __uint_as_float(o[e]) * factor;
          if (!meet()) {
            alive = false;
            break;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (e < width) {
              float sum = 0.f;
              for (int p = 0; p < fold; ++p) sum += scratch[(p * (kRowsA / fold) + row) * S::kScratchRow + part * width + e];
              f[e] = empty ? 0.f : sum * inv;
            }
        }
        if (live) {
          const int col = 32 * k + (fold == 1 ? 0 : part * width);
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            if (e < width) {
              if (direct) {
                *reinterpret_cast<uint4*>(out + col + e) =
                    make_uint4(Num<T>::pack(f[e], f[e + 1]), Num<T>::pack(f[e + 2], f[e + 3]), Num<T>::pack(f[e + 4], f[e + 5]),
                               Num<T>::pack(f[e + 6], f[e + 7]));
              } else {
                reinterpret_cast<float4*>(part_o + col + e)[0] = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
                reinterpret_cast<float4*>(part_o + col + e)[1] = make_float4(f[e + 4], f[e + 5], f[e + 6], f[e + 7]);
              }
            }
        }
        if (fold > 1 && !meet()) {
          alive = false;
          break;
        }
      }
      if (!alive) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kOEmpty]);
    }
  }

  if (tid == 0) {
    if (count == 0) a.cuts[8 * blockIdx.x] = 0;
    if (blockIdx.x == 0) *reinterpret_cast<unsigned long long*>(a.cuts + 8 * kMaxCtas) = W;
  }
  __syncthreads();
  // lengths that the table does not hold
  if (blockIdx.x == 0)
    for (int r = tid; r < a.num_reqs; r += kThreadsA)
      if (plan.ntok(r) > 0 && plan.len(plan.seq(r)) < plan.seq(r)) report(a.status, IDX_ST_LEN_CLAMPED);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemColsA);
  }
}

// Joins the partial rows of the segments that the stretches cut.  Block x
// acts where stretch x + 1 begins inside a segment that the stretch before it
// began; a warp joins a row: the largest reference maximum, then the weighted
// sums.
constexpr int kJoinWarps = 8;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) k_tree_combine(const __grid_constant__ TreeArgs a, int ctas) {
  pdl_enter();
  __shared__ float weight[kJoinWarps][kMaxCtas];
  using u64 = unsigned long long;
  const int x = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t* cut = a.cuts + 8 * x;
  if (cut[0] == 0) return;
  const u64 W = *reinterpret_cast<const u64*>(a.cuts + 8 * kMaxCtas);
  const u64 u0 = reinterpret_cast<const u64*>(cut)[2], u1 = reinterpret_cast<const u64*>(cut)[3];
  auto start = [&](int y) { return W * (u64)y / (u64)ctas; };
  auto cta_of = [&](u64 u) { return (int)(((u + 1) * (u64)ctas - 1) / W); };
  const int from = cta_of(start(x) - 1), to = cta_of(u1 - 1);
  if (start(from) > u0) return;  // an earlier block joins this segment
  const int row = blockIdx.y * kJoinWarps + warp, rows = cut[2] * a.group;
  if (row >= rows) return;
  // slot 2y, but 2y + 1 where the segment is not its stretch's first
  const int first_slot = 2 * from + (u0 > start(from) ? 1 : 0);
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
  float big = -INFINITY;
  for (int y = from + lane; y <= to; y += 32)
    if (start(y) < start(y + 1)) big = fmaxf(big, ml[(int64_t)(y == from ? first_slot : 2 * y) * kRowsA + row].x);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
  float sum = 0.f;
  for (int y = from + lane; y <= to; y += 32) {
    float w = 0.f;
    if (start(y) < start(y + 1)) {
      const float2 p = ml[(int64_t)(y == from ? first_slot : 2 * y) * kRowsA + row];
      if (p.x != -INFINITY) w = ex2(p.x - big), sum += w * p.y;
    }
    weight[warp][y - from] = w;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  __syncwarp();
  constexpr int kE = D / 32;
  float acc[kE] = {};
#pragma unroll 4
  for (int y = from; y <= to; ++y) {
    const float w = weight[warp][y - from];
    if (w == 0.f) continue;
    const float* o = a.part_o + ((int64_t)(y == from ? first_slot : 2 * y) * kRowsA + row) * D + lane * kE;
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] = fmaf(w, o[e], acc[e]);
  }
  const int t = cut[1] + row / a.group, h = cut[3] * a.group + row % a.group;
  const bool empty = sum == 0.f;
  const float inv = empty ? 0.f : 1.f / sum;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + (int64_t)t * a.o_ts + (int64_t)h * a.o_hs + lane * kE);
#pragma unroll
  for (int e = 0; e < kE; e += 2) out[e / 2] = empty ? 0u : Num<T>::pack(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && a.lse != nullptr) a.lse[(int64_t)t * a.q_heads + h] = empty ? -INFINITY : (big + log2f(sum)) * 0.6931471805599453f;
}

// The union of a block's page lists.  One CTA per (token, list) looks whether
// the token begins a block, gathers the lists of the block's tokens, and keeps
// of each page its first appearance with the tokens that list it.
constexpr int kUnionThreads = 128;
__global__ void __launch_bounds__(kUnionThreads) k_list_pages(const __grid_constant__ TreeArgs a) {
  pdl_enter();
  __shared__ int page_s[kMaxListTokens * 64];
  __shared__ int kept, warp_kept[kUnionThreads / 32];
  const int t = blockIdx.x, lh = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const Plan plan(a);
  // the request: the last one whose tokens begin at or before t (a probe of 32 places a step)
  int lo = 0, hi = a.num_reqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const uint32_t ok = __ballot_sync(0xFFFFFFFFu, at < hi && plan.tok0(at) <= t);
    const int k = 31 - __clz(ok | 1u);
    const int nlo = lo + k * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  const int r = lo, t0 = plan.tok0(r), n = plan.ntok(r), node = t - t0;
  if (node < 0 || node >= n || node % a.block_tokens != 0) return;
  const int m = min(a.block_tokens, n - node), total = m * a.per;
  const int len = plan.len(plan.seq(r)), used = (int)(((int64_t)len + a.page - 1) / a.page);
  for (int e = tid; e < total; e += kUnionThreads) {
    const int p = a.pages[((int64_t)(t + e / a.per) * a.lists + lh) * a.per + e % a.per];
    page_s[e] = p >= 0 && p < used ? p : -1;
  }
  if (tid == 0) kept = 0;
  __syncthreads();
  ListEntry* out = a.entries + ((int64_t)t * a.lists + (int64_t)lh * m) * a.per;
  bool bad = false;
  for (int base = 0; base < total; base += kUnionThreads) {
    const int e = base + tid;
    const int p = e < total ? page_s[e] : -1;
    uint32_t tokens = 0;
    bool take = p >= 0;
    int blk = -1;
    if (take) {
      blk = a.bt[r * a.bt_stride + p];
      for (int f = 0; f < total; ++f)
        if (page_s[f] == p) {
          if (f < e) take = false;
          tokens |= 1u << (f / a.per);
        }
      if (blk < 0 || blk >= a.num_blocks) bad = true, take = false;
    }
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, take);
    if (lane == 0) warp_kept[tid >> 5] = __popc(b);
    __syncthreads();
    int at = kept;
    for (int w = 0; w < tid >> 5; ++w) at += warp_kept[w];
    if (take) out[at + __popc(b & ((1u << lane) - 1u))] = ListEntry{blk, p, tokens, 0};
    __syncthreads();
    if (tid == 0)
      for (int w = 0; w < kUnionThreads / 32; ++w) kept += warp_kept[w];
    __syncthreads();
  }
  if (tid == 0) a.counts[(int64_t)t * a.lists + lh] = kept;
  if (bad) report(a.status, IDX_ST_BLOCK_OOR);
}

// Workspace: cuts, partial maxima and sums, partial rows, then the lists.
struct Layout {
  size_t part_ml, part_o, counts, entries, bytes;
};
Layout layout_of(int32_t num_tokens, int32_t head_dim, int32_t lists, int32_t per) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Layout w{};
  size_t at = up((size_t)kMaxCtas * 32 + 32);
  w.part_ml = at, at += up((size_t)2 * kMaxCtas * kRowsA * 8);
  w.part_o = at, at += up((size_t)2 * kMaxCtas * kRowsA * head_dim * 4);
  w.counts = at, at += up((size_t)num_tokens * lists * 4);
  w.entries = at, at += up((size_t)num_tokens * lists * per * sizeof(ListEntry));
  w.bytes = at;
  return w;
}

template <typename T, int D>
int launch_tree(const TreeArgs& a, cudaStream_t s) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return IDX_E_CUDA;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(k_tree_attention<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes) != cudaSuccess ||
        cudaFuncSetAttribute(k_tree_attention<T, D>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             (int)cudaSharedmemCarveoutMaxShared) != cudaSuccess)
      return IDX_E_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  const int sms = device_sms();
  if (sms < 1) return IDX_E_CUDA;
  const int ctas = std::min(sms, kMaxCtas);
  // a dimension of one place has any stride
  auto bytes = [](int64_t stride, int64_t n) { return (cuuint64_t)(n > 1 ? stride * 2 : 16); };
  CUtensorMap qmap, kmap, vmap;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.q_heads, (cuuint64_t)a.num_tokens};
    const cuuint64_t strides[2] = {bytes(a.q_hs, a.q_heads), bytes(a.q_ts, a.num_tokens)};
    const cuuint32_t box[3] = {64u, (cuuint32_t)a.group, 1u};
    if (!encode_tensor_map(&qmap, Num<T>::kMap, 3, a.q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return IDX_E_BAD_SHAPE;
  }
  {
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)a.kv_heads, (cuuint64_t)a.page, (cuuint64_t)a.num_blocks};
    const cuuint64_t strides[3] = {bytes(a.c_hs, a.kv_heads), bytes(a.c_ts, a.page), bytes(a.c_bs, a.num_blocks)};
    const cuuint32_t box[4] = {64u, 1u, (cuuint32_t)std::min(a.page, kTile), 1u};
    if (!encode_tensor_map(&kmap, Num<T>::kMap, 4, a.kc, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tensor_map(&vmap, Num<T>::kMap, 4, a.vc, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return IDX_E_BAD_SHAPE;
  }
  if (a.pages != nullptr) {
    launch_pdl(k_list_pages, dim3((unsigned)a.num_tokens, (unsigned)a.lists), dim3(kUnionThreads), 0, s, a);
    if (const int rc = launch_result()) return rc;
  }
  launch_pdl(k_tree_attention<T, D>, dim3(ctas), dim3(kThreadsA), Smem<D>::kBytes, s, qmap, kmap, vmap, a);
  if (const int rc = launch_result()) return rc;
  if (ctas > 1) launch_pdl(k_tree_combine<T, D>, dim3(ctas - 1, kRowsA / kJoinWarps), dim3(kJoinWarps * 32), 0, s, a, ctas);
  return launch_result();
}

}  // namespace
}  // namespace idx

extern "C" size_t idx_tree_attention_workspace_bytes(int32_t num_reqs, int32_t num_tokens, int32_t q_heads,
                                                     int32_t kv_heads, int32_t head_dim, int32_t page_lists,
                                                     int32_t pages_per_list) {
  if (num_reqs <= 0 || num_tokens <= 0 || q_heads <= 0 || kv_heads <= 0 || head_dim <= 0 || page_lists < 0 || pages_per_list < 0)
    return 0;
  return idx::layout_of(num_tokens, head_dim, page_lists, pages_per_list).bytes;
}

extern "C" int idx_tree_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_cache,
                                  const void* v_cache, int64_t num_blocks, int32_t page_tokens, int64_t c_block_stride,
                                  int64_t c_token_stride, int64_t c_head_stride, const int32_t* block_table,
                                  int64_t bt_stride, int32_t max_blocks, const int32_t* seq_lens,
                                  const int32_t* cu_tokens, int32_t num_reqs, int32_t num_tokens, int32_t q_heads,
                                  int32_t kv_heads, int32_t head_dim, const uint64_t* tree_mask, const int32_t* pages,
                                  int32_t page_lists, int32_t pages_per_list, float scale, int32_t dtype, void* out,
                                  int64_t o_token_stride, int64_t o_head_stride, float* lse, void* workspace,
                                  size_t workspace_bytes, int32_t* status, void* stream) {
  using namespace idx;
  if (num_reqs < 0 || num_tokens < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || max_blocks < 0 ||
      num_blocks < 0 || bt_stride < max_blocks || !std::isfinite(scale))
    return IDX_E_BAD_SHAPE;
  if (head_dim != 64 && head_dim != 128) return IDX_E_BAD_SHAPE;
  if (page_tokens != 16 && page_tokens != 32 && page_tokens != 64 && (page_tokens < 128 || page_tokens % 128 != 0))
    return IDX_E_BAD_SHAPE;
  if (dtype != IDX_BF16 && dtype != IDX_F16) return IDX_E_BAD_SHAPE;
  if (pages != nullptr && (page_lists < 1 || kv_heads % page_lists != 0 || pages_per_list < 1)) return IDX_E_BAD_SHAPE;
  for (int64_t s : {q_token_stride, q_head_stride, c_block_stride, c_token_stride, c_head_stride, o_token_stride, o_head_stride})
    if (s < 0 || s % 8 != 0) return IDX_E_BAD_SHAPE;
  if ((q_heads > 1 && o_head_stride < head_dim) || (num_tokens > 1 && o_token_stride < head_dim)) return IDX_E_BAD_SHAPE;
  if (num_reqs > 65535 || q_heads / kv_heads > 128 || kv_heads > 65535 || num_blocks > 0x7FFFFFFF) return IDX_E_TOO_LARGE;
  if (pages != nullptr && (pages_per_list > 64 || page_lists > 65535 ||
                           (int64_t)num_tokens * page_lists * pages_per_list > 0x7FFFFFFF))
    return IDX_E_TOO_LARGE;
  if (num_tokens == 0 || num_reqs == 0) return num_tokens == 0 ? IDX_OK : IDX_E_BAD_SHAPE;
  if (!q || !out || !seq_lens || !cu_tokens) return IDX_E_NULL_PTR;
  if (!k_cache || !v_cache || (max_blocks > 0 && !block_table)) return IDX_E_NULL_PTR;
  if (num_blocks < 1) return IDX_E_BAD_SHAPE;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(cu_tokens, 4) || !aligned(tree_mask, 8) || !aligned(pages, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 256) || !aligned(status, 4))
    return IDX_E_MISALIGNED;
  const Layout w = layout_of(num_tokens, head_dim, pages ? page_lists : 0, pages ? pages_per_list : 0);
  if (workspace == nullptr || workspace_bytes < w.bytes) return IDX_E_WORKSPACE;
  int rc;
  if ((rc = check_device()) != IDX_OK) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  TreeArgs a{};
  a.q = q, a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.kc = k_cache, a.vc = v_cache;
  a.num_blocks = num_blocks, a.page = page_tokens, a.c_bs = c_block_stride, a.c_ts = c_token_stride, a.c_hs = c_head_stride;
  a.bt = block_table, a.bt_stride = bt_stride, a.max_blocks = max_blocks, a.seq_lens = seq_lens, a.cu = cu_tokens;
  a.num_reqs = num_reqs, a.num_tokens = num_tokens, a.q_heads = q_heads, a.kv_heads = kv_heads, a.group = q_heads / kv_heads;
  a.mask = tree_mask, a.pages = pages, a.lists = page_lists, a.per = pages_per_list, a.scale = scale;
  a.out = out, a.o_ts = o_token_stride, a.o_hs = o_head_stride, a.lse = lse, a.status = status;
  a.cuts = reinterpret_cast<int32_t*>(ws);
  a.part_ml = reinterpret_cast<float*>(ws + w.part_ml), a.part_o = reinterpret_cast<float*>(ws + w.part_o);
  a.counts = reinterpret_cast<int32_t*>(ws + w.counts), a.entries = reinterpret_cast<ListEntry*>(ws + w.entries);
  a.block_tokens = pages != nullptr ? std::min(kMaxListTokens, kRowsA / a.group) : kRowsA / a.group;
  a.polls = wait_polls();
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == IDX_BF16) return head_dim == 128 ? launch_tree<__nv_bfloat16, 128>(a, s) : launch_tree<__nv_bfloat16, 64>(a, s);
  return head_dim == 128 ? launch_tree<__half, 128>(a, s) : launch_tree<__half, 64>(a, s);
}
