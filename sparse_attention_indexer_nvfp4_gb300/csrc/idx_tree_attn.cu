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
// below 128 places).  All segments form one line of units, kSegCost for a
// segment's begin and end (~7,000 cycles against ~2,800 of a tile, of which
// some overlap) and one for each of its tiles; each of the
// persistent CTAs, one an SM, takes an equal stretch of it.  A segment cut by a
// stretch's end leaves partial (O, M, l) in the workspace, which
// k_tree_combine joins.
//
// Roles of a CTA (thirteen warps), which pass tiles on through mbarriers:
//   warps 0-7  a row's scores of a tile go to two threads, one in warps 0-3
//              for places 0-63 and one in warps 4-7 for places 64-127: scores
//              from TMEM, softmax, weights back into the scores' columns, and
//              at a segment's end the rows' results.  The two halves have
//              their own (O, M, l), so no tile needs them to meet;
//   warp 8     the plan: records of up to kChunk tiles at once, a lane a tile
//              (block ids, places, what is masked), kSlots chunks ahead;
//   warps 9-11 TMA: keys, values (a ring of tiles each), queries;
//   warp 12    MMA: S = Q K^T (both from shared memory), double buffered, so
//              tile i+1's scores form during tile i's softmax, and O += P V
//              (P in TMEM, V as it lies, places along K).  Its lanes test the
//              barriers, one each, and the first issues what is ready.
// An instruction of a warp that works alone takes 10-30 cycles, a barrier's
// test 200-300: with the plan made tile by tile by the warp that issues the
// copies, that warp set the pace (5,300 cycles a tile against the 2,800 that
// HBM needs; the softmax takes 1,400), hence the many small roles.
// With at most 64 (32) live rows the queries stand two (four) times in the
// 128 rows, and copy c of a row takes the softmax of the c-th part of each
// half tile, its weights for the others being zero: all warps share the work
// that otherwise a few would do, and the copies' (O, M, l) join at the end.
//
// The bound is HBM for up to ~128 rows a KV head (4 D flops a row and key
// against 4 D bytes a key: 128 flops a byte, below the ridge of ~280); beyond,
// each block of a request goes through its tiles again and a CTA's pace a tile,
// ~2,600 cycles with 128 live rows, is the bound (blocks taken side by side by
// neighbouring CTAs, so that the second read comes from L2: 163 us for 169 on 5
// requests of up to 61 tokens, but 58.6 for 55.7 on 64 tokens over 16,384
// places).  Measured with 64 query and 4 KV heads of 128 in bf16:
//     64 requests, 8 tokens each over 1,024 to 16,384 places   213 us, 5.9 TB/s
//     one request, 8 tokens over 500,000 places                168 us, 6.1 TB/s
//     64 requests, one token each over 8,192 places            177 us, 6.1 TB/s
//     one request, 64 tokens over 65,536 places                160 us, 859 TFLOP/s
//     one request, 2,048 tokens (a chain) after 16,384        1351 us, 865 TFLOP/s
//     64 requests, 8 tokens each, 16 of their pages a list     132 us
//     one request, one token over 1,000 places                 16.3 us
// With heads of 64 a tile has half the bytes and takes nearly as long: 156 us
// (3.5 TB/s) for the first, 137 us (3.9) for the third.
// What the last spends: launches of the kernel and the join (~5 us), the
// setup up to the first copy (~8 us), then a tile's latency from copy to row.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "idx_common.cuh"
#include "idx_internal.h"
#include "idx_tc.cuh"

namespace idx {
namespace {

constexpr int kRowsA = 128;         // rows of an MMA
constexpr int kTile = 128;          // places of a tile
constexpr int kMaxCtas = 160;       // persistent CTAs at most (workspace sizes depend on it)
// Key and value tiles in flight.  A key tile is held for its load and one MMA,
// a value tile too where it does not come early; one ring for both would load
// a value tile long before its softmax is done.
template <int D>
struct Ring {
  static constexpr int kKeys = D == 128 ? 3 : 5, kValues = D == 128 ? 2 : 5;
};
constexpr int kMaxStages = 5;
constexpr int kSegCost = 4;         // units of a segment's begin and end
constexpr int kSoftWarps = 8;
constexpr int kPlanWarp = 8, kKeyTma = 9, kValueTma = 10, kQueryTma = 11, kMmaWarpA = 12;
constexpr int kThreadsA = 13 * 32;
constexpr int kHalf = kTile / 2;    // places of a half tile
constexpr int kChunk = 16;          // tiles planned at once, all of one segment
constexpr int kSlots = 4;           // chunks planned ahead
constexpr int kSlotUsers = kSoftWarps + 4;  // warps that read a chunk
constexpr int kRecWords = 32;
constexpr int kSlotWords = (kChunk + 1) * kRecWords;  // a header, then the tiles
constexpr int kGroup = 16;          // places of a record's group
constexpr int kMaxListTokens = 32;  // tokens of a block with page lists (bits of a mask)
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kScratchRow = 20;     // floats: 16 columns, and 4 that keep rows on different banks

// TMEM columns: two score tiles, whose halves the weights overwrite (two to a
// column), and the two halves' O.
constexpr uint32_t kColS = 0, kColO = 256, kTmemColsA = 512;

// A segment that several stretches share, noted by the one that cuts it first:
// its rows (0: none), first token, KV head, the stretches' first and last, the
// first one's partial slot, and whether some stretch between may be empty.
enum CutWord { kCRows, kCTok0, kCHead, kCFrom, kCTo, kCSlot, kCHoles };
// A chunk's header, and a tile's record.
enum HeadWord { kHTiles, kHTok0, kHTokens, kHHead, kHCtx, kHNew, kHNode0, kHLen, kHOut, kHFold };
enum RecWord { kRFlags, kROffset, kRPos = 8, kRMask = 16, kRBox = 24 };
constexpr int kFlagFirst = 1, kFlagLast = 2, kKindShift = 2;
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
  uint32_t group_inv;  // ceil(2^16 / group): x / group for rows x < 128
  const uint64_t* mask;
  const int32_t* pages;
  int32_t lists, per;
  float scale;
  void* out;
  int64_t o_ts, o_hs;
  float* lse;
  int32_t* status;
  // workspace
  int32_t* cuts;       // [kMaxCtas][8]: the segment to join that was cut first at each stretch's begin (see CutWord)
  float* part_ml;      // [2 * kMaxCtas][128][2]
  float* part_o;       // [2 * kMaxCtas][128][D]
  int32_t* counts;     // [num_tokens * lists], at a block's first token
  ListEntry* entries;  // [num_tokens * lists * per]
  int32_t block_tokens;
  uint32_t polls;
};

// The token of a block's row.
__device__ __forceinline__ int token_of(const TreeArgs& a, int row) { return (int)(((uint32_t)row * a.group_inv) >> 16); }

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
  // units of a request: for each segment kSegCost, then its tiles
  __device__ unsigned long long units(int n, int t0, int s) const {
    const int nl = a.pages != nullptr ? a.lists : 1;
    unsigned long long sum = 0;
    for (int b = 0; b < blocks(n); ++b)
      for (int l = 0; l < nl; ++l) sum += (unsigned long long)(kSegCost + tiles(s, n, t0, b, l));
    return sum * (unsigned)(a.kv_heads / nl);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two values at once: a * b + c, and a + b.
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
// The four softmax warps of both halves, none of which can be missing here.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// The four softmax warps of one half.
__device__ __forceinline__ void half_sync(int half) { asm volatile("bar.sync %0, 128;" ::"r"(2 + half) : "memory"); }
__device__ __forceinline__ bool soft_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
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

// kRescale: powers of two that a score may exceed the reference maximum before O
// is rescaled; kLift: powers of two that all weights are larger by.
template <typename T>
struct Num;
template <>
struct Num<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static constexpr CUtensorMapDataType kMap = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  static constexpr float kLift = 0.f, kRescale = 8.f;
  // Two values rounded to nearest: outputs, and the weights of the product with
  // v, whose two operands the tensor core wants in one 16-bit type.  That is the
  // one rounding before the output's: against 64 bits outputs are off by 0.0023
  // (bf16) and 0.00029 (fp16) of their size, with weights in fp32 by 0.0017 and
  // 0.00021.
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
  // Weights (and their sum) are 2^7 larger, which an output's quotient drops
  // again: the smallest that fp16 keeps is then 2^-32 of a row's largest.  With
  // 2^-25 a long tail below one key was lost in O while the sum counted it.  4
  // powers until a rescale leave 5 below fp16's largest number.
  static constexpr float kLift = 7.f, kRescale = 4.f;
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
constexpr int kBarSet = 64;  // barriers of a run over the stretch
template <int D>
struct Smem {
  static constexpr int kQ = kRowsA * D * 2, kKv = kTile * D * 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffKv = kOffQ + kQ;
  static constexpr int kOffV = kOffKv + Ring<D>::kKeys * kKv;
  static constexpr int kOffScratch = kOffV + Ring<D>::kValues * kKv;
  static constexpr int kOffStats = kOffScratch + kSoftWarps * 32 * kScratchRow * 4;
  static constexpr int kOffRec = kOffStats + kSoftWarps * 32 * 8;
  static constexpr int kOffBar = kOffRec + kSlots * kSlotWords * 4;
  static constexpr int kOffMisc = kOffBar + 2 * kBarSet * 8;
  static constexpr int kBytes = kOffMisc + 256 + 1024;
  // in a careful run (see take_out) the scratch holds marks between segments' ends
  static constexpr int kMarkWords = D / 16;  // of a place or row
  static_assert(2 * 128 * kMarkWords <= kSoftWarps * 32 * kScratchRow, "places' and rows' marks fit");
};
enum BarsA { kKFullA = 0, kKEmptyA = kKFullA + kMaxStages, kVFullA = kKEmptyA + kMaxStages, kVEmptyA = kVFullA + kMaxStages,
             kQFullA = kVEmptyA + kMaxStages, kQEmptyA, kSFull, kPFull = kSFull + 2,
             kPvDone = kPFull + 2, kOEmpty = kPvDone + 2, kMerge, kSlotFull, kSlotEmpty = kSlotFull + kSlots, kDrainA = kSlotEmpty + kSlots,
             kNumBarsA };
static_assert(kNumBarsA <= kBarSet, "barriers fit");

struct MiscA {
  uint32_t tmem_base;
  int abort_flag;
  int soft_dead;  // a softmax warp gave up
  int careful;    // some row's result is not finite though its scores are
  int bad[2];     // (careful) whether a tile has a value that is not finite
  int issued[2];  // key and value tiles whose copies were issued
  int begin[4];   // the request of the stretch's first unit: number, tokens, first token, length
  unsigned long long rem;
  unsigned long long warp_units[kThreadsA / 32];
  uint32_t odd[kRowsA / 32];  // rows whose result is not finite
};

// A warp's way through the planned tiles: all its lanes call next() for each
// tile and done() after it.
struct Walk {
  uint32_t* recs;
  uint64_t* bars;
  volatile int* abort_flag;
  int32_t* status;
  uint32_t polls;
  int chunk = -1, k = 0, n = 0;
  bool ended = false;
  const volatile uint32_t* head = nullptr;
  const volatile uint32_t* rec = nullptr;
  __device__ Walk(uint32_t* r, uint64_t* b, volatile int* f, int32_t* s, uint32_t p)
      : recs(r), bars(b), abort_flag(f), status(s), polls(p) {}
  __device__ bool next() {
    if (k == n) {
      ++chunk;
      const int slot = chunk % kSlots;
      const bool ok = timed_wait_flag(&bars[kSlotFull + slot], (uint32_t)(chunk / kSlots) & 1u, abort_flag, status, polls);
      if (!__all_sync(0xFFFFFFFFu, ok)) return false;
      head = recs + slot * kSlotWords;
      rec = head;
      n = (int)head[kHTiles], k = 0;
      if (n == 0) {  // the stretch's end
        ended = true;
        return false;
      }
    }
    rec += kRecWords;
    ++k;
    return true;
  }
  __device__ void done() {
    __syncwarp();
    if (k == n && lane_id() == 0) mbar_arrive(&bars[kSlotEmpty + chunk % kSlots]);
  }
};

static_assert(sizeof(MiscA) <= 256, "fits its place");

// The barriers of a run over the stretch, by one thread.
__device__ __forceinline__ void init_bars(uint64_t* bars) {
  for (int s = 0; s < kMaxStages; ++s) {
    mbar_init(&bars[kKFullA + s], 1);
    mbar_init(&bars[kKEmptyA + s], 1);
    mbar_init(&bars[kVFullA + s], 1);
    mbar_init(&bars[kVEmptyA + s], 1);
  }
  mbar_init(&bars[kQFullA], 1);
  mbar_init(&bars[kQEmptyA], 1);
  for (int s = 0; s < 2; ++s) {
    mbar_init(&bars[kSFull + s], 1);
    mbar_init(&bars[kPFull + s], kSoftWarps);
    mbar_init(&bars[kPvDone + s], 1);
  }
  mbar_init(&bars[kOEmpty], kSoftWarps);
  mbar_init(&bars[kMerge], kSoftWarps);
  mbar_init(&bars[kDrainA], 1);
  for (int s = 0; s < kSlots; ++s) {
    mbar_init(&bars[kSlotFull + s], 1);
    mbar_init(&bars[kSlotEmpty + s], kSlotUsers);
  }
  fence_mbar_init();
}

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

// One half tile's softmax for a thread whose row stands F times: kCols scores
// in, their weights out.  Updates the row's reference maximum m (of raw
// scores) and its sum l.
template <typename T, int D, int F>
__device__ __forceinline__ bool soft_tile(uint32_t half_s, uint32_t half_o, const volatile uint32_t* rec, const RowState& st,
                                          bool tree, bool lists, float c, bool negate, int col0, int copy, bool first, float& m,
                                          float& l, uint64_t* pv_prev, uint32_t pv_parity, volatile int* abort_flag,
                                          int32_t* status, uint32_t polls) {
  constexpr int kCols = kHalf / F;
  const int kind = (rec[kRFlags] >> kKindShift) & 3;
  uint32_t v[kCols];
#pragma unroll
  for (int k = 0; k < kCols; k += 16) tmem_ld16(half_s + (uint32_t)(copy * kCols + k), v + k);
  tmem_wait_ld();
  if (negate) {
#pragma unroll
    for (int e = 0; e < kCols; ++e) v[e] ^= 0x80000000u;
  }
  if (kind == kRowMask) {
    if (!((rec[kRMask] >> st.token) & 1u)) {
#pragma unroll
      for (int e = 0; e < kCols; ++e) v[e] = 0xFF800000u;
    }
  } else if (kind == kGeneral) {
#pragma unroll
    for (int k = 0; k < kCols; k += kGroup) {
      const int g = (col0 + k) / kGroup;
      const uint32_t bits = group_bits((int)rec[kRPos + g], rec[kRMask + g], st, tree, lists);
#pragma unroll
      for (int e = 0; e < kGroup; ++e)
        if (!((bits >> e) & 1u)) v[k + e] = 0xFF800000u;
    }
  }
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < kCols; ++e) top[e & 3] = fmaxf(top[e & 3], __uint_as_float(v[e]));
  const float big = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));

  float scale = 1.f;
  if (big > m && (m == -INFINITY || (big - m) * c > Num<T>::kRescale)) {
    scale = m == -INFINITY ? 1.f : ex2((m - big) * c);  // with no score so far O and l are zero
    m = big;
  }
  if (!first && __any_sync(0xFFFFFFFFu, scale != 1.f)) {
    // O is complete up to the tile before
    const bool ok = timed_wait_flag(pv_prev, pv_parity, abort_flag, status, polls);
    if (!__all_sync(0xFFFFFFFFu, ok)) return false;
    tc_fence_after();
    l *= scale;
#pragma unroll 1
    for (int k = 0; k < D; k += 16) {
      uint32_t o[16];
      tmem_ld16(half_o + (uint32_t)k, o);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scale);
      tmem_st8(half_o + (uint32_t)k, o);
      tmem_st8(half_o + (uint32_t)k + 8, o + 8);
    }
  }
  const float mc = m == -INFINITY ? 0.f : fmaf(m, c, -Num<T>::kLift);
  const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
  float2 sum[2] = {};
#pragma unroll
  for (int k = 0; k < kCols; k += 16) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float2 x = fma2(make_float2(__uint_as_float(v[k + e]), __uint_as_float(v[k + e + 1])), c2, mc2);
      const float2 y = make_float2(ex2(x.x), ex2(x.y));
      sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], y);
      w[e >> 1] = Num<T>::pack(y.x, y.y);
    }
    tmem_st8(half_s + (uint32_t)((copy * kCols + k) / 2), w);
  }
  if (F > 1) {
    // the places of the other copies
    const uint32_t zero[8] = {};
#pragma unroll
    for (int k = 0; k < F; ++k)
      if (k != copy) {
#pragma unroll
        for (int e = 0; e < kCols / 2; e += 8) tmem_st8(half_s + (uint32_t)(k * kCols / 2 + e), zero);
      }
  }
  const float2 both = add2(sum[0], sum[1]);
  l += both.x + both.y;
  return true;
}

// The rows of a segment whose row stands F times: this warp's half of the
// columns of both halves' O, weighed by g0 and g1, summed over the copies and
// written, 16 columns a round.  Warps w and w + 4 reach the same TMEM lanes, so
// the halves join in registers; copies lie in other lanes and join through
// shared memory, which also turns the rows so that four lanes write one row's
// columns (row by row a thread would write pieces of 32 rows at a time: 4 us a
// segment against 1).  Sets `odd` for rows with a value that is not finite.
template <typename T, int D, int F>
__device__ __forceinline__ bool write_rows(const TreeArgs& a, uint32_t tmem_o, float* scratch, uint32_t* odd_rows, int half, float g0,
                                           float g1, int rows, int tok0, int kvh, uint32_t slot) {
  constexpr int kPer = kRowsA / F, kItems = 4 / F;  // rows, items (a row's four columns) of a thread
  const int tid = threadIdx.x, lane = tid & 31, in_half = tid & (kRowsA - 1);
  const bool direct = slot == 0xFFFFFFFFu;
  float4* own = reinterpret_cast<float4*>(scratch + tid * kScratchRow);
  const float* base = scratch + half * kRowsA * kScratchRow + 4 * (lane & 3);
  const uint32_t tmem = tmem_o + (uint32_t)(half * (D / 2));
  uint32_t x[16], y[16];
  tmem_ld16(tmem, x);
  tmem_ld16(tmem + D, y);
  T* out[kItems];
  float* part[kItems];
  int row[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    row[i] = F == 1 ? (in_half & ~31) + 8 * i + (lane >> 2) : 32 * i + (in_half >> 2);
    const int tk = token_of(a, row[i]), t = tok0 + tk, h = kvh * a.group + row[i] - tk * a.group;
    const int col = half * (D / 2) + 4 * (lane & 3);
    out[i] = static_cast<T*>(a.out) + (int64_t)t * a.o_ts + (int64_t)h * a.o_hs + col;
    part[i] = a.part_o + ((int64_t)(direct ? 0 : slot) * kRowsA + row[i]) * D + col;
  }
  float worst[kItems] = {};  // sums of magnitudes: not finite where a value is not
#pragma unroll 1
  for (int k = 0; k < D / 2; k += 16) {
    tmem_wait_ld();
    float4 f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float* v = reinterpret_cast<float*>(&f[e]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = (g0 == 0.f ? 0.f : __uint_as_float(x[4 * e + j]) * g0) + (g1 == 0.f ? 0.f : __uint_as_float(y[4 * e + j]) * g1);
    }
    if (k + 16 < D / 2) {  // the next round's columns, meanwhile
      tmem_ld16(tmem + (uint32_t)(k + 16), x);
      tmem_ld16(tmem + (uint32_t)(D + k + 16), y);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) own[e] = f[e];
    if (F == 1) __syncwarp();
    else half_sync(half);
    // all loads before any store, so that none waits for another
    float4 z[kItems][F];
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
      for (int c = 0; c < F; ++c) z[i][c] = *reinterpret_cast<const float4*>(base + (row[i] + c * kPer) * kScratchRow);
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
      for (int c = 1; c < F; ++c) z[i][0].x += z[i][c].x, z[i][0].y += z[i][c].y, z[i][0].z += z[i][c].z, z[i][0].w += z[i][c].w;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const float4 u = z[i][0];
      worst[i] += (fabsf(u.x) + fabsf(u.y)) + (fabsf(u.z) + fabsf(u.w));
      if (row[i] < rows) {
        if (direct) *reinterpret_cast<uint2*>(out[i] + k) = make_uint2(Num<T>::pack(u.x, u.y), Num<T>::pack(u.z, u.w));
        else *reinterpret_cast<float4*>(part[i] + k) = u;
      }
    }
    if (F == 1) __syncwarp();
    else half_sync(half);
  }
  bool odd = false;
#pragma unroll
  for (int i = 0; i < kItems; ++i)
    if (row[i] < rows && !(worst[i] < INFINITY)) {
      atomicOr(&odd_rows[row[i] >> 5], 1u << (row[i] & 31));
      odd = true;
    }
  return odd;
}

// Values that are not finite.  A weight of zero does not take an infinity or
// NaN out of the tensor core's sum, so a row can come out not finite because of
// a value that it does not see.  That shows at the segment's end; the CTA then
// goes through its stretch a second time, carefully: it takes such values out
// of each value tile before the product, marks their places' columns, and adds
// up for each row the marks of the places that it sees, which say what those
// columns are.  That costs a CTA's stretch two to three times its usual time,
// more where nearly every place holds one (64 requests of 8 tokens over 8,192
// places: 219 us, 690 with one such value a request, 3.1 ms with one a place).

// 64 columns of a place, as they lie in shared memory (16-byte pieces in the
// order of the 128-byte swizzle): zeros in the stead of infinities and NaN,
// marked in pos (+inf), neg (-inf) or both (NaN).
template <typename T>
__device__ __forceinline__ bool take_out(uint4* v, int place, uint32_t (&pos)[2], uint32_t (&neg)[2]) {
  constexpr uint32_t kExp = Num<T>::kBf16 ? 0x7F80u : 0x7C00u;
  pos[0] = pos[1] = neg[0] = neg[1] = 0u;
  bool any = false;
#pragma unroll 1
  for (int k = 0; k < 8; ++k) {
    uint4 x = v[k];
    uint32_t* w = reinterpret_cast<uint32_t*>(&x);
    bool here = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = (w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
      if ((h & kExp) == kExp) {
        const int col = 8 * (k ^ (place & 7)) + e;
        const uint32_t bit = 1u << (col & 31);
        const bool nan = (h & 0x7FFFu) != kExp;
        if (nan || !(h & 0x8000u)) pos[col >> 5] |= bit;
        if (nan || (h & 0x8000u)) neg[col >> 5] |= bit;
        w[e >> 1] &= ~(0xFFFFu << (16 * (e & 1)));
        here = true;
      }
    }
    if (here) v[k] = x, any = true;
  }
  return any;
}

// Rows of a padded batch, past the last request: a warp of each CTA that is done
// long before the others clears its share.
template <typename T, int D>
__device__ __noinline__ void clear_rest(const TreeArgs& a) {
  const int lane = (int)lane_id();
  const int64_t all = (int64_t)a.num_tokens * a.q_heads;
  for (int64_t x = (int64_t)Plan(a).tok0(a.num_reqs) * a.q_heads + blockIdx.x; x < all; x += gridDim.x) {
    const int64_t t = x / a.q_heads, h = x - t * a.q_heads;
    if (lane < D / 8) *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + t * a.o_ts + h * a.o_hs + 8 * lane) = make_uint4(0, 0, 0, 0);
    if (lane == 0 && a.lse != nullptr) a.lse[x] = -INFINITY;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsA, 1)
    k_tree_attention(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeArgs a) {
  using S = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* const all_bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  MiscA* misc = reinterpret_cast<MiscA*>(smem + S::kOffMisc);
  uint32_t* recs = reinterpret_cast<uint32_t*>(smem + S::kOffRec);
  volatile int* abort_flag = &misc->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Plan plan(a);
  const bool lists = a.pages != nullptr, tree = a.mask != nullptr;

  if (tid == 0) {
    misc->abort_flag = 0;
    misc->soft_dead = 0;
    misc->issued[0] = misc->issued[1] = 0;
    misc->careful = misc->bad[0] = misc->bad[1] = 0;
    for (int s = 0; s < kRowsA / 32; ++s) misc->odd[s] = 0;
    init_bars(all_bars);
  }
  if (tid == 32) {  // a cold descriptor costs a copy a microsecond
    asm volatile("prefetch.tensormap [%0];" ::"l"(&qmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
  }
  __syncwarp();
  if (warp == 0) tmem_alloc(&misc->tmem_base, kTmemColsA);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem_base;
  pdl_enter();  // before any global-memory access
  // The line of units, cut into stretches [w0, w1): who holds unit w0, and the
  // units before it in that request.
  unsigned long long W = 0, w0 = 0, w1 = 0;
  auto cut = [&](unsigned long long all) {  // (64-bit divisions take some hundred cycles each)
    const uint32_t x = blockIdx.x, g = gridDim.x;
    W = all;
    if (W < (1u << 23)) w0 = (uint32_t)W * x / g, w1 = (uint32_t)W * (x + 1) / g;
    else w0 = W * x / g, w1 = W * (x + 1) / g;
  };
  {
    // a request a thread, or a run of them
    const int run = (a.num_reqs + kThreadsA - 1) / kThreadsA, r0 = tid * run;
    unsigned long long mine = 0;
    int n = 0, t0 = 0, s = 0;
#pragma unroll 1
    for (int r = r0; r < min(r0 + run, a.num_reqs); ++r) {
      n = plan.ntok(r), t0 = plan.tok0(r), s = plan.seq(r);
      mine += plan.units(n, t0, s);
    }
    unsigned long long incl = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) misc->warp_units[warp] = incl;
    __syncthreads();
    unsigned long long all = 0, before = incl - mine;
#pragma unroll 1
    for (int k = 0; k < kThreadsA / 32; ++k) {
      const unsigned long long y = misc->warp_units[k];
      if (k < warp) before += y;
      all += y;
    }
    cut(all);
    if (w0 < w1 && before <= w0 && w0 < before + mine) {
      int r = min(r0 + run, a.num_reqs) - 1;
      if (run > 1)  // which of the run
        for (r = r0;; ++r) {
          n = plan.ntok(r), t0 = plan.tok0(r), s = plan.seq(r);
          const unsigned long long u = plan.units(n, t0, s);
          if (w0 < before + u) break;
          before += u;
        }
      misc->begin[0] = r, misc->begin[1] = n, misc->begin[2] = t0, misc->begin[3] = s;
      misc->rem = w0 - before;
    }
    __syncthreads();
  }

  // A run over the stretch: once, or a second time where some value was not
  // finite (see take_out), with barriers of its own, which no arrival of the
  // first run can reach.  Code of its own as well: with both runs in one loop the
  // warps' way to their barriers was longer, 168 us for 160 on 64 tokens over
  // 65,536 places.
  auto run = [&](auto how) {
    constexpr bool kCareful = decltype(how)::value;
    uint64_t* const bars = all_bars + (kCareful ? kBarSet : 0);
    if (warp == kPlanWarp) {
      const bool some = w0 < w1;
      int r = some ? misc->begin[0] : 0, n = some ? misc->begin[1] : 0, t0 = some ? misc->begin[2] : 0, s = some ? misc->begin[3] : 0;
      unsigned long long rem = some ? misc->rem : 0;
      // and its block, head and tile; all lanes hold the same cursor
      int b = 0, kvh = 0;
      const int per_list = lists ? a.kv_heads / a.lists : a.kv_heads;
      int tiles = some ? plan.tiles(s, n, t0, 0, 0) : 0;
      while (some && rem >= (unsigned)(kSegCost + tiles)) {
        rem -= (unsigned)(kSegCost + tiles);
        if (++kvh == a.kv_heads) kvh = 0, ++b;
        tiles = plan.tiles(s, n, t0, b, kvh / per_list);
      }
      // the segment's units begin at u0; the stretch's part of it are the tiles from `tile` on
      unsigned long long u0 = w0 - rem;
      int tile = max(0, (int)rem - kSegCost);
      const int bs = min(a.page, kTile), boxes = kTile / bs;  // places of a box, boxes of a tile
      const int page_tiles = max(1, a.page / kTile);
      // the segment that the stretch begins in, for its note below
      const int tile0 = tile, tiles0 = tiles, rows0 = min(a.block_tokens, n - b * a.block_tokens) * a.group, kvh0 = kvh;
      const int tok00 = t0 + b * a.block_tokens;
      const unsigned long long u00 = u0;
      int seg = 0, piece_first = tile, chunk = 0;
      bool bad_block = false, gave_up = false;
      while (some && u0 < w1) {
        // tiles of the segment up to the stretch's end
        const int piece_end = (int)min((unsigned long long)tiles, w1 > u0 + kSegCost ? w1 - u0 - kSegCost : 0ull);
        if (tile >= piece_end) break;  // the stretch ends before the segment's first tile
        const int len = plan.len(s), ctx = s - n;
        const int m = min(a.block_tokens, n - b * a.block_tokens), tok = t0 + b * a.block_tokens;
        const int rows = m * a.group;
        const int fold_code = rows <= kRowsA / 4 ? 2 : rows <= kRowsA / 2 ? 1 : 0;
        const int lh = lists ? kvh / per_list : 0;
        const int64_t list = ((int64_t)tok * a.lists + (int64_t)lh * m) * a.per;
        const int entries = lists ? min(a.counts[(int64_t)tok * a.lists + lh], m * a.per) : 0;
        const int here = min(kChunk, piece_end - tile);  // tiles of this chunk
        const int slot = chunk % kSlots;
        const bool ok = chunk < kSlots || timed_wait_flag(&bars[kSlotEmpty + slot], ((uint32_t)(chunk / kSlots) & 1u) ^ 1u, abort_flag,
                                                          a.status, a.polls);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          gave_up = true;
          break;
        }
        uint32_t* head = recs + slot * kSlotWords;
        if (lane == 31) {
          head[kHTiles] = (uint32_t)here, head[kHTok0] = (uint32_t)tok, head[kHTokens] = (uint32_t)m, head[kHHead] = (uint32_t)kvh;
          head[kHCtx] = (uint32_t)ctx, head[kHNew] = (uint32_t)n, head[kHNode0] = (uint32_t)(b * a.block_tokens);
          head[kHLen] = (uint32_t)len, head[kHFold] = (uint32_t)fold_code;
          // partial results: slot 2x for the first segment of stretch x, 2x + 1 for the last; -1: the whole segment is here
          head[kHOut] = piece_first == 0 && piece_end == tiles ? 0xFFFFFFFFu : (uint32_t)(2 * blockIdx.x + (seg > 0 ? 1 : 0));
        }
        if (lane < here) {
          const int my = tile + lane;
          uint32_t* rec = head + (1 + lane) * kRecWords;
          const uint32_t every = m >= 32 ? 0xFFFFFFFFu : (1u << m) - 1u;
          const int page0 = boxes > 1 ? my * boxes : my / page_tiles, offset = boxes > 1 ? 0 : (my % page_tiles) * kTile;
          bool all_cached = true, all_tokens = true;
          for (int x = 0; x < boxes; ++x) {
            int blk = -1, pg = page0 + x;
            uint32_t tokens = 0xFFFFFFFFu;
            if (lists) {
              if (pg < entries) {
                const ListEntry en = a.entries[list + pg];
                blk = en.block, pg = en.page, tokens = en.tokens;
              }
            } else if ((int64_t)pg * a.page < len) {
              blk = a.bt[r * a.bt_stride + pg];
              if (blk < 0 || blk >= a.num_blocks) bad_block = true, blk = -1;
            }
            rec[kRBox + x] = (uint32_t)(blk < 0 ? (int)a.num_blocks : blk);  // a block outside the pool reads as zeros
            const int pos = pg * a.page + offset;
            all_cached = all_cached && blk >= 0 && (int64_t)pos + bs <= ctx && (int64_t)pos + bs <= len;
            all_tokens = all_tokens && (tokens & every) == every;
            for (int g = 0; g < bs / kGroup; ++g) {
              rec[kRPos + x * (bs / kGroup) + g] = (uint32_t)(blk < 0 ? -1 : pos + g * kGroup);
              rec[kRMask + x * (bs / kGroup) + g] = tokens;
            }
          }
          const int kind = all_cached && all_tokens ? kFull : all_cached && boxes == 1 ? kRowMask : kGeneral;
          rec[kROffset] = (uint32_t)offset;
          rec[kRFlags] = (uint32_t)((my == piece_first ? kFlagFirst : 0) | (my + 1 == piece_end ? kFlagLast : 0) | (kind << kKindShift));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kSlotFull + slot]);
        ++chunk;
        tile += here;
        if (tile == tiles) {
          // next segment
          u0 += (unsigned)(kSegCost + tiles);
          tile = 0;
          piece_first = 0;
          ++seg;
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
          if (u0 < w1) tiles = plan.tiles(s, n, t0, b, kvh / per_list);
        } else if (tile == piece_end) {
          break;
        }
      }
      if (!gave_up) {
        const int slot = chunk % kSlots;
        const bool ok =
            timed_wait_flag(&bars[kSlotEmpty + slot], ((uint32_t)(chunk / kSlots) & 1u) ^ 1u, abort_flag, a.status, a.polls);
        if (__all_sync(0xFFFFFFFFu, ok) && lane == 0) {
          recs[slot * kSlotWords + kHTiles] = 0;  // the end
          mbar_arrive(&bars[kSlotFull + slot]);
        }
        __syncwarp();
      }
      if (lane == 0) {
        int32_t* cut = a.cuts + 8 * blockIdx.x;
        int rows = 0;
        if (some && tile0 > 0) {
          // stretch y begins at unit W y / ctas and holds unit u for y = ((u + 1) ctas - 1) / W
          const unsigned long long ctas = gridDim.x, u1 = u00 + kSegCost + tiles0;
          const int from = (int)((w0 * ctas - 1) / W), to = (int)((u1 * ctas - 1) / W);
          const unsigned long long begin = W * from / ctas;
          if (begin <= u00 + kSegCost) {  // else the segment was cut before
            rows = rows0;
            cut[kCTok0] = tok00, cut[kCHead] = kvh0, cut[kCFrom] = from, cut[kCTo] = to;
            // slot 2y, but 2y + 1 where the segment is not its stretch's first
            cut[kCSlot] = 2 * from + (u00 > begin ? 1 : 0);
            cut[kCHoles] = W < ctas ? 1 : 0;
          }
        }
        cut[kCRows] = rows;
      }
      if (bad_block) report(a.status, IDX_ST_BLOCK_OOR);
      __syncwarp();
      if constexpr (!kCareful) clear_rest<T, D>(a);
    } else if (warp == kKeyTma || warp == kValueTma) {
      const bool keys = warp == kKeyTma;
      const CUtensorMap* map = keys ? &kmap : &vmap;
      const int bs = min(a.page, kTile), boxes = kTile / bs;
      const int bx = lane % boxes, sub = lane / boxes;
      const bool mine = lane < boxes * (D / 64);
      const int stages = keys ? Ring<D>::kKeys : Ring<D>::kValues;
      uint64_t *full = &bars[keys ? kKFullA : kVFullA], *empty = &bars[keys ? kKEmptyA : kVEmptyA];
      uint8_t* dst = smem + (keys ? S::kOffKv : S::kOffV) + sub * (kTile * 128) + bx * bs * 128;
      Walk w(recs, bars, abort_flag, a.status, a.polls);
      int i = 0, stage = 0;
      uint32_t phase = 0;
      for (; w.next(); ++i) {
        const int kvh = (int)w.head[kHHead], offset = (int)w.rec[kROffset], box = (int)w.rec[kRBox + bx];
        const bool ok = timed_wait_flag(&empty[stage], phase ^ 1u, abort_flag, a.status, a.polls);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], (uint32_t)S::kKv);
        __syncwarp();
        if (mine) tma_load_4d(dst + stage * S::kKv, map, sub * 64, kvh, offset, box, &full[stage]);
        w.done();
        if (++stage == stages) stage = 0, phase ^= 1u;
      }
      if (lane == 0) misc->issued[keys ? 0 : 1] = i;
    } else if (warp == kQueryTma) {
      Walk w(recs, bars, abort_flag, a.status, a.polls);
      int queries = 0;
      while (w.next()) {
        if (w.rec[kRFlags] & kFlagFirst) {
          for (int k = lane; k < (int)w.head[kHTokens] * (D / 64); k += 32)  // into L2 while the queries before are in use
            asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(&qmap), "r"(k % (D / 64) * 64),
                         "r"((int)w.head[kHHead] * a.group), "r"((int)w.head[kHTok0] + k / (D / 64))
                         : "memory");
          bool ok = true;
          if (queries > 0) ok = timed_wait_flag(&bars[kQEmptyA], (uint32_t)(queries - 1) & 1u, abort_flag, a.status, a.polls);
          if (!__all_sync(0xFFFFFFFFu, ok)) break;
          const int m = (int)w.head[kHTokens], fold = 1 << (int)w.head[kHFold], tok = (int)w.head[kHTok0], kvh = (int)w.head[kHHead];
          const int loads = m * fold * (D / 64);
          if (lane == 0) mbar_arrive_expect_tx(&bars[kQFullA], (uint32_t)(loads * a.group * 128));
          __syncwarp();
          for (int k = lane; k < loads; k += 32) {
            const int sub = k % (D / 64), tk = k / (D / 64) % m, copy = k / (D / 64) / m;
            tma_load_3d(smem + S::kOffQ + sub * (kRowsA * 128) + (copy * (kRowsA / fold) + tk * a.group) * 128, &qmap, sub * 64,
                        kvh * a.group, tok + tk, &bars[kQFullA]);
          }
          ++queries;
        }
        w.done();
      }
      if (lane == 0 && queries > 0) mbar_wait(&bars[kQFullA], (uint32_t)(queries - 1) & 1u, nullptr);
    } else if (warp == kMmaWarpA) {
      constexpr uint32_t kIdS = idesc_16(Num<T>::kBf16, kRowsA, kTile, false);
      constexpr uint32_t kIdO = idesc_16(Num<T>::kBf16, kRowsA, D, true);
      Walk w(recs, bars, abort_flag, a.status, a.polls);
      // A barrier's test takes 200-300 cycles even where the phase is long
      // complete; one after another this warp's tests (up to six a tile) set the
      // pace, 2,850 cycles a tile.  So its lanes test all that the next scores (of
      // tile i) and the next rows (of tile j) wait for at once, a barrier a lane,
      // and whatever is ready is issued (64 drafted tokens over 65,536 places:
      // 168 -> 161 us; one token over 5,000: 16.5 -> 16.1).
      int i = 0, j = 0;              // tiles whose scores, whose rows have been issued
      int seg_s = 0, seg_o = 0;      // segments whose scores, whose rows have been issued
      uint32_t flags[3] = {};        // of tiles i, i - 1, i - 2
      int k_stage = 0, v_stage = 0;
      uint32_t k_phase = 0, v_phase = 0;
      bool issued = false;
      bool more = w.next();
      if (more) flags[0] = w.rec[kRFlags], w.done();
      const uint64_t limit = a.polls == 0 ? 1ull : (uint64_t)a.polls << 10;
      uint64_t idle = 0;  // tests since the last issue
      while (more || j < i) {
        const uint32_t row_flags = i - j == 2 ? flags[2] : flags[1];  // of tile j
        int bar = -1;       // nothing to wait for
        uint32_t phase = 0;
        if (lane == 0) bar = kKFullA + k_stage, phase = k_phase;
        if (lane == 1 && i >= 2) bar = kPvDone + (i & 1), phase = (uint32_t)((i >> 1) - 1) & 1u;  // the weights of tile i - 2 are read
        if (lane == 2 && (flags[0] & kFlagFirst)) bar = kQFullA, phase = (uint32_t)seg_s & 1u;
        if (lane == 3) bar = kVFullA + v_stage, phase = v_phase;
        if (lane == 4) bar = kPFull + (j & 1), phase = (uint32_t)(j >> 1) & 1u;
        if (lane == 5 && (row_flags & kFlagFirst) && seg_o > 0) bar = kOEmpty, phase = (uint32_t)(seg_o - 1) & 1u;  // the rows before are read
        const bool ready = bar < 0 || mbar_try_wait_nosuspend(&bars[bar], phase);
        const uint32_t got = __ballot_sync(0xFFFFFFFFu, ready);
        const bool do_scores = more && (got & 7u) == 7u;
        // scores come first: rows wait while all that scores lack is the end of
        // the product just issued, or the next softmax would wait instead
        const bool hold = more && i - j == 1 && (got & 7u) == 5u;
        const bool do_rows = j < i && (got & 0x38u) == 0x38u && !hold;
        if (!do_rows && !do_scores) {
          const bool stop = ++idle >= limit || ((idle & 63u) == 0 && *abort_flag);
          if (__any_sync(0xFFFFFFFFu, stop)) {
            if (lane == 0 && !*abort_flag) {
              *abort_flag = 1;
              report(a.status, IDX_ST_TIMEOUT);
            }
            break;
          }
          continue;
        }
        idle = 0;
        __syncwarp();  // what each lane has seen complete is so for the lane that issues
        tc_fence_after();
        if (lane == 0) {
          if (do_scores) {
            const uint64_t qd = sw128_desc(sbase + S::kOffQ), kd = sw128_desc(sbase + S::kOffKv + k_stage * S::kKv);
            const uint32_t d = tmem + kColS + (uint32_t)(i & 1) * kTile;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint64_t step = (uint64_t)((k / 4) * (kRowsA * 128 / 16) + (k % 4) * 2);
              mma_16(d, qd + step, kd + step, kIdS, k > 0 ? 1u : 0u);
            }
            // a tile's stage is given back before anybody can learn that the
            // tile is done: the ring's waits count on that order
            mma_commit(&bars[kKEmptyA + k_stage]);
            if (flags[0] & kFlagLast) mma_commit(&bars[kQEmptyA]);
            mma_commit(&bars[kSFull + (i & 1)]);
          }
          if (do_rows) {
            const uint64_t vd = sw128_desc_nmajor(sbase + S::kOffV + v_stage * S::kKv);
            const uint32_t p = tmem + kColS + (uint32_t)(j & 1) * kTile, old = row_flags & kFlagFirst ? 0u : 1u;
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k) {
              const int half = k / (kHalf / 16);
              mma_16_ta(tmem + kColO + (uint32_t)(half * D), p + (uint32_t)(half * kHalf + 8 * (k % (kHalf / 16))),
                        vd + (uint64_t)(k * (2048 / 16)), kIdO, k % (kHalf / 16) > 0 ? 1u : old);
            }
            mma_commit(&bars[kVEmptyA + v_stage]);
            mma_commit(&bars[kPvDone + (j & 1)]);
          }
        }
        __syncwarp();
        issued = true;
        if (do_rows) {
          if (row_flags & kFlagLast) ++seg_o;
          if (++v_stage == Ring<D>::kValues) v_stage = 0, v_phase ^= 1u;
          ++j;
        }
        if (do_scores) {
          if (flags[0] & kFlagLast) ++seg_s;
          if (++k_stage == Ring<D>::kKeys) k_stage = 0, k_phase ^= 1u;
          ++i;
          flags[2] = flags[1], flags[1] = flags[0];
          more = w.next();
          if (more) flags[0] = w.rec[kRFlags], w.done();
          else if (!w.ended) break;
        }
      }
      if (issued) {
        if (lane == 0) mma_commit(&bars[kDrainA]);
        __syncwarp();
        mbar_wait(&bars[kDrainA], 0, nullptr);
      }
    } else if (warp < kSoftWarps) {
      const int lane_row = tid & (kRowsA - 1), half = warp >> 2;
      const uint32_t tmem_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t half_o = tmem_row + kColO + (uint32_t)(half * D);
      float* scratch = reinterpret_cast<float*>(smem + S::kOffScratch);
      float2* stats = reinterpret_cast<float2*>(smem + S::kOffStats);
      const bool negate = a.scale < 0.f;
      // scores in powers of two; a scale of 0 becomes one that still hides masked places
      const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
      float m = -INFINITY, l = 0.f;
      RowState st{};
      int meets = 0;
      int row = 0, copy = 0, fold = 1, col0 = 0, rows = 0;
      bool warp_live = true, met = false;
      // All eight warps meet, those that gave up among them (see below); the wait
      // ends for all or for none, so that no warp misses a later barrier.  False:
      // one gave up.
      auto meet = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kMerge]);
        const bool all = mbar_wait(&bars[kMerge], (uint32_t)meets & 1u, nullptr);
        ++meets;
        return __all_sync(0xFFFFFFFFu, all) && !*reinterpret_cast<volatile int*>(&misc->soft_dead);
      };
      uint32_t* place_marks = reinterpret_cast<uint32_t*>(scratch);  // [place][+ columns, - columns]
      uint32_t* row_marks = place_marks + kTile * S::kMarkWords;
      if (kCareful)
        for (int k = tid; k < kRowsA * S::kMarkWords; k += kSoftWarps * 32) row_marks[k] = 0;
      Walk w(recs, bars, abort_flag, a.status, a.polls);
      for (int i = 0; w.next(); ++i) {
        const uint32_t s_par = (uint32_t)(i >> 1) & 1u;
        const volatile uint32_t *rec = w.rec, *head = w.head;
        const uint32_t flags = rec[kRFlags];
        const bool first = (flags & kFlagFirst) != 0;
        if (first) {
          rows = (int)head[kHTokens] * a.group;
          fold = 1 << (int)head[kHFold];
          row = lane_row & (kRowsA / fold - 1), copy = lane_row / (kRowsA / fold);
          col0 = half * kHalf + copy * (kHalf / fold);
          warp_live = (row & ~31) < rows;
          m = -INFINITY, l = 0.f;
          st.token = min(token_of(a, row), (int)head[kHTokens] - 1);  // rows past the block's compute on the last token's mask
          st.ctx = (int)head[kHCtx], st.len = (int)head[kHLen];
          const int n = (int)head[kHNew];
          st.chain_end = st.ctx + (int)head[kHNode0] + st.token + 1;
          st.tree = tree ? a.mask[(int)head[kHTok0] + st.token] & (n >= 64 ? ~0ull : (1ull << n) - 1ull) : 0ull;
        }
        bool ok = timed_wait_flag(&bars[kSFull + (i & 1)], s_par, abort_flag, a.status, a.polls);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        tc_fence_after();
        const uint32_t half_s = tmem_row + kColS + (uint32_t)((i & 1) * kTile + half * kHalf);
        uint64_t* pv_prev = &bars[kPvDone + ((i + 1) & 1)];
        const uint32_t pv_par = (uint32_t)((i - 1) >> 1) & 1u;
        if (warp_live) {  // a warp without a live row leaves what lies there: its rows are not read
          if (fold == 4)
            ok = soft_tile<T, D, 4>(half_s, half_o, rec, st, tree, lists, c, negate, col0, copy, first, m, l, pv_prev, pv_par, abort_flag,
                                    a.status, a.polls);
          else if (fold == 2)
            ok = soft_tile<T, D, 2>(half_s, half_o, rec, st, tree, lists, c, negate, col0, copy, first, m, l, pv_prev, pv_par, abort_flag,
                                    a.status, a.polls);
          else
            ok = soft_tile<T, D, 1>(half_s, half_o, rec, st, tree, lists, c, negate, col0, copy, first, m, l, pv_prev, pv_par, abort_flag,
                                    a.status, a.polls);
        }
        if (!ok) break;
        if (((flags >> kKindShift) & 3) == kGeneral && half < D / 64) {
          // values at places that do not exist may be anything: zeros in their stead
          const int pos = (int)rec[kRPos + lane_row / kGroup];
          if (pos >= 0 && pos + lane_row % kGroup >= st.len) {
            const int stage = i % Ring<D>::kValues;
            ok = timed_wait_flag(&bars[kVFullA + stage], (uint32_t)(i / Ring<D>::kValues) & 1u, abort_flag, a.status, a.polls);
            if (ok) {
              uint4* vrow = reinterpret_cast<uint4*>(smem + S::kOffV + stage * S::kKv + half * (kTile * 128) + lane_row * 128);
#pragma unroll
              for (int e = 0; e < 8; ++e) vrow[e] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          if (!__all_sync(0xFFFFFFFFu, ok)) break;
        }
        if constexpr (kCareful) {
          const int stage = i % Ring<D>::kValues;
          ok = timed_wait_flag(&bars[kVFullA + stage], (uint32_t)(i / Ring<D>::kValues) & 1u, abort_flag, a.status, a.polls);
          if (!__all_sync(0xFFFFFFFFu, ok)) break;
          if (half < D / 64) {
            uint32_t pos[2], neg[2];
            uint4* v = reinterpret_cast<uint4*>(smem + S::kOffV + stage * S::kKv + half * (kTile * 128) + lane_row * 128);
            if (take_out<T>(v, lane_row, pos, neg)) misc->bad[i & 1] = 1;
            uint32_t* mark = place_marks + lane_row * S::kMarkWords + 2 * half;
            mark[0] = pos[0], mark[1] = pos[1], mark[D / 32] = neg[0], mark[D / 32 + 1] = neg[1];
            fence_proxy_async_smem();
          }
          if (!meet()) {
            met = true;
            break;
          }
          if (*reinterpret_cast<volatile int*>(&misc->bad[i & 1]) && row < rows) {
            // the marks of this thread's places that the row sees
            const int kind = (flags >> kKindShift) & 3;
            for (int p = col0; p < col0 + kHalf / fold; ++p) {
              bool seen = kind == kFull || (kind == kRowMask && ((rec[kRMask] >> st.token) & 1u));
              if (kind == kGeneral)
                seen = (group_bits((int)rec[kRPos + p / kGroup], rec[kRMask + p / kGroup], st, tree, lists) >> (p % kGroup)) & 1u;
              for (int k = 0; seen && k < S::kMarkWords; ++k) {
                const uint32_t x = place_marks[p * S::kMarkWords + k];
                if (x) atomicOr(&row_marks[row * S::kMarkWords + k], x);
              }
            }
          }
          if (tid == 0) misc->bad[(i + 1) & 1] = 0;
          if (!meet()) {
            met = true;
            break;
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kPFull + (i & 1)]);
        if (!(flags & kFlagLast)) {
          w.done();
          continue;
        }

        // the segment's rows
        ok = timed_wait_flag(&bars[kPvDone + (i & 1)], s_par, abort_flag, a.status, a.polls);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        tc_fence_after();
        stats[tid] = make_float2(m, l);
        if (!meet()) {
          met = true;
          break;
        }
        // the row's parts: two halves of `fold` copies
        const int per = kRowsA / fold;
        auto row_of = [&](int x, float& sum) {  // the row's largest maximum, and its sum
          float top = -INFINITY;
          sum = 0.f;
#pragma unroll 1
          for (int p = x; p < kRowsA; p += per) top = fmaxf(top, fmaxf(stats[p].x, stats[kRowsA + p].x));
#pragma unroll 1
          for (int p = x; p < kRowsA; p += per) {
            const float2 u = stats[p], v = stats[kRowsA + p];
            // (a part without a maximum has the sum 0, or NaN where all scores that it sees are NaN)
            sum += u.x != -INFINITY ? u.y * ex2((u.x - top) * c) : u.y;
            sum += v.x != -INFINITY ? v.y * ex2((v.x - top) * c) : v.y;
          }
          return top;
        };
        float sum_l;
        const float big = row_of(row, sum_l);
        const uint32_t slot = head[kHOut];
        const bool direct = slot == 0xFFFFFFFFu, empty = sum_l == 0.f;
        const bool lost = sum_l != sum_l;  // some score is NaN: so is the row, whichever part saw it
        // what this lane's two halves weigh in the row
        const float inv = empty ? 0.f : direct || lost ? 1.f / sum_l : 1.f, m0 = stats[lane_row].x, m1 = stats[kRowsA + lane_row].x;
        const float g0 = m0 == -INFINITY && !lost ? 0.f : ex2((m0 - big) * c) * inv;
        const float g1 = m1 == -INFINITY && !lost ? 0.f : ex2((m1 - big) * c) * inv;
        const int tok0 = (int)head[kHTok0], kvh = (int)head[kHHead];
        if (row < rows && half == 0 && copy == 0) {
          const int tk = token_of(a, row), t = tok0 + tk, h = kvh * a.group + row - tk * a.group;
          const float ref = empty ? -INFINITY : lost ? sum_l : fmaf(big, c, -Num<T>::kLift);
          if (!direct) reinterpret_cast<float2*>(a.part_ml)[(int64_t)slot * kRowsA + row] = make_float2(ref, sum_l);
          else if (a.lse != nullptr)
            a.lse[(int64_t)t * a.q_heads + h] = empty ? -INFINITY : (ref + __log2f(sum_l)) * 0.6931471805599453f;
        }
        const bool sum_ok = sum_l > 0.f && sum_l < INFINITY;  // else its scores are not finite, or it sees nothing
        uint32_t pos[D / 64] = {}, neg[D / 64] = {};  // marks of the row's columns of this half
        if constexpr (kCareful) {
          if (row < rows && copy == 0 && sum_ok) {
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
              pos[k] = row_marks[row * S::kMarkWords + half * (D / 64) + k];
              neg[k] = row_marks[row * S::kMarkWords + D / 32 + half * (D / 64) + k];
            }
          }
          soft_sync();  // the scratch is free
        }
        bool odd;
        if (fold == 4) odd = write_rows<T, D, 4>(a, tmem_row + kColO, scratch, misc->odd, half, g0, g1, rows, tok0, kvh, slot);
        else if (fold == 2) odd = write_rows<T, D, 2>(a, tmem_row + kColO, scratch, misc->odd, half, g0, g1, rows, tok0, kvh, slot);
        else odd = write_rows<T, D, 1>(a, tmem_row + kColO, scratch, misc->odd, half, g0, g1, rows, tok0, kvh, slot);
        if constexpr (kCareful) {
          soft_sync();  // the rows are written
          const int tk = token_of(a, row), t = tok0 + tk, h = kvh * a.group + row - tk * a.group;
          T* to = static_cast<T*>(a.out) + (int64_t)t * a.o_ts + (int64_t)h * a.o_hs + half * (D / 2);
          float* part = a.part_o + ((int64_t)(direct ? 0 : slot) * kRowsA + row) * D + half * (D / 2);
#pragma unroll
          for (int k = 0; k < D / 64; ++k)
            for (uint32_t left = pos[k] | neg[k]; left; left &= left - 1u) {
              const int e = __ffs((int)left) - 1;
              const bool up = (pos[k] >> e) & 1u, down = (neg[k] >> e) & 1u;
              const float x = up && down ? NAN : up ? INFINITY : -INFINITY;
              if (direct) to[32 * k + e] = (T)x;
              else part[32 * k + e] = x;
            }
          for (int k = tid; k < kRowsA * S::kMarkWords; k += kSoftWarps * 32) row_marks[k] = 0;
        } else if (soft_any(odd)) {  // rare
          if (row < rows && sum_ok && ((*reinterpret_cast<volatile uint32_t*>(&misc->odd[row >> 5]) >> (row & 31)) & 1u)) misc->careful = 1;
          soft_sync();
          if (tid < kRowsA / 32) misc->odd[tid] = 0;
          soft_sync();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kOEmpty]);
        w.done();
      }
      if (!w.ended && !met && lane == 0) {
        // gave up: say so, then take this warp's place at the barrier that the others may wait at
        *reinterpret_cast<volatile int*>(&misc->soft_dead) = 1;
        mbar_arrive(&bars[kMerge]);
      }
    }

    if constexpr (!kCareful) {
      if (tid == 0 && blockIdx.x == 0) *reinterpret_cast<unsigned long long*>(a.cuts + 8 * kMaxCtas) = W;
      // lengths that the table does not hold
      if (blockIdx.x == 0)
        for (int r = tid; r < a.num_reqs; r += kThreadsA)
          if (plan.ntok(r) > 0 && plan.len(plan.seq(r)) < plan.seq(r)) report(a.status, IDX_ST_LEN_CLAMPED);
    }
    __syncwarp();
    __syncthreads();  // all copies have landed, all products are done
  };
  run(std::false_type{});
  bool careful = false;
  if (!*abort_flag && *reinterpret_cast<volatile int*>(&misc->careful)) {
    careful = true;
    if (tid == 0) {
      misc->issued[0] = misc->issued[1] = 0;
      init_bars(all_bars + kBarSet);
    }
    __syncthreads();
    run(std::true_type{});
  }

  if (*abort_flag) {
    if (tid < 2) {
      // never leave with a copy in flight: the last ones of each ring
      uint64_t* const bars = all_bars + (careful ? kBarSet : 0);
      const int stages = tid == 0 ? Ring<D>::kKeys : Ring<D>::kValues;
      for (int i = max(0, misc->issued[tid] - stages); i < misc->issued[tid]; ++i)
        mbar_wait(&bars[(tid == 0 ? kKFullA : kVFullA) + i % stages], (uint32_t)(i / stages) & 1u, nullptr);
    }
    __syncwarp();
    __syncthreads();
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemColsA);
  }
}

// Joins the partial rows of the segments that the stretches share: block
// (x, y) those that stretch x + 1 cut first, a warp a row: the largest
// reference maximum, then the weighted sums.
constexpr int kJoinWarps = 4;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) k_tree_combine(const __grid_constant__ TreeArgs a, int ctas) {
  pdl_enter();
  __shared__ float weight[kJoinWarps][kMaxCtas];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 c0 = *reinterpret_cast<const int4*>(a.cuts + 8 * (blockIdx.x + 1));
  const int4 c1 = *reinterpret_cast<const int4*>(a.cuts + 8 * (blockIdx.x + 1) + 4);
  const int row = blockIdx.y * kJoinWarps + warp;
  if (row >= c0.x) return;
  const int from = c0.w, to = c1.x, first_slot = c1.y;
  const bool holes = c1.z != 0;
  const unsigned long long W = holes ? *reinterpret_cast<const unsigned long long*>(a.cuts + 8 * kMaxCtas) : 0ull;
  auto there = [&](int y) {  // stretch y has units
    return !holes || W * (unsigned)y / (unsigned)ctas < W * (unsigned)(y + 1) / (unsigned)ctas;
  };
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
  constexpr int kMost = (kMaxCtas + 31) / 32;
  float2 part[kMost];
  float big = -INFINITY;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int y = from + 32 * k + lane;
    part[k] = y <= to && there(y) ? ml[(int64_t)(y == from ? first_slot : 2 * y) * kRowsA + row] : make_float2(-INFINITY, 0.f);
    big = fmaxf(big, part[k].x);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    float w = part[k].x != -INFINITY ? ex2(part[k].x - big) : 0.f;
    if (w == 0.f && part[k].x != -INFINITY) w = 1e-45f;  // an infinity that is seen keeps its place in the sum
    sum += w * part[k].y;
    if (from + 32 * k + lane <= to) weight[warp][32 * k + lane] = w;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  __syncwarp();
  constexpr int kE = D / 32;
  float acc[kE] = {};
  for (int y = from; y <= to; y += 4) {
    float w[4], o[4][kE];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = y + k <= to ? weight[warp][y + k - from] : 0.f;
      const float* src = a.part_o + ((int64_t)(y + k == from ? first_slot : 2 * (y + k)) * kRowsA + row) * D + lane * kE;
#pragma unroll
      for (int e = 0; e < kE; ++e) o[k][e] = w[k] != 0.f ? src[e] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[e] = fmaf(w[k], o[k][e], acc[e]);
  }
  const int t = c0.y + row / a.group, h = c0.z * a.group + row % a.group;
  const bool empty = sum == 0.f;
  const float inv = empty ? 0.f : 1.f / sum;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + (int64_t)t * a.o_ts + (int64_t)h * a.o_hs + lane * kE);
#pragma unroll
  for (int e = 0; e < kE; e += 2) out[e / 2] = empty ? 0u : Num<T>::pack(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && a.lse != nullptr) a.lse[(int64_t)t * a.q_heads + h] = empty ? -INFINITY : (big + log2f(sum)) * 0.6931471805599453f;
}

// The union of a block's page lists: of each page its first appearance, with
// the tokens that list it.  A CTA takes the blocks of a request (every
// gridDim.z-th) and a list; a thread compares its entries with all of the
// block's, four at a time from shared memory.
constexpr int kUnionThreads = 128;
__global__ void __launch_bounds__(kUnionThreads) k_list_pages(const __grid_constant__ TreeArgs a) {
  pdl_enter();
  __shared__ __align__(16) int page_s[kMaxListTokens * 64];
  __shared__ int warp_kept[2][kUnionThreads / 32];
  const int r = blockIdx.x, lh = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Plan plan(a);
  const int t0 = plan.tok0(r), n = plan.ntok(r), s = plan.seq(r);
  const int len = plan.len(s), used = (int)(((int64_t)len + a.page - 1) / a.page);
  const int per4 = (a.per + 3) / 4 * 4;  // entries a token in shared memory
  bool bad = false;
  for (int node = blockIdx.z * a.block_tokens; node < n; node += gridDim.z * a.block_tokens) {
    const int m = min(a.block_tokens, n - node), t = t0 + node, total = m * per4;
    for (int e = tid; e < total; e += kUnionThreads) {
      const int tk = e / per4, j = e - tk * per4;
      const int p = j < a.per ? a.pages[((int64_t)(t + tk) * a.lists + lh) * a.per + j] : -1;
      page_s[e] = p >= 0 && p < used ? p : -1;
    }
    __syncthreads();
    ListEntry* out = a.entries + ((int64_t)t * a.lists + (int64_t)lh * m) * a.per;
    int kept = 0;
    for (int base = 0, round = 0; base < total; base += kUnionThreads, ++round) {
      const int e = base + tid;
      const int p = e < total ? page_s[e] : -1;
      const int blk = p >= 0 ? a.bt[r * a.bt_stride + p] : -1;
      uint32_t tokens = 0;
      int first = total;
      for (int tk = m - 1; tk >= 0; --tk) {
        const int4* row = reinterpret_cast<const int4*>(page_s + tk * per4);
        uint32_t hit = 0;
        for (int j = 0; j < per4 / 4; ++j) {
          const int4 x = row[j];
          const int k = x.x == p ? 0 : x.y == p ? 1 : x.z == p ? 2 : x.w == p ? 3 : -1;
          if (k >= 0) {
            if (!hit) first = tk * per4 + 4 * j + k;
            hit = 1;
          }
        }
        tokens |= hit << tk;
      }
      bool take = p >= 0 && first == e;
      if (p >= 0 && (blk < 0 || blk >= a.num_blocks)) bad = true, take = false;
      const uint32_t b = __ballot_sync(0xFFFFFFFFu, take);
      if (lane == 0) warp_kept[round & 1][warp] = __popc(b);
      __syncthreads();
      int at = kept;
#pragma unroll
      for (int w = 0; w < kUnionThreads / 32; ++w) {
        if (w < warp) at += warp_kept[round & 1][w];
        kept += warp_kept[round & 1][w];
      }
      if (take) out[at + __popc(b & ((1u << lane) - 1u))] = ListEntry{blk, p, tokens, 0};
    }
    if (tid == 0) a.counts[(int64_t)t * a.lists + lh] = kept;
    __syncthreads();  // page_s is used up
  }
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
    const int64_t blocks = ((int64_t)a.num_tokens + a.block_tokens - 1) / a.block_tokens;
    const unsigned z = (unsigned)std::max<int64_t>(1, std::min<int64_t>(64, blocks / a.num_reqs));  // CTAs a request and list
    launch_pdl(k_list_pages, dim3((unsigned)a.num_reqs, (unsigned)a.lists, z), dim3(kUnionThreads), 0, s, a);
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
  a.group_inv = (65536u + a.group - 1) / a.group;
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
