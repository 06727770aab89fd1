// What becomes of cached rows and pages after a step: rows of the drafts that
// stand are moved together, requests fork, pages go back to the free list.
//
// A cache is a set of planes (layers, keys and values) of the same blocks, a
// token's row in a plane contiguous; several caches (the index-K pages' codes
// and scales among them) go through one call.
//
// k_settle: the i-th node that stands, number n_i of its request, goes to the
// place of node 1 + i.  A path has n_i >= 1 + i, so a row is never written
// before it was read where the rows are taken in order; every thread has one
// piece of a plane's row and takes the path's nodes in order, kMoveS rows
// loaded before they are stored, and no thread needs another's.
//
// k_fork: one launch; the blocks that the forks take follow from a count over
// the forks before, formed in each CTA (at most IDX_MAX_FORKS).
//
// k_release, k_push: a page's holders beyond the first are counted in refs.
// Each release takes one off; what falls below zero goes back.  The order in
// which atomics come would show in the free list, so a second kernel collects
// the blocks below zero by id: a cluster of CTAs counts its stretches, then
// writes, and the result is the same each time.
//
// All three are bound by latency, or, with many layers, by HBM: 64 forks of 16
// requests over 48 layers take 98 us (363 MB written; the parents' pages, 84 MB, are
// read 2.5 times, the other forks find them in L2: 66 at HBM's rate with one reading
// each, 107 with one a fork), 64 trees of 24 settled over 48 layers 8.2 us (12.7 with
// eight rows in flight a thread and 256 threads), 187,000 pages of 1,021 requests
// released 12.4 us (15 with a cluster of 8); the smallest calls 4 to 6 us.
#include "idx_common.cuh"
#include "idx_internal.h"

namespace idx {
namespace {

constexpr int kThreadsC = 256;
constexpr int kThreadsM = 128;  // of k_settle
constexpr int kMoveS = 4;      // rows in flight a thread
constexpr int kStageS = 64;    // nodes of a path looked up together
constexpr int kPartsF = 16;    // CTAs a page of a plane, at most
constexpr int kThreadsU = 1024;
constexpr int kClusterU = 16;
constexpr int kUnrollU = 16;   // words of refs in flight a warp

struct Cache {
  char* base;
  int64_t plane_stride, block_stride, token_stride;  // bytes
  int32_t planes, row_bytes, piece, pieces;          // piece: bytes of an access; pieces of a row
};
struct Caches {
  Cache c[IDX_MAX_CACHES];
  int32_t num;
  int32_t planes;      // of all
  int64_t per_token;   // pieces of a token's rows in all planes
  int64_t num_blocks;
  int32_t page;
};

template <typename F>
__device__ __forceinline__ void by_piece(int piece, F&& f) {
  switch (piece) {
    case 16: f(uint4{}); break;
    case 8: f(uint2{}); break;
    case 4: f(uint32_t{}); break;
    case 2: f(uint16_t{}); break;
    default: f(uint8_t{}); break;
  }
}

struct SettleArgs {
  const int64_t* slots;
  const int32_t *cu, *out_tokens, *out_nodes, *accepted, *ctx;
  int32_t num_reqs, num_tokens, max_out;
  int32_t* ctx_out;
  int32_t* counts;
  int64_t counts_stride;
  int32_t vocab;
  int32_t* status;
};

__global__ void __launch_bounds__(kThreadsM) k_settle(const __grid_constant__ SettleArgs a, const __grid_constant__ Caches cs) {
  pdl_enter();
  __shared__ int from_block[kStageS], from_tok[kStageS], to_block[kStageS], to_tok[kStageS];
  const int r = blockIdx.y, tid = threadIdx.x;
  const int t0 = max(0, min(a.cu[r], a.num_tokens)), n = max(0, min(a.cu[r + 1], a.num_tokens) - t0);
  const int stands = max(0, min(a.accepted[r], min(n, a.max_out) - 1));
  if (blockIdx.x == 0) {
    if (tid == 0) a.ctx_out[r] = a.ctx[r] + (n > 0 ? 1 + stands : 0);
    if (a.counts != nullptr && n > 0)
      for (int i = tid; i <= stands; i += kThreadsM) {
        const int x = a.out_tokens[(int64_t)r * a.max_out + i];
        if (x >= 0 && x < a.vocab) atomicAdd(a.counts + (int64_t)r * a.counts_stride + x, 1);
      }
  }
  // this thread's piece of a row
  int64_t at = (int64_t)blockIdx.x * kThreadsM + tid;
  int c = 0;
  while (c < cs.num && at >= (int64_t)cs.c[c].planes * cs.c[c].pieces) at -= (int64_t)cs.c[c].planes * cs.c[c].pieces, ++c;
  const bool live = c < cs.num;
  const Cache& k = cs.c[live ? c : 0];
  const int plane = live ? (int)(at / k.pieces) : 0, piece = live ? (int)(at - (int64_t)plane * k.pieces) : 0;
  char* base = k.base + plane * k.plane_stride + (int64_t)piece * k.piece;
  const int64_t places = cs.num_blocks * cs.page;
  for (int i0 = 0; i0 < stands; i0 += kStageS) {
    const int m = min(kStageS, stands - i0);
    __syncthreads();
    if (tid < m) {
      const int i = i0 + tid, node = a.out_nodes[(int64_t)r * a.max_out + i];
      int64_t from = -1, to = -1;
      if (node < i + 1 || node >= n) {
        if (blockIdx.x == 0) report(a.status, IDX_ST_BAD_TREE);
      } else if (node != i + 1 && cs.num > 0) {  // (without caches no row has a place, and slots may be NULL)
        from = a.slots[t0 + node], to = a.slots[t0 + 1 + i];
        if ((from >= places || to >= places) && blockIdx.x == 0) report(a.status, IDX_ST_BLOCK_OOR);
        if (from < 0 || to < 0 || from >= places || to >= places) from = -1;
      }
      from_block[tid] = from < 0 ? -1 : (int)(from / cs.page), from_tok[tid] = from < 0 ? 0 : (int)(from % cs.page);
      to_block[tid] = from < 0 ? -1 : (int)(to / cs.page), to_tok[tid] = from < 0 ? 0 : (int)(to % cs.page);
    }
    __syncthreads();
    if (!live) continue;
    by_piece(k.piece, [&](auto one) {
      using P = decltype(one);
      for (int j = 0; j < m; j += kMoveS) {
        P x[kMoveS];
#pragma unroll
        for (int u = 0; u < kMoveS; ++u)
          if (j + u < m && from_block[j + u] >= 0)
            x[u] = *reinterpret_cast<const P*>(base + from_block[j + u] * k.block_stride + from_tok[j + u] * k.token_stride);
#pragma unroll
        for (int u = 0; u < kMoveS; ++u)
          if (j + u < m && from_block[j + u] >= 0) *reinterpret_cast<P*>(base + to_block[j + u] * k.block_stride + to_tok[j + u] * k.token_stride) = x[u];
      }
    });
  }
}

struct ForkArgs {
  const int32_t *parents, *children;
  int32_t num_forks, num_reqs;
  int32_t *ctx, *owned, *bt;
  int64_t bt_stride;
  int32_t max_blocks;
  int32_t* refs;
  const int32_t* free_blocks;
  int32_t num_free;
  const int32_t* cursor;
  int32_t* cursor_out;
  int32_t* status;
  int32_t parts;
};

__global__ void __launch_bounds__(kThreadsC) k_fork(const __grid_constant__ ForkArgs a, const __grid_constant__ Caches cs) {
  pdl_enter();
  extern __shared__ uint32_t bits[];  // requests that are a child, then those that no fork may make
  __shared__ int sums[kThreadsC / 32][2];
  const int tid = threadIdx.x, fork = blockIdx.y, words = (a.num_reqs + 31) / 32;
  uint32_t* child = bits;
  uint32_t* bad = bits + words;
  for (int w = tid; w < 2 * words; w += kThreadsC) bits[w] = 0;
  __syncthreads();
  for (int j = tid; j < a.num_forks; j += kThreadsC) {
    const int c = a.children[j], p = a.parents[j];
    if (c >= 0 && c < a.num_reqs && (atomicOr(&child[c >> 5], 1u << (c & 31)) >> (c & 31) & 1u)) atomicOr(&bad[c >> 5], 1u << (c & 31));
    if (c != -1 && p >= 0 && p < a.num_reqs) atomicOr(&bad[p >> 5], 1u << (p & 31));
  }
  __syncthreads();
  // tokens of fork j; -1: it is not made
  auto length = [&](int j, int& report_bits) {
    const int c = a.children[j], p = a.parents[j];
    if (c == -1) return -1;  // none
    if (c < 0 || c >= a.num_reqs || p < 0 || p >= a.num_reqs || (bad[c >> 5] >> (c & 31) & 1u)) {
      report_bits |= IDX_ST_BAD_FORK;
      return -1;
    }
    const int own = min(max(a.owned[p], 0), a.max_blocks), ctx = max(a.ctx[p], 0);
    if (ctx > (int64_t)own * cs.page) {
      report_bits |= IDX_ST_LEN_CLAMPED;
      return own * cs.page;
    }
    return ctx;
  };
  int before = 0, all = 0, said = 0;
  for (int j = tid; j < a.num_forks; j += kThreadsC) {
    const int len = length(j, said), takes = len > 0 && len % cs.page != 0;
    all += takes, before += j < fork ? takes : 0;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o), all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  if ((tid & 31) == 0) sums[tid >> 5][0] = before, sums[tid >> 5][1] = all;
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int w = 0; w < kThreadsC / 32; ++w) before += sums[w][0], all += sums[w][1];
  const int cursor = min(max(*a.cursor, 0), a.num_free);
  const bool first = blockIdx.x == 0;
  if (first && fork == 0) {
    if (tid == 0) *a.cursor_out = (int)min((int64_t)cursor + all, (int64_t)a.num_free);
    if (said) report(a.status, said);
  }
  if (fork >= a.num_forks) return;
  int none = 0;
  const int len = length(fork, none);
  if (len < 0) return;
  const int p = a.parents[fork], c = a.children[fork];
  const int full = len / cs.page, rest = len - full * cs.page;
  const int32_t* row = a.bt + p * a.bt_stride;
  int block = -1;
  if (rest > 0) {
    const int64_t src = (int64_t)cursor + before;
    if (src < a.num_free) block = a.free_blocks[src];
    if (block < 0 || block >= cs.num_blocks) {  // no block for the last page: not made
      if (first && tid == 0) {
        report(a.status, src < a.num_free ? IDX_ST_BLOCK_OOR : IDX_ST_NO_BLOCKS);
        a.ctx[c] = 0, a.owned[c] = 0;
      }
      return;
    }
  }
  if (first) {
    int32_t* to = a.bt + c * a.bt_stride;
    for (int i = tid; i < full; i += kThreadsC) {
      const int id = row[i];
      to[i] = id;
      if (id >= 0 && id < cs.num_blocks) atomicAdd(a.refs + id, 1);
      else report(a.status, IDX_ST_BLOCK_OOR);
    }
    if (tid == 0) {
      if (rest > 0) to[full] = block;
      a.ctx[c] = len, a.owned[c] = full + (rest > 0);
    }
  }
  if (rest == 0) return;
  // the last page's rows, plane by plane
  const int last = row[full];
  if (last < 0 || last >= cs.num_blocks) {
    if (first && tid == 0) report(a.status, IDX_ST_BLOCK_OOR);
    return;
  }
  const int part = blockIdx.x % a.parts;
  for (int plane = blockIdx.x / a.parts; plane < cs.planes; plane += gridDim.x / a.parts) {
    int ci = 0, pl = plane;
    while (pl >= cs.c[ci].planes) pl -= cs.c[ci].planes, ++ci;
    const Cache& k = cs.c[ci];
    const char* src = k.base + pl * k.plane_stride + last * k.block_stride;
    char* dst = k.base + pl * k.plane_stride + block * k.block_stride;
    by_piece(k.piece, [&](auto one) {
      using P = decltype(one);
      const uint32_t pieces = (uint32_t)k.pieces, total = (uint32_t)rest * pieces;  // a page's rows of a plane stay below 4 GB
      const bool dense = k.token_stride == k.row_bytes;
      // (one piece a thread and turn: two took 105 us for 64 forks over 48 layers, four 140)
      for (int64_t i = part * kThreadsC + tid; i < total; i += a.parts * kThreadsC) {
        const uint32_t tok = dense ? 0u : (uint32_t)i / pieces;
        const int64_t off = tok * k.token_stride + (i - (int64_t)tok * pieces) * (int64_t)sizeof(P);
        *reinterpret_cast<P*>(dst + off) = *reinterpret_cast<const P*>(src + off);
      }
    });
  }
}

struct ReleaseArgs {
  const int32_t *keep, *owned, *bt;
  int64_t bt_stride;
  int32_t max_blocks, num_reqs, page;
  int32_t* refs;
  int64_t num_blocks;
  int32_t* free_blocks;
  int32_t num_free;
  const int32_t* cursor;
  int32_t *cursor_out, *pages_out, *status;
};

__global__ void __launch_bounds__(kThreadsC) k_release(const __grid_constant__ ReleaseArgs a) {
  pdl_enter();
  const int r = blockIdx.y;
  const int own = min(max(a.owned[r], 0), a.max_blocks);
  const int kept = (int)min((int64_t)own, ((int64_t)max(a.keep[r], 0) + a.page - 1) / a.page);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.pages_out[r] = kept;
  bool oor = false;
  const int32_t* row = a.bt + r * a.bt_stride;
  for (int i = kept + (int)(blockIdx.x * kThreadsC + threadIdx.x); i < own; i += (int)(gridDim.x * kThreadsC)) {
    const int id = row[i];
    if (id >= 0 && id < a.num_blocks) atomicSub(a.refs + id, 1);
    else oor |= id != -1;
  }
  if (oor) report(a.status, IDX_ST_BLOCK_OOR);
}

// Blocks below zero, by id, into the free list's entries before the cursor.
__global__ void __launch_bounds__(kThreadsU) k_push(const __grid_constant__ ReleaseArgs a) {
  pdl_enter();
  __shared__ int warp_sum[kThreadsU / 32];
  __shared__ unsigned long long cta_sum[kClusterU];
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // stretches of whole words of 32, one a warp of the cluster, kUnrollU words in flight
  const int64_t all_words = (a.num_blocks + 31) / 32, w = (int64_t)rank * (kThreadsU / 32) + warp, warps = kClusterU * (kThreadsU / 32);
  const int64_t lo = all_words * w / warps * 32, hi = min(all_words * (w + 1) / warps * 32, a.num_blocks);
  auto load = [&](int64_t b, int (&v)[kUnrollU]) {
#pragma unroll
    for (int e = 0; e < kUnrollU; ++e) v[e] = b + 32 * e + lane < hi ? a.refs[b + 32 * e + lane] : 0;
  };
  int mine = 0;
  for (int64_t b = lo; b < hi; b += 32 * kUnrollU) {
    int v[kUnrollU];
    load(b, v);
#pragma unroll
    for (int e = 0; e < kUnrollU; ++e) mine += v[e] < 0;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
  if (lane == 0) warp_sum[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    int sum = warp_sum[lane];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    // every CTA of the cluster runs before its shared memory is written
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (lane < kClusterU)
      asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.u64 [a], %2;\n\t}" ::"r"(smem_u32(&cta_sum[rank])),
                   "r"(lane), "l"((unsigned long long)sum)
                   : "memory");
    __syncwarp();
  } else {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  int64_t total = 0, at = 0;
  for (int c = 0; c < kClusterU; ++c) total += (int64_t)cta_sum[c], at += c < (int)rank ? (int64_t)cta_sum[c] : 0;
  for (int k = 0; k < warp; ++k) at += warp_sum[k];
  const int cursor = min(max(*a.cursor, 0), a.num_free);
  const int64_t begin = cursor - total;  // below 0: more than were taken
  if (rank == 0 && tid == 0) {
    *a.cursor_out = (int)max((int64_t)0, begin);
    if (begin < 0) report(a.status, IDX_ST_BAD_OUTPUT);
  }
  at += begin;
  for (int64_t b = lo; b < hi; b += 32 * kUnrollU) {
    int v[kUnrollU];
    load(b, v);
#pragma unroll
    for (int e = 0; e < kUnrollU; ++e) {
      const uint32_t gone = __ballot_sync(0xFFFFFFFFu, v[e] < 0);
      const int64_t to = at + __popc(gone & ((1u << lane) - 1u));
      if (v[e] < 0) {
        if (to >= 0) a.free_blocks[to] = (int)(b + 32 * e + lane);
        a.refs[b + 32 * e + lane] = 0;
      }
      at += __popc(gone);
    }
  }
}

// The caches as the kernels take them; IDX_OK or what is wrong with them.
int take_caches(const idx_cache* caches, int32_t num, int64_t num_blocks, int32_t page, Caches* out) {
  if (num < 0 || num_blocks < 0 || page < 1) return IDX_E_BAD_SHAPE;
  if (num > IDX_MAX_CACHES || num_blocks > 0x7FFFFFFF) return IDX_E_TOO_LARGE;
  if (num > 0 && !caches) return IDX_E_NULL_PTR;
  out->num = 0, out->planes = 0, out->per_token = 0, out->num_blocks = num_blocks, out->page = page;
  for (int i = 0; i < num; ++i) {
    const idx_cache& c = caches[i];
    if (c.planes < 0 || c.row_bytes < 0 || c.plane_stride < 0 || c.block_stride < 0 || c.token_stride < 0) return IDX_E_BAD_SHAPE;
    if (c.planes == 0 || c.row_bytes == 0 || num_blocks == 0) continue;
    if (!c.base) return IDX_E_NULL_PTR;
    // different planes, blocks and tokens must not share bytes
    if ((c.planes > 1 && c.plane_stride < c.row_bytes) || (num_blocks > 1 && c.block_stride < c.row_bytes) || (page > 1 && c.token_stride < c.row_bytes))
      return IDX_E_BAD_SHAPE;
    if ((int64_t)page * c.row_bytes >= (1ll << 32)) return IDX_E_TOO_LARGE;
    if (out->planes > 0x7FFFFFFF - c.planes) return IDX_E_TOO_LARGE;
    int64_t fit = (int64_t)(reinterpret_cast<uintptr_t>(c.base) | (uintptr_t)c.plane_stride | (uintptr_t)c.block_stride | (uintptr_t)c.token_stride |
                            (uintptr_t)c.row_bytes | 16u);
    const int piece = (int)(fit & -fit);  // the lowest bit set: what all are multiples of
    out->c[out->num++] = Cache{static_cast<char*>(c.base), c.plane_stride, c.block_stride, c.token_stride, c.planes, c.row_bytes, piece, c.row_bytes / piece};
    out->planes += c.planes;
    out->per_token += (int64_t)c.planes * (c.row_bytes / piece);
  }
  return IDX_OK;
}

}  // namespace
}  // namespace idx

extern "C" int idx_settle_drafts(const idx_cache* caches, int32_t num_caches, int64_t num_blocks, int32_t page_tokens, const int64_t* slots,
                                 const int32_t* cu_tokens, int32_t num_reqs, int32_t num_tokens, const int32_t* out_tokens,
                                 const int32_t* out_nodes, int32_t max_out, const int32_t* num_accepted, const int32_t* ctx_lens, int32_t* ctx_out,
                                 int32_t* counts, int64_t counts_stride, int32_t vocab, int32_t* status, void* stream) {
  using namespace idx;
  if (num_reqs < 0 || num_tokens < 0 || max_out < 1) return IDX_E_BAD_SHAPE;
  if (counts && (vocab < 1 || (num_reqs > 1 && counts_stride < vocab))) return IDX_E_BAD_SHAPE;
  if (num_reqs > 65535) return IDX_E_TOO_LARGE;
  Caches cs{};
  int rc = take_caches(caches, num_caches, num_blocks, page_tokens, &cs);
  if (rc != IDX_OK) return rc;
  if (num_reqs == 0) return IDX_OK;
  if (!cu_tokens || !out_nodes || !num_accepted || !ctx_lens || !ctx_out || (counts && !out_tokens) || (num_tokens > 0 && cs.num > 0 && !slots))
    return IDX_E_NULL_PTR;
  for (const void* p : {(const void*)cu_tokens, (const void*)out_tokens, (const void*)out_nodes, (const void*)num_accepted, (const void*)ctx_lens,
                        (const void*)ctx_out, (const void*)counts, (const void*)status})
    if (!aligned(p, 4)) return IDX_E_MISALIGNED;
  if (!aligned(slots, 8)) return IDX_E_MISALIGNED;
  const int64_t ctas = (cs.per_token + kThreadsM - 1) / kThreadsM;
  if (ctas > 0x7FFFFFFF) return IDX_E_TOO_LARGE;
  if ((rc = check_device()) != IDX_OK) return rc;
  const SettleArgs a{slots, cu_tokens, out_tokens, out_nodes, num_accepted, ctx_lens, num_reqs, num_tokens, max_out, ctx_out, counts, counts_stride, vocab, status};
  launch_pdl(k_settle, dim3((unsigned)(ctas > 0 ? ctas : 1), (unsigned)num_reqs), dim3(kThreadsM), 0, (cudaStream_t)stream, a, cs);
  return launch_result();
}

extern "C" int idx_fork_pages(const idx_cache* caches, int32_t num_caches, int64_t num_blocks, int32_t page_tokens, const int32_t* parents,
                              const int32_t* children, int32_t num_forks, int32_t* ctx_lens, int32_t* owned_pages, int32_t num_reqs,
                              int32_t* block_table, int64_t bt_stride, int32_t max_blocks, int32_t* refs, const int32_t* free_blocks,
                              int32_t num_free, const int32_t* free_cursor, int32_t* cursor_out, int32_t* status, void* stream) {
  using namespace idx;
  if (num_forks < 0 || num_reqs < 0 || max_blocks < 0 || bt_stride < max_blocks || num_free < 0) return IDX_E_BAD_SHAPE;
  if (num_reqs > 65535 || num_forks > IDX_MAX_FORKS) return IDX_E_TOO_LARGE;
  Caches cs{};
  int rc = take_caches(caches, num_caches, num_blocks, page_tokens, &cs);
  if (rc != IDX_OK) return rc;
  if ((num_forks > 0 && (!parents || !children)) || !free_cursor || !cursor_out || (num_free > 0 && !free_blocks)) return IDX_E_NULL_PTR;
  if (num_reqs > 0 && (!ctx_lens || !owned_pages || (max_blocks > 0 && !block_table) || (num_blocks > 0 && !refs))) return IDX_E_NULL_PTR;
  if (free_cursor == cursor_out) return IDX_E_BAD_SHAPE;
  for (const void* p : {(const void*)parents, (const void*)children, (const void*)ctx_lens, (const void*)owned_pages, (const void*)block_table,
                        (const void*)refs, (const void*)free_blocks, (const void*)free_cursor, (const void*)cursor_out, (const void*)status})
    if (!aligned(p, 4)) return IDX_E_MISALIGNED;
  if ((rc = check_device()) != IDX_OK) return rc;
  // a page of a plane for several CTAs while that leaves SMs without any
  const int sms = max(device_sms(), 1), planes = max(cs.planes, 1);
  const int parts = (int)max((int64_t)1, min((int64_t)kPartsF, (int64_t)sms * 4 / ((int64_t)planes * max(num_forks, 1))));
  const ForkArgs a{parents, children, num_forks, num_reqs, ctx_lens, owned_pages, block_table, bt_stride, max_blocks, refs, free_blocks, num_free,
                   free_cursor, cursor_out, status, parts};
  const size_t smem = (size_t)((num_reqs + 31) / 32) * 8;
  const int x = parts * (int)min((int64_t)planes, max((int64_t)1, (int64_t)sms * 64 / max(num_forks, 1)));
  launch_pdl(k_fork, dim3((unsigned)x, (unsigned)max(num_forks, 1)), dim3(kThreadsC), smem, (cudaStream_t)stream, a, cs);
  return launch_result();
}

extern "C" int idx_release_pages(const int32_t* keep_lens, const int32_t* owned_pages, int32_t num_reqs, const int32_t* block_table,
                                 int64_t bt_stride, int32_t max_blocks, int32_t* refs, int64_t num_blocks, int32_t* free_blocks, int32_t num_free,
                                 const int32_t* free_cursor, int32_t* cursor_out, int32_t* pages_out, int32_t page_tokens, int32_t* status,
                                 void* stream) {
  using namespace idx;
  if (num_reqs < 0 || max_blocks < 0 || bt_stride < max_blocks || num_blocks < 0 || num_free < 0 || page_tokens < 1) return IDX_E_BAD_SHAPE;
  if (num_reqs > 65535 || num_blocks > 0x7FFFFFFF) return IDX_E_TOO_LARGE;
  if (!free_cursor || !cursor_out || (num_free > 0 && !free_blocks) || (num_blocks > 0 && !refs)) return IDX_E_NULL_PTR;
  if (num_reqs > 0 && (!keep_lens || !owned_pages || !pages_out || (max_blocks > 0 && !block_table))) return IDX_E_NULL_PTR;
  if (free_cursor == cursor_out || (num_reqs > 0 && (owned_pages == pages_out || keep_lens == pages_out))) return IDX_E_BAD_SHAPE;
  for (const void* p : {(const void*)keep_lens, (const void*)owned_pages, (const void*)block_table, (const void*)refs, (const void*)free_blocks,
                        (const void*)free_cursor, (const void*)cursor_out, (const void*)pages_out, (const void*)status})
    if (!aligned(p, 4)) return IDX_E_MISALIGNED;
  int rc;
  if ((rc = check_device()) != IDX_OK) return rc;
  const ReleaseArgs a{keep_lens, owned_pages, block_table, bt_stride, max_blocks, num_reqs, page_tokens, refs, num_blocks, free_blocks, num_free,
                      free_cursor, cursor_out, pages_out, status};
  cudaStream_t s = (cudaStream_t)stream;
  if (num_reqs > 0) {
    const int x = max(1, min((max_blocks + kThreadsC - 1) / kThreadsC, max(1, 8 * max(device_sms(), 1) / num_reqs)));
    launch_pdl(k_release, dim3((unsigned)x, (unsigned)num_reqs), dim3(kThreadsC), 0, s, a);
    if ((rc = launch_result()) != IDX_OK) return rc;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kClusterU);
  cfg.blockDim = dim3(kThreadsU);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kClusterU, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaFuncSetAttribute(k_push, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  cudaLaunchKernelEx(&cfg, k_push, a);
  return launch_result();
}
