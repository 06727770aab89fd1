// Block tables, slot maps, positions and tree masks from request lengths.
//
// Two exclusive sums over the requests place everything: the step's tokens
// (cu_tokens) and the blocks taken from the free list.  One launch, no
// scratch: every CTA walks all requests in chunks of kChunk, scans both
// sums in shared memory, and fills the chunk's tokens and table entries that
// are its own (tokens in slices of equal length, taken blocks interleaved).
// The walk is repeated in every CTA because it is short (a chunk of 1,024
// requests is three 4 KB loads from L2 and one scan) while a second launch
// that waits for the first costs more than a small call: 4.5 us for 512 tokens
// of 64 trees, all latency.  A million tokens of 1,021 requests take 12.7 us,
// where HBM would take 2.0 for their 13 MB: there the instructions set the pace
// (61% of the issue slots): the scan in 64 bits in each of 608 CTAs, a search for
// each four tokens, a division by the page size a token.
#include "idx_common.cuh"
#include "idx_internal.h"

namespace idx {
namespace {

constexpr int kThreadsS = 256;
constexpr int kPerThread = 4;
constexpr int kChunk = kThreadsS * kPerThread;
constexpr int kTreeNodes = 64;  // bits of a mask

struct SlotArgs {
  const int32_t *ctx_lens, *new_lens, *owned;
  int32_t num_reqs;
  int32_t* bt;
  int64_t bt_stride;
  int32_t max_blocks;
  const int32_t* free_blocks;
  int32_t num_free;
  const int32_t* cursor;
  int64_t num_blocks;
  int32_t page;
  const int32_t* parents;
  int32_t num_tokens;
  int32_t *cu, *seq, *pages_out, *cursor_out, *pos;
  int64_t* slots;
  uint64_t* mask;
  int32_t* status;
  bool wide;  // the tokens' outputs are 16-byte aligned
};

// Greatest i in [0, n) with key[i] <= x; key[0] <= x, key non-decreasing.
__device__ __forceinline__ int last_le(const long long* key, int n, long long x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (key[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// kPer: consecutive tokens a thread takes at a time
template <int kPer>
__global__ void __launch_bounds__(kThreadsS) k_build_slots(const __grid_constant__ SlotArgs a) {
  pdl_enter();
  __shared__ long long tok0[kChunk];  // first token of each request of the chunk
  __shared__ long long blk0[kChunk];  // first taken block, counted from the cursor
  __shared__ int ctx_s[kChunk], own_s[kChunk], need_s[kChunk];
  __shared__ long long warp_tok[kThreadsS / 32], warp_blk[kThreadsS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long cap = a.num_tokens;
  // slices of whole kPer
  const long long pers = (cap + kPer - 1) / kPer;
  const long long t_lo = kPer * (pers * blockIdx.x / gridDim.x), t_hi = min(cap, kPer * (pers * (blockIdx.x + 1) / gridDim.x));
  const int cursor = min(max(*a.cursor, 0), a.num_free);
  long long tok_sum = 0, blk_sum = 0;  // of the chunks before
  int bits = 0;

  for (int base = 0; base < a.num_reqs; base += kChunk) {
    const int n = min(kChunk, a.num_reqs - base);
    long long tk[kPerThread], bk[kPerThread], tk_all = 0, bk_all = 0;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const int i = tid * kPerThread + e;
      long long fresh = 0, take = 0;
      if (i < n) {
        const int ctx = max(a.ctx_lens[base + i], 0), own = min(max(a.owned[base + i], 0), a.max_blocks);
        fresh = max(a.new_lens[base + i], 0);
        const long long pages = (ctx + fresh + a.page - 1) / a.page;
        const int need = (int)min(pages, (long long)a.max_blocks);
        take = max(0, need - own);
        ctx_s[i] = ctx, own_s[i] = own, need_s[i] = need;
      }
      tk[e] = tk_all, bk[e] = bk_all;
      tk_all += fresh, bk_all += take;
    }
    long long ti = tk_all, bi = bk_all;  // inclusive over the warp's threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xFFFFFFFFu, ti, o), y = __shfl_up_sync(0xFFFFFFFFu, bi, o);
      if (lane >= o) ti += x, bi += y;
    }
    if (lane == 31) warp_tok[warp] = ti, warp_blk[warp] = bi;
    __syncthreads();
    long long tw = 0, bw = 0, tok_all = 0, blk_all = 0;
#pragma unroll
    for (int w = 0; w < kThreadsS / 32; ++w) {
      if (w < warp) tw += warp_tok[w], bw += warp_blk[w];
      tok_all += warp_tok[w], blk_all += warp_blk[w];
    }
    const long long t0 = tok_sum + tw + ti - tk_all, b0 = blk_sum + bw + bi - bk_all;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const int i = tid * kPerThread + e;
      if (i < n) tok0[i] = t0 + tk[e], blk0[i] = b0 + bk[e];
    }
    __syncthreads();

    // per request: one CTA a chunk, turn by turn
    if ((base / kChunk) % gridDim.x == blockIdx.x) {
      for (int i = tid; i < n; i += kThreadsS) {
        const int r = base + i;
        const long long fresh = max(a.new_lens[r], 0), total = ctx_s[i] + fresh;
        a.cu[r] = (int)min(tok0[i], cap);
        a.seq[r] = (int)min(total, 0x7FFFFFFFll);
        const long long take = max(0, need_s[i] - own_s[i]);
        const long long got = min(take, max(0ll, (long long)a.num_free - cursor - blk0[i]));
        a.pages_out[r] = own_s[i] + (int)got;
        if (got < take) bits |= IDX_ST_NO_BLOCKS;
        if (total > (long long)a.max_blocks * a.page) bits |= IDX_ST_LEN_CLAMPED;
      }
    }
    // taken blocks into the table
    for (long long k = (long long)blockIdx.x * kThreadsS + tid; k < blk_all; k += (long long)gridDim.x * kThreadsS) {
      const int i = last_le(blk0, n, blk_sum + k);
      const long long at = blk_sum + k;
      const long long col = own_s[i] + (at - blk0[i]);
      const long long src = cursor + at;
      a.bt[(base + i) * a.bt_stride + col] = src < a.num_free ? a.free_blocks[src] : -1;
    }
    // the tokens of this CTA's slice, kPer a thread: one search, and a load of
    // a block id where the page changes
    const long long lo = max(t_lo, tok_sum), hi = min(t_hi, tok_sum + tok_all);
    for (long long t4 = lo / kPer * kPer + kPer * tid; t4 < hi; t4 += kPer * kThreadsS) {
      const long long from = max(t4, lo);
      int i = last_le(tok0, n, from), r_at = -1;
      uint32_t pg_at = 0;
      int64_t block = -1;
      int64_t slot[kPer] = {};
      int pos[kPer] = {};
      uint64_t mask[kPer] = {};
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const long long t = t4 + e;
        if (t < lo || t >= hi) continue;
        while (i + 1 < n && tok0[i + 1] <= t) ++i;
        const int node = (int)(t - tok0[i]);
        const uint32_t place = (uint32_t)ctx_s[i] + (uint32_t)node;  // below 2^32
        const uint32_t pg = place / (uint32_t)a.page;
        if (i != r_at || pg != pg_at) {
          r_at = i, pg_at = pg, block = -1;
          if (pg < (uint32_t)own_s[i]) {
            block = a.bt[(int64_t)(base + i) * a.bt_stride + pg];
          } else if (pg < (uint32_t)need_s[i]) {
            const long long src = cursor + blk0[i] + (pg - (uint32_t)own_s[i]);
            if (src < a.num_free) block = a.free_blocks[src];
          }
          if (block < -1 || block >= a.num_blocks) {
            bits |= IDX_ST_BLOCK_OOR;
            block = -1;
          }
        }
        slot[e] = block < 0 ? -1 : block * a.page + (place - pg * (uint32_t)a.page);
        int depth = node;
        if (a.parents != nullptr) {
          // up the tree: a parent below its child's index, so the walk ends
          uint64_t m = 0;
          if (node < kTreeNodes) {
            depth = -1;
            for (int j = node; j >= 0;) {
              m |= 1ull << j;
              ++depth;
              const int up = a.parents[tok0[i] + j];
              if (up < -1 || up >= j) bits |= IDX_ST_BAD_TREE;
              j = up >= -1 && up < j ? up : -1;
            }
          } else {
            bits |= IDX_ST_BAD_TREE;
          }
          mask[e] = m;
        }
        pos[e] = (int)min((long long)ctx_s[i] + depth, 0x7FFFFFFFll);
      }
      bool written = false;
      if (kPer == 4 && a.wide && t4 >= lo && t4 + 4 <= hi) {
        written = true;
        *reinterpret_cast<int4*>(a.pos + t4) = make_int4(pos[0], pos[1 % kPer], pos[2 % kPer], pos[3 % kPer]);
        reinterpret_cast<longlong2*>(a.slots + t4)[0] = make_longlong2(slot[0], slot[1 % kPer]);
        reinterpret_cast<longlong2*>(a.slots + t4)[1] = make_longlong2(slot[2 % kPer], slot[3 % kPer]);
        if (a.mask != nullptr) {
          reinterpret_cast<ulonglong2*>(a.mask + t4)[0] = make_ulonglong2(mask[0], mask[1 % kPer]);
          reinterpret_cast<ulonglong2*>(a.mask + t4)[1] = make_ulonglong2(mask[2 % kPer], mask[3 % kPer]);
        }
      }
      if (!written) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const long long t = t4 + e;
          if (t < lo || t >= hi) continue;
          a.pos[t] = pos[e], a.slots[t] = slot[e];
          if (a.mask != nullptr) a.mask[t] = mask[e];
        }
      }
    }
    tok_sum += tok_all, blk_sum += blk_all;
    __syncthreads();  // the chunk's arrays are used up
  }

  if (blockIdx.x == 0 && tid == 0) {
    a.cu[a.num_reqs] = (int)min(tok_sum, cap);
    *a.cursor_out = (int)min(cursor + blk_sum, (long long)a.num_free);
    if (tok_sum > cap) bits |= IDX_ST_LEN_CLAMPED;
  }
  // a padded batch's tail
  for (long long t = max(t_lo, tok_sum) + tid; t < t_hi; t += kThreadsS) {
    a.slots[t] = -1;
    a.pos[t] = 0;
    if (a.mask != nullptr) a.mask[t] = 0;
  }
  if (bits) report(a.status, bits);
}

}  // namespace
}  // namespace idx

extern "C" int idx_build_slots(const int32_t* ctx_lens, const int32_t* new_lens, const int32_t* owned_pages,
                               int32_t num_reqs, int32_t* block_table, int64_t bt_stride, int32_t max_blocks,
                               const int32_t* free_blocks, int32_t num_free, const int32_t* free_cursor,
                               int64_t num_blocks, int32_t page_tokens, const int32_t* parents, int32_t num_tokens,
                               int32_t* cu_tokens, int32_t* seq_lens, int32_t* pages_out, int32_t* cursor_out,
                               int32_t* positions, int64_t* slots, uint64_t* tree_mask, int32_t* status,
                               void* stream) {
  using namespace idx;
  if (num_reqs < 0 || num_tokens < 0 || max_blocks < 0 || num_free < 0 || num_blocks < 0 || page_tokens < 1 ||
      bt_stride < max_blocks)
    return IDX_E_BAD_SHAPE;
  if (num_reqs > 65535) return IDX_E_TOO_LARGE;
  if (!cu_tokens || !free_cursor || !cursor_out) return IDX_E_NULL_PTR;
  if (num_reqs > 0 && (!ctx_lens || !new_lens || !owned_pages || !seq_lens || !pages_out)) return IDX_E_NULL_PTR;
  if (num_reqs > 0 && max_blocks > 0 && !block_table) return IDX_E_NULL_PTR;
  if (num_free > 0 && !free_blocks) return IDX_E_NULL_PTR;
  if (num_tokens > 0 && (!positions || !slots)) return IDX_E_NULL_PTR;
  if (num_tokens > 0 && (parents == nullptr) != (tree_mask == nullptr)) return IDX_E_NULL_PTR;
  if (free_cursor == cursor_out || (num_reqs > 0 && (owned_pages == pages_out || ctx_lens == seq_lens)))
    return IDX_E_BAD_SHAPE;
  for (const void* p : {(const void*)ctx_lens, (const void*)new_lens, (const void*)owned_pages,
                        (const void*)block_table, (const void*)free_blocks, (const void*)free_cursor,
                        (const void*)parents, (const void*)cu_tokens, (const void*)seq_lens, (const void*)pages_out,
                        (const void*)cursor_out, (const void*)positions, (const void*)status})
    if (!aligned(p, 4)) return IDX_E_MISALIGNED;
  if (!aligned(slots, 8) || !aligned(tree_mask, 8)) return IDX_E_MISALIGNED;
  int rc;
  if ((rc = check_device()) != IDX_OK) return rc;
  SlotArgs a{ctx_lens,  new_lens, owned_pages, num_reqs,   block_table, bt_stride, max_blocks, free_blocks,
             num_free,  free_cursor, num_blocks, page_tokens, parents,  num_tokens, cu_tokens, seq_lens,
             pages_out, cursor_out,  positions,  slots,       tree_mask, status,
             aligned(positions, 16) && aligned(slots, 16) && aligned(tree_mask, 16)};
  // a wave of CTAs (four an SM), a token a thread as long as that takes them
  // all, else four (a million tokens: 12.7 us against 16.5, and 6.2 against 4.6
  // for 512, whose loads follow one another)
  const int wave = 4 * max(device_sms(), 1);
  if (num_tokens <= wave * kThreadsS)
    launch_pdl(k_build_slots<1>, dim3(max(1, (num_tokens + kThreadsS - 1) / kThreadsS)), dim3(kThreadsS), 0, (cudaStream_t)stream, a);
  else
    launch_pdl(k_build_slots<4>, dim3(wave), dim3(kThreadsS), 0, (cudaStream_t)stream, a);
  return launch_result();
}
