// Attention of a step's tokens over the paged cache (simple form).
#include <cuda_bf16.h>

#include "idx_common.cuh"
#include "idx_internal.h"

namespace idx {
namespace {

constexpr int kThreadsA = 128;

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
  int32_t num_reqs, num_tokens, q_heads, kv_heads;
  const uint64_t* mask;
  const int32_t* pages;
  int32_t lists, per;
  float scale;
  void* out;
  int64_t o_ts, o_hs;
  float* lse;
  int32_t* status;
};

__device__ __forceinline__ float tf(__half x) { return __half2float(x); }
__device__ __forceinline__ float tf(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsA) k_tree_simple(const __grid_constant__ TreeArgs a) {
  pdl_enter();
  __shared__ float qs[D], ps[kThreadsA], red[8];
  __shared__ int64_t rows[kThreadsA];
  const int tid = threadIdx.x;
  const int t = blockIdx.x, h = blockIdx.y, hk = h / (a.q_heads / a.kv_heads);
  T* out = static_cast<T*>(a.out) + t * a.o_ts + h * a.o_hs;
  int r = 0;
  while (r < a.num_reqs && !(a.cu[r] <= t && t < a.cu[r + 1])) ++r;
  int n = 0, node = 0, seq = 0, ctx = 0;
  if (r < a.num_reqs) n = a.cu[r + 1] - a.cu[r], node = t - a.cu[r], seq = max(0, a.seq_lens[r]), ctx = seq - n;
  const uint64_t bits = a.mask != nullptr ? a.mask[t] : 0;
  for (int i = tid; i < D; i += kThreadsA) qs[i] = tf(static_cast<const T*>(a.q)[t * a.q_ts + h * a.q_hs + i]);
  const int used = min((int64_t)(seq + a.page - 1) / a.page, (int64_t)a.max_blocks);
  if (tid == 0 && (int64_t)seq > (int64_t)a.max_blocks * a.page) report(a.status, IDX_ST_LEN_CLAMPED);
  const int entries = a.pages != nullptr ? a.per : used;
  const int32_t* list = a.pages != nullptr ? a.pages + ((int64_t)t * a.lists + hk / (a.kv_heads / a.lists)) * a.per : nullptr;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int e = 0; e < entries; ++e) {
    const int pg = list != nullptr ? list[e] : e;
    if (pg < 0 || pg >= used) continue;
    bool again = false;
    for (int f = 0; list != nullptr && f < e; ++f) again |= list[f] == pg;
    if (again) continue;
    const int64_t blk = a.bt[r * a.bt_stride + pg];
    if (blk < 0 || blk >= a.num_blocks) {
      if (tid == 0) report(a.status, IDX_ST_BLOCK_OOR);
      continue;
    }
    for (int b = 0; b < a.page; b += kThreadsA) {
      __syncthreads();
      const int off = b + tid;
      const int64_t place = (int64_t)pg * a.page + off;
      const int64_t j = place - ctx;
      const bool seen = off < a.page && place < seq &&
                        (j < 0 || (a.mask != nullptr ? j < 64 && ((bits >> j) & 1) : j <= node));
      const int64_t row = blk * a.c_bs + off * a.c_ts + hk * a.c_hs;
      float s = -INFINITY;
      if (seen) {
        float acc = 0.f;
        for (int d = 0; d < D; ++d) acc += qs[d] * tf(static_cast<const T*>(a.kc)[row + d]);
        s = acc * a.scale;
      }
      rows[tid] = seen ? row : -1;
      float mx = s;
      for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
      if ((tid & 31) == 0) red[tid >> 5] = mx;
      __syncthreads();
      mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
      const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.f : mn;
      const float p = seen ? expf(s - base) : 0.f;
      ps[tid] = p;
      float sum = p;
      for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
      if ((tid & 31) == 0) red[4 + (tid >> 5)] = sum;
      __syncthreads();
      const float f = m == -INFINITY ? 0.f : expf(m - base);
      l = l * f + red[4] + red[5] + red[6] + red[7];
      o *= f;
      m = mn;
      if (tid < D)
        for (int x = 0; x < kThreadsA; ++x)
          if (rows[x] >= 0) o += ps[x] * tf(static_cast<const T*>(a.vc)[rows[x] + tid]);
    }
  }
  if (tid < D) put(out + tid, l == 0.f ? 0.f : o / l);
  if (tid == 0 && a.lse != nullptr) a.lse[(int64_t)t * a.q_heads + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace
}  // namespace idx

extern "C" size_t idx_tree_attention_workspace_bytes(int32_t num_reqs, int32_t num_tokens, int32_t q_heads,
                                                     int32_t kv_heads, int32_t head_dim, int32_t page_lists,
                                                     int32_t pages_per_list) {
  if (num_reqs <= 0 || num_tokens <= 0 || q_heads <= 0 || kv_heads <= 0 || head_dim <= 0 || page_lists < 0 || pages_per_list < 0)
    return 0;
  return 256;
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
      num_blocks < 0 || bt_stride < max_blocks)
    return IDX_E_BAD_SHAPE;
  if (head_dim != 64 && head_dim != 128) return IDX_E_BAD_SHAPE;
  if (page_tokens != 16 && page_tokens != 32 && page_tokens != 64 && (page_tokens < 128 || page_tokens % 128 != 0))
    return IDX_E_BAD_SHAPE;
  if (dtype != IDX_BF16 && dtype != IDX_F16) return IDX_E_BAD_SHAPE;
  if (pages != nullptr && (page_lists < 1 || kv_heads % page_lists != 0 || pages_per_list < 1)) return IDX_E_BAD_SHAPE;
  for (int64_t s : {q_token_stride, q_head_stride, c_block_stride, c_token_stride, c_head_stride, o_token_stride, o_head_stride})
    if (s < 0 || s % 8 != 0) return IDX_E_BAD_SHAPE;
  if ((q_heads > 1 && o_head_stride < head_dim) || (num_tokens > 1 && o_token_stride < head_dim)) return IDX_E_BAD_SHAPE;
  if (num_reqs > 65535 || q_heads / kv_heads > 128 || kv_heads > 65535 || (pages != nullptr && pages_per_list > 64) ||
      num_blocks > 0x7FFFFFFF)
    return IDX_E_TOO_LARGE;
  if (num_tokens == 0) return IDX_OK;
  if (!q || !out || (num_reqs > 0 && (!seq_lens || !cu_tokens))) return IDX_E_NULL_PTR;
  if (num_reqs > 0 && max_blocks > 0 && num_blocks > 0 && (!block_table || !k_cache || !v_cache)) return IDX_E_NULL_PTR;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(cu_tokens, 4) || !aligned(tree_mask, 8) || !aligned(pages, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 256) || !aligned(status, 4))
    return IDX_E_MISALIGNED;
  const size_t need = idx_tree_attention_workspace_bytes(num_reqs, num_tokens, q_heads, kv_heads, head_dim, pages ? page_lists : 0,
                                                         pages ? pages_per_list : 0);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return IDX_E_WORKSPACE;
  int rc;
  if ((rc = check_device()) != IDX_OK) return rc;
  TreeArgs a{q, q_token_stride, q_head_stride, k_cache, v_cache, num_blocks, page_tokens, c_block_stride, c_token_stride,
             c_head_stride, block_table, bt_stride, max_blocks, seq_lens, cu_tokens, num_reqs, num_tokens, q_heads, kv_heads,
             tree_mask, pages, page_lists, pages_per_list, scale, out, o_token_stride, o_head_stride, lse, status};
  const dim3 grid(num_tokens, q_heads), block(kThreadsA);
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == IDX_BF16 && head_dim == 128) launch_pdl(k_tree_simple<__nv_bfloat16, 128>, grid, block, 0, s, a);
  else if (dtype == IDX_BF16) launch_pdl(k_tree_simple<__nv_bfloat16, 64>, grid, block, 0, s, a);
  else if (head_dim == 128) launch_pdl(k_tree_simple<__half, 128>, grid, block, 0, s, a);
  else launch_pdl(k_tree_simple<__half, 64>, grid, block, 0, s, a);
  return launch_result();
}
