// Attention of a round's tokens over a shared prefix and each request's own
// pages of a paged key/value cache: for query token i of request r and head h,
//   x_j = scale q . k_j over the prefix's keys and the request's keys up to the
//   token's own position, out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),
//   lse = m + ln sum_j e^(x_j - m), m = max_j x_j.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace dspark {

struct AttnParams {
  int R, T, Hq, Hkv, page, n_pages, max_pages, prefix_len;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int32_t* prefix_pages;
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* kv_len;
  float rate;  // scale log2(e)
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
};

// One warp a (token, query head): the running maximum and sum of the softmax over one key at a time.
template <int D>
__global__ void __launch_bounds__(256) attention_rows_kernel(AttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (int r = threadIdx.x; r < p.R; r += blockDim.x)
      if (p.q_start[r] < 0 || p.q_start[r + 1] < p.q_start[r] || p.q_start[r + 1] > p.T || p.kv_len[r] < 0 ||
          p.kv_len[r] > (long long)p.max_pages * p.page)
        set_status(p.status, DSPARK_ERR_RANGE);
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (long long)p.T * p.Hq) return;
  const int t = (int)(row / p.Hq), hq = (int)(row % p.Hq), h = hq / (p.Hq / p.Hkv);
  int lo = 0, hi = p.R;
  while (lo < hi) {  // the first request that ends after t
    const int mid = (lo + hi) >> 1;
    if (p.q_start[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  if (lo >= p.R || t < p.q_start[lo]) return;
  const int r = lo, n = p.q_start[r + 1] - p.q_start[r];
  const long long len = min((long long)p.kv_len[r], (long long)p.max_pages * p.page);
  const long long seen = max(0ll, min(len, len - n + (t - p.q_start[r]) + 1));
  float q[E], o[E] = {}, m = -INFINITY, z = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(p.q[row * D + lane * E + e]);
  for (int part = 0; part < 2; ++part) {
    const long long keys = part ? seen : p.prefix_len;
    const int32_t* pages = part ? p.table + (size_t)r * p.max_pages : p.prefix_pages;
    for (long long j = 0; j < keys; ++j) {
      const int pg = pages[j / p.page];
      if (pg < 0 || pg >= p.n_pages) { set_status(p.status, DSPARK_ERR_RANGE); continue; }
      const size_t at = (((size_t)pg * p.page + j % p.page) * p.Hkv + h) * D + lane * E;
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x = fmaf(q[e], __bfloat162float(p.k[at + e]), x);
      x = warp_sum(x) * p.rate;
      const float mn = fmaxf(m, x), a = exp2f(m - mn), w = exp2f(x - mn);
      m = mn;
      z = z * a + w;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * __bfloat162float(p.v[at + e]);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) p.out[row * D + lane * E + e] = __float2bfloat16_rn(z > 0.f ? o[e] / z : 0.f);
  if (p.lse && lane == 0) p.lse[row] = z > 0.f ? (m + log2f(z)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_attention_workspace_bytes(int32_t R, int32_t T, int32_t n_heads, int32_t n_kv_heads,
                                                   int32_t head_dim) {
  if (R < 1 || T < 0 || n_heads < 1 || n_kv_heads < 1 || head_dim < 1) return 0;
  return 256;
}

extern "C" dspark_status dspark_prefix_attention(int32_t R, int32_t T, int32_t n_heads, int32_t n_kv_heads,
                                                 int32_t head_dim, int32_t page_size, int32_t n_pages,
                                                 int32_t max_pages, int32_t prefix_len, const void* q,
                                                 const void* k_cache, const void* v_cache, const int32_t* prefix_pages,
                                                 const int32_t* block_table, const int32_t* q_start,
                                                 const int32_t* kv_len, float scale, void* out, float* lse,
                                                 void* workspace, size_t workspace_bytes, dspark_stream_t stream) {
  note_launches(0);
  if (R < 1 || T < 0 || n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > 128 ||
      (head_dim != 64 && head_dim != 128) || page_size < 16 || page_size > 4096 || (page_size & (page_size - 1)) != 0 ||
      n_pages < 1 || max_pages < 1 || prefix_len < 0 || !(scale > 0.f) || !isfinite(scale))
    return DSPARK_ERR_INVALID_ARG;
  if (!q || !k_cache || !v_cache || (prefix_len > 0 && !prefix_pages) || !block_table || !q_start || !kv_len || !out)
    return DSPARK_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
       reinterpret_cast<uintptr_t>(out)) & 15)
    return DSPARK_ERR_INVALID_ARG;
  const size_t need = dspark_attention_workspace_bytes(R, T, n_heads, n_kv_heads, head_dim);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < need)
    return DSPARK_ERR_WORKSPACE;
  if (T == 0) return DSPARK_OK;
  AttnParams p{R, T, n_heads, n_kv_heads, page_size, n_pages, max_pages, prefix_len,
               (const __nv_bfloat16*)q, (const __nv_bfloat16*)k_cache, (const __nv_bfloat16*)v_cache, prefix_pages,
               block_table, q_start, kv_len, scale * 1.4426950408889634f, (__nv_bfloat16*)out, lse,
               static_cast<uint32_t*>(workspace)};
  const int grid = ceil_div((long long)T * n_heads, 8);
  if (head_dim == 128) attention_rows_kernel<128><<<grid, 256, 0, (cudaStream_t)stream>>>(p);
  else attention_rows_kernel<64><<<grid, 256, 0, (cudaStream_t)stream>>>(p);
  note_launches(1);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
