// Paged key/value cache upkeep around a round: pages and slots of the tokens
// that enter the cache (the anchor and the scheduled draft tokens of every
// request), and the copy of their keys and values into it.
//
// page_plan_kernel  request r holds have = ceil(c / p) pages for its c cached
//   tokens and needs ceil((c + n) / p) for n more (page size p). The missing
//   ones are taken from the list of free pages in request order, so a request's
//   first entry is the sum of the missing pages before it, and its first token's
//   index the sum of n before it. A request that the token capacity cuts asks for
//   what is left of it, the later ones for nothing. Each CTA plans kPlanReqs requests and forms
//   both sums over all earlier requests itself: at 8,192 requests that reads at
//   most 64 KB from L2 in a CTA, and no CTA waits for another. The list ends at its first
//   negative id, which each CTA looks for among the entries that its requests and the
//   earlier ones ask for (35 KB there). Bound by latency:
//   128 requests, 1,144 tokens 8 us a call (the launch's host side; 5.9 on the GPU), 8,192 requests,
//   73,720 tokens 12 us (1.05 MB, 0.16 us of bandwidth; 10.8 on the GPU, of which the list's end 0.9,
//   looked for an entry at a time 1.8).
// kv_append_kernel  one 16-byte piece of one token's key and value row a thread
//   step; bound by bytes (each read once and written once): 15,904 tokens of 8 heads
//   of 128 bf16 (130 MB) 23 us, 5.6 TB/s, 0.83 of the measured copy bandwidth.
#include <algorithm>
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace dspark {

constexpr int kPlanThreads = 512;
constexpr int kPlanReqs = 128;

struct PlanParams {
  int R, page, max_pages, n_free, capacity;
  const int32_t* cached;
  const int32_t* fresh;
  const int32_t* free_pages;
  int32_t* table;
  int32_t* q_start;
  int32_t* kv_len;
  int32_t* positions;
  long long* slots;
  int32_t* used;
  uint32_t* status;
};

__device__ __forceinline__ long long block_sum_ll(long long v, long long* sh) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane == 0) sh[w] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < nw; ++i) v += sh[i];
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(PlanParams p) {
  __shared__ long long sh[32];
  __shared__ long long s_tok[kPlanReqs + 1], s_pg[kPlanReqs + 1];  // token / free-list starts of this CTA's requests
  __shared__ long long s_warp[kPlanReqs / 32];
  __shared__ int s_c[kPlanReqs], s_have[kPlanReqs];
  __shared__ int s_end;  // where the list of free pages ends: at its first negative id
  const int tid = threadIdx.x, r0 = blockIdx.x * kPlanReqs, nr = min(kPlanReqs, p.R - r0);
  bool bad = false;
  if (tid == 0) s_end = p.n_free;
  // Every CTA looks for the list's end among the entries that its requests and the earlier ones ask for, four at a time: the
  // first 4 kPlanThreads in flight with the lengths. (Entries past what is asked for do no harm.)
  const int lead = (int)((16 - (reinterpret_cast<uintptr_t>(p.free_pages) & 15)) & 15) / 4;  // before the first 16-byte boundary
  auto entries = [&](int i) {
    const long long at = lead + 4ll * i;
    if (at + 4 <= p.n_free) return __ldg(reinterpret_cast<const int4*>(p.free_pages + at));
    auto one = [&](long long k) { return k < p.n_free ? __ldg(p.free_pages + k) : 0; };
    return make_int4(one(at), one(at + 1), one(at + 2), one(at + 3));
  };
  auto first_negative = [&](const int4& ids, int i) {
    const int at = ids.x < 0 ? 0 : ids.y < 0 ? 1 : ids.z < 0 ? 2 : 3;
    return (ids.x | ids.y | ids.z | ids.w) < 0 ? lead + 4 * i + at : INT_MAX;
  };
  auto ends_at = [&](int at) {  // the lowest of a warp's
    at = __reduce_min_sync(0xffffffffu, at);
    if ((tid & 31) == 0 && at < INT_MAX) atomicMin(&s_end, at);
  };
  const int4 head = entries(tid);
  const int loose = tid < min(lead, p.n_free) ? __ldg(p.free_pages + tid) : 0;
  auto lengths = [&](int r, int& c, int& n) {
    c = __ldg(p.cached + r);
    n = __ldg(p.fresh + r);
    bad |= c < 0 || n < 0;
    c = max(c, 0);
    n = max(n, 0);
  };
  // lengths are below 2^31, their sums below 2^32: 32-bit divisions, the quotients formed once a request
  const uint32_t page = (uint32_t)p.page;
  auto pages_of = [&](uint32_t x) { return x / page + (x % page != 0 ? 1u : 0u); };
  auto missing = [&](int c, int n) { return (long long)pages_of((uint32_t)c + (uint32_t)n) - (long long)pages_of((uint32_t)c); };
  long long tok = 0, pg = 0;
#pragma unroll 4
  for (int r = tid; r < r0; r += kPlanThreads) {
    int c, n;
    lengths(r, c, n);
    tok += n;
    pg += missing(c, n);
  }
  if (r0 > 0) {
    tok = block_sum_ll(tok, sh);
    pg = block_sum_ll(pg, sh);
  }
  // This CTA's requests: running sums over four warps. Tokens first: the capacity may cut a request's.
  auto running = [&](long long a, long long first, long long* to) {  // to[i] = first + the sum of a over requests 0..i-1
    if (tid < kPlanReqs) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, o);
        if ((tid & 31) >= o) a += x;
      }
      if ((tid & 31) == 31) s_warp[tid >> 5] = a;
    }
    __syncthreads();
    if (tid < kPlanReqs) {
      for (int w = 0; w < (tid >> 5); ++w) a += s_warp[w];
      to[tid + 1] = first + a;
      if (tid == 0) to[0] = first;
    }
    __syncthreads();
  };
  int c = 0, n = 0;
  if (tid < nr) lengths(r0 + tid, c, n);
  running(n, tok, s_tok);
  long long miss = 0;
  if (tid < nr) {
    const int fit = (int)max(0ll, min((long long)n, p.capacity - s_tok[tid]));
    miss = missing(c, fit);
    s_c[tid] = c;
    s_have[tid] = (int)pages_of((uint32_t)c);
    const long long end = (long long)c + fit;
    bad |= end > 0x7fffffffll;
    p.kv_len[r0 + tid] = (int)min(end, 0x7fffffffll);
  }
  ends_at(loose < 0 ? tid : first_negative(head, tid));  // (s_end was set before the barriers of the first running sum)
  running(miss, pg, s_pg);
  const int asked = (int)min(s_pg[nr], (long long)p.n_free);
  if (asked > lead + 4 * kPlanThreads) {
    int at = INT_MAX;
#pragma unroll 4
    for (int i = kPlanThreads + tid; lead + 4ll * i < asked; i += kPlanThreads) at = min(at, first_negative(entries(i), i));
    ends_at(at);
    __syncthreads();
  }
  const int list_end = s_end;
  // new entries of the block table: -1 where the list has run out
  bool full = false;
  const int warp = tid >> 5, lane = tid & 31;
  for (int i = warp; i < nr; i += kPlanThreads / 32) {
    const int have = s_have[i];
    const long long n_new = s_pg[i + 1] - s_pg[i];
    full |= have + n_new > p.max_pages;
    for (long long j = lane; j < n_new && have + j < p.max_pages; j += 32) {
      const long long at = s_pg[i] + j;
      const int id = at < list_end ? __ldg(p.free_pages + at) : -1;  // (a list may end early: dspark_page_collect's do)
      full |= id < 0;
      p.table[(size_t)(r0 + i) * p.max_pages + have + j] = id;
    }
  }
  if (tid < nr) p.q_start[r0 + tid] = (int)min(s_tok[tid], (long long)p.capacity);
  const long long t_end = s_tok[nr];
  full |= t_end > p.capacity;
  // the tokens of this CTA's requests
  for (long long t = s_tok[0] + tid; t < min(t_end, (long long)p.capacity); t += kPlanThreads) {
    int lo = 0, hi = nr - 1;  // the last request that starts at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_tok[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    const uint32_t pos = (uint32_t)s_c[lo] + (uint32_t)(t - s_tok[lo]);
    const uint32_t col = pos / page;
    int id = -1;
    if (col < (uint32_t)p.max_pages) {
      if (col < (uint32_t)s_have[lo]) {
        id = __ldg(p.table + (size_t)(r0 + lo) * p.max_pages + col);
      } else {
        const long long at = s_pg[lo] + col - s_have[lo];
        if (at < list_end) id = __ldg(p.free_pages + at);
      }
    }
    p.positions[t] = (int)pos;
    p.slots[t] = id < 0 ? -1ll : (long long)id * p.page + pos % page;
  }
  // pages are taken up to the CTA in which the capacity is reached (pg of the later ones is not their start: a request
  // that the capacity cuts counts in full there)
  if (tid == 0 && (r0 == 0 || s_tok[0] < p.capacity) && (t_end >= p.capacity || r0 + nr == p.R))
    p.used[0] = (int)min(s_pg[nr], (long long)list_end);
  if (r0 + nr == p.R) {
    if (tid == 0) p.q_start[p.R] = (int)min(t_end, (long long)p.capacity);
    for (long long t = t_end + tid; t < p.capacity; t += kPlanThreads) {
      p.positions[t] = -1;
      p.slots[t] = -1ll;
    }
  }
  if (bad) set_status(p.status, DSPARK_ERR_RANGE);
  if (full) set_status(p.status, DSPARK_ERR_CAPACITY);
}

// ---------------------------------------------------------------------------
template <class Tv>
__global__ void __launch_bounds__(256)
    kv_append_kernel(long long n_vec, int per_row, const Tv* __restrict__ k, const Tv* __restrict__ v,
                     const long long* __restrict__ slots, long long n_slots, Tv* __restrict__ k_cache,
                     Tv* __restrict__ v_cache, uint32_t* status) {
  // piece i is piece `off` of token t; both advance by a fixed step, so the divisions are made once
  const long long step = (long long)gridDim.x * blockDim.x;
  long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long t_step = step / per_row, t0 = i / per_row;
  const int off_step = (int)(step - t_step * per_row);
  int off = (int)(i - t0 * per_row);
  for (long long t = t0; i < n_vec; i += step) {
    const Tv a = k[i], b = v[i];  // read whatever the slot says: in flight together with it
    const long long slot = __ldg(slots + t);
    if (slot >= n_slots) {
      set_status(status, DSPARK_ERR_RANGE);
    } else if (slot >= 0) {
      k_cache[slot * per_row + off] = a;
      v_cache[slot * per_row + off] = b;
    }
    t += t_step;
    off += off_step;
    if (off >= per_row) { off -= per_row; ++t; }
  }
}

}  // namespace dspark

using namespace dspark;

extern "C" dspark_status dspark_page_plan(int32_t R, int32_t page_size, int32_t max_pages, int32_t n_free,
                                          int32_t capacity, const int32_t* cached_len, const int32_t* new_len,
                                          const int32_t* free_pages, int32_t* block_table, int32_t* q_start,
                                          int32_t* kv_len, int32_t* positions, int64_t* slots, int32_t* used,
                                          void* workspace, size_t workspace_bytes, dspark_stream_t stream) {
  note_launches(0);
  if (R < 1 || page_size < 1 || max_pages < 1 || n_free < 0 || capacity < 0 || !cached_len || !new_len ||
      (n_free > 0 && !free_pages) || !block_table || !q_start || !kv_len || (capacity > 0 && (!positions || !slots)) ||
      !used)
    return DSPARK_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < 256)
    return DSPARK_ERR_WORKSPACE;
  PlanParams p{R, page_size, max_pages, n_free, capacity, cached_len, new_len, free_pages, block_table, q_start,
               kv_len, positions, reinterpret_cast<long long*>(slots), used, static_cast<uint32_t*>(workspace)};
  page_plan_kernel<<<ceil_div(R, kPlanReqs), kPlanThreads, 0, (cudaStream_t)stream>>>(p);
  note_launches(1);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

extern "C" dspark_status dspark_kv_append(int32_t T, int32_t n_kv_heads, int32_t head_dim, int32_t dtype, const void* k,
                                          const void* v, const int64_t* slots, int64_t n_slots, void* k_cache,
                                          void* v_cache, void* workspace, size_t workspace_bytes,
                                          dspark_stream_t stream) {
  note_launches(0);
  if (T < 0 || n_kv_heads < 1 || head_dim < 1 || (long long)n_kv_heads * head_dim > (1 << 24) ||
      (dtype != DSPARK_FP32 && dtype != DSPARK_BF16) || n_slots < 0 || n_slots > (1ll << 40))
    return DSPARK_ERR_INVALID_ARG;
  if (T > 0 && (!k || !v || !slots || !k_cache || !v_cache)) return DSPARK_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < 256)
    return DSPARK_ERR_WORKSPACE;
  if (T == 0) return DSPARK_OK;
  const int elem = dtype == DSPARK_BF16 ? 2 : 4;
  const int row = n_kv_heads * head_dim * elem;
  const uintptr_t at = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
                       reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache);
  const int unit = ((at | (uintptr_t)row) & 15) == 0 ? 16 : elem;  // bytes a thread copies at a time
  const long long n_vec = (long long)T * (row / unit);
  const int grid = (int)std::min<long long>((n_vec + 255) / 256, 152 * 16);
  uint32_t* status = static_cast<uint32_t*>(workspace);
  const long long* sl = reinterpret_cast<const long long*>(slots);
  cudaStream_t s = (cudaStream_t)stream;
  if (unit == 16)
    kv_append_kernel<<<grid, 256, 0, s>>>(n_vec, row / unit, (const uint4*)k, (const uint4*)v, sl, (long long)n_slots,
                                          (uint4*)k_cache, (uint4*)v_cache, status);
  else if (unit == 4)
    kv_append_kernel<<<grid, 256, 0, s>>>(n_vec, row / unit, (const uint32_t*)k, (const uint32_t*)v, sl,
                                          (long long)n_slots, (uint32_t*)k_cache, (uint32_t*)v_cache, status);
  else
    kv_append_kernel<<<grid, 256, 0, s>>>(n_vec, row / unit, (const uint16_t*)k, (const uint16_t*)v, sl,
                                          (long long)n_slots, (uint16_t*)k_cache, (uint16_t*)v_cache, status);
  note_launches(1);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
