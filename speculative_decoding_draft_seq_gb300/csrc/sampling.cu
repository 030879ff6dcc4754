// The target's sampling rule (temperature, top-k, top-p, min-p) on rows of
// logits: one token a row from a given uniform, or the row with every entry
// outside the kept set masked.
//
// Weights of a row with maximum M at temperature T: w = 2^((l - M) log2(e)/T)
// in float32, each operation rounded once, and their masses the integers
// floor(w 2^40). Sums of masses are integer sums, so they do not depend on an
// order, and every comparison below is exact. With the row sorted by (logit
// descending, index ascending), top-k keeps the first k entries; top-p keeps,
// of these, the entries whose mass before them is below floor(p S), S the mass
// of the top-k set; min-p keeps the entries with w >= min_p. So the kept set is
// a threshold on (logit, index) and one on w. The threshold is found by radix
// selection on the logits' order-preserving integer keys: histograms of counts
// and masses over a shrinking key range.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace dspark {

constexpr int kSThreads = 1024;
constexpr int kSBins = 2048;

struct SampleParams {
  int V;
  const void* logits;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const double* u;
  int32_t* tokens;
  float* prob;
  void* out;
  uint32_t* status;
};

__device__ __forceinline__ uint32_t logit_key(float x) {  // larger logit, larger key; -0 and +0 alike
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ float rule_weight(float x, float M, float rate) {
  return x == -INFINITY ? 0.f : exp2f(__fmul_rn(__fsub_rn(x, M), rate));
}
// floor(x S) for x in [0, 1), x to 53 bits
__device__ __forceinline__ unsigned long long scale_mass(double x, unsigned long long S) {
  if (!(x > 0.0)) x = 0.0;
  if (x > 1.0 - 0x1p-53) x = 1.0 - 0x1p-53;
  return scale_u53((unsigned long long)__double2ull_rz(x * 0x1p53), S);
}

__device__ __forceinline__ unsigned long long block_sum_u64(unsigned long long v, unsigned long long* sh) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane == 0) sh[w] = v;
  __syncthreads();
  v = lane < nw ? sh[lane] : 0ull;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Inclusive scan over the block's threads.
__device__ __forceinline__ unsigned long long block_scan_u64(unsigned long long v, unsigned long long* sh) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) sh[w] = v;
  __syncthreads();
  unsigned long long s = lane < nw ? sh[lane] : 0ull;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  const unsigned long long before = __shfl_sync(0xffffffffu, s, w > 0 ? w - 1 : 0);
  return w > 0 ? v + before : v;
}

struct Threshold {
  uint32_t key;             // the last kept key
  unsigned long long ties;  // entries of this key that are kept, in index order
  unsigned long long count, above;  // entries of this key; the mass of the larger keys
};

// The key at which the running count (by_mass = false) or mass of the row in descending order first
// reaches `target`, among the keys lo..hi.
template <class Tin>
__device__ Threshold select_key(const Tin* row, int V, float M, float rate, bool by_mass, unsigned long long target,
                                uint32_t lo, uint32_t hi, uint32_t* h_cnt, unsigned long long* h_mass,
                                unsigned long long* sh, unsigned long long* s_pick) {
  unsigned long long c_above = 0, m_above = 0;
  const int tid = threadIdx.x;
  for (;;) {
    const uint32_t span = hi - lo;
    const int bits = 32 - __clz(span), shift = bits > 11 ? bits - 11 : 0;
    for (int b = tid; b < kSBins; b += kSThreads) { h_cnt[b] = 0; h_mass[b] = 0; }
    __syncthreads();
    for (int v = tid; v < V; v += kSThreads) {
      const float x = ld_elem(row, v);
      const uint32_t k = logit_key(x);
      if (k < lo || k > hi) continue;
      const uint32_t b = (hi - k) >> shift;
      atomicAdd(&h_cnt[b], 1u);
      atomicAdd(&h_mass[b], fx40(rule_weight(x, M, rate)));
    }
    __syncthreads();
    const unsigned long long c0 = h_cnt[2 * tid], c1 = h_cnt[2 * tid + 1];
    const unsigned long long m0 = h_mass[2 * tid], m1 = h_mass[2 * tid + 1];
    const unsigned long long ci = block_scan_u64(c0 + c1, sh) + c_above, mi = block_scan_u64(m0 + m1, sh) + m_above;
    const unsigned long long end1 = by_mass ? mi : ci, v1 = by_mass ? m1 : c1, v0 = by_mass ? m0 : c0;
    const unsigned long long end0 = end1 - v1, start = end0 - v0;
    if (start < target && end1 >= target) {
      const bool second = end0 < target;
      s_pick[0] = 2 * tid + (second ? 1 : 0);
      s_pick[1] = ci - c1 - (second ? 0 : c0);
      s_pick[2] = mi - m1 - (second ? 0 : m0);
      s_pick[3] = second ? c1 : c0;
    }
    __syncthreads();
    const uint32_t b = (uint32_t)s_pick[0];
    c_above = s_pick[1];
    m_above = s_pick[2];
    const unsigned long long cnt = s_pick[3];
    __syncthreads();
    if (shift == 0) {
      Threshold t;
      t.key = hi - b;
      t.count = cnt;
      t.above = m_above;
      const unsigned long long w = fx40(rule_weight(key_logit(t.key), M, rate));
      t.ties = by_mass ? (target - m_above + w - 1) / w : target - c_above;
      if (t.ties > cnt) t.ties = cnt;
      return t;
    }
    const uint32_t top = hi - (b << shift);
    lo = max(lo, top - ((1u << shift) - 1));
    hi = top;
  }
}

template <class Tin>
__global__ void __launch_bounds__(kSThreads) sampling_rule_kernel(SampleParams p) {
  __shared__ uint32_t h_cnt[kSBins];
  __shared__ unsigned long long h_mass[kSBins];
  __shared__ unsigned long long sh[32], s_pick[4];
  __shared__ float shf[32];
  __shared__ int shi[32];
  const int tid = threadIdx.x, V = p.V;
  const size_t r = blockIdx.x;
  const Tin* row = static_cast<const Tin*>(p.logits) + r * V;
  Tin* out = p.out ? static_cast<Tin*>(p.out) + r * V : nullptr;
  const float T = p.temperature[r];
  // the maximum and its first index
  float M = -INFINITY;
  int at = 0x7fffffff, bad = 0;
  for (int v = tid; v < V; v += kSThreads) {
    const float x = ld_elem(row, v);
    bad |= !(x < INFINITY);
    if (x > M) { M = x; at = v; }
  }
  block_argmax(M, at, shf, shi);
  bad = __syncthreads_or(bad) | (M == -INFINITY);
  if (bad) {  // a NaN or +inf, or nothing finite: no distribution
    if (tid == 0) set_status(p.status, DSPARK_ERR_NONFINITE);
    if (p.tokens && tid == 0) {
      p.tokens[r] = -1;
      if (p.prob) p.prob[r] = 0.f;
    }
    if (out)
      for (int v = tid; v < V; v += kSThreads) out[v] = row[v];
    return;
  }
  M = __fadd_rn(M, 0.f);
  const bool greedy = !(T > 0.f);
  const float rate = fminf(__fdiv_rn(1.4426950408889634f, T), 1e30f);
  uint32_t key = 0;                      // kept: keys above `key`, and `key` itself up to index `cut`
  int cut = V;
  const float min_w = fminf(fmaxf(p.min_p[r], 0.f), 1.f);
  if (greedy) {
    key = logit_key(M);
    cut = at + 1;
  } else {
    const int k = p.top_k[r];
    const float tp = p.top_p[r];
    Threshold th;
    bool have = false;
    const uint32_t hi = logit_key(M);
    uint32_t lo = logit_key(-INFINITY);
    unsigned long long S = 0;
    if (k > 0 && k < V) {
      th = select_key(row, V, M, rate, false, (unsigned long long)k, lo, hi, h_cnt, h_mass, sh, s_pick);
      have = true;
      lo = th.key;
      S = th.above + th.ties * fx40(rule_weight(key_logit(th.key), M, rate));
    }
    if (tp < 1.f) {
      if (!have) {
        for (int v = tid; v < V; v += kSThreads) S += fx40(rule_weight(ld_elem(row, v), M, rate));
        S = block_sum_u64(S, sh);
      }
      const unsigned long long limit = max(1ull, scale_mass((double)fminf(tp, 1.f - 0x1p-24f), S));
      th = select_key(row, V, M, rate, true, limit, lo, hi, h_cnt, h_mass, sh, s_pick);
      have = true;
    }
    if (have) {
      key = th.key;
      if (th.ties < th.count) {  // the index of the last tie that is kept
        const int len = ceil_div(V, kSThreads), b = min(tid * len, V), e = min(b + len, V);
        unsigned long long n = 0;
        for (int v = b; v < e; ++v) n += logit_key(ld_elem(row, v)) == key;
        unsigned long long c = block_scan_u64(n, sh) - n;
        if (c < th.ties && c + n >= th.ties)
          for (int v = b; v < e; ++v)
            if (logit_key(ld_elem(row, v)) == key && ++c == th.ties) s_pick[0] = v + 1;
        __syncthreads();
        cut = (int)s_pick[0];
      }
    }
  }
  auto kept = [&](float x, int v, float w) {
    const uint32_t k = logit_key(x);
    return (k > key || (k == key && v < cut)) && (greedy || w >= min_w) && x > -INFINITY;
  };
  if (out) {
    const Tin lowest = sizeof(Tin) == 2 ? Tin(-3.3895313892515355e38f) : Tin(-3.4028234663852886e38f);
    for (int v = tid; v < V; v += kSThreads) {
      const float x = ld_elem(row, v);
      out[v] = kept(x, v, greedy ? 1.f : rule_weight(x, M, rate)) ? row[v] : lowest;
    }
  }
  if (p.tokens) {
    if (greedy) {
      if (tid == 0) {
        p.tokens[r] = at;
        if (p.prob) p.prob[r] = 1.f;
      }
      return;
    }
    const int len = ceil_div(V, kSThreads), b = min(tid * len, V), e = min(b + len, V);
    unsigned long long m = 0;
    for (int v = b; v < e; ++v) {
      const float x = ld_elem(row, v), w = rule_weight(x, M, rate);
      if (kept(x, v, w)) m += fx40(w);
    }
    const unsigned long long end = block_scan_u64(m, sh), Z = block_sum_u64(m, sh);
    const unsigned long long t = scale_mass(p.u[r], Z);
    unsigned long long c = end - m;
    if (c <= t && end > t) {
      for (int v = b; v < e; ++v) {
        const float x = ld_elem(row, v), w = rule_weight(x, M, rate);
        if (!kept(x, v, w)) continue;
        c += fx40(w);
        if (c > t) {
          p.tokens[r] = v;
          if (p.prob) p.prob[r] = (float)((double)fx40(w) / (double)Z);
          break;
        }
      }
    }
  }
}

static dspark_status sampling_entry(int32_t N, int32_t V, int32_t dtype, const void* logits, const float* temperature,
                                    const int32_t* top_k, const float* top_p, const float* min_p, const double* u,
                                    int32_t* tokens, float* prob, void* out, void* workspace, size_t workspace_bytes,
                                    dspark_stream_t stream) {
  note_launches(0);
  if (N < 0 || V < 1 || V > (1 << 20) || (dtype != DSPARK_FP32 && dtype != DSPARK_BF16)) return DSPARK_ERR_INVALID_ARG;
  if (N > 0 && (!logits || !temperature || !top_k || !top_p || !min_p)) return DSPARK_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < 256)
    return DSPARK_ERR_WORKSPACE;
  if (N == 0) return DSPARK_OK;
  SampleParams p{V, logits, temperature, top_k, top_p, min_p, u, tokens, prob, out, static_cast<uint32_t*>(workspace)};
  if (dtype == DSPARK_BF16)
    sampling_rule_kernel<__nv_bfloat16><<<N, kSThreads, 0, (cudaStream_t)stream>>>(p);
  else
    sampling_rule_kernel<float><<<N, kSThreads, 0, (cudaStream_t)stream>>>(p);
  note_launches(1);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // namespace dspark

using namespace dspark;

extern "C" dspark_status dspark_sample(int32_t N, int32_t V, int32_t dtype, const void* logits, const float* temperature,
                                       const int32_t* top_k, const float* top_p, const float* min_p, const double* u,
                                       int32_t* tokens, float* prob, void* workspace, size_t workspace_bytes,
                                       dspark_stream_t stream) {
  if (N > 0 && (!u || !tokens)) return DSPARK_ERR_INVALID_ARG;
  return sampling_entry(N, V, dtype, logits, temperature, top_k, top_p, min_p, u, tokens, prob, nullptr, workspace,
                        workspace_bytes, stream);
}

extern "C" dspark_status dspark_truncate(int32_t N, int32_t V, int32_t dtype, const void* logits,
                                         const float* temperature, const int32_t* top_k, const float* top_p,
                                         const float* min_p, void* out, void* workspace, size_t workspace_bytes,
                                         dspark_stream_t stream) {
  if (N > 0 && !out) return DSPARK_ERR_INVALID_ARG;
  return sampling_entry(N, V, dtype, logits, temperature, top_k, top_p, min_p, nullptr, nullptr, nullptr, out, workspace,
                        workspace_bytes, stream);
}
