// Verification of drafted tokens against rows of probabilities, from given
// uniforms ("DSpark: Aceleração da inferência de LLM com speculative decoding
// [pdf]" (GeekNews), "Definição do problema"), for any drafter: its rows of
// probabilities are an input, or it has none (its token had probability 1).
//
// Draft x_k stands iff u_k Q_k(x_k) < P_{k-1}(x_k), the product in float64, so that the
// test is the same wherever it is made. The first draft that does not is
// replaced by a draw from w = max(0, fl32(P - Q)) of its row (from P if that has no
// mass); if all stand, one is drawn from the row after the last. The draw is the first v
// whose mass up to and including v exceeds floor(u Z), masses the integers
// floor(min(w, 1) 2^40) and Z their sum: integer sums do not depend on an order.
//
// A cluster of CTAs takes a request. Every CTA walks the request's chain itself (a
// warp, a lane a draft; three dependent loads), then sums a contiguous share of the one row
// that matters, warp by warp; the warps' sums go to all CTAs, and the warp whose
// share holds the token reads that share once more to find it.
#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"
#include "verify_common.cuh"

namespace dspark {

constexpr int kVpThreads = 512;
constexpr int kVpWarps = kVpThreads / 32;
constexpr int kVpMaxCluster = 8;

struct VerifyProbsParams {
  int gamma, V, T, C;
  const void* target;
  const int32_t* q_start;
  const void* draft;  // or null
  const int32_t* tokens;
  const double* u;
  int32_t* out_tokens;
  int32_t* accepted;
  float* p_tok;
  uint32_t* status;
};

// floor(x S) for x in [0, 1), exactly (x has at most 53 bits); below 0 and NaN count as 0, 1 and above as the largest
// value below 1.
__device__ __forceinline__ unsigned long long draw_goal(double x, unsigned long long S) {
  const double k = floor(x * 0x1p53);
  const unsigned long long most = (1ull << 53) - 1;
  return scale_u53(!(k > 0.0) ? 0ull : k >= 0x1p53 ? most : (unsigned long long)k, S);
}

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Entries of the row that is drawn from: the target's, less the drafter's where a draft was rejected.
template <class T>
struct DrawRow {
  static constexpr int E = 16 / sizeof(T);
  const T* p;
  const T* q;    // or null
  int token;     // of a rejected draft without a row of its own: Q is 1 there (else -1)
  __device__ __forceinline__ float at(int v) const {
    float w = ld_elem(p, v);
    if (q) w = __fsub_rn(w, ld_elem(q, v));
    return v == token ? __fsub_rn(w, 1.f) : w;
  }
};

__device__ __forceinline__ unsigned long long mass40(float w) { return fx40(fminf(fmaxf(w, 0.f), 1.f)); }

template <class T>
__global__ void __launch_bounds__(kVpThreads) verify_probs_kernel(VerifyProbsParams p) {
  constexpr int E = 16 / sizeof(T);
  __shared__ unsigned long long sums[2][kVpMaxCluster * kVpWarps];  // one set a pass
  __shared__ int s_start, s_n, s_accepted;
  const int rank = (int)cluster_rank(), C = p.C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster_arrive();
  const size_t r = blockIdx.x / C;
  const T* target = static_cast<const T*>(p.target);
  const T* draft = static_cast<const T*>(p.draft);
  const size_t V = p.V;

  if (warp == 0) {
    const int a = __ldg(p.q_start + r), b = __ldg(p.q_start + r + 1);
    const bool wrong = a < 0 || b < a || b > p.T || b - a - 1 > p.gamma;
    const int n = a < 0 || b < a || b > p.T ? 0 : min(b - a, p.gamma + 1);
    if (wrong && rank == 0 && lane == 0) set_status(p.status, DSPARK_ERR_RANGE);
    int accepted = 0;
    bool go = true;  // no draft rejected so far
    for (int k0 = 0; k0 < p.gamma; k0 += 32) {
      const int k = k0 + lane;
      bool ok = false;
      float pt = 0.f;
      if (k < n - 1) {
        const int x = __ldg(p.tokens + r * p.gamma + k);
        if (x >= 0 && x < p.V) {
          pt = ld_elem(target, (size_t)(a + k) * V + x);
          const float qt = draft ? ld_elem(draft, (r * p.gamma + k) * V + x) : 1.f;
          ok = __dmul_rn(__ldg(p.u + r * (p.gamma + 1) + k), (double)qt) < (double)pt;
          if (rank == 0 && !(fabsf(pt) + fabsf(qt) < INFINITY)) set_status(p.status, DSPARK_ERR_NONFINITE);
        } else if (rank == 0) {
          set_status(p.status, DSPARK_ERR_RANGE);
        }
      }
      if (rank == 0 && k < p.gamma) p.p_tok[r * p.gamma + k] = pt;
      const uint32_t fails = ~__ballot_sync(0xffffffffu, ok);
      if (go) accepted += fails ? __ffs(fails) - 1 : 32;
      go &= fails == 0;
      if (!go && rank != 0) break;  // CTA 0 goes on: it writes the probabilities
    }
    if (lane == 0) {
      s_start = a;
      s_n = n;
      s_accepted = accepted;
    }
  }
  __syncthreads();
  const int n = s_n, A = s_accepted;
  int32_t* out = p.out_tokens + r * (p.gamma + 1);
  if (rank == 0) {
    for (int i = threadIdx.x; i <= p.gamma; i += kVpThreads)
      if (i != A || n == 0) out[i] = i < A ? __ldg(p.tokens + r * p.gamma + i) : -1;
    if (threadIdx.x == 0) p.accepted[r] = A;
  }
  cluster_wait();
  if (n == 0) return;  // (the whole cluster)

  DrawRow<T> row{target + (size_t)(s_start + A) * V, nullptr, -1};
  if (A < n - 1) {
    const int x = __ldg(p.tokens + r * p.gamma + A);
    if (x >= 0 && x < p.V) {
      if (draft) row.q = draft + (r * p.gamma + A) * V;
      else row.token = x;
    }
  }
  const double u = __ldg(p.u + r * (p.gamma + 1) + p.gamma);
  // this warp's share: whole multiples of a warp's step, so that wide loads stay possible
  const int shares = C * kVpWarps;
  const int share = ceil_div(ceil_div(p.V, shares), 32 * E) * 32 * E;
  const int mine = rank * kVpWarps + warp;
  const int v0 = (int)min((long long)mine * share, (long long)p.V), v1 = (int)min((long long)v0 + share, (long long)p.V);

  for (int pass = 0; pass < 2; ++pass) {
    unsigned long long m = 0;
    float finite = 0.f;
    for (int v = v0 + lane; v < v1; v += 32) {
      const float w = row.at(v);
      finite = __fmaf_rn(w, 0.f, finite);
      m += mass40(w);
    }
    if (finite != 0.f) set_status(p.status, DSPARK_ERR_NONFINITE);
    m = warp_sum_u64(m);
    if (lane < C) store_peer(peer_address(&sums[pass][mine], lane), m);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    unsigned long long before = 0, Z = 0;  // the mass of the shares before this one, and of all
    for (int i = lane; i < shares; i += 32) {
      const unsigned long long x = sums[pass][i];
      Z += x;
      if (i < mine) before += x;
    }
    Z = warp_sum_u64(Z);
    before = warp_sum_u64(before);
    if (Z == 0) {  // the same in every warp
      if (pass == 0 && (row.q || row.token >= 0)) {
        row.q = nullptr;
        row.token = -1;
        continue;
      }
      if (rank == 0 && threadIdx.x == 0) {
        out[A] = -1;
        set_status(p.status, DSPARK_ERR_NONFINITE);
      }
      return;
    }
    const unsigned long long goal = draw_goal(u, Z);
    if (goal < before || goal - before >= m) return;
    unsigned long long left = goal - before;
    for (int v = v0; v < v1; v += 32) {
      const unsigned long long x = v + lane < v1 ? mass40(row.at(v + lane)) : 0ull;
      unsigned long long c = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, c > left);
      if (hit) {
        if (lane == 0) out[A] = v + __ffs(hit) - 1;
        return;
      }
      left -= __shfl_sync(0xffffffffu, c, 31);
    }
    return;
  }
}

template <class T>
static cudaError_t launch_verify_probs(const VerifyProbsParams& p, int R, cudaStream_t s) {
  return launch_clusters(verify_probs_kernel<T>, p, (unsigned)R * p.C, p.C, kVpThreads, 0, s);
}

}  // namespace dspark

using namespace dspark;

extern "C" dspark_status dspark_verify_probs(int32_t R, int32_t gamma, int32_t V, int32_t T, int32_t dtype,
                                             const void* target_probs, const int32_t* q_start, const void* draft_probs,
                                             const int32_t* draft_tokens, const double* u, int32_t* out_tokens,
                                             int32_t* accepted_len, float* p_tok, void* workspace,
                                             size_t workspace_bytes, dspark_stream_t stream) {
  note_launches(0);
  if (R < 1 || R > (1 << 24) || gamma < 1 || gamma > (1 << 20) || V < 1 || V > (1 << 20) || T < 0 ||
      (dtype != DSPARK_FP32 && dtype != DSPARK_BF16))
    return DSPARK_ERR_INVALID_ARG;
  if ((T > 0 && !target_probs) || !q_start || !draft_tokens || !u || !out_tokens || !accepted_len || !p_tok)
    return DSPARK_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < 256)
    return DSPARK_ERR_WORKSPACE;
  const VerifyProbsParams p{gamma, V, T, kVpMaxCluster, target_probs, q_start, draft_probs, draft_tokens, u, out_tokens,
                            accepted_len, p_tok, static_cast<uint32_t*>(workspace)};
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = dtype == DSPARK_BF16 ? launch_verify_probs<__nv_bfloat16>(p, R, s) : launch_verify_probs<float>(p, R, s);
  note_launches(1);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
