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
// warp, a lane a draft; two dependent loads), then sums a contiguous share of the one row
// that matters, warp by warp; the warps' sums go to all CTAs, and the warp whose
// share holds the token reads a part of that share once more to find it. The rows come through
// a ring of asynchronous copies a warp: they keep the loads going while a step is added up, and
// let rows of any alignment be copied in whole pieces and put together in shared memory (with loads to registers an
// odd row length took twice the time of an even one).
//
// Bound by bytes where requests fill the GPU, by its chain of dependent steps (row numbers, draft, probability,
// row, exchange, token) where they do not. 128 requests over 129,280 float32 entries, up to 16 drafts: 28 us, 117
// MB (0.62 of the measured copy bandwidth), odd row length 31, bf16 20; without rows of the drafter's 20; one request 8.5,
// over 32,000 entries 6. CTAs a request: 8, 4, 2, 1 as the SMs hold them (16 requests: 9.6 us with 8,
// 12.7 with 4; 512 over 32,000: 24 with 1, 31 with 2).
#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"
#include "mass.cuh"

namespace dspark {

constexpr int kVpThreads = 256;
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

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
  // 27 bits at a time: 32 of them add up to 32 bits
  const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x7ffffffu);
  const uint32_t b = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 27) & 0x7ffffffu);
  const uint32_t c = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 54));
  return a + ((unsigned long long)b << 27) + ((unsigned long long)c << 54);
}

// Entries of the row that is drawn from: the target's, less the drafter's where a draft was rejected.
template <class T>
struct DrawRow {
  static constexpr int E = 16 / sizeof(T);
  const T* p;
  const T* q;  // or null
  int token;   // of a rejected draft without a row of its own: Q is 1 there (else -1)
  __device__ __forceinline__ float at(int v) const {
    float w = ld_elem(p, v);
    if (q) w = __fsub_rn(w, ld_elem(q, v));
    return v == token ? __fsub_rn(w, 1.f) : w;
  }
  // entries of a row before its first 16-byte boundary
  static __device__ __forceinline__ int lead(const T* row) {
    return (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T);
  }
  static __device__ __forceinline__ void split(const uint4& a, float (&x)[E]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (E == 4) {
        x[i] = __uint_as_float(w[i]);
      } else {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
};

// Mass of w clamped to [0, 1] (NaN: 0): the subtraction's saturation does it.
__device__ __forceinline__ unsigned long long mass40(float w) { return fx40(__saturatef(w)); }

// Masses of the E entries of a piece (w before they are clamped), added up; `finite` stays 0 while all are finite.
template <int E>
__device__ __forceinline__ void add_masses(MassSum& m, float (&w)[E], float& finite) {
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    finite = __fmaf_rn(w[i], 0.f, finite);
    finite = __fmaf_rn(w[i + 1], 0.f, finite);
    m.add(MassPair(__saturatef(w[i]), __saturatef(w[i + 1])));
  }
}

// The 16 bytes that begin d entries after the start of the pair (a, b), d < 16 / sizeof(T).
template <class T>
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int d) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const int bytes = d * (int)sizeof(T);
  if (bytes & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (bytes & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (bytes & 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kStretches = 4;  // parts of a warp's share whose masses its lanes keep

constexpr int kLane = 2;       // pieces of a row that a lane takes in a step
constexpr int kAhead = 2;      // steps of a warp that are on their way to shared memory
// a step's pieces: the target's, and the drafter's with the one after the last (whole lines: copies to unaligned ones are
// slower)
struct __align__(128) StepBuffer {
  uint4 p[32 * kLane], q[32 * kLane + 8];
};
constexpr int kVpSmem = kVpWarps * kAhead * (int)sizeof(StepBuffer);

__device__ __forceinline__ void copy_piece(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

// part[s] = this lane's mass in stretch s of its warp's share, of `stretch` steps of kLane pieces a lane from entry v0 (which
// may lie before the row: pieces begin at the target row's 16-byte boundaries). The drafter's row has a boundary
// d entries before each piece's start: a piece of it is put together from two. Pieces go through the warp's ring in shared memory.
template <class T>
__device__ __forceinline__ void share_masses(const DrawRow<T>& row, int V, int v0, int stretch, int d, StepBuffer* ring,
                                             unsigned long long (&part)[kStretches], float& finite) {
  constexpr int E = 16 / sizeof(T);
  const int lane = threadIdx.x & 31, steps = stretch * kStretches;
  const auto in_row = [&](int at) { return at >= 0 && at + E <= V; };
  const auto issue = [&](int step) {
    StepBuffer& s = ring[step % kAhead];
    if (step < steps) {
#pragma unroll
      for (int i = 0; i < kLane; ++i) {
        const int k = i * 32 + lane, at = v0 + (step * 32 * kLane + k) * E;
        if (in_row(at)) copy_piece(s.p + k, row.p + at);
        if (row.q) {
          if (in_row(at - d)) copy_piece(s.q + k, row.q + at - d);
          if (d && k == 32 * kLane - 1 && in_row(at - d + E)) copy_piece(s.q + k + 1, row.q + at - d + E);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) issue(i);
  int step = 0;
#pragma unroll
  for (int s = 0; s < kStretches; ++s) {
    part[s] = 0;
#pragma unroll 1
    for (int t = 0; t < stretch; ++t, ++step) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
      __syncwarp();
      const StepBuffer& from = ring[step % kAhead];
      MassSum sum;
#pragma unroll
      for (int i = 0; i < kLane; ++i) {
        const int k = i * 32 + lane, at = v0 + (step * 32 * kLane + k) * E;
        float w[E];
        if (in_row(at) && (!row.q || (in_row(at - d) && (d == 0 || in_row(at - d + E))))) {
          DrawRow<T>::split(from.p[k], w);
          if (row.q) {
            float x[E];
            DrawRow<T>::split(d ? shifted<T>(from.q[k], from.q[k + 1], d) : from.q[k], x);
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = __fsub_rn(w[e], x[e]);
          }
          if ((unsigned)(row.token - at) < (unsigned)E) {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (at + e == row.token) w[e] = __fsub_rn(w[e], 1.f);
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) w[e] = at + e >= 0 && at + e < V ? row.at(at + e) : 0.f;
        }
        add_masses(sum, w, finite);
      }
      part[s] += sum.total();
      __syncwarp();  // everyone has read: the buffer may be filled again
      issue(step + kAhead);
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
}

template <class T>
__global__ void __launch_bounds__(kVpThreads, 4) verify_probs_kernel(VerifyProbsParams p) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ __align__(128) StepBuffer rings[];
  __shared__ unsigned long long sums[2][kVpMaxCluster * kVpWarps];  // one set a pass
  __shared__ int s_start, s_n, s_accepted, s_token;
  const int rank = (int)cluster_rank(), C = p.C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster_arrive();
  const size_t r = blockIdx.x / C;
  const T* target = static_cast<const T*>(p.target);
  const T* draft = static_cast<const T*>(p.draft);
  const size_t V = p.V;

  if (warp == 0) {
    const int a = __ldg(p.q_start + r), b = __ldg(p.q_start + r + 1);
    // the first drafts and uniforms, in flight together with the row numbers
    const int x0 = lane < p.gamma ? __ldg(p.tokens + r * p.gamma + lane) : -1;
    const double u0 = lane < p.gamma ? __ldg(p.u + r * (p.gamma + 1) + lane) : 0.0;
    const bool wrong = a < 0 || b < a || b > p.T || b - a - 1 > p.gamma;
    const int n = a < 0 || b < a || b > p.T ? 0 : min(b - a, p.gamma + 1);
    if (wrong && rank == 0 && lane == 0) set_status(p.status, DSPARK_ERR_RANGE);
    int accepted = 0, token = -1;
    bool go = true;  // no draft rejected so far
    for (int k0 = 0; k0 < p.gamma; k0 += 32) {
      const int k = k0 + lane;
      bool ok = false;
      float pt = 0.f;
      int x = -1;
      if (k < n - 1) {
        x = k0 == 0 ? x0 : __ldg(p.tokens + r * p.gamma + k);
        const double u = k0 == 0 ? u0 : __ldg(p.u + r * (p.gamma + 1) + k);
        if (x >= 0 && x < p.V) {
          pt = ld_elem(target, (size_t)(a + k) * V + x);
          const float qt = draft ? ld_elem(draft, (r * p.gamma + k) * V + x) : 1.f;
          ok = __dmul_rn(u, (double)qt) < (double)pt;
          if (rank == 0 && !(fabsf(pt) + fabsf(qt) < INFINITY)) set_status(p.status, DSPARK_ERR_NONFINITE);
        } else if (rank == 0) {
          set_status(p.status, DSPARK_ERR_RANGE);
        }
      }
      if (rank == 0 && k < p.gamma) p.p_tok[r * p.gamma + k] = pt;
      const uint32_t fails = ~__ballot_sync(0xffffffffu, ok);
      if (go) accepted += fails ? __ffs(fails) - 1 : 32;
      if (go && fails) token = __shfl_sync(0xffffffffu, x, __ffs(fails) - 1);  // (-1 past the last draft)
      go &= fails == 0;
      if (!go && rank != 0) break;  // CTA 0 goes on: it writes the probabilities
    }
    if (lane == 0) {
      s_start = a;
      s_n = n;
      s_accepted = accepted;
      s_token = token;
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
  if (const int x = s_token; x >= 0 && x < p.V) {
    if (draft) row.q = draft + (r * p.gamma + A) * V;
    else row.token = x;
  }
  const double u = __ldg(p.u + r * (p.gamma + 1) + p.gamma);
  // this warp's share, in steps of a piece a lane, and the steps in kStretches stretches; entries are numbered from the
  // piece that holds the row's first one
  const int shares = C * kVpWarps;
  const int origin = DrawRow<T>::lead(row.p) ? DrawRow<T>::lead(row.p) - E : 0;
  const int stretch = ceil_div(ceil_div(p.V - origin, shares), kStretches * 32 * kLane * E), steps = stretch * kStretches;
  const int mine = rank * kVpWarps + warp;
  const int v0 = (int)min(origin + (long long)mine * steps * 32 * kLane * E, (long long)p.V);

  for (int pass = 0; pass < 2; ++pass) {
    const int d = row.q ? (int)(reinterpret_cast<uintptr_t>(row.q + (origin + E)) & 15) / (int)sizeof(T) : 0;
    unsigned long long part[kStretches];
    float finite = 0.f;
    share_masses(row, p.V, v0, stretch, d, rings + warp * kAhead, part, finite);
    unsigned long long m = 0;
#pragma unroll
    for (int s = 0; s < kStretches; ++s) m += part[s];
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
    const unsigned long long goal = scale_mass(u, Z);
    if (goal < before || goal - before >= m) return;
    // the stretch that holds it, then its steps from memory
    unsigned long long left = goal - before;
    int at = 0;
#pragma unroll
    for (int s = 0; s < kStretches; ++s) {
      const unsigned long long x = warp_sum_u64(part[s]);
      if (at == s && left >= x) {
        left -= x;
        ++at;
      }
    }
    for (int v = v0 + at * stretch * 32 * kLane * E; v < p.V; v += 32 * E) {
      float w[E];
      unsigned long long own = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int k = v + lane * E + e;
        w[e] = k >= 0 && k < p.V ? row.at(k) : 0.f;
        own += mass40(w[e]);
      }
      const unsigned long long step = warp_sum_u64(own);
      if (left >= step) {
        left -= step;
        continue;
      }
      unsigned long long c = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += y;
      }
      if (lane == __ffs(__ballot_sync(0xffffffffu, c > left)) - 1) {
        c -= own;
        int token = v + lane * E;
#pragma unroll
        for (int e = 0; e < E - 1; ++e) {
          c += mass40(w[e]);
          token += c <= left;
        }
        out[A] = token;
      }
      return;
    }
    return;
  }
}

template <class T>
static cudaError_t launch_verify_probs(const VerifyProbsParams& p, int R, cudaStream_t s) {
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = set_smem_limit_once((const void*)verify_probs_kernel<T>, kVpSmem, attr);
  if (e != cudaSuccess) return e;
  return launch_clusters(verify_probs_kernel<T>, p, (unsigned)R * p.C, p.C, kVpThreads, kVpSmem, s);
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
  const int elem = dtype == DSPARK_BF16 ? 2 : 4;
  const long long drafts = (long long)R * gamma;
  if (!separate({span(target_probs, (long long)T * V, elem), span(q_start, R + 1ll), span(draft_probs, drafts, V * elem),
                 span(draft_tokens, drafts), span(u, drafts + R)},
                {span(out_tokens, drafts + R), span(accepted_len, R), span(p_tok, drafts)}))
    return DSPARK_ERR_INVALID_ARG;
  // CTAs a request: what the SMs hold at once, four each (more leave each warp too little to pay for its chain and exchange)
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSPARK_ERR_CUDA;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int C = kVpMaxCluster;
  while (C > 1 && (long long)R * C > 4 * sms) C /= 2;
  const VerifyProbsParams p{gamma, V, T, C, target_probs, q_start, draft_probs, draft_tokens, u, out_tokens,
                            accepted_len, p_tok, static_cast<uint32_t*>(workspace)};
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = dtype == DSPARK_BF16 ? launch_verify_probs<__nv_bfloat16>(p, R, s) : launch_verify_probs<float>(p, R, s);
  note_launches(1);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
