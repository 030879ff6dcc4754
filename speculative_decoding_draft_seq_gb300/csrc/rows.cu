// Softmax over whole rows of logits: their probabilities under one temperature a
// row, and a drafter's divergence from a teacher's top logits with its gradient.
//
// Both need a row's maximum M and Z = sum 2^((x - M) r) before they can write
// anything of the row's size, and are bound by bytes (a row in, a row out) if the row is read
// once. So a cluster of CTAs holds a row in registers, kPieces 16-byte pieces a
// thread: every warp forms the maximum and the sum of its own pieces, the warps of all
// CTAs exchange these pairs through distributed shared memory, and after one cluster
// barrier each thread combines them in the same order and writes its pieces. A row too long
// for the registers of a cluster is read again instead (kHold false).
#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"
#include "verify_common.cuh"

namespace dspark {

constexpr int kRowThreads = 512;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kPieces = 8;       // 16-byte pieces of a row that a thread holds
constexpr int kMaxCluster = 8;   // the portable limit
constexpr int kMaxTop = 1024;    // listed teacher entries of a row

__device__ __forceinline__ float nan_max(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// One row of V elements as this thread sees it: 16-byte pieces, of which it owns number
// (i C + rank) NT + tid, i = 0, 1, .., and the loose elements before the first and after the last
// piece, one each for the first threads of CTA 0.
template <class T>
struct RowPart {
  static constexpr int E = 16 / sizeof(T);
  const T* row;
  int V, a0, n, C, rank;
  __device__ RowPart(const T* r, int V_, int C_, int rank_) : row(r), V(V_), C(C_), rank(rank_) {
    const int off = (int)((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(T));
    a0 = min(off ? E - off : 0, V);
    n = (V - a0) / E;
  }
  __device__ __forceinline__ int loose() const { return V - n * E; }
  __device__ __forceinline__ int loose_index(int i) const { return i < a0 ? i : i + n * E; }
  __device__ __forceinline__ int piece(int i) const { return (i * C + rank) * kRowThreads + (int)threadIdx.x; }
  __device__ __forceinline__ int steps() const { return ceil_div(n, C * kRowThreads); }
  __device__ __forceinline__ uint4 load(int g) const {
    uint4 q;
    const void* p = row + a0 + (size_t)g * E;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "l"(p) : "memory");
    return q;
  }
  // whether this thread owns a loose element, and which
  __device__ __forceinline__ int own_loose() const { return rank == 0 && (int)threadIdx.x < loose() ? loose_index(threadIdx.x) : -1; }
  // owner of element v: CTA, and the local number of its piece (step * NT + thread); loose ones: -1 - number
  __device__ __forceinline__ int owner(int v, int& local, int& at) const {
    if (v < a0 || v >= a0 + n * E) {
      local = -1 - (v < a0 ? v : v - n * E);
      at = 0;
      return 0;
    }
    const int g = (v - a0) / E;
    at = (v - a0) % E;
    const int step = g / (C * kRowThreads), t = g - step * C * kRowThreads;
    local = step * kRowThreads + t % kRowThreads;
    return t / kRowThreads;
  }
};
template <class T>
__device__ __forceinline__ float row_elem(const T* p) {
  if constexpr (sizeof(T) == 4) return *p;
  else return __uint_as_float((uint32_t)*reinterpret_cast<const unsigned short*>(p) << 16);
}
template <class T>
__device__ __forceinline__ void split_piece(const uint4& q, float (&x)[16 / sizeof(T)]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <class T>
__device__ __forceinline__ uint4 empty_piece() {  // -inf throughout
  const uint32_t e = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
  return make_uint4(e, e, e, e);
}
template <class T>
__device__ __forceinline__ float piece_max(const uint4& q) {
  float x[16 / sizeof(T)];
  split_piece<T>(q, x);
  float m = x[0];
#pragma unroll
  for (int e = 1; e < (int)(16 / sizeof(T)); ++e) m = nan_max(m, x[e]);
  return m;
}
__device__ __forceinline__ float warp_nan_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = nan_max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <class T>
__device__ __forceinline__ void store_elem(T* p, float v) {
  if constexpr (sizeof(T) == 4) *p = v;
  else *p = __float2bfloat16_rn(v);
}
// E neighbouring results to out[0..E-1]; `wide`: out + any piece's first element is 16-byte aligned
template <class To, int E>
__device__ __forceinline__ void store_piece(To* out, const float (&y)[E], bool wide) {
  if (wide) {
    if constexpr (sizeof(To) == 4) {
#pragma unroll
      for (int i = 0; i < E; i += 4)
        __stcs(reinterpret_cast<float4*>(out + i), make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]));
    } else {
      uint32_t w[E / 2];
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if constexpr (E == 8) __stcs(reinterpret_cast<uint4*>(out), make_uint4(w[0], w[1], w[2], w[3]));
      else __stcs(reinterpret_cast<uint2*>(out), make_uint2(w[0], w[1]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) store_elem(out + i, y[i]);
  }
}

// The exponent of an entry's weight: (x - M) r, as fma(x, h, -M h) (r / h) with h = 1, or 1/2 for rates so small
// that differences past float32's range count.
struct Weigher {
  float h, Mh, rate;
  __device__ __forceinline__ Weigher(float M, float h_, float rate_) : h(h_), Mh(M * h_), rate(rate_) {}
  __device__ __forceinline__ float exponent(float x) const { return __fmul_rn(__fmaf_rn(x, h, -Mh), rate); }
  __device__ __forceinline__ float operator()(float x) const { return ex2_approx(exponent(x)); }
};

// (maximum, sum) of a warp's pieces, continued over chunks of pieces; `listed` the part of the sum that is marked.
struct WarpSum {
  float m = -INFINITY, z = 0.f, listed = 0.f;
};
template <class T, int P, class Marks>
__device__ __forceinline__ void add_pieces(WarpSum& s, const uint4 (&q)[P], float loose, float h, float rate, Marks marks) {
  constexpr int E = 16 / sizeof(T);
  float m = loose;
#pragma unroll
  for (int i = 0; i < P; ++i) m = nan_max(m, piece_max<T>(q[i]));
  m = nan_max(s.m, warp_nan_max(m));
  if (m == -INFINITY) return;  // (the whole warp)
  const Weigher w(m, h, rate);
  if (s.m != -INFINITY) {
    const float f = w(s.m);
    s.z *= f;
    s.listed *= f;
  }
  s.m = m;
  float a = 0.f, b = 0.f, l = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    float x[E];
    split_piece<T>(q[i], x);
    const uint32_t bits = marks(i);
    if (bits == 0) {
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        a += w(x[e]);
        b += w(x[e + 1]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float y = w(x[e]);
        if (bits >> e & 1) l += y;
        else a += y;
      }
    }
  }
  if (loose != -INFINITY) {
    const float y = w(loose);
    if (marks(-1)) l += y;
    else a += y;
  }
  s.z += a + b;
  s.listed += l;
}

// The row's maximum and sums from those of all warps of the cluster, the same in every thread: combined in float64
// (a warp's lanes each take every 32nd entry, then a fixed tree).
struct RowSum {
  float M;
  double z, listed;
};
__device__ __forceinline__ double warp_add_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ RowSum exchange(WarpSum s, float4* all, int C, int rank, float h, float rate) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  s.z = warp_sum(s.z);
  s.listed = warp_sum(s.listed);
  if (lane < C) store_peer(peer_address(all + rank * kRowWarps + warp, lane), make_float4(s.m, s.z, s.listed, 0.f));
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  RowSum r{-INFINITY, 0.0, 0.0};
  for (int i = lane; i < C * kRowWarps; i += 32) r.M = nan_max(r.M, all[i].x);
  r.M = warp_nan_max(r.M);
  if (r.M == -INFINITY) return r;
  const Weigher w(r.M, h, rate);
  for (int i = lane; i < C * kRowWarps; i += 32) {
    const float4 t = all[i];
    if (t.x == -INFINITY) continue;
    const float f = w(t.x);
    r.z += (double)t.y * f;
    r.listed += (double)t.z * f;
  }
  r.z = warp_add_d(r.z);
  r.listed = warp_add_d(r.listed);
  return r;
}

// ---------------------------------------------------------------------------
struct ProbsParams {
  int V, C;
  const void* logits;
  const float* temperature;
  void* probs;
  uint32_t* status;
};

template <class T, class To, bool kHold>
__global__ void __launch_bounds__(kRowThreads) probabilities_kernel(ProbsParams p) {
  constexpr int E = 16 / sizeof(T);
  __shared__ float4 all[kMaxCluster * kRowWarps];
  __shared__ uint32_t first[kMaxCluster * kRowWarps];
  const int rank = (int)cluster_rank(), C = p.C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster_arrive();  // the others' shared memory is theirs once they run: waited for before the exchange
  const size_t r = blockIdx.x / C;
  const RowPart<T> part(static_cast<const T*>(p.logits) + r * p.V, p.V, C, rank);
  To* out = static_cast<To*>(p.probs) + r * p.V;
  const bool wide = (reinterpret_cast<uintptr_t>(out + part.a0) & (E * sizeof(To) < 16 ? E * sizeof(To) - 1 : 15)) == 0;
  const float T_ = __ldg(p.temperature + r);
  const bool greedy = !(T_ > 0.f);
  // the smallest rate (T = inf) still takes an entry of -inf to weight 0
  const float rate0 = greedy ? 1.f : fmaxf(fminf(__fdiv_rn(1.44269504088896340736f, T_), 1e30f), 1e-45f);
  const float h = rate0 < 1e-36f ? 0.5f : 1.f, rate = rate0 < 1e-36f ? 2.f * rate0 : rate0;
  const int loose_at = part.own_loose();
  const float loose = loose_at >= 0 ? row_elem(part.row + loose_at) : -INFINITY;
  const auto unmarked = [](int) { return 0u; };

  uint4 q[kPieces];
  WarpSum s;
  const int chunks = kHold ? 1 : ceil_div(part.steps(), kPieces);
  const auto fetch = [&](int c) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int g = part.piece(c * kPieces + i);
      q[i] = g < part.n ? part.load(g) : empty_piece<T>();
    }
  };
  for (int c = 0; c < max(chunks, 1); ++c) {
    fetch(c);
    add_pieces<T>(s, q, c == 0 ? loose : -INFINITY, h, rate, unmarked);
  }
  cluster_wait();
  const RowSum sum = exchange(s, all, C, rank, h, rate);
  const bool bad = !(fabsf(sum.M) < INFINITY);
  if (bad && rank == 0 && threadIdx.x == 0) set_status(p.status, DSPARK_ERR_NONFINITE);

  int top = INT_MAX;  // greedy: the first maximum
  if (greedy && !bad) {
    for (int c = 0; c < max(chunks, 1); ++c) {
      if (!kHold) fetch(c);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        float x[E];
        split_piece<T>(q[i], x);
        const int g = part.piece(c * kPieces + i);
#pragma unroll
        for (int e = E - 1; e >= 0; --e)
          if (g < part.n && x[e] == sum.M) top = min(top, part.a0 + g * E + e);
      }
    }
    if (loose_at >= 0 && loose == sum.M) top = min(top, loose_at);
    top = warp_min_i(top);
    if (lane < C) store_peer(peer_address(first + rank * kRowWarps + warp, lane), (uint32_t)top);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    top = INT_MAX;
    for (int i = lane; i < C * kRowWarps; i += 32) top = min(top, (int)first[i]);
    top = warp_min_i(top);
  }

  const Weigher w(sum.M, h, rate);
  const float inv = bad ? 0.f : (float)(1.0 / sum.z);
  const auto result = [&](float x, int v) { return bad ? 0.f : greedy ? (v == top ? 1.f : 0.f) : w(x) * inv; };
  for (int c = 0; c < max(chunks, 1); ++c) {
    if (!kHold) fetch(c);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int g = part.piece(c * kPieces + i);
      if (g >= part.n) continue;
      float x[E];
      split_piece<T>(q[i], x);
      const int v = part.a0 + g * E;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = result(x[e], v + e);
      store_piece<To, E>(out + v, x, wide);
    }
  }
  if (loose_at >= 0) store_elem(out + loose_at, result(loose, loose_at));
}

// ---------------------------------------------------------------------------
struct DistillParams {
  int V, K, C, marks;  // marks: bytes of the marked-entry map
  const void* logits;
  const int32_t* ids;
  const float* teacher;
  const float* teacher_lse;
  const float* weight;
  float tau;
  float* loss;
  void* grad;
  uint32_t* status;
};

__device__ __forceinline__ double block_sum_dd(double v, double* sh) {
  v = warp_add_d(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < kRowWarps; ++i) v += sh[i];
  return v;
}

template <class T, bool kHold>
__global__ void __launch_bounds__(kRowThreads) distill_kernel(DistillParams p) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ float4 all[kMaxCluster * kRowWarps];
  __shared__ double sums[kRowWarps];
  __shared__ float maxima[kRowWarps];
  __shared__ uint32_t loose_marks;
  __shared__ int twice;
  // of the listed entries: id (-1: none), teacher's logit, the student's, the teacher's probability
  int* s_id = reinterpret_cast<int*>(dyn);
  float* s_t = reinterpret_cast<float*>(s_id + p.K);
  float* s_x = s_t + p.K;
  double* s_p = reinterpret_cast<double*>(dyn + (((size_t)p.K * 12 + 15) & ~(size_t)15));
  uint32_t* s_marks = reinterpret_cast<uint32_t*>(s_p + p.K);
  const int rank = (int)cluster_rank(), C = p.C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster_arrive();
  const size_t r = blockIdx.x / C;
  const T* row = static_cast<const T*>(p.logits) + r * p.V;
  const RowPart<T> part(row, p.V, C, rank);
  const bool with_rest = p.teacher_lse != nullptr;
  const float rate = __fdiv_rn(1.44269504088896340736f, p.tau);
  const int loose_at = part.own_loose();
  const float loose = loose_at >= 0 ? row_elem(row + loose_at) : -INFINITY;

  uint4 q[kPieces];
  const auto fetch = [&](int c) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int g = part.piece(c * kPieces + i);
      q[i] = g < part.n ? part.load(g) : empty_piece<T>();
    }
  };
  fetch(0);
  // the listed entries, in every CTA; those of this CTA's pieces are marked
  for (int i = tid; i < p.marks / 4; i += kRowThreads) s_marks[i] = 0;
  if (tid == 0) {
    loose_marks = 0;
    twice = 0;
  }
  __syncthreads();
  bool out_of_range = false;
  float t_max = -INFINITY;
  for (int j = tid; j < p.K; j += kRowThreads) {
    int id = __ldg(p.ids + r * p.K + j);
    out_of_range |= id >= p.V;
    if (id >= p.V) id = -1;
    float t = __ldg(p.teacher + r * p.K + j);
    if (id < 0) {
      id = -1;
      t = -INFINITY;
    }
    s_id[j] = id;
    s_t[j] = t;
    s_x[j] = id >= 0 ? row_elem(row + id) : -INFINITY;
    t_max = nan_max(t_max, t);
    if (id >= 0) {
      int local, at;
      if (part.owner(id, local, at) == rank) {
        bool again;
        if (local < 0) {
          const uint32_t bit = 1u << (-1 - local);
          again = atomicOr(&loose_marks, bit) & bit;
        } else {
          const uint32_t bit = 1u << ((local & 3) * 8 + at);
          again = atomicOr(s_marks + (local >> 2), bit) & bit;
        }
        if (again) twice = 1;
      }
    }
  }
  if (out_of_range) set_status(p.status, DSPARK_ERR_RANGE);
  t_max = warp_nan_max(t_max);
  if (lane == 0) maxima[warp] = t_max;
  __syncthreads();
  t_max = maxima[0];
#pragma unroll
  for (int i = 1; i < kRowWarps; ++i) t_max = nan_max(t_max, maxima[i]);
  const double lse = with_rest ? (double)__ldg(p.teacher_lse + r) : 0.0;
  const bool none = t_max == -INFINITY;
  const bool bad_teacher = !(t_max < INFINITY) || (with_rest && !(fabs(lse) < (double)INFINITY));
  // the teacher's probabilities: float64, since what they leave of 1 and the logarithms' differences may be small
  const double per_tau = 1.0 / (double)p.tau;
  double share = 0.0;
  for (int j = tid; j < p.K; j += kRowThreads) {
    const double y = with_rest ? (double)s_t[j] * per_tau - lse : ((double)s_t[j] - (double)t_max) * per_tau;
    const double e = none || bad_teacher || s_id[j] < 0 ? 0.0 : exp(y);
    s_p[j] = e;
    share += e;
  }
  share = block_sum_dd(share, sums);
  const double norm = with_rest || share == 0.0 ? 1.0 : 1.0 / share;
  const double p_rest = with_rest ? fmax(0.0, 1.0 - share) : 0.0;

  WarpSum s;
  const int chunks = kHold ? 1 : max(ceil_div(part.steps(), kPieces), 1);
  for (int c = 0; c < chunks; ++c) {
    if (c > 0) fetch(c);
    const auto marks = [&](int i) -> uint32_t {
      if (!with_rest) return 0u;
      if (i < 0) return loose_marks >> tid & 1u;
      const int local = (c * kPieces + i) * kRowThreads + tid;
      return local < p.marks ? s_marks[local >> 2] >> ((local & 3) * 8) & 255u : 0u;
    };
    add_pieces<T>(s, q, c == 0 ? loose : -INFINITY, 1.f, rate, marks);
  }
  cluster_wait();
  const RowSum sum = exchange(s, all, C, rank, 1.f, rate);
  const double z = sum.z + sum.listed, z_rest = sum.z;
  const bool bad = !(fabsf(sum.M) < INFINITY) || bad_teacher;
  const bool some = p_rest > 0.0 && z_rest > 0.0;  // a rest without mass on either side counts for nothing
  const Weigher w(sum.M, 1.f, rate);

  if (rank == 0) {
    const double step = (double)rate * 0.69314718055994530942;  // 1 / tau as the weights have it
    double a = 0.0;
    for (int j = tid; j < p.K; j += kRowThreads) {
      const double e = s_p[j];
      if (e > 0.0) {
        const double y = with_rest ? (double)s_t[j] * per_tau - lse : ((double)s_t[j] - (double)t_max) * per_tau;
        a += e * (y - ((double)s_x[j] - (double)sum.M) * step);
      }
    }
    a = block_sum_dd(a, sums);
    if (tid == 0) {
      double loss = 0.0;
      const double ln_z = log(z);
      if (with_rest) {
        loss = a + share * ln_z;
        if (some) loss += p_rest * (log(p_rest) - log(z_rest) + ln_z);
      } else if (share > 0.0) {
        loss = a * norm + ln_z - log(share);
      }
      p.loss[r] = bad ? NAN : (float)loss;
      if (bad) set_status(p.status, DSPARK_ERR_NONFINITE);
    }
  }
  if (!p.grad) return;

  // d loss / d x_v = (1/tau) (s_v total - [rest] s_v p_rest / s_rest - p_v)
  T* grad = static_cast<T*>(p.grad) + r * p.V;
  const bool wide = (reinterpret_cast<uintptr_t>(grad + part.a0) & 15) == 0;
  const double scale = (p.weight ? (double)__ldg(p.weight + r) : 1.0) * per_tau;
  const double total = with_rest ? share + (some ? p_rest : 0.0) : (share > 0.0 ? 1.0 : 0.0);
  const float listed_f = bad ? 0.f : (float)(scale * total / z);
  const float rest_f = bad ? 0.f : (float)(scale * (total / z - (some ? p_rest / z_rest : 0.0)));
  for (int c = 0; c < chunks; ++c) {
    if (!kHold) fetch(c);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int g = part.piece(c * kPieces + i);
      if (g >= part.n) continue;
      float x[E];
      split_piece<T>(q[i], x);
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = bad ? 0.f : w(x[e]) * rest_f;
      store_piece<T, E>(grad + part.a0 + (size_t)g * E, x, wide);
    }
  }
  if (loose_at >= 0) store_elem(grad + loose_at, bad ? 0.f : w(loose) * rest_f);
  if (bad) return;
  // the listed entries of this CTA over what was just written
  __syncthreads();
  for (int j = tid; j < p.K; j += kRowThreads) {
    const int id = s_id[j];
    int local, at;
    if (id < 0 || part.owner(id, local, at) != rank) continue;
    double e = s_p[j];
    if (twice) {  // an id that comes more than once: every occurrence writes the sum of all
      e = 0.0;
      for (int i = 0; i < p.K; ++i)
        if (s_id[i] == id) e += s_p[i];
    }
    store_elem(grad + id, (float)((double)(w(s_x[j]) * listed_f) - scale * norm * e));
  }
}

// ---------------------------------------------------------------------------
static int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// CTAs a row: as few as hold it, more while the rows leave SMs idle.
static int row_cluster(int N, int V, int elem, int sms, bool& hold) {
  const long long pieces = (long long)V * elem / 16;
  int C = 1;
  while (C < kMaxCluster && (pieces > (long long)C * kRowThreads * kPieces || ((long long)N * C * 2 <= sms && pieces > (long long)C * kRowThreads)))
    C *= 2;
  hold = pieces <= (long long)C * kRowThreads * kPieces;
  return C;
}

template <class T, class To>
static cudaError_t launch_probs(const ProbsParams& p, int N, bool hold, cudaStream_t s) {
  return launch_clusters(hold ? probabilities_kernel<T, To, true> : probabilities_kernel<T, To, false>, p, (unsigned)N * p.C, p.C,
                         kRowThreads, 0, s);
}

constexpr size_t kDistillSmem = (size_t)kMaxTop * 20 + 16 + ((1 << 20) / 4 / kMaxCluster + kRowThreads);  // float32 rows of 2^20

template <class T, bool kHold>
static cudaError_t launch_distill(const DistillParams& p, int N, cudaStream_t s) {
  static std::atomic<unsigned long long> attr{0};
  const size_t smem = (((size_t)p.K * 12 + 15) & ~(size_t)15) + (size_t)p.K * 8 + p.marks;
  const cudaError_t e = set_smem_limit_once((const void*)distill_kernel<T, kHold>, (int)kDistillSmem, attr);
  if (e != cudaSuccess) return e;
  return launch_clusters(distill_kernel<T, kHold>, p, (unsigned)N * p.C, p.C, kRowThreads, smem, s);
}

static bool row_args(int32_t N, int32_t V, int32_t dtype) {
  return N >= 0 && N <= (1 << 24) && V >= 1 && V <= (1 << 20) && (dtype == DSPARK_FP32 || dtype == DSPARK_BF16);
}
static bool workspace_ok(const void* ws, size_t bytes) {
  return ws && (reinterpret_cast<uintptr_t>(ws) & 255) == 0 && bytes >= 256;
}

}  // namespace dspark

using namespace dspark;

extern "C" dspark_status dspark_probabilities(int32_t N, int32_t V, int32_t dtype, const void* logits,
                                              const float* temperature, int32_t probs_dtype, void* probs, void* workspace,
                                              size_t workspace_bytes, dspark_stream_t stream) {
  note_launches(0);
  if (!row_args(N, V, dtype) || (probs_dtype != DSPARK_FP32 && probs_dtype != DSPARK_BF16)) return DSPARK_ERR_INVALID_ARG;
  if (N > 0 && (!logits || !temperature || !probs)) return DSPARK_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes)) return DSPARK_ERR_WORKSPACE;
  if (N == 0) return DSPARK_OK;
  const int sms = sm_count();
  if (sms == 0) return DSPARK_ERR_CUDA;
  bool hold;
  const int C = row_cluster(N, V, dtype == DSPARK_BF16 ? 2 : 4, sms, hold);
  const ProbsParams p{V, C, logits, temperature, probs, static_cast<uint32_t*>(workspace)};
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (dtype == DSPARK_BF16)
    e = probs_dtype == DSPARK_BF16 ? launch_probs<__nv_bfloat16, __nv_bfloat16>(p, N, hold, s)
                                   : launch_probs<__nv_bfloat16, float>(p, N, hold, s);
  else
    e = probs_dtype == DSPARK_BF16 ? launch_probs<float, __nv_bfloat16>(p, N, hold, s) : launch_probs<float, float>(p, N, hold, s);
  note_launches(1);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

extern "C" dspark_status dspark_distill(int32_t N, int32_t V, int32_t K, int32_t dtype, const void* logits,
                                        const int32_t* ids, const float* teacher, const float* teacher_lse,
                                        const float* weight, float temperature, float* loss, void* grad, void* workspace,
                                        size_t workspace_bytes, dspark_stream_t stream) {
  note_launches(0);
  if (!row_args(N, V, dtype) || K < 1 || K > kMaxTop || !(temperature >= 1e-6f && temperature <= 1e6f))
    return DSPARK_ERR_INVALID_ARG;
  if (N > 0 && (!logits || !ids || !teacher || !loss)) return DSPARK_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes)) return DSPARK_ERR_WORKSPACE;
  if (N == 0) return DSPARK_OK;
  const int sms = sm_count();
  if (sms == 0) return DSPARK_ERR_CUDA;
  bool hold;
  const int elem = dtype == DSPARK_BF16 ? 2 : 4;
  const int C = row_cluster(N, V, elem, sms, hold);
  // one byte a piece of this CTA, whole steps of the block
  const int marks = ceil_div((long long)V * elem / 16, (long long)C * kRowThreads) * kRowThreads;
  const DistillParams p{V, K, C, marks, logits, ids, teacher, teacher_lse, weight, temperature, loss, grad,
                        static_cast<uint32_t*>(workspace)};
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (dtype == DSPARK_BF16) e = hold ? launch_distill<__nv_bfloat16, true>(p, N, s) : launch_distill<__nv_bfloat16, false>(p, N, s);
  else e = hold ? launch_distill<float, true>(p, N, s) : launch_distill<float, false>(p, N, s);
  note_launches(1);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
