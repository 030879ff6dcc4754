// Softmax over whole rows of logits: their probabilities under one temperature a
// row, and a drafter's divergence from a teacher's top logits with its gradient.
//
// Both need a row's maximum M and Z = sum 2^((x - M) r) before they can write
// anything of the row's size, and are bound by bytes (a row in, a row out) if the row is read
// once. So a cluster of CTAs holds a row in shared memory: every thread copies its own 16-byte
// pieces there (asynchronously; nobody else reads them, so it waits for itself only), every warp forms
// the maximum and the sum of its pieces, the warps of all CTAs exchange these pairs through
// distributed shared memory, and after one cluster barrier each thread combines them in the
// same order and writes its pieces. At kPieces pieces a thread three CTAs of an SM load, wait and write
// independently of each other. A row longer than a cluster holds is taken in windows, which are read again for
// the results.
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
static_assert(kRowThreads == 512 && kMaxCluster == 8, "RowPart takes logarithms of both");
constexpr int kMaxTop = 1024;    // listed teacher entries of a row

__device__ __forceinline__ float nan_max(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float warp_nan_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = nan_max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ unsigned long long pair_mul(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long pair_add(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void copy_async(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <class T>
__device__ __forceinline__ float row_elem(const T* p) {
  if constexpr (sizeof(T) == 4) return *p;
  else return __uint_as_float((uint32_t)*reinterpret_cast<const unsigned short*>(p) << 16);
}
template <class T>
__device__ __forceinline__ void store_elem(T* p, float v) {
  if constexpr (sizeof(T) == 4) *p = v;
  else *p = __float2bfloat16_rn(v);
}

// One row of V elements as this thread sees it: 16-byte pieces, of which it owns number
// (i C + rank) NT + tid, i = 0, 1, .., and the loose elements before the first and after the last
// piece, one each for the first threads of CTA 0.
template <class T>
struct RowPart {
  static constexpr int E = 16 / sizeof(T);
  const T* row;
  int a0, n, shift, rank;  // C NT = 2^shift, C a power of two up to kMaxCluster
  __device__ RowPart(const T* r, int V, int C, int rank_) : row(r), shift(9 + (C >= 2) + (C >= 4) + (C >= 8)), rank(rank_) {
    const int off = (int)((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(T));
    a0 = min(off ? E - off : 0, V);
    n = (V - a0) / E;
  }
  __device__ __forceinline__ int piece(int i) const { return (i << shift) + rank * kRowThreads + (int)threadIdx.x; }
  // pieces that this thread owns
  __device__ __forceinline__ int own() const {
    return (n - 1 - piece(0) + (1 << shift)) >> shift;
  }
  __device__ __forceinline__ int steps() const { return (n + (1 << shift) - 1) >> shift; }
  // the loose element that this thread owns, or -1
  __device__ __forceinline__ int own_loose(int V) const {
    const int i = threadIdx.x;
    return rank == 0 && i < V - n * E ? (i < a0 ? i : i + n * E) : -1;
  }
  // owner of element v: CTA, and the local number of its piece (step * NT + thread); loose ones: -1 - number
  __device__ __forceinline__ int owner(int v, int& local, int& at) const {
    if (v < a0 || v >= a0 + n * E) {
      local = -1 - (v < a0 ? v : v - n * E);
      at = 0;
      return 0;
    }
    const int g = (v - a0) / E, t = g & ((1 << shift) - 1);
    at = (v - a0) % E;
    local = (g >> shift) * kRowThreads + t % kRowThreads;
    return t / kRowThreads;
  }
  // starts the copies of this thread's pieces i0 .. min(i0 + kPieces, own) - 1
  __device__ __forceinline__ void fetch(uint4* held, int i0) const {
    const int m = min(own() - i0, kPieces);
    for (int i = 0; i < m; ++i) copy_async(held + i * kRowThreads + threadIdx.x, row + a0 + (size_t)piece(i0 + i) * E);
  }
};

// The two logits of each 32-bit word of a piece (of each two words, float32).
template <class T>
__device__ __forceinline__ void split_piece(const uint4& q, unsigned long long (&x)[8 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    x[0] = (unsigned long long)q.y << 32 | q.x;
    x[1] = (unsigned long long)q.w << 32 | q.z;
  } else {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (unsigned long long)(w[i] & 0xffff0000u) << 32 | w[i] << 16;
  }
}
template <class T>
__device__ __forceinline__ float piece_max(const uint4& q) {
  if constexpr (sizeof(T) == 4) {
    return nan_max(nan_max(__uint_as_float(q.x), __uint_as_float(q.y)), nan_max(__uint_as_float(q.z), __uint_as_float(q.w)));
  } else {
    uint32_t a, b;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(q.x), "r"(q.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(q.z), "r"(q.w));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    return nan_max(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
}
// E neighbouring results to out[0..E-1]; `wide`: aligned to their size
template <class To, int E>
__device__ __forceinline__ void store_piece(To* out, const float (&y)[E], bool wide) {
  if (wide) {
    if constexpr (sizeof(To) == 4 && E == 8) {
      asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]),
                   "f"(y[5]), "f"(y[6]), "f"(y[7])
                   : "memory");
    } else if constexpr (sizeof(To) == 4) {
      __stcs(reinterpret_cast<float4*>(out), make_float4(y[0], y[1], y[2], y[3]));
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
// that differences past float32's range count. One entry, or two at a time with the same bits.
struct Weigher {
  float h, Mh, rate;
  __device__ __forceinline__ Weigher(float M, float h_, float rate_) : h(h_), Mh(M * h_), rate(rate_) {}
  __device__ __forceinline__ float operator()(float x) const { return ex2_approx(__fmul_rn(__fmaf_rn(x, h, -Mh), rate)); }
  __device__ __forceinline__ unsigned long long both(unsigned long long x) const {
    const unsigned long long y = pair_mul(f32x2_fma(x, f32x2_pack(h, h), f32x2_pack(-Mh, -Mh)), f32x2_pack(rate, rate));
    float a, b;
    f32x2_unpack(y, a, b);
    return f32x2_pack(ex2_approx(a), ex2_approx(b));
  }
};

// f(i) for i < m <= kPieces, U at a time.
template <int U, class F>
__device__ __forceinline__ void for_pieces(int m, F f) {
  int i = 0;
#pragma unroll 1
  for (; i + U <= m; i += U) {
#pragma unroll
    for (int j = 0; j < U; ++j) f(i + j);
  }
#pragma unroll 1
  for (; i < m; ++i) f(i);
}

// (maximum, sum) of a warp's pieces, continued over windows; `listed` the part of the sum that is marked.
struct WarpSum {
  float m = -INFINITY, z = 0.f, listed = 0.f;
};
// Adds the window's m pieces of this thread and its loose element (-inf: none). marks(i): the listed entries of piece i as
// bits, marks(-1): whether the loose one is.
template <class T, bool kMarks, class Marks>
__device__ __forceinline__ void add_pieces(WarpSum& s, const uint4* held, int m, float loose, float h, float rate, Marks marks) {
  constexpr int W = 8 / sizeof(T);
  const uint4* mine = held + threadIdx.x;
  float top = loose;
  for_pieces<4>(m, [&](int i) { top = nan_max(top, piece_max<T>(mine[i * kRowThreads])); });
  top = nan_max(s.m, warp_nan_max(top));
  if (top == -INFINITY) return;  // (the whole warp)
  const Weigher w(top, h, rate);
  if (s.m != -INFINITY) {
    const float f = w(s.m);
    s.z *= f;
    s.listed *= f;
  }
  s.m = top;
  unsigned long long a = 0, b = 0;
  float l = 0.f;
  for_pieces<2>(m, [&](int i) {
    unsigned long long x[W];
    split_piece<T>(mine[i * kRowThreads], x);
#pragma unroll
    for (int e = 0; e < W; ++e) x[e] = w.both(x[e]);
    if (kMarks) {
      const uint32_t bits = marks(i);
      if (bits) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
          float y0, y1;
          f32x2_unpack(x[e], y0, y1);
          if (bits >> (2 * e) & 1) l += y0, y0 = 0.f;
          if (bits >> (2 * e + 1) & 1) l += y1, y1 = 0.f;
          x[e] = f32x2_pack(y0, y1);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < W; e += 2) {
      a = pair_add(a, x[e]);
      b = pair_add(b, x[e + 1]);
    }
  });
  float a0, a1, b0, b1;
  f32x2_unpack(a, a0, a1);
  f32x2_unpack(b, b0, b1);
  if (loose != -INFINITY) {
    const float y = w(loose);
    if (kMarks && marks(-1)) l += y;
    else a0 += y;
  }
  s.z += (a0 + a1) + (b0 + b1);
  s.listed += l;
}

// The row's maximum and sums from those of all warps of the cluster, the same in every thread (a warp's lanes each
// take every 32nd entry, then a fixed tree).
struct RowSum {
  float M, z, listed;
};
__device__ __forceinline__ RowSum exchange(WarpSum s, float4* all, int C, int rank, float h, float rate) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  s.z = warp_sum(s.z);
  s.listed = warp_sum(s.listed);
  if (lane < C) store_peer(peer_address(all + rank * kRowWarps + warp, lane), make_float4(s.m, s.z, s.listed, 0.f));
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  RowSum r{-INFINITY, 0.f, 0.f};
  for (int i = lane; i < C * kRowWarps; i += 32) r.M = nan_max(r.M, all[i].x);
  r.M = warp_nan_max(r.M);
  if (r.M == -INFINITY) return r;
  const Weigher w(r.M, h, rate);
  for (int i = lane; i < C * kRowWarps; i += 32) {
    const float4 t = all[i];
    if (t.x == -INFINITY) continue;
    const float f = w(t.x);
    r.z += t.y * f;
    r.listed += t.z * f;
  }
  r.z = warp_sum(r.z);
  r.listed = warp_sum(r.listed);
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

template <class T, class To>
__global__ void __launch_bounds__(kRowThreads, 3) probabilities_kernel(ProbsParams p) {
  constexpr int E = 16 / sizeof(T), W = E / 2;
  extern __shared__ __align__(16) uint4 held[];
  __shared__ float4 all[kMaxCluster * kRowWarps];
  __shared__ uint32_t first[kMaxCluster * kRowWarps];
  const int rank = (int)cluster_rank(), C = p.C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster_arrive();  // the others' shared memory is theirs once they run: waited for before the exchange
  const size_t r = blockIdx.x / C;
  const RowPart<T> part(static_cast<const T*>(p.logits) + r * p.V, p.V, C, rank);
  part.fetch(held, 0);
  To* out = static_cast<To*>(p.probs) + r * p.V;
  const bool wide = (reinterpret_cast<uintptr_t>(out + part.a0) & (E * sizeof(To) - 1)) == 0;
  const float T_ = __ldg(p.temperature + r);
  const bool greedy = !(T_ > 0.f);
  // the smallest rate (T = inf) still takes an entry of -inf to weight 0
  const float rate0 = greedy ? 1.f : fmaxf(fminf(__fdiv_rn(1.44269504088896340736f, T_), 1e30f), 1e-45f);
  const float h = rate0 < 1e-36f ? 0.5f : 1.f, rate = rate0 < 1e-36f ? 2.f * rate0 : rate0;
  const int loose_at = part.own_loose(p.V), own = part.own();
  const float loose = loose_at >= 0 ? row_elem(part.row + loose_at) : -INFINITY;
  const int windows = max(1, (part.steps() + kPieces - 1) / kPieces);

  WarpSum s;
  for (int c = 0; c < windows; ++c) {
    if (c > 0) part.fetch(held, c * kPieces);
    copies_done();
    add_pieces<T, false>(s, held, min(own - c * kPieces, kPieces), c == 0 ? loose : -INFINITY, h, rate, [](int) { return 0u; });
  }
  cluster_wait();
  const RowSum sum = exchange(s, all, C, rank, h, rate);
  const bool bad = !(fabsf(sum.M) < INFINITY);
  if (bad && rank == 0 && threadIdx.x == 0) set_status(p.status, DSPARK_ERR_NONFINITE);
  // f(piece's number in the window's memory, first element) for this thread's pieces
  const auto each = [&](auto f) {
    for (int c = 0; c < windows; ++c) {
      if (windows > 1) {
        part.fetch(held, c * kPieces);
        copies_done();
      }
      const int m = min(own - c * kPieces, kPieces);
      for_pieces<2>(m, [&](int i) { f(held[i * kRowThreads + threadIdx.x], part.a0 + part.piece(c * kPieces + i) * E); });
    }
  };

  if (bad || greedy) {
    int top = INT_MAX;  // the first maximum
    if (!bad) {
      each([&](const uint4& q, int v) {
        unsigned long long x[W];
        split_piece<T>(q, x);
#pragma unroll
        for (int e = 0; e < W; ++e) {
          float x0, x1;
          f32x2_unpack(x[e], x0, x1);
          if (x0 == sum.M) top = min(top, v + 2 * e);
          if (x1 == sum.M) top = min(top, v + 2 * e + 1);
        }
      });
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
    for (int i = 0; i < own; ++i) {
      const int v = part.a0 + part.piece(i) * E;
      float y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = v + e == top ? 1.f : 0.f;
      store_piece<To, E>(out + v, y, wide);
    }
    if (loose_at >= 0) store_elem(out + loose_at, loose_at == top ? 1.f : 0.f);
    return;
  }
  const Weigher w(sum.M, h, rate);
  const float inv = __fdiv_rn(1.f, sum.z);
  each([&](const uint4& q, int v) {
    unsigned long long x[W];
    split_piece<T>(q, x);
    float y[E];
#pragma unroll
    for (int e = 0; e < W; ++e) f32x2_unpack(pair_mul(w.both(x[e]), f32x2_pack(inv, inv)), y[2 * e], y[2 * e + 1]);
    store_piece<To, E>(out + v, y, wide);
  });
  if (loose_at >= 0) store_elem(out + loose_at, w(loose) * inv);
}

// ---------------------------------------------------------------------------
struct DistillParams {
  int V, K, C, held, marks;  // bytes of the held pieces and of the map of marked entries
  const void* logits;
  const int32_t* ids;
  const float* teacher;
  const float* teacher_lse;
  const float* weight;
  double per_tau;      // 1 / temperature
  float k_hi, k_lo;    // log2(e) / temperature
  float* loss;
  void* grad;
  uint32_t* status;
};

__device__ __forceinline__ double warp_add_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// a b as a float and what its rounding left
struct Split {
  float hi, lo;
};
__device__ __forceinline__ Split product(float a, float b_hi, float b_lo) {
  const float p = __fmul_rn(a, b_hi);
  return {p, __fmaf_rn(a, b_lo, __fmaf_rn(a, b_hi, -p))};
}
// 2^(a - b) to float32's precision whatever the size of a and b: the difference with what rounding cut off, the power
// of its fraction
__device__ __forceinline__ float exp2_difference(Split a, Split b) {
  const float d = __fsub_rn(a.hi, b.hi), v = __fsub_rn(d, a.hi);
  const float cut = __fsub_rn(__fsub_rn(a.hi, __fsub_rn(d, v)), __fadd_rn(b.hi, v));
  const float n = fmaxf(rintf(d), -160.f);
  return ldexpf(exp2f(__fadd_rn(__fsub_rn(d, n), __fadd_rn(cut, __fsub_rn(a.lo, b.lo)))), (int)n);
}

template <class T, bool kRest>
__global__ void __launch_bounds__(kRowThreads, 3) distill_kernel(DistillParams p) {
  constexpr int E = 16 / sizeof(T), W = E / 2;
  extern __shared__ __align__(16) uint4 held[];
  __shared__ float4 all[kMaxCluster * kRowWarps];
  __shared__ double sums[kRowWarps];
  __shared__ float4 s_teacher;  // from CTA 0 of the cluster: 1 / share (or 1), share, what it leaves of 1, their sum
  __shared__ float maxima[kRowWarps];
  __shared__ uint32_t loose_marks;
  __shared__ int twice;
  // of the listed entries: the teacher's probability (CTA 0), its logit, the student's, the id (-1: none); then the map
  double* s_p = reinterpret_cast<double*>(reinterpret_cast<char*>(held) + p.held);
  float* s_t = reinterpret_cast<float*>(s_p + p.K);
  float* s_x = s_t + p.K;
  int* s_id = reinterpret_cast<int*>(s_x + p.K);
  uint32_t* s_marks = reinterpret_cast<uint32_t*>(s_id + p.K);
  const int rank = (int)cluster_rank(), C = p.C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster_arrive();
  const size_t r = blockIdx.x / C;
  const T* row = static_cast<const T*>(p.logits) + r * p.V;
  const RowPart<T> part(row, p.V, C, rank);
  part.fetch(held, 0);
  const float rate = p.k_hi;
  const int loose_at = part.own_loose(p.V), own = part.own();
  const float loose = loose_at >= 0 ? row_elem(row + loose_at) : -INFINITY;

  // the listed entries, in every CTA; those of this CTA's pieces are marked
  for (int i = tid; i < p.marks / 4; i += kRowThreads) s_marks[i] = 0;
  if (tid == 0) {
    loose_marks = 0;
    twice = 0;
  }
  __syncthreads();
  float t_max = -INFINITY;
  for (int j = tid; j < p.K; j += kRowThreads) {
    int id = __ldg(p.ids + r * p.K + j);
    float t = __ldg(p.teacher + r * p.K + j);
    if (id >= p.V) set_status(p.status, DSPARK_ERR_RANGE);
    if (id < 0 || id >= p.V) {
      id = -1;
      t = -INFINITY;
    }
    s_id[j] = id;
    s_t[j] = t;
    s_x[j] = id >= 0 ? row_elem(row + id) : -INFINITY;
    t_max = nan_max(t_max, t);
    int local, at;
    if (id >= 0 && part.owner(id, local, at) == rank) {
      uint32_t* word = local < 0 ? &loose_marks : s_marks + (local >> 2);
      const uint32_t bit = local < 0 ? 1u << (-1 - local) : 1u << ((local & 3) * 8 + at);
      if (atomicOr(word, bit) & bit) twice = 1;
    }
  }
  t_max = warp_nan_max(t_max);
  if (lane == 0) maxima[warp] = t_max;
  __syncthreads();
  t_max = lane < kRowWarps ? maxima[lane] : -INFINITY;
  t_max = warp_nan_max(t_max);
  const float lse = kRest ? __ldg(p.teacher_lse + r) : t_max;
  const bool none = t_max == -INFINITY;
  const bool bad_teacher = !(t_max < INFINITY) || (kRest && !(fabsf(lse) < INFINITY));
  const bool listless = none || bad_teacher;
  const Split ref = kRest ? product(lse, 1.44269502e+00f, 1.92596303e-08f) : product(lse, p.k_hi, p.k_lo);
  // an entry's share before it is scaled: relative to the largest entry, or to the teacher's sum
  const auto share_of = [&](int j) {
    const float t = s_t[j];
    return t == -INFINITY || listless ? 0.f : exp2_difference(product(t, p.k_hi, p.k_lo), ref);
  };
  const auto ln_p = [&](float t) { return kRest ? (double)t * p.per_tau - (double)lse : ((double)t - (double)lse) * p.per_tau; };
  // CTA 0: in float64, since what they leave of 1, and the logarithms' differences, may be small
  if (rank == 0) {
    if (warp * 32 < p.K) {
      double share = 0.0;
      for (int j = tid; j < p.K; j += kRowThreads) {
        const double e = listless || s_id[j] < 0 ? 0.0 : exp(ln_p(s_t[j]));
        s_p[j] = e;
        share += e;
      }
      share = warp_add_d(share);
      if (lane == 0) sums[warp] = share;
    }
    __syncthreads();
  }

  WarpSum s;
  const int windows = max(1, (part.steps() + kPieces - 1) / kPieces);
  for (int c = 0; c < windows; ++c) {
    if (c > 0) part.fetch(held, c * kPieces);
    copies_done();
    const auto marks = [&](int i) -> uint32_t {
      if (i < 0) return loose_marks >> tid & 1u;
      const int local = (c * kPieces + i) * kRowThreads + tid;
      return s_marks[local >> 2] >> ((local & 3) * 8) & 255u;
    };
    add_pieces<T, kRest>(s, held, min(own - c * kPieces, kPieces), c == 0 ? loose : -INFINITY, 1.f, rate, marks);
  }
  cluster_wait();
  double share = 0.0;
  if (rank == 0 && warp == 0) {
    for (int i = 0; i < min((p.K + 31) / 32, kRowWarps); ++i) share += sums[i];
    const double left = kRest ? fmax(0.0, 1.0 - share) : 0.0;
    if (lane < C)
      store_peer(peer_address(&s_teacher, lane),
                 make_float4(kRest ? 1.f : share > 0.0 ? __fdiv_rn(1.f, (float)share) : 0.f, (float)share, (float)left, (float)(share + left)));
  }
  const RowSum sum = exchange(s, all, C, rank, 1.f, rate);
  const bool bad = !(fabsf(sum.M) < INFINITY) || bad_teacher;
  const Weigher w(sum.M, 1.f, rate);
  const float z = sum.z + sum.listed, z_rest = sum.z;
  const float norm = s_teacher.x, p_rest = s_teacher.z;
  const bool some = kRest && p_rest > 0.f && z_rest > 0.f;  // a rest without mass on either side counts for nothing

  if (p.grad) {
    // d loss / d x_v = (1/tau) (s_v total - [rest] s_v p_rest / s_rest - p_v)
    T* grad = static_cast<T*>(p.grad) + r * p.V;
    const bool wide = (reinterpret_cast<uintptr_t>(grad + part.a0) & 15) == 0;
    const float scale = __fmul_rn(p.weight ? __ldg(p.weight + r) : 1.f, (float)p.per_tau);
    const float total = kRest ? (some ? s_teacher.w : s_teacher.y) : norm > 0.f ? 1.f : 0.f;
    const float per_z = total / z;
    const float listed_f = bad ? 0.f : scale * per_z;
    const float rest_f = bad ? 0.f : scale * (per_z - (some ? p_rest / z_rest : 0.f));
    for (int c = 0; c < windows; ++c) {
      if (windows > 1) {
        part.fetch(held, c * kPieces);
        copies_done();
      }
      const int m = min(own - c * kPieces, kPieces);
      for_pieces<2>(m, [&](int i) {
        unsigned long long x[W];
        split_piece<T>(held[i * kRowThreads + tid], x);
        float y[E];
#pragma unroll
        for (int e = 0; e < W; ++e) {
          f32x2_unpack(pair_mul(w.both(x[e]), f32x2_pack(rest_f, rest_f)), y[2 * e], y[2 * e + 1]);
          if (bad) y[2 * e] = y[2 * e + 1] = 0.f;
        }
        store_piece<T, E>(grad + part.a0 + (size_t)part.piece(c * kPieces + i) * E, y, wide);
      });
    }
    if (loose_at >= 0) store_elem(grad + loose_at, bad ? 0.f : w(loose) * rest_f);
    // the listed entries of this CTA over what was just written
    __syncthreads();
    for (int j = tid; j < p.K && !bad; j += kRowThreads) {
      const int id = s_id[j];
      int local, at;
      if (id < 0 || part.owner(id, local, at) != rank) continue;
      float e = share_of(j);
      if (twice) {  // an id that comes more than once: every occurrence writes the sum of all
        e = 0.f;
        for (int i = 0; i < p.K; ++i)
          if (s_id[i] == id) e += share_of(i);
      }
      store_elem(grad + id, __fmaf_rn(-scale * norm, e, w(s_x[j]) * listed_f));
    }
  }

  if (rank == 0 && warp == 0) {
    const double step = (double)rate * 0.69314718055994530942;  // 1 / tau as the weights have it
    double a = 0.0;
    for (int j = lane; j < p.K; j += 32) {
      const double e = s_p[j];
      if (e > 0.0) a += e * (ln_p(s_t[j]) - ((double)s_x[j] - (double)sum.M) * step);
    }
    a = warp_add_d(a);
    if (lane == 0) {
      double loss = 0.0;
      if (kRest) {
        const double left = fmax(0.0, 1.0 - share);
        loss = a + share * log((double)z);
        if (some) loss += left * log(left * ((double)z / (double)z_rest));
      } else if (share > 0.0) {
        loss = a / share + log((double)z / share);
      }
      p.loss[r] = bad ? NAN : (float)loss;
      if (bad) set_status(p.status, DSPARK_ERR_NONFINITE);
    }
  }
}

// ---------------------------------------------------------------------------
static int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// CTAs a row: as few as hold it, more while the rows leave SMs idle. `held`: the bytes that a CTA keeps of it.
static int row_cluster(int N, int V, int elem, int sms, int& held) {
  const long long pieces = (long long)V * elem / 16;
  int C = 1;
  while (C < kMaxCluster && (pieces > (long long)C * kRowThreads * kPieces || ((long long)N * C * 2 <= sms && pieces > (long long)C * kRowThreads)))
    C *= 2;
  held = std::min(kPieces, ceil_div(pieces, (long long)C * kRowThreads)) * kRowThreads * 16;
  return C;
}

template <class T, class To>
static cudaError_t launch_probs(const ProbsParams& p, int N, int held, cudaStream_t s) {
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = set_smem_limit_once((const void*)probabilities_kernel<T, To>, kPieces * kRowThreads * 16, attr);
  if (e != cudaSuccess) return e;
  return launch_clusters(probabilities_kernel<T, To>, p, (unsigned)N * p.C, p.C, kRowThreads, held, s);
}

// the pieces, 20 bytes a listed entry, and a byte for each piece of a row of 2^20 float32
constexpr int kDistillSmem = kPieces * kRowThreads * 16 + kMaxTop * 20 + (1 << 20) / 4 / kMaxCluster + kRowThreads;

template <class T, bool kRest>
static cudaError_t launch_distill(const DistillParams& p, int N, cudaStream_t s) {
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = set_smem_limit_once((const void*)distill_kernel<T, kRest>, kDistillSmem, attr);
  if (e != cudaSuccess) return e;
  return launch_clusters(distill_kernel<T, kRest>, p, (unsigned)N * p.C, p.C, kRowThreads, (size_t)p.held + (size_t)p.K * 20 + p.marks, s);
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
  int held;
  const int C = row_cluster(N, V, dtype == DSPARK_BF16 ? 2 : 4, sms, held);
  const ProbsParams p{V, C, logits, temperature, probs, static_cast<uint32_t*>(workspace)};
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (dtype == DSPARK_BF16)
    e = probs_dtype == DSPARK_BF16 ? launch_probs<__nv_bfloat16, __nv_bfloat16>(p, N, held, s)
                                   : launch_probs<__nv_bfloat16, float>(p, N, held, s);
  else
    e = probs_dtype == DSPARK_BF16 ? launch_probs<float, __nv_bfloat16>(p, N, held, s) : launch_probs<float, float>(p, N, held, s);
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
  int held;
  const int elem = dtype == DSPARK_BF16 ? 2 : 4;
  const int C = row_cluster(N, V, elem, sms, held);
  // one byte a piece of this CTA, whole steps of the block
  const int marks = ceil_div((long long)V * elem / 16, (long long)C * kRowThreads) * kRowThreads;
  const double k = 1.44269504088896340736 / (double)temperature;
  const DistillParams p{V, K, C, held, marks, logits, ids, teacher, teacher_lse, weight, 1.0 / (double)temperature, (float)k,
                        (float)(k - (double)(float)k), loss, grad,
                        static_cast<uint32_t*>(workspace)};
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (dtype == DSPARK_BF16) e = teacher_lse ? launch_distill<__nv_bfloat16, true>(p, N, s) : launch_distill<__nv_bfloat16, false>(p, N, s);
  else e = teacher_lse ? launch_distill<float, true>(p, N, s) : launch_distill<float, false>(p, N, s);
  note_launches(1);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
