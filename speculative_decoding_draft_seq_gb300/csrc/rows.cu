// Softmax over whole rows of logits: their probabilities under one temperature a
// row, and a drafter's divergence from a teacher's top logits with its gradient.
//
// Both need a row's maximum M and Z = sum 2^((x - M) r) before they can write
// anything of the row's size, and are bound by bytes (a row in, a row out) if the row is read
// once. So a cluster of CTAs holds a row in shared memory: every thread copies its own 16-byte
// pieces there (asynchronously; nobody else reads them, so it waits for itself only) and adds them up a group
// at a time as they arrive, the warps of all CTAs exchange their maxima and sums through
// distributed shared memory, and after one cluster barrier each thread combines them in the
// same order and writes its pieces. At kPieces pieces a thread three CTAs of an SM load, wait and write
// independently of each other (held in registers, one CTA an SM, the same took 2.5 times as long). A row longer than a
// cluster holds is taken in windows, which are read again for the results.
//
// Statistics are float32: a thread adds a group's weights in four chains (8 additions each for bf16, 4 for float32), joins these and a
// loose entry (3), groups one by one, then trees (5 over a warp, 7 over the cluster): at most 27 roundings in a sum over a row that is
// held at once (4 groups), 51 for 2^20 float32 (32). The loss of a distilled row is a small
// difference of large terms, so what it is made of (the listed entries' shares and sums, the logarithms) is kept in pairs of
// floats; float64, at 1/64 of the rate, took a third of the time.
//
// Measured (129,280 entries): 1,152 rows of bf16 to float32 probabilities 136 us (6.55 TB/s, 0.97 of the measured copy
// bandwidth), to bf16 100 (5.95); 2,048 rows of bf16 distilled with 64 entries each 196 us (5.4 TB/s, 0.80), 1,024 of float32
// 181 (0.87), the loss alone 117 (4.5 TB/s), with a rest 254 (the marks, the weights' second sum, and instructions that the cache
// does not hold; 248 without what far rests need), its loss alone 162; 256 entries a row 239, with a rest 333. All rows' rests
// far: 391, the loss alone 290. Lists of 1,024: 700, with a rest 513 (without one, repeated ids are found pairwise).
// One row of 32,000: probabilities 4.1 us. What holds the distillation below the copy rate: instructions (0.48 of the issue
// slots, at 30 warps an SM) and the meeting of a row's CTAs, once a row; the loss alone waits for the meetings most.
#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"
#include "mass.cuh"
#include "verify_common.cuh"

namespace dspark {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kPieces = 16;      // 16-byte pieces of a row that a thread holds
constexpr int kGroup = 4;        // pieces that are waited for and added together
constexpr int kGroups = kPieces / kGroup;
constexpr int kMaxCluster = 8;   // the portable limit
static_assert(kMaxCluster == 8, "RowPart takes its logarithm");
constexpr int kMaxTop = 1024;    // listed teacher entries of a row

__device__ __forceinline__ float nan_max(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float warp_nan_max(float v) {
  float d;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ void copy_async(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_done() {  // all groups but the last kLeft
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

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
  int a0, n, shift, rank;  // C = 2^shift, up to kMaxCluster
  __device__ RowPart(const T* r, int V, int C, int rank_) : row(r), shift((C >= 2) + (C >= 4) + (C >= 8)), rank(rank_) {
    const int off = (int)((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(T));
    a0 = min(off ? E - off : 0, V);
    n = (V - a0) / E;
  }
  __device__ __forceinline__ int piece(int i) const { return ((i << shift) + rank) * kRowThreads + (int)threadIdx.x; }
  // pieces that this thread owns
  __device__ __forceinline__ int own() const {
    return (n - 1 - (int)threadIdx.x + kRowThreads) / kRowThreads + (1 << shift) - 1 - rank >> shift;
  }
  __device__ __forceinline__ int steps() const { return ((n + kRowThreads - 1) / kRowThreads + (1 << shift) - 1) >> shift; }
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
    const int g = (v - a0) / E, block = g / kRowThreads;
    at = (v - a0) % E;
    local = (block >> shift) * kRowThreads + g % kRowThreads;
    return block & ((1 << shift) - 1);
  }
  // the word of the map that holds the marks of a piece with this local number, and the piece's byte in it
  static __device__ __forceinline__ int mark_word(int local) { return local / kRowThreads / kGroup * kRowThreads + local % kRowThreads; }
  static __device__ __forceinline__ int mark_byte(int local) { return local / kRowThreads % kGroup; }
  // starts the copies of group g of this thread's pieces i0 .. i0 + m - 1
  __device__ __forceinline__ void fetch_group(uint4* held, int i0, int m, int g) const {
    const T* from = row + a0 + (size_t)piece(i0) * E;
    const size_t step = (size_t)(E * kRowThreads) << shift;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const int k = g * kGroup + i;
      if (k < m) copy_async(held + k * kRowThreads + threadIdx.x, from + k * step);
    }
    copies_group();
  }
  __device__ __forceinline__ void fetch(uint4* held, int i0, int m) const {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) fetch_group(held, i0, m, g);
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
__device__ __forceinline__ uint4 empty_piece() {  // -inf throughout
  const uint32_t e = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
  return make_uint4(e, e, e, e);
}
// The piece with its marked entries at -inf.
template <class T>
__device__ __forceinline__ uint4 without_marked(const uint4& q, uint32_t marked) {
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      if (marked >> i & 1) w[i] = 0xff800000u;
    } else {
      if (marked >> (2 * i) & 1) w[i] = (w[i] & 0xffff0000u) | 0xff80u;
      if (marked >> (2 * i + 1) & 1) w[i] = (w[i] & 0xffffu) | 0xff800000u;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <class T>
__device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b) {  // of one float32 or two bf16
  uint32_t d;
  if constexpr (sizeof(T) == 4) d = __float_as_uint(nan_max(__uint_as_float(a), __uint_as_float(b)));
  else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <class T, int N>
__device__ __forceinline__ float pieces_max(const uint4 (&q)[N]) {
  uint32_t m = word_max<T>(word_max<T>(q[0].x, q[0].y), word_max<T>(q[0].z, q[0].w));
#pragma unroll
  for (int i = 1; i < N; ++i) m = word_max<T>(m, word_max<T>(word_max<T>(q[i].x, q[i].y), word_max<T>(q[i].z, q[i].w)));
  return sizeof(T) == 4 ? __uint_as_float(m) : nan_max(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
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

// Weights of a row's entries relative to its maximum M. Where M rate is of an ordinary size they are 2^(x rate - c), c the
// whole number nearest to M rate: the exponent is one fma, rounded once at its own size, and sums relative to other maxima
// differ by exact powers of two. Else they are 2^((x - M) rate), as fma(x, h, -M h) (rate / h), with h = 1/2 for rates so
// small that differences past float32's range count.
struct Rate {
  float h, rate;  // rate / h
};
__device__ __forceinline__ bool plain_exponent(const Rate& r, float M) { return r.h == 1.f && fabsf(M * r.rate) < 0x1p20f; }
__device__ __forceinline__ float origin(const Rate& r, float M) { return rintf(__fmul_rn(M, r.rate)); }
template <bool kPlain>
struct Weigher {
  float a, b, rate;
  __device__ __forceinline__ Weigher(const Rate& r, float M) : a(kPlain ? r.rate : r.h), b(kPlain ? -origin(r, M) : -M * r.h), rate(r.rate) {}
  __device__ __forceinline__ float operator()(float x) const {
    const float y = __fmaf_rn(x, a, b);
    return ex2_approx(kPlain ? y : __fmul_rn(y, rate));
  }
  __device__ __forceinline__ unsigned long long both(unsigned long long x) const {  // two entries, the same bits
    unsigned long long y = f32x2_fma(x, f32x2_pack(a, a), f32x2_pack(b, b));
    if (!kPlain) y = f32x2_mul(y, f32x2_pack(rate, rate));
    float y0, y1;
    f32x2_unpack(y, y0, y1);
    return f32x2_pack(ex2_approx(y0), ex2_approx(y1));
  }
};
// What a sum relative to x is multiplied by to be one relative to M >= x.
__device__ __forceinline__ float rescale(const Rate& r, float x, float M) {
  const bool plain_x = plain_exponent(r, x), plain_M = plain_exponent(r, M);
  if (plain_x && plain_M) {
    const float d = origin(r, x) - origin(r, M);
    return d < -126.f ? 0.f : __int_as_float((int)(127.f + d) << 23);
  }
  float y = __fmul_rn(__fmaf_rn(x, r.h, -M * r.h), r.rate);
  if (plain_x) y -= __fmaf_rn(x, r.rate, -origin(r, x));
  if (plain_M) y += __fmaf_rn(M, r.rate, -origin(r, M));
  return ex2_approx(y);
}

// (maximum, sum) of a thread's entries so far; `listed` the part of the sum that is marked.
struct ThreadSum {
  float m = -INFINITY, z = 0.f, listed = 0.f;
};
// Adds kGroup pieces and a loose element (-inf: none). marks: the marked entries of each piece, a byte each;
// loose_mark: whether the loose one is.
template <class T, bool kMarks, bool kPlain>
__device__ __forceinline__ void add_weights(ThreadSum& s, const uint4 (&q)[kGroup], float loose, const Rate& r, uint32_t marks, bool loose_mark) {
  constexpr int W = 8 / sizeof(T);
  const Weigher<kPlain> w(r, s.m);
  unsigned long long a = 0, b = 0;
  float l = 0.f;
#pragma unroll
  for (int i = 0; i < kGroup; ++i) {
    unsigned long long x[W];
    split_piece<T>(q[i], x);
#pragma unroll
    for (int e = 0; e < W; ++e) x[e] = w.both(x[e]);
    if (kMarks) {
      const uint32_t marked = marks >> (8 * i) & 255u;
      if (marked) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
          float y0, y1;
          f32x2_unpack(x[e], y0, y1);
          if (marked >> (2 * e) & 1) l += y0, y0 = 0.f;
          if (marked >> (2 * e + 1) & 1) l += y1, y1 = 0.f;
          x[e] = f32x2_pack(y0, y1);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < W; e += 2) {
      a = f32x2_add(a, x[e]);
      b = f32x2_add(b, x[e + 1]);
    }
  }
  float a0, a1, b0, b1;
  f32x2_unpack(a, a0, a1);
  f32x2_unpack(b, b0, b1);
  if (loose != -INFINITY) {
    const float y = w(loose);
    if (kMarks && loose_mark) l += y;
    else a0 += y;
  }
  s.z += (a0 + a1) + (b0 + b1);
  if (kMarks) s.listed += l;
}
template <class T, bool kMarks>
__device__ __forceinline__ void add_pieces(ThreadSum& s, const uint4 (&q)[kGroup], float loose, const Rate& r, uint32_t marks, bool loose_mark) {
  const float top = nan_max(nan_max(s.m, loose), pieces_max<T>(q));
  if (top == -INFINITY) return;
  if (top != s.m) {
    if (s.m != -INFINITY) {
      const float f = rescale(r, s.m, top);
      s.z *= f;
      if (kMarks) s.listed *= f;
    }
    s.m = top;
  }
  if (plain_exponent(r, top)) add_weights<T, kMarks, true>(s, q, loose, r, marks, loose_mark);
  else add_weights<T, kMarks, false>(s, q, loose, r, marks, loose_mark);
}
template <class T, bool kMarks>
__device__ __forceinline__ void add_group(ThreadSum& s, const uint4* mine, int m, float loose, const Rate& r, uint32_t marks, bool loose_mark) {
  static_assert(kGroup == 4, "a byte a piece");
  uint4 q[kGroup];
#pragma unroll
  for (int i = 0; i < kGroup; ++i) q[i] = i < m ? mine[i * kRowThreads] : empty_piece<T>();
  add_pieces<T, kMarks>(s, q, loose, r, marks, loose_mark);
}
// A window's pieces, a group as soon as it has arrived; marks(g): the marked entries of group g; after(g) may start another
// group's copies over group g's (kRefill).
template <class T, bool kMarks, bool kRefill, int g, class Marks, class After>
__device__ __forceinline__ void add_groups(ThreadSum& s, const uint4* mine, int m, float loose, const Rate& r, Marks marks, bool loose_mark,
                                           After after) {
  copies_done<kRefill ? kGroups - 1 : kGroups - 1 - g>();
  if (g == 0 || m > g * kGroup)
    add_group<T, kMarks>(s, mine + g * kGroup * kRowThreads, m - g * kGroup, g == 0 ? loose : -INFINITY, r, kMarks ? marks(g) : 0u,
                         loose_mark);
  after(g);
  if constexpr (g + 1 < kGroups) add_groups<T, kMarks, kRefill, g + 1>(s, mine, m, loose, r, marks, loose_mark, after);
}

// A value as a float and what its rounding left.
struct Split {
  float hi, lo;
};
__device__ __forceinline__ Split two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), v = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v))};
}
__device__ __forceinline__ Split product(float a, float b_hi, float b_lo) {
  const float p = __fmul_rn(a, b_hi);
  return {p, __fmaf_rn(a, b_lo, __fmaf_rn(a, b_hi, -p))};
}
__device__ __forceinline__ Split add(Split a, Split b) {
  const Split s = two_sum(a.hi, b.hi);
  const float lo = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)), hi = __fadd_rn(s.hi, lo);
  return {hi, __fsub_rn(lo, __fsub_rn(hi, s.hi))};
}
__device__ __forceinline__ Split warp_add(Split v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = add(v, Split{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}

// Where every warp's part of the unlisted entries' sum, relative to the row's maximum, is below this, they are summed once more,
// relative to their own maximum. Down to it what weights lose below 2^-126 is 2^-60 of the sum an entry, and no quotient
// by the sum overflows; below, the sum would first lose entries and then be 0, where its logarithm and its entries' shares in it
// are of an ordinary size. (Of parts, not of their sum: every thread of the cluster has to find the same, those that sum pairs of
// floats too.)
constexpr float kFarRest = 0x1p-66f;

// The row's maximum and sums from those of all warps of the cluster, the same in every thread (a warp's lanes each
// take every 32nd entry, then a fixed tree).
struct RowSum {
  float M, z, listed;
  bool far;  // kMarks: z is below kFarRest, all warps' parts of it are
  float z_lo, listed_lo;  // kPair: what the sums' roundings left
};
template <bool kMarks>
__device__ __forceinline__ void send(const ThreadSum& s, float4* all, int C, int rank, const Rate& rate) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float m = warp_nan_max(s.m);
  const float f = s.m == -INFINITY ? 0.f : rescale(rate, s.m, m);
  const float zw = warp_sum(s.z * f), lw = kMarks ? warp_sum(s.listed * f) : 0.f;
  if (lane < C) store_peer(peer_address(all + rank * kRowWarps + warp, lane), make_float4(m, zw, lw, 0.f));
  __syncwarp();
}
template <bool kMarks, bool kPair>
__device__ __forceinline__ RowSum combine(const float4* all, int C, const Rate& rate) {
  const int lane = threadIdx.x & 31;
  RowSum r{-INFINITY, 0.f, 0.f, false, 0.f, 0.f};
  const int n = C * kRowWarps;
  constexpr int L = kMaxCluster * kRowWarps / 32;  // entries a lane
  float4 t[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    t[i] = lane + 32 * i < n ? all[lane + 32 * i] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    r.M = nan_max(r.M, t[i].x);
  }
  r.M = warp_nan_max(r.M);
  if (r.M == -INFINITY) return r;
  bool near = !(fabsf(r.M) < INFINITY);
  if constexpr (kPair) {
    Split z{0.f, 0.f}, l = z;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const float g = t[i].x == -INFINITY ? 0.f : rescale(rate, t[i].x, r.M);
      near |= __fmul_rn(t[i].y, g) >= kFarRest;
      z = add(z, product(t[i].y, g, 0.f));
      if (kMarks) l = add(l, product(t[i].z, g, 0.f));
    }
    z = warp_add(z);
    r.z = z.hi, r.z_lo = z.lo;
    if (kMarks) l = warp_add(l), r.listed = l.hi, r.listed_lo = l.lo;
  } else {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const float g = t[i].x == -INFINITY ? 0.f : rescale(rate, t[i].x, r.M);
      near |= __fmul_rn(t[i].y, g) >= kFarRest;
      r.z = __fmaf_rn(t[i].y, g, r.z);
      if (kMarks) r.listed = __fmaf_rn(t[i].z, g, r.listed);
    }
    r.z = warp_sum(r.z);
    if (kMarks) r.listed = warp_sum(r.listed);
  }
  if (kMarks) r.far = !__any_sync(0xffffffffu, near);
  return r;
}

template <bool kMarks>
__device__ __forceinline__ RowSum receive(const float4* all, int C, const Rate& rate) {
  cluster_arrive();
  cluster_wait();
  return combine<kMarks, false>(all, C, rate);
}

// ---------------------------------------------------------------------------
struct ProbsParams {
  int V, C;
  const void* logits;
  const float* temperature;
  void* probs;
  uint32_t* status;
};

template <class T, class To, bool kPlain>
__device__ __forceinline__ void scaled_piece(const uint4& q, const Weigher<kPlain>& w, float by, To* out, bool wide) {
  constexpr int E = 16 / sizeof(T), W = E / 2;
  unsigned long long x[W];
  split_piece<T>(q, x);
  float y[E];
#pragma unroll
  for (int e = 0; e < W; ++e) f32x2_unpack(f32x2_mul(w.both(x[e]), f32x2_pack(by, by)), y[2 * e], y[2 * e + 1]);
  store_piece<To, E>(out, y, wide);
}
// out[v] = weight of entry v times `by`, for this thread's pieces and its loose element; after(g) as above.
template <class T, class To, bool kPlain, class After>
__device__ __forceinline__ void write_weights(const RowPart<T>& part, uint4* held, int own, int windows, const Weigher<kPlain>& w, float by,
                                              To* out, bool wide, int loose_at, float loose, After after) {
  constexpr int E = 16 / sizeof(T);
  static_assert(kGroup % 2 == 0, "pieces two at a time");
  const size_t step = (size_t)(E * kRowThreads) << part.shift;
  for (int c = 0; c < windows; ++c) {
    const int m = min(own - c * kPieces, kPieces);
    if (windows > 1) {
      part.fetch(held, c * kPieces, m);
      copies_done<0>();
    }
    To* to = out + part.a0 + (size_t)part.piece(c * kPieces) * E;
    const uint4* mine = held + threadIdx.x;
#pragma unroll 1
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int i = 0; i < kGroup; i += 2) {
        if (g * kGroup + i + 1 < m) {
          const uint4 q0 = mine[i * kRowThreads], q1 = mine[(i + 1) * kRowThreads];
          scaled_piece<T>(q0, w, by, to + i * step, wide);
          scaled_piece<T>(q1, w, by, to + (i + 1) * step, wide);
        } else if (g * kGroup + i < m) {
          scaled_piece<T>(mine[i * kRowThreads], w, by, to + i * step, wide);
        }
      }
      after(g);
      to += kGroup * step;
      mine += kGroup * kRowThreads;
    }
  }
  if (loose_at >= 0) store_elem(out + loose_at, w(loose) * by);
}
// out[v] = 1 at v = top, else 0
template <class T, class To>
__device__ __forceinline__ void write_one(const RowPart<T>& part, int own, int top, To* out, bool wide, int loose_at) {
  constexpr int E = 16 / sizeof(T);
#pragma unroll 1
  for (int i = 0; i < own; ++i) {
    const int v = part.a0 + part.piece(i) * E;
    float y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = v + e == top ? 1.f : 0.f;
    store_piece<To, E>(out + v, y, wide);
  }
  if (loose_at >= 0) store_elem(out + loose_at, loose_at == top ? 1.f : 0.f);
}

template <class T, class To>
__global__ void __launch_bounds__(kRowThreads, 3) probabilities_kernel(ProbsParams p) {
  constexpr int E = 16 / sizeof(T), W = E / 2;
  extern __shared__ __align__(128) uint4 held[];  // (copies to unaligned lines take a tenth longer)
  __shared__ float4 all[kMaxCluster * kRowWarps];
  __shared__ uint32_t first[kMaxCluster * kRowWarps];
  const int rank = (int)cluster_rank(), C = p.C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster_arrive_relaxed();  // the others' shared memory is theirs once they run: waited for before the exchange
  const size_t r = blockIdx.x / C;
  const RowPart<T> part(static_cast<const T*>(p.logits) + r * p.V, p.V, C, rank);
  const int own = part.own();
  part.fetch(held, 0, min(own, kPieces));
  To* out = static_cast<To*>(p.probs) + r * p.V;
  const bool wide = (reinterpret_cast<uintptr_t>(out + part.a0) & (E * sizeof(To) - 1)) == 0;
  const float T_ = __ldg(p.temperature + r);
  const bool greedy = !(T_ > 0.f);
  // the smallest rate (T = inf) still takes an entry of -inf to weight 0
  const float rate0 = greedy ? 1.f : fmaxf(fminf(__fdiv_rn(1.44269504088896340736f, T_), 1e30f), 1e-45f);
  const Rate rate{rate0 < 1e-36f ? 0.5f : 1.f, rate0 < 1e-36f ? 2.f * rate0 : rate0};
  const int loose_at = part.own_loose(p.V);
  const float loose = loose_at >= 0 ? row_elem(part.row + loose_at) : -INFINITY;
  const int windows = max(1, (part.steps() + kPieces - 1) / kPieces);

  ThreadSum s;
  for (int c = 0; c < windows; ++c) {
    const int m = min(own - c * kPieces, kPieces);
    if (c > 0) part.fetch(held, c * kPieces, m);
    add_groups<T, false, false, 0>(s, held + threadIdx.x, m, c == 0 ? loose : -INFINITY, rate, [](int) { return 0u; }, false, [](int) {});
  }
  cluster_wait();
  send<false>(s, all, C, rank, rate);
  const RowSum sum = receive<false>(all, C, rate);
  const bool bad = !(fabsf(sum.M) < INFINITY);
  if (bad && rank == 0 && threadIdx.x == 0) set_status(p.status, DSPARK_ERR_NONFINITE);
  if (bad) {
    write_one(part, own, -1, out, wide, loose_at);
  } else if (greedy) {
    int top = INT_MAX;  // the first maximum
    for (int c = 0; c < windows; ++c) {
      const int m = min(own - c * kPieces, kPieces);
      if (windows > 1) {
        part.fetch(held, c * kPieces, m);
        copies_done<0>();
      }
#pragma unroll 1
      for (int i = 0; i < m; ++i) {
        const int v = part.a0 + part.piece(c * kPieces + i) * E;
        unsigned long long x[W];
        split_piece<T>(held[i * kRowThreads + threadIdx.x], x);
#pragma unroll
        for (int e = 0; e < W; ++e) {
          float x0, x1;
          f32x2_unpack(x[e], x0, x1);
          if (x0 == sum.M) top = min(top, v + 2 * e);
          if (x1 == sum.M) top = min(top, v + 2 * e + 1);
        }
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
    write_one(part, own, warp_min_i(top), out, wide, loose_at);
  } else if (plain_exponent(rate, sum.M)) {
    write_weights(part, held, own, windows, Weigher<true>(rate, sum.M), __fdiv_rn(1.f, sum.z), out, wide, loose_at, loose, [](int) {});
  } else {
    write_weights(part, held, own, windows, Weigher<false>(rate, sum.M), __fdiv_rn(1.f, sum.z), out, wide, loose_at, loose, [](int) {});
  }
}

// ---------------------------------------------------------------------------
struct DistillParams {
  int N, V, K, C, windows, held, marks;  // held, marks: bytes of the held pieces and of the map of marked entries
  const void* logits;
  const int32_t* ids;
  const float* teacher;
  const float* teacher_lse;
  const float* weight;
  float per_tau;       // 1 / temperature
  float k_hi, k_lo;    // log2(e) / temperature
  float* loss;
  void* grad;
  uint32_t* status;
};

__device__ __forceinline__ Split times(Split a, Split b) {
  const float p = __fmul_rn(a.hi, b.hi);
  return {p, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.hi, -p)))};
}
constexpr float kLn2 = 0.693147182f, kLn2Lo = -1.90465421e-9f;
// 2^(a - b) within 2^-27 of it, whatever the size of a and b: float64 would do it on 1/64 of the lanes. With
// a - b = n + f and u = f ln 2, |u| < 0.35, the exponential series of u: its first three terms with what their roundings
// leave, the rest (to u^9 / 9!, below 2^-37) in float32.
__device__ __forceinline__ Split exp2_difference(Split a, Split b, Split& difference) {
  const Split d = two_sum(a.hi, -b.hi);
  difference = {d.hi, __fadd_rn(d.lo, __fsub_rn(a.lo, b.lo))};
  if (d.hi < -150.f) return {0.f, 0.f};
  const float n = rintf(d.hi);
  const Split f = two_sum(__fsub_rn(d.hi, n), difference.lo);  // (the subtraction is exact)
  const float u = __fmul_rn(f.hi, kLn2), u_lo = __fmaf_rn(f.lo, kLn2, __fmaf_rn(f.hi, kLn2Lo, __fmaf_rn(f.hi, kLn2, -u)));
  const float s = __fmul_rn(u, u), s_lo = __fmaf_rn(2.f * u, u_lo, __fmaf_rn(u, u, -s));
  float q = 1.f / 362880.f;
  q = __fmaf_rn(q, u, 1.f / 40320.f);
  q = __fmaf_rn(q, u, 1.f / 5040.f);
  q = __fmaf_rn(q, u, 1.f / 720.f);
  q = __fmaf_rn(q, u, 1.f / 120.f);
  q = __fmaf_rn(q, u, 1.f / 24.f);
  q = __fmaf_rn(q, u, 1.f / 6.f);
  const Split w = two_sum(0.5f * s, __fmul_rn(__fmul_rn(s, u), q));
  const Split v = two_sum(1.f, u), t = two_sum(v.hi, w.hi);
  const float lo = __fadd_rn(__fadd_rn(t.lo, v.lo), __fadd_rn(w.lo, __fadd_rn(u_lo, 0.5f * s_lo)));
  return {ldexpf(__fadd_rn(t.hi, lo), (int)n), ldexpf(__fsub_rn(lo, __fsub_rn(__fadd_rn(t.hi, lo), t.hi)), (int)n)};
}
// ln v, v > 0, within 2^-27 whatever its size: the logarithm of v's fraction to float32, and what its power leaves of the
// fraction
__device__ __forceinline__ Split ln_of(Split v) {
  int e;
  float m = frexpf(v.hi, &e);  // [1/2, 1)
  if (m < 0.70710678f) m *= 2.f, --e;
  const float y = logf(m);
  Split unused;
  const Split q = times(exp2_difference(Split{0.f, 0.f}, product(y, 1.44269502e+00f, 1.92596299e-08f), unused), Split{m, 0.f});  // m e^-y
  const float left = __fadd_rn(add(q, Split{-1.f, 0.f}).hi, __fdiv_rn(v.lo, v.hi));
  return add(product((float)e, kLn2, kLn2Lo), two_sum(y, left));
}
__device__ __forceinline__ Split negative(Split v) { return {-v.hi, -v.lo}; }
__device__ __forceinline__ Split quotient(Split a, Split b) {
  const float inv = __fdiv_rn(1.f, b.hi), q = __fmul_rn(a.hi, inv);
  return two_sum(q, __fmul_rn(add(a, negative(times(b, Split{q, 0.f}))).hi, inv));
}

// What a CTA knows of those of a row's listed entries that lie in its pieces: the sum of their shares e, and of e log2 e
// and e x. As pairs of floats, since what the shares leave of 1, and differences of logarithms, may be small (a float64
// instruction takes the SM 16 cycles a warp).
enum { kNoList = 1, kBadList = 2 };  // (of the whole row) nothing listed has a share; a NaN or infinity among the teacher's numbers
constexpr float kFar = 1e32f;  // teacher's logits count up to here, so that none times log2(e) / tau overflows (masked ones do not differ)
__device__ __forceinline__ float clamped(float t) { return fminf(fmaxf(t, -kFar), kFar); }
constexpr float kSmall = 0x1p-40f;
struct __align__(16) ListSums {
  Split share, e_log_e;
  Split e_x;  // times kSmall: masked entries hold the type's lowest value, of which a sum would overflow
  int flags, unused;
};
// A listed entry as the gradient needs it.
struct Listed {
  float e, x;  // the teacher's share (before that, its logit) and the drafter's logit
  int id;      // -1: none
};

constexpr int kListThreads = 64;
constexpr int kDistillThreads = kRowThreads + kListThreads;
template <int kId, int kThreads>
__device__ __forceinline__ void named_sync() { asm volatile("barrier.cta.sync %0, %1;" ::"n"(kId), "n"(kThreads) : "memory"); }
template <int kId, int kThreads>
__device__ __forceinline__ void named_arrive() { asm volatile("barrier.cta.arrive %0, %1;" ::"n"(kId), "n"(kThreads) : "memory"); }
enum { kMarksReady = 1, kRowWritten = 2, kListSync = 3 };  // named barriers

// What a row with a far rest needs besides, as functions of their own: in line their registers cost the other rows time (the loss
// alone of 2,048 rows 166 us for 162, with the gradient 255.6 for 255; without any of it 156 and 249).
// The streaming threads' part: each one's unlisted entries, from the row itself (what held it may already hold the next one), then
// the cluster's exchange. loose: the loose element (-inf: none, or listed).
template <class T>
__device__ __noinline__ RowSum unlisted_sum(RowPart<T> part, int own, float loose, Rate r, const uint32_t* s_marks, int words, float4* apart) {
  ThreadSum s;
#pragma unroll 1
  for (int i0 = 0; i0 < own || i0 == 0; i0 += kGroup) {
    const int word = i0 / kGroup * kRowThreads + (int)threadIdx.x;
    const uint32_t marks = word < words ? s_marks[word] : 0u;
    uint4 q[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      q[i] = empty_piece<T>();
      if (i0 + i < own) q[i] = *reinterpret_cast<const uint4*>(part.row + part.a0 + (size_t)part.piece(i0 + i) * RowPart<T>::E);
      q[i] = without_marked<T>(q[i], marks >> (8 * i) & 255u);
    }
    add_pieces<T, false>(s, q, i0 == 0 ? loose : -INFINITY, r, 0u, false);
  }
  const int C = 1 << part.shift;
  send<false>(s, apart, C, part.rank, r);
  return receive<false>(apart, C, r);
}
// The list's warps take part in that exchange: the sum.
__device__ __noinline__ float unlisted_received(const float4* apart, int C, Rate r) {
  cluster_arrive();
  cluster_wait();
  return combine<false, false>(apart, C, r).z;
}
// The same after it, with what its roundings left.
__device__ __noinline__ RowSum unlisted_pair(const float4* apart, int C, Rate r) { return combine<false, true>(apart, C, r); }
// p_R (ln p_R - ln s_R) times kSmall, with p_R = left, ln_z the logarithm of the row's sum relative to its maximum M. (One thread's.)
__device__ __noinline__ Split far_term(RowSum rest, Rate r, float M, Split left, Split ln_z) {
  const bool plain_rest = plain_exponent(r, rest.M), plain_M = plain_exponent(r, M);
  const Split k{r.rate, 0.f};
  // in octaves, times kSmall: what a weight of 1 relative to rest.M is relative to M
  const auto level = [&](float x, bool plain) { return plain ? Split{origin(r, x) * kSmall, 0.f} : times(Split{x * kSmall, 0.f}, k); };
  const Split octaves = plain_rest || plain_M ? add(level(rest.M, plain_rest), negative(level(M, plain_M)))
                                              : times(two_sum(rest.M * kSmall, -M * kSmall), k);
  const Split near = add(add(ln_of(left), negative(ln_of(Split{rest.z, rest.z_lo}))), ln_z);
  return times(left, add(Split{near.hi * kSmall, near.lo * kSmall}, negative(times(octaves, Split{kLn2, kLn2Lo}))));
}

// What the weights of a row are multiplied by in its gradient: entries of the rest, listed ones; and the teacher's shares.
// z_rest: the rest's sum, relative to an origin at which a weight of 1 is one of to_M relative to the row's maximum; the rest's
// weights are to be relative to it too.
struct Factors {
  float rest, listed, teacher;
  bool bad, some;  // some: a rest without mass on either side counts for nothing
};
template <bool kRest>
__device__ __forceinline__ Factors factors(const ListSums* of, int C, const RowSum& sum, float z_rest, float to_M, float weight, float per_tau) {
  Split share{0.f, 0.f};
  for (int c = 0; c < C; ++c) share = add(share, of[c].share);
  const Split rest = two_sum(1.f, -share.hi);
  const float left = kRest ? fmaxf(0.f, __fadd_rn(rest.hi, __fsub_rn(rest.lo, share.lo))) : 0.f, all = __fadd_rn(share.hi, share.lo);
  const int flags = of[0].flags;
  Factors f;
  f.bad = !(fabsf(sum.M) < INFINITY) || flags & kBadList;
  f.some = kRest && left > 0.f && z_rest > 0.f;
  const float scale = __fmul_rn(weight, per_tau);
  const float per_z = __fdiv_rn(kRest ? (f.some ? fmaxf(1.f, all) : all) : flags & kNoList ? 0.f : 1.f, sum.z + sum.listed);
  f.listed = scale * per_z;
  f.rest = scale * (kRest ? __fmaf_rn(per_z, to_M, f.some ? -__fdiv_rn(left, z_rest) : 0.f) : per_z);
  f.teacher = kRest ? scale : flags & kNoList ? 0.f : scale * __fdiv_rn(1.f, all);
  return f;
}

// A cluster takes rows cluster, cluster + clusters, .. one after the other. kRowThreads threads of a CTA stream: a row's
// pieces are overwritten by the next row's as soon as they have been used for the last time, so that the next row
// arrives while this one's gradient leaves. Two more warps look after the listed entries: they load and mark the next
// row's and form its sums while this row is written, then put this row's listed entries over what was written. The two groups
// meet once a row, at the cluster's exchange (with a rest also where the marks have to be ready).
template <class T, bool kRest, bool kGrad>
__global__ void __launch_bounds__(kDistillThreads, 3) distill_kernel(DistillParams p) {
  extern __shared__ __align__(128) uint4 held[];  // (copies to unaligned lines take a tenth longer)
  // two sets each: a CTA may write the next row's while another still reads this one's
  __shared__ float4 all[2][kMaxCluster * kRowWarps];
  __shared__ ListSums teachers[2][kMaxCluster];
  __shared__ Split sums[kListThreads / 32][3];
  __shared__ int counts[2][kListThreads / 32];
  __shared__ float maxima[kListThreads / 32];
  __shared__ uint32_t loose_marks;
  __shared__ int twice[2];
  __shared__ float4 apart[kRest ? kMaxCluster * kRowWarps : 1];  // of the unlisted entries, relative to their own maxima
  const int half = (p.K + 1) / 2;  // a warp's part of a list
  Listed* lists = reinterpret_cast<Listed*>(reinterpret_cast<char*>(held) + p.held);  // two rows' two parts
  uint32_t* s_marks = reinterpret_cast<uint32_t*>(lists + 4 * half);
  const int rank = (int)cluster_rank(), C = p.C, tid = threadIdx.x, lane = tid & 31;
  cluster_arrive_relaxed();
  const int clusters = gridDim.x / C;
  const Rate rate{1.f, p.k_hi};
  const T* logits = static_cast<const T*>(p.logits);
  const auto part_of = [&](int r) { return RowPart<T>(logits + (size_t)r * p.V, p.V, C, rank); };
  int r = blockIdx.x / C;

  if (tid < kRowThreads) {
    RowPart<T> part = part_of(r);
    int own = part.own();
    if (p.windows == 1) part.fetch(held, 0, own);
    cluster_wait();
#pragma unroll 1
    for (int turn = 0; r < p.N; turn ^= 1) {
      const int loose_at = part.own_loose(p.V);
      const float loose = loose_at >= 0 ? row_elem(part.row + loose_at) : -INFINITY;
      const int r_next = r + clusters;
      const RowPart<T> follow = part_of(min(r_next, p.N - 1));
      const int own_next = r_next < p.N && p.windows == 1 ? follow.own() : 0;
      const auto refill = [&](int g) { follow.fetch_group(held, 0, own_next, g); };
      if (kRest) named_sync<kMarksReady, kDistillThreads>();
      ThreadSum s;
      const bool loose_mark = kRest && loose_at >= 0 && (loose_marks >> tid & 1u);
      if (p.windows == 1) {
        const auto marks = [&](int g) { return g * kRowThreads + tid < p.marks / 4 ? s_marks[g * kRowThreads + tid] : 0u; };
        if constexpr (kGrad) add_groups<T, kRest, false, 0>(s, held + tid, own, loose, rate, marks, loose_mark, [](int) {});
        else add_groups<T, kRest, true, 0>(s, held + tid, own, loose, rate, marks, loose_mark, refill);
      } else {
        for (int c = 0; c < p.windows; ++c) {
          const int m = min(own - c * kPieces, kPieces);
          part.fetch(held, c * kPieces, m);
          add_groups<T, kRest, false, 0>(s, held + tid, m, c == 0 ? loose : -INFINITY, rate,
                                         [&](int g) {
                                           const int word = (c * kGroups + g) * kRowThreads + tid;
                                           return word < p.marks / 4 ? s_marks[word] : 0u;
                                         },
                                         loose_mark, [](int) {});
        }
      }
      send<kRest>(s, all[turn], C, rank, rate);
      const RowSum sum = receive<kRest>(all[turn], C, rate);
      float rest_M = sum.M;  // the entry that the rest's weights are relative to
      const auto row_factors = [&](float z_rest, float to_M) {
        return factors<kRest>(teachers[turn], C, sum, z_rest, to_M, p.weight ? __ldg(p.weight + r) : 1.f, p.per_tau);
      };
      Factors f{};
      if constexpr (kGrad) f = row_factors(sum.z, 1.f);
      if constexpr (kRest) {
        if (sum.far) {
          const RowSum unlisted = unlisted_sum(part, own, loose_mark ? -INFINITY : loose, rate, s_marks, p.marks / 4, apart);
          if (kGrad && unlisted.M != -INFINITY) {
            rest_M = unlisted.M;
            f = row_factors(unlisted.z, rescale(rate, rest_M, sum.M));
          }
        }
      }
      if constexpr (kGrad) {
        // d loss / d x_v = (1/tau) (s_v total - [rest] s_v p_rest / s_rest - p_v), here without the last term
        T* grad = static_cast<T*>(p.grad) + (size_t)r * p.V;
        const bool wide = (reinterpret_cast<uintptr_t>(grad + part.a0) & 15) == 0;
        const auto after = [&](int g) {
          if (p.windows == 1) refill(g);
        };
        if (f.bad) {
          write_one(part, own, -1, grad, wide, loose_at);
#pragma unroll 1
          for (int g = 0; g < kGroups; ++g) after(g);
        } else if (plain_exponent(rate, rest_M)) {
          write_weights(part, held, own, p.windows, Weigher<true>(rate, rest_M), f.rest, grad, wide, loose_at, loose, after);
        } else {
          write_weights(part, held, own, p.windows, Weigher<false>(rate, rest_M), f.rest, grad, wide, loose_at, loose, after);
        }
        named_arrive<kRowWritten, kDistillThreads>();
      }
      r = r_next;
      part = follow;
      own = part.own();
    }
    copies_done<0>();
    return;
  }

  // The listed entries: each warp goes through half of the list and keeps, in order, those in this CTA's pieces.
  const int j0 = tid - kRowThreads, warp = j0 >> 5;
  struct Row {
    int n, flags;  // entries kept by this warp
  };
  const auto list_of = [&](int turn, int w) { return lists + (turn * 2 + w) * half; };
  // The first kEarly entries of the warp's half, loaded ahead of their use: ids and logits, then the drafter's logits.
  constexpr int kEarly = 64;
  struct Early {
    int id[kEarly / 32];
    float t[kEarly / 32], x[kEarly / 32];
  };
  const int first = warp * half, last = min(first + half, p.K);
  const auto load = [&](int r, Early& e) {
#pragma unroll
    for (int i = 0; i < kEarly / 32; ++i) {
      const int j = first + 32 * i + lane;
      e.id[i] = -1;
      e.t[i] = -INFINITY;
      if (r < p.N && j < last) {
        asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(e.id[i]) : "l"(p.ids + (size_t)r * p.K + j));
        asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(e.t[i]) : "l"(p.teacher + (size_t)r * p.K + j));
      }
    }
  };
  const auto is_mine = [&](const RowPart<T>& part, int id) {
    int local, at;
    return id >= 0 && id < p.V && part.owner(id, local, at) == rank;
  };
  const auto gather = [&](int r, Early& e) {
    const RowPart<T> part = part_of(r);
#pragma unroll
    for (int i = 0; i < kEarly / 32; ++i) e.x[i] = is_mine(part, e.id[i]) ? row_elem(part.row + e.id[i]) : -INFINITY;
  };
  const auto prepare = [&](int r, int turn, const Early& early) {
    Listed* list = list_of(turn, warp);
    const RowPart<T> part = part_of(r);
    float t_max = -INFINITY;
    int n = 0;
    const auto keep = [&](int id, float t, float x) {
      if (id >= p.V) set_status(p.status, DSPARK_ERR_RANGE);
      const bool valid = id >= 0 && id < p.V, mine = is_mine(part, id);
      if (valid) t_max = nan_max(t_max, t);
      const uint32_t b = __ballot_sync(0xffffffffu, mine);
      if (mine) list[n + __popc(b & ((1u << lane) - 1u))] = Listed{t, x, id};
      n += __popc(b);
    };
#pragma unroll
    for (int i = 0; i < kEarly / 32; ++i) keep(early.id[i], early.t[i], early.x[i]);
    for (int base = first + kEarly; base < last; base += 128) {
      int id[4];
      float t[4], x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = base + 32 * i + lane;
        id[i] = j < last ? __ldg(p.ids + (size_t)r * p.K + j) : -1;
        t[i] = j < last ? __ldg(p.teacher + (size_t)r * p.K + j) : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = is_mine(part, id[i]) ? row_elem(part.row + id[i]) : -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) keep(id[i], t[i], x[i]);
    }
    if (j0 == 0) twice[turn] = 0;
    t_max = warp_nan_max(t_max);
    if (lane == 0) {
      maxima[warp] = t_max;
      counts[turn][warp] = n;
    }
    named_sync<kListSync, kListThreads>();
    t_max = nan_max(maxima[0], maxima[1]);
    static_assert(kListThreads == 64, "two warps");
    for (int k = lane; k < n; k += 32) {
      const int id = list[k].id;
      if (kRest) {
        int local, at;
        part.owner(id, local, at);
        uint32_t* word = local < 0 ? &loose_marks : s_marks + part.mark_word(local);
        const uint32_t bit = local < 0 ? 1u << (-1 - local) : 1u << (part.mark_byte(local) * 8 + at);
        if (atomicOr(word, bit) & bit) twice[turn] = 1;
      } else {  // nobody else needs the map
        int same = 0;
        for (int w = 0; w < 2; ++w)
          for (int i = 0; i < counts[turn][w]; ++i) same += list_of(turn, w)[i].id == id;
        if (same > 1) twice[turn] = 1;
      }
    }
    if (kRest) named_arrive<kMarksReady, kDistillThreads>();
    const float lse = kRest ? __ldg(p.teacher_lse + r) : clamped(t_max);
    const bool bad = !(t_max < INFINITY) || (kRest && !(fabsf(lse) < kFar));
    const bool none = t_max == -INFINITY || bad;
    // an entry's share before it is scaled: relative to the largest entry, or to the teacher's sum
    const Split ref = kRest ? product(lse, 1.44269502e+00f, 1.92596299e-08f) : product(lse, p.k_hi, p.k_lo);
    Split a{0.f, 0.f}, b = a, c = a;
    bool infinite = false;  // a listed entry to which the drafter gives nothing (apart from the sum: -inf less -inf is NaN)
    for (int k = lane; k < n; k += 32) {
      const float t = list[k].e;
      Split e{0.f, 0.f}, y = e;
      if (t != -INFINITY && !none) e = exp2_difference(product(clamped(t), p.k_hi, p.k_lo), ref, y);
      list[k].e = e.hi;
      if (e.hi > 0.f) {
        a = add(a, e);
        b = add(b, times(e, y));
        const float x = list[k].x;
        if (x == -INFINITY) infinite = true;
        else c = add(c, times(e, Split{x * kSmall, 0.f}));
      }
    }
    if (n > 0) {
      a = warp_add(a);
      b = warp_add(b);
      c = __any_sync(0xffffffffu, infinite) ? Split{-INFINITY, 0.f} : warp_add(c);
    }
    if (lane == 0) sums[warp][0] = a, sums[warp][1] = b, sums[warp][2] = c;
    named_sync<kListSync, kListThreads>();
    return Row{n, (none ? kNoList : 0) | (bad ? kBadList : 0)};
  };
  if (kRest) {
    for (int i = j0; i < p.marks / 4; i += kListThreads) s_marks[i] = 0;
    if (j0 == 0) loose_marks = 0;
    named_sync<kListSync, kListThreads>();
  }
  Early early;
  load(r, early);
  gather(r, early);
  Row now = prepare(r, 0, early);
  cluster_wait();
#pragma unroll 1
  for (int turn = 0; r < p.N; turn ^= 1) {
    if (warp == 0) {
      const auto both = [&](int i) {
        const Split u = sums[0][i], v = sums[1][i];
        return u.hi == -INFINITY || v.hi == -INFINITY ? Split{-INFINITY, 0.f} : add(u, v);
      };
      const Split a = both(0), b = both(1), c = both(2);
      if (lane < C) {
        ListSums* to = &teachers[turn][rank];
        store_peer(peer_address(to, lane), make_float4(a.hi, a.lo, b.hi, b.lo));
        store_peer(peer_address(&to->e_x, lane), make_float4(c.hi, c.lo, __int_as_float(now.flags), 0.f));
      }
    }
    __syncwarp();
    const int r_next = r + clusters;
    load(r_next, early);
    cluster_arrive();
    gather(min(r_next, p.N - 1), early);  // (past the last row: no ids)
    cluster_wait();
    const RowSum sum = combine<kRest, true>(all[turn], C, rate);
    // (of a far rest the streaming threads read the marks before that)
    const float z_rest = kRest && sum.far ? unlisted_received(apart, C, rate) : sum.z;
    const Factors f = factors<kRest>(teachers[turn], C, sum, z_rest, 1.f, p.weight ? __ldg(p.weight + r) : 1.f, p.per_tau);
    const RowPart<T> part = part_of(r);
    const Listed* list = list_of(turn, warp);

    // the marks are taken back and the next row's set
    if (kRest) {
      for (int k = lane; k < now.n; k += 32) {
        int local, at;
        part.owner(list[k].id, local, at);
        if (local >= 0) s_marks[part.mark_word(local)] = 0;
      }
      if (j0 == 0) loose_marks = 0;
      named_sync<kListSync, kListThreads>();
    }
    Row next{0, 0};
    if (r_next < p.N) next = prepare(r_next, turn ^ 1, early);

    RowSum rest = sum;  // its z: the unlisted entries', relative to its M
    if (kRest && sum.far) rest = unlisted_pair(apart, C, rate);  // (by whole warps)
    // the loss: the last CTA's
    if (rank == C - 1 && j0 == 32) {
      Split share{0.f, 0.f}, a = share, x = share;
      bool infinite = false;  // a listed entry to which the drafter gives nothing
      for (int c = 0; c < C; ++c) {
        const ListSums& of = teachers[turn][c];
        share = add(share, of.share);
        a = add(a, of.e_log_e);
        infinite |= of.e_x.hi == -INFINITY;
        x = add(x, of.e_x);
      }
      // sum of e (log2 e - log2 of the drafter's weight), then ln 2 of it; rate and origin as the weights have them
      const bool plain = plain_exponent(rate, sum.M);
      const Split from = times(share, Split{(plain ? origin(rate, sum.M) : sum.M) * kSmall, 0.f});
      const Split k{rate.rate, 0.f};
      const Split below = plain ? add(times(x, k), negative(from)) : times(add(x, negative(from)), k);
      const auto small = [](Split v) { return Split{v.hi * kSmall, v.lo * kSmall}; };
      a = times(add(small(a), negative(below)), Split{kLn2, kLn2Lo});
      const Split z{sum.z, sum.z_lo}, ln_z = ln_of(add(z, Split{sum.listed, sum.listed_lo}));
      Split loss{0.f, 0.f};  // times kSmall
      if (kRest) {
        const Split left = add(Split{1.f, 0.f}, negative(share));
        loss = add(a, small(times(share, ln_z)));
        if (f.some && sum.far) loss = add(loss, far_term(rest, rate, sum.M, left, ln_z));
        else if (f.some) loss = add(loss, small(times(left, add(add(ln_of(left), negative(ln_of(z))), ln_z))));
      } else if (share.hi > 0.f) {
        loss = add(quotient(a, share), small(add(ln_z, negative(ln_of(share)))));
      }
      loss.hi /= kSmall;
      if (infinite) loss.hi = INFINITY;
      p.loss[r] = f.bad ? NAN : loss.hi;
      if (f.bad) set_status(p.status, DSPARK_ERR_NONFINITE);
    }

    if constexpr (kGrad) {  // the listed entries of this CTA over what was written
      named_sync<kRowWritten, kDistillThreads>();
      T* grad = static_cast<T*>(p.grad) + (size_t)r * p.V;
      const bool plain = plain_exponent(rate, sum.M);
      for (int k = lane; k < now.n && !f.bad; k += 32) {
        float e = list[k].e;
        if (twice[turn]) {  // an id that comes more than once: every occurrence writes the sum of all
          e = 0.f;
          for (int w = 0; w < 2; ++w)
            for (int i = 0; i < counts[turn][w]; ++i)
              if (list_of(turn, w)[i].id == list[k].id) e += list_of(turn, w)[i].e;
        }
        const float x = list[k].x;
        const float y = plain ? Weigher<true>(rate, sum.M)(x) : Weigher<false>(rate, sum.M)(x);
        store_elem(grad + list[k].id, __fmaf_rn(-f.teacher, e, y * f.listed));
      }
      named_sync<kListSync, kListThreads>();
    }
    r = r_next;
    now = next;
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

// the pieces, two rows' listed entries, and a byte for each piece of a row of 2^20 float32
constexpr int kDistillSmem = kPieces * kRowThreads * 16 + kMaxTop * 2 * (int)sizeof(Listed) + (1 << 20) / 4 / kMaxCluster + kGroup * kRowThreads;

// Rows are taken in equal turns by as many clusters as the GPU holds at once (more would begin when those end).
template <class T, bool kRest, bool kGrad>
static cudaError_t launch_distill(const DistillParams& p, cudaStream_t s) {
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = set_smem_limit_once((const void*)distill_kernel<T, kRest, kGrad>, kDistillSmem, attr);
  if (e != cudaSuccess) return e;
  const size_t smem = (size_t)p.held + (size_t)((p.K + 1) / 2) * 4 * sizeof(Listed) + p.marks;
  int resident = 0;
  const cudaError_t f = resident_clusters((const void*)distill_kernel<T, kRest, kGrad>, p.C, kDistillThreads, smem, resident);
  if (f != cudaSuccess) return f;
  const int turns = ceil_div(p.N, resident);
  return launch_clusters(distill_kernel<T, kRest, kGrad>, p, (unsigned)(ceil_div(p.N, turns) * p.C), p.C, kDistillThreads, smem, s);
}
template <class T>
static cudaError_t launch_distill(const DistillParams& p, cudaStream_t s) {
  if (p.teacher_lse) return p.grad ? launch_distill<T, true, true>(p, s) : launch_distill<T, true, false>(p, s);
  return p.grad ? launch_distill<T, false, true>(p, s) : launch_distill<T, false, false>(p, s);
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
  const int elem = dtype == DSPARK_BF16 ? 2 : 4;
  const long long entries = (long long)N * V;
  const bool in_place = probs == logits && probs_dtype == dtype;
  if (!separate({span(logits, in_place ? 0 : entries, elem), span(temperature, N)}, {span(probs, entries, probs_dtype == DSPARK_BF16 ? 2 : 4)}))
    return DSPARK_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms == 0) return DSPARK_ERR_CUDA;
  int held;
  const int C = row_cluster(N, V, elem, sms, held);
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
  const int elem = dtype == DSPARK_BF16 ? 2 : 4;
  const long long entries = (long long)N * V, listed = (long long)N * K;
  if (!separate({span(logits, grad == logits ? 0 : entries, elem), span(ids, listed), span(teacher, listed), span(teacher_lse, N), span(weight, N)},
                {span(loss, N), span(grad, entries, elem)}))
    return DSPARK_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms == 0) return DSPARK_ERR_CUDA;
  int held;
  const int C = row_cluster(N, V, elem, sms, held);
  // with a rest, the map of listed entries: a byte for each piece of this CTA, a word for a group of a thread's
  const int steps = ceil_div((long long)V * elem / 16, (long long)C * kRowThreads);
  const int marks = teacher_lse ? ceil_div(steps, kGroup) * kRowThreads * 4 : 0;
  const double k = 1.44269504088896340736 / (double)temperature;
  const int windows = std::max(1, ceil_div(steps, kPieces));
  const DistillParams p{N, V, K, C, windows, held, marks, logits, ids, teacher, teacher_lse, weight, (float)(1.0 / (double)temperature),
                        (float)k, (float)(k - (double)(float)k), loss, grad, static_cast<uint32_t*>(workspace)};
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = dtype == DSPARK_BF16 ? launch_distill<__nv_bfloat16>(p, s) : launch_distill<float>(p, s);
  note_launches(1);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
