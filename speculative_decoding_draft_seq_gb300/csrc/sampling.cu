// The target's sampling rule (temperature, top-k, top-p, min-p) on rows of
// logits: one token a row from a given uniform, or the row with every entry
// outside the kept set masked.
//
// Weights of a row with maximum M at temperature T: w = 2^((l - M) log2(e)/T)
// in float32 (difference and product rounded once, the power by ex2.approx, within
// 2^-22 of it), and their masses the integers floor(w 2^40). Sums of masses are
// integer sums, so they do not depend on an order, and every comparison below is exact. With the row sorted by (logit
// descending, index ascending), top-k keeps the first k entries; top-p keeps,
// of these, the entries whose mass before them is below floor(p S), S the mass
// of the top-k set; min-p keeps the entries with w >= min_p. All three are
// prefixes of that order, so the kept set is "logit above x*, or equal to it
// and index below cut": one threshold, found in three steps.
//   1  the row streams in once from memory: its maximum, and for top-k and top-p an
//      estimate of its distribution in 2048 bins, 16 an octave of weight for top-k (a
//      rank may lie far down), 64 for top-p. The largest entry of each 16-byte piece
//      is counted once; for top-p the piece's first entry, if it is another one,
//      stands for the rest of all pieces. (A shared-memory add for every entry bounds
//      the pass: 15 us a row of 129,280 instead of 6.)
//   2  the estimate says down to which logit top-k reaches (at least k pieces have
//      a larger one), or between which two logits top-p ends, with a margin; a
//      second pass (from L2) collects the entries of that range, or all from its
//      lower end up where they fit, in shared memory, and forms exactly the masses
//      that the answer needs. They prove the range right; a range that was not is
//      moved by what they show, and collected again.
//   3  exact selection among the collected entries: by comparing all pairs of a
//      short list, else by radix selection on order-preserving integer keys
//      (1024-bin histograms of counts or masses over a shrinking key range).
// A draw needs the kept masses in index order: those above the collected range are kept
// by runs of 128 pieces in the second pass, the list's are added to them, and only the run
// that holds the token is read again. Without such a pass (top-p off) the row is.
// Where no range fits the list (thousands of equal entries, logits hundreds of
// octaves apart), the radix selection runs on the row itself. One block a row: a
// row of 129,280 bf16 is 258 KB, and the rows in flight stay in L2 between passes.
//
// What bounds it: issue slots. A pass that only compares takes 6,500 cycles a row of
// 129,280 bf16 entries on an SM of its own, one that weighs every entry 19,000, and one that also
// adds up what lies above the range and collects 38,000; the serial steps between
// (bins, selection, ties) are 25,000. 128 such rows drawn, one an SM: greedy 9 us, top-k
// 50 19, top-k 1000 27, top-p 0.95 48, top-p 0.99 52, all entries 21 (floor 4.9, the bytes);
// 128 rows of mixed parameters 51. 2,176 rows truncated, two blocks an SM: greedy 236 us (4.8 TB/s),
// top-k 50 329, top-p 0.95 555, mixed 350 (3.2 TB/s, 0.48 of the measured copy
// bandwidth). 288 rows of 32,003 float32 truncated, mixed: 50 us. Float32, 129,280 entries, mixed: 128 rows drawn
// 60 us (floor 9.8), 256 rows truncated 112 (floor 39). One row, drawn: 32,000 bf16 9 to 25, by its parameters.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mass.cuh"
#include "verify_common.cuh"

namespace dspark {

constexpr int kSBits = 10;               // key bits that a selection round settles
constexpr int kSBins = 1 << kSBits;
constexpr int kWBins = 2048;    // weight bins, 16 (top-k) or 64 (top-p) an octave
constexpr int kSList = 7168;    // collected entries (80 KB with all else: two blocks an SM leave 64 KB to L1)
constexpr int kRun = 128;       // neighbouring pieces whose mass above the collected range is kept for the draw
constexpr int kRuns = kSBins;
constexpr uint32_t kSSmem = kWBins * 4 + kWBins * 4 + kSList * 8 + kRuns * 8;
static_assert(kRuns == kSBins, "find_bin looks the token's run up");
static_assert(kSBins * 12 <= kWBins * 8, "the selection's arrays lie over the weight bins");

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
// The next smaller logit. The key below 0's would be -0's, which no entry has: -0 is equal to 0 in every comparison.
__device__ __forceinline__ float logit_below(float x) {
  const uint32_t k = logit_key(x) - 1u;
  return key_logit(k == 0x7fffffffu ? k - 1u : k);
}
// (A distance that overflows is multiplied at half its size. That matters to rates below kTinyRate alone: at larger ones
// 2^(-inf) = 0 and 2^(-3.4e38 rate) = 0 are the same weight.)
constexpr float kTinyRate = 1e-36f;
__device__ __forceinline__ float rule_exponent(float x, float M, float rate) {
  const float d = __fsub_rn(x, M);
  const float y = d == -INFINITY ? 2.f * __fmul_rn(__fsub_rn(0.5f * x, 0.5f * M), rate) : __fmul_rn(d, rate);
  return x == -INFINITY ? -INFINITY : y;
}
// Every mass, wherever it is added, subtracted or walked over, is that of this weight or of the packed pair of it (the
// same three instructions on two entries), so that they agree to the last bit.
__device__ __forceinline__ float rule_weight(float x, float M, float rate) { return ex2_approx(rule_exponent(x, M, rate)); }
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
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

// A row in 16-byte pieces, the entries before the first and after the last aligned one on their own.
// Plain loads: dspark_truncate may write the row in place. U pieces a thread are in flight.
template <class Tin, int U>
struct RowView {
  static constexpr int E = 16 / (int)sizeof(Tin), kInFlight = U;
  static_assert(U % 4 == 0, "after() follows four rows of pieces");
  const Tin* row;
  int V, a0, nv;
  __device__ RowView(const Tin* r, int n) : row(r), V(n) {
    a0 = min(n, (int)(((16 - (reinterpret_cast<uintptr_t>(r) & 15)) & 15) / sizeof(Tin)));
    nv = (n - a0) / E;
  }
  static __device__ __forceinline__ float elem(const float* p) { return *p; }
  static __device__ __forceinline__ float elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ __forceinline__ float at(int v) const { return elem(row + v); }
  __device__ __forceinline__ uint4 piece(int g) const { return *reinterpret_cast<const uint4*>(row + a0 + (size_t)g * E); }
  static __device__ __forceinline__ void split(const uint4& q, float (&x)[E]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (E == 8) {
        x[(2 * i) % E] = __uint_as_float(w[i] << 16);
        x[(2 * i + 1) % E] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        x[i % E] = __uint_as_float(w[i]);
      }
    }
  }
  // The largest entry of a piece (NaN if there is one).
  static __device__ __forceinline__ float largest(const uint4& q) {
    if (E == 8) {
      const uint32_t m = bf16x2_max_nan(bf16x2_max_nan(q.x, q.y), bf16x2_max_nan(q.z, q.w));
      return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
    return max_nan(max_nan(__uint_as_float(q.x), __uint_as_float(q.y)), max_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
  }
  // A piece of -inf, in place of one past the end.
  static __device__ __forceinline__ uint4 nothing() {
    const uint32_t w = E == 8 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(w, w, w, w);
  }
  // f(piece, first index, is it one) for the pieces g0 <= g < g1, the tid-th of every nt; the lanes of a warp stay
  // together. after(g) follows every four pieces, g the first of them, `gap` apart: nt, or with kByRun 32, so that a
  // warp's four rows of pieces are kRun neighbours (6% slower where the row comes from memory).
  struct Nothing {
    __device__ __forceinline__ void operator()(int) const {}
  };
  template <bool kByRun = false, class F, class After = Nothing>
  __device__ __forceinline__ void pieces(int g0, int g1, int tid, int nt, F f, After after = After()) const {
    if (g0 >= g1) return;
    const int gap = kByRun ? 32 : nt, at = kByRun ? (tid >> 5) * 32 * U + (tid & 31) : tid;
    uint4 q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + at + u * gap;
      q[u] = g < g1 ? piece(g) : nothing();
    }
    for (int b = g0; b < g1; b += U * nt) {  // the next loads are on their way while these are looked at
      uint4 next[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int g = b + at + U * nt + u * gap;
        next[u] = g < g1 ? piece(g) : nothing();
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int g = b + at + u * gap;
        f(q[u], a0 + g * E, g < g1);
        if (u % 4 == 3) after(g - 3 * gap);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) q[u] = next[u];
    }
  }
  // f(x, v) for the loose entries at both ends
  template <class F>
  __device__ __forceinline__ void loose(int tid, int nt, F f) const {
    for (int i = tid; i < V - nv * E; i += nt) {
      const int v = i < a0 ? i : i + nv * E;
      f(at(v), v);
    }
  }
  // f(x, v) for all entries
  template <class F>
  __device__ __forceinline__ void all(F f) const {
    pieces(0, nv, threadIdx.x, blockDim.x, [&](const uint4& q, int v, bool ok) {
      if (!ok) return;
      float x[E];
      split(q, x);
#pragma unroll
      for (int e = 0; e < E; ++e) f(x[e], v + e);
    });
    loose(threadIdx.x, blockDim.x, f);
  }
};

// 64-bit sums of a selection round in two words: shared memory adds 32 bits natively (a 64-bit add is a
// compare-and-swap loop, and equal logits all add to one bin).
struct MassBin {
  uint32_t lo, hi;
  __device__ __forceinline__ unsigned long long value() const { return ((unsigned long long)hi << 32) | lo; }
};
__device__ __forceinline__ void add_mass(MassBin* b, unsigned long long m) {
  const uint32_t lo = (uint32_t)m, old = atomicAdd(&b->lo, lo);
  const uint32_t hi = (uint32_t)(m >> 32) + (old + lo < old ? 1u : 0u);
  if (hi) atomicAdd(&b->hi, hi);
}

struct Threshold {
  uint32_t key;   // the last kept key
  uint32_t ties;  // entries of this key that are kept, in index order
  uint32_t count; // entries of this key
};

__device__ __forceinline__ uint32_t block_scan_u32(uint32_t v, uint32_t* sh) {  // inclusive, over the block's threads
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) sh[w] = v;
  __syncthreads();
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < w && lane < nw ? sh[lane] : 0u);
  return v + before;
}

// The first of kSBins bins at which the running sum, from `above` on, reaches `target`: pick[0], and the sum
// before it: pick[1]. A warp adds up neighbouring bins; the warp that the target falls to scans its own.
template <class Value>
__device__ __forceinline__ void find_bin(Value value, unsigned long long target, unsigned long long above, unsigned long long* sh,
                                         unsigned long long* pick) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5, per = kSBins / nw;
  unsigned long long v = 0;
  for (int i = lane; i < per; i += 32) v += value(w * per + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) sh[w] = v;
  __syncthreads();
  unsigned long long at = above;
  for (int i = 0; i < w; ++i) at += sh[i];
  if (at < target && at + v >= target) {
    for (int i = lane; i < per; i += 32) {
      const unsigned long long n = value(w * per + i);
      unsigned long long x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (at + x - n < target && at + x >= target) {
        pick[0] = w * per + i;
        pick[1] = at + x - n;
      }
      at += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
}

struct SelectScratch {
  uint32_t* cnt;              // [kSBins]
  MassBin* mass;              // [kSBins]
  unsigned long long* sh;     // [32]
  unsigned long long* pick;   // [4]
};

// The key at which the running count or (kByMass) mass in descending order first reaches `target`, among
// the keys lo..hi of the entries that `source` enumerates; `above`: that of the larger keys it leaves out.
// The keys' lowest kUnit bits are the same for all keys of one sign (bf16 logits: 16): bins of 2^kUnit hold one key.
template <bool kByMass, int kUnit, class Source, class Mass>
__device__ Threshold select_key(Source source, Mass mass_of, unsigned long long target, unsigned long long above, uint32_t lo,
                                uint32_t hi, const SelectScratch& s) {
  const int tid = threadIdx.x, nt = blockDim.x;
  for (int round = 0;; ++round) {
    const uint32_t span = hi - lo;
    const int bits = 32 - __clz(span), shift = max(bits - kSBits, kUnit);
    // the key of a bin of one: of a logit below 0 its low bits are ones, also where hi's are not
    auto key_of = [&](uint32_t b) {
      const uint32_t k = hi - (b << shift);
      return kUnit > 0 && k < 0x80000000u ? (k - 1u) | ((1u << kUnit) - 1u) : k;
    };
    __syncthreads();
    for (int b = tid; b < kSBins; b += nt) {
      s.cnt[b] = 0;
      if (kByMass) s.mass[b] = MassBin{0, 0};
    }
    __syncthreads();
    source([&](uint32_t k) {
      if (k < lo || k > hi) return;
      const uint32_t b = (hi - k) >> shift;
      atomicAdd(&s.cnt[b], 1u);
      if (kByMass && shift > kUnit) add_mass(&s.mass[b], mass_of(k));
    });
    __syncthreads();
    auto value = [&](int b) -> unsigned long long {
      if (!kByMass) return s.cnt[b];
      if (shift > kUnit) return s.mass[b].value();
      const unsigned long long n = s.cnt[b];  // a bin of one key
      return n ? n * mass_of(key_of((uint32_t)b)) : 0ull;
    };
    find_bin(value, target, above, s.sh, s.pick);
    const uint32_t b = (uint32_t)s.pick[0];
    above = s.pick[1];
    if (shift == kUnit || round == 32) {  // (a round settles kSBits of at most 32 bits)
      Threshold t;
      t.key = key_of(b);
      t.count = s.cnt[b];
      const unsigned long long w = kByMass ? mass_of(t.key) : 1ull;
      t.ties = (uint32_t)min((unsigned long long)t.count, (target - above + w - 1) / w);
      __syncthreads();
      return t;
    }
    const uint32_t top = hi - (b << shift);
    lo = max(lo, top - ((1u << shift) - 1));
    hi = top;
  }
}

// Entry tid of a short list: how many entries come before it in an order, and their mass. All pairs are
// compared, kRanked threads an entry's share each.
constexpr int kRanked = 256;
struct RankScratch {
  unsigned long long* mass;  // [kRanked]
  MassBin* before;           // [kRanked]
  uint32_t* rank;            // [kRanked]
};
struct Ranked {
  int rank;
  unsigned long long mass, before;
};
template <class Mass, class First>
__device__ Ranked rank_entries(const uint2* list, int n, Mass mass_of, First first, const RankScratch& s) {
  const int tid = threadIdx.x, e = tid & (kRanked - 1), parts = blockDim.x / kRanked;
  __syncthreads();
  if (tid < n) {
    s.mass[tid] = mass_of(list[tid].x);
    s.before[tid] = MassBin{0, 0};
    s.rank[tid] = 0;
  }
  __syncthreads();
  if (e < n) {
    const uint2 me = list[e];
    uint32_t rank = 0;
    unsigned long long m = 0;
#pragma unroll 4
    for (int j = tid / kRanked; j < n; j += parts) {
      const bool b = first(list[j], me);
      rank += b ? 1u : 0u;
      m += b ? s.mass[j] : 0ull;
    }
    atomicAdd(&s.rank[e], rank);
    add_mass(&s.before[e], m);
  }
  __syncthreads();
  Ranked r{0, 0, 0};
  if (tid < n) r = Ranked{(int)s.rank[tid], s.mass[tid], s.before[tid].value()};
  return r;
}

// Magic-number rounding to whole bins: float32 values from 2^23 on are integers.
struct WeightBins {
  float c, off;  // bin of x: round(c x + off) - 2^23, clamped to the bins
  __device__ __forceinline__ float pos(float x) const {
    return fminf(fmaxf(__fmaf_rn(x, c, off), 8388608.f), 8388608.f + (kWBins - 1));
  }
  static __device__ __forceinline__ int index(float t) { return (int)(__float_as_uint(t) & (kWBins - 1)); }
  static __device__ __forceinline__ float edge(int bin) { return 8388608.f + (float)bin; }
};

template <class Tin, int NT, int kBlocks, bool kDraw>
__global__ void __launch_bounds__(NT, kBlocks) sampling_rule_kernel(SampleParams p) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  __shared__ unsigned long long sh[32], s_pick[4];
  __shared__ float shf[32];
  __shared__ int shi[32];
  __shared__ uint2 s_range[32];
  uint32_t* cum_c = reinterpret_cast<uint32_t*>(s_raw);        // [kWBins] estimated counts, from the top bin down
  float* cum_m = reinterpret_cast<float*>(cum_c + kWBins);     // [kWBins] estimated masses, relative to the maximum's
  uint2* list = reinterpret_cast<uint2*>(cum_m + kWBins);      // [kSList] (key, index)
  // the selection's arrays, over the bins (no longer needed then)
  MassBin* s_mass = reinterpret_cast<MassBin*>(s_raw);
  const SelectScratch scratch{reinterpret_cast<uint32_t*>(s_mass + kSBins), s_mass, sh, s_pick};
  unsigned long long* s_u64 = reinterpret_cast<unsigned long long*>(s_raw);
  const RankScratch few{s_u64, reinterpret_cast<MassBin*>(s_u64 + kRanked), reinterpret_cast<uint32_t*>(s_u64 + 2 * kRanked)};
  uint2* few_list = reinterpret_cast<uint2*>(s_u64 + 3 * kRanked);
  MassBin* run_mass = reinterpret_cast<MassBin*>(list + kSList);  // [kRuns]
  const int tid = threadIdx.x, V = p.V;
  constexpr int nt = NT, kUnit = sizeof(Tin) == 2 ? 16 : 0;
  const size_t r = blockIdx.x;
  const RowView<Tin, (kBlocks > 1 ? 4 : 8)> row(static_cast<const Tin*>(p.logits) + r * V, V);
  const float T = __ldg(p.temperature + r), tp = __ldg(p.top_p + r);
  const float min_w = fminf(fmaxf(__ldg(p.min_p + r), 0.f), 1.f);
  const int k = __ldg(p.top_k + r);
  const bool greedy = !(T > 0.f), by_k = !greedy && k > 0 && k < V, by_p = !greedy && tp < 1.f;
  const float rate = fminf(__fdiv_rn(1.4426950408889634f, T), 1e30f);  // (0 at T = inf)
  const bool tiny = rate < kTinyRate;  // weights by rule_weight alone: the packed ones know no distance past float32's range

  // ---- 1: maximum and weight bins ----
  using Row = RowView<Tin, (kBlocks > 1 ? 4 : 8)>;
  const float octave = by_k ? 16.f : 64.f, bin = 1.f / octave;  // bins an octave, and octaves a bin
  WeightBins bins{octave * rate, 0.f};
  bool binned = by_k || by_p;
  float M = -INFINITY, mine = -INFINITY;  // the row's maximum; a greedy row: this thread's, and the piece it is in
  int first_at = V;
  if (binned) {
    for (int b = tid; b < kWBins; b += nt) cum_c[b] = 0;
    // the bins' origin: the largest entry of the first stretch, which stays in registers
    constexpr int U = Row::kInFlight;
    uint4 q0[U];
    float m0 = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) q0[u] = tid + u * nt < row.nv ? row.piece(tid + u * nt) : Row::nothing();
    row.loose(tid, nt, [&](float x, int) { m0 = fmaxf(m0, x); });
#pragma unroll
    for (int u = 0; u < U; ++u) m0 = fmaxf(m0, Row::largest(q0[u]));
    m0 = block_max(m0, shf);
    if (!(fabsf(m0) < INFINITY)) m0 = 0.f;
    const float o = rintf(m0 * bins.c);
    binned = fabsf(o) <= 524288.f && !tiny;  // else too far from 0 for whole bins in float32
    bins.off = 8388608.f + (by_k ? kWBins / 2 : kWBins - 6 * 64) - o;
    auto count = [&](float x, uint32_t n) { atomicAdd(&cum_c[kWBins - 1 - WeightBins::index(bins.pos(x))], n); };
    auto visit = [&](const uint4& q, int, bool ok) {
      const float g = Row::largest(q);
      M = max_nan(M, g);
      if (ok) count(g, 1u);
      if (!by_k) {  // of E entries that are not the largest with chance 1 - 1/E, E - 1 to stand for
        const float x = Row::E == 8 ? __uint_as_float(q.x << 16) : __uint_as_float(q.x);
        if (x < g) count(x, (uint32_t)Row::E);
      }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) visit(q0[u], 0, tid + u * nt < row.nv);
    row.pieces(U * nt, row.nv, tid, nt, visit);
    row.loose(tid, nt, [&](float x, int) {
      M = max_nan(M, x);
      count(x, 1u);
    });
  } else {
    float best = -INFINITY;
    row.pieces(0, row.nv, tid, nt, [&](const uint4& q, int v, bool) {
      const float g = Row::largest(q);
      M = max_nan(M, g);
      if (g > best) { best = g; first_at = v; }
    });
    row.loose(tid, nt, [&](float x, int v) {
      M = max_nan(M, x);
      if (x > best || (x == best && v < first_at)) { best = x; first_at = v; }
    });
    mine = best;
  }
  __syncthreads();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
  if ((tid & 31) == 0) shf[tid >> 5] = M;
  __syncthreads();
  for (int i = 0; i < (nt >> 5); ++i) M = max_nan(M, shf[i]);
  if (!(M < INFINITY) || M == -INFINITY) {  // a NaN or +inf, or nothing finite: no distribution
    if (tid == 0) {
      set_status(p.status, DSPARK_ERR_NONFINITE);
      if (kDraw) p.tokens[r] = -1;
      if (kDraw && p.prob) p.prob[r] = 0.f;
    }
    if (!kDraw) {
      Tin* out = static_cast<Tin*>(p.out) + r * V;
      for (int v = tid; v < V; v += nt) out[v] = row.row[v];
    }
    return;
  }
  M = __fadd_rn(M, 0.f);
  const unsigned long long neg_m = f32x2_pack(-M, -M), rate2 = f32x2_pack(rate, rate);
  auto weights = [&](float x0, float x1) {  // rule_weight of two entries, as masses
    float y0, y1;
    f32x2_unpack(f32x2_mul(f32x2_add(f32x2_pack(x0, x1), neg_m), rate2), y0, y1);
    return MassPair(ex2_approx(y0), ex2_approx(y1));
  };
  auto mass_of = [&](uint32_t key) { return fx40(rule_weight(key_logit(key), M, rate)); };
  auto from_row = [&](auto f) { row.all([&](float x, int) { f(logit_key(x)); }); };

  // the kept set: logits above key_logit(key), and those equal to it up to index `cut`
  uint32_t key = logit_key(-INFINITY) + 1;
  int cut = V;
  bool headed = false;  // the list holds every kept entry
  // each warp fills a part of the list of its own (no atomics)
  constexpr int kPart = kSList / (NT / 32);
  uint2* part = list + (tid >> 5) * kPart;
  int n_part = 0, n_list = 0;  // entries of the warp's part, and of all
  // run_mass: each run's mass above run_hi, where the list holds every kept entry up to it; loose entries go with
  // the first and the last run
  const int n_runs = max(1, (row.nv + kRun - 1) / kRun);
  const bool by_run = kDraw && row.nv > 0 && n_runs <= kRuns;
  auto run_of = [&](int v) { return min(max(v - row.a0, 0) / (kRun * Row::E), n_runs - 1); };
  float run_hi = -INFINITY;
  if (greedy) {
    int at = block_min_i(mine == M ? first_at : V, shi);
    while (at < V - 1 && row.at(at) != M) ++at;  // within the piece
    key = logit_key(M);
    cut = at + 1;
  } else if (by_k || by_p) {
    const uint32_t hi = logit_key(M), lowest = logit_key(-INFINITY);
    const float tm = __fmaf_rn(M, bins.c, bins.off - 8388608.f);  // the maximum's place on the bins' axis
    binned = binned && tm > 0.f;
    Threshold th{0, 0, 0};
    bool found = false;
    unsigned long long S = 0, want = 0, above = 0;  // top-p's whole, its limit, and what lies above the list
    unsigned long long below_before = 0;                // the mass down to the end of the range before
    // the mass of the top-k set that ends at `th`
    auto top_mass = [&](auto source) {
      unsigned long long m = 0;
      source([&](uint32_t q) { m += q > th.key ? mass_of(q) : 0ull; });
      return block_sum_u64(m, sh) + th.ties * mass_of(th.key);
    };
    auto no_mass = [](uint32_t) { return 1ull; };
    // ---- 2: the bins in question ----
    if (binned) {
      // running sums from the top bin down, a stretch of neighbouring bins a warp
      constexpr int per = kWBins / (NT / 32);
      const int lane = tid & 31, w0 = (tid >> 5) * per;
      auto weight = [&](int j) { return j == 0 && tm >= kWBins - 1 ? 1.f : ex2_approx(((float)(kWBins - 1 - j) - tm) * bin); };
      uint32_t c = 0;
      float m = 0.f;
#pragma unroll 4
      for (int i = lane; i < per; i += 32) {
        const uint32_t n = cum_c[w0 + i];
        c += n;
        if (!by_k) m += (float)n * weight(w0 + i);
      }
      c = __reduce_add_sync(0xffffffffu, c);
      m = warp_sum(m);
      if (lane == 0) s_range[tid >> 5] = make_uint2(c, __float_as_uint(m));
      __syncthreads();
      c = 0;
      m = 0.f;
      for (int i = 0; i < (tid >> 5); ++i) {
        c += s_range[i].x;
        m += __uint_as_float(s_range[i].y);
      }
#pragma unroll 2
      for (int i = lane; i < per; i += 32) {
        const uint32_t n = cum_c[w0 + i];
        uint32_t x = n;
        float y = by_k ? 0.f : (float)n * weight(w0 + i);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t xo = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += xo;
          if (!by_k) {
            const float yo = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += yo;
          }
        }
        cum_c[w0 + i] = c + x;
        c += __shfl_sync(0xffffffffu, x, 31);
        if (!by_k) {
          cum_m[w0 + i] = m + y;
          m += __shfl_sync(0xffffffffu, y, 31);
        }
      }
      __syncthreads();
      // the first bin (from the top) whose sum reaches `goal` (warp-wide, 32 bins a step)
      auto first = [&](const auto* cum, auto goal) {
        int lo = 0, n = kWBins;
        while (n > 1) {
          n = (n + 31) / 32;
          const int at = min(lo + ((tid & 31) + 1) * n - 1, kWBins - 1);
          const uint32_t ok = __ballot_sync(0xffffffffu, cum[at] >= goal);
          lo = min(lo + (ok ? __ffs(ok) - 1 : 31) * n, kWBins - 1);
        }
        return lo;
      };
      const float origin = bins.off - 8388608.f;
      // the logit `j` bins down from the top of the first one
      auto logit_at = [&](float j) { return j >= (float)kWBins ? -INFINITY : ((float)kWBins - 0.5f - j - origin) / bins.c; };
      auto est_at = [&](float x) {  // the estimated mass above a logit
        const float j = fminf(fmaxf((float)kWBins - 0.5f - (x * bins.c + origin), 0.f), (float)kWBins);
        const int i = min((int)j, kWBins - 1);
        const float a = i > 0 ? cum_m[i - 1] : 0.f;
        return a + (j - (float)i) * (cum_m[i] - a);
      };
      const float est = by_k ? 0.f : cum_m[kWBins - 1];  // of the whole row
      float goal = fminf(tp, 1.f) * est;  // top-p's limit in the estimate's measure
      float slack = est * 0.0156f;
      float r_lo = 0.f, r_hi = 0.f;  // the range before
      int move = 0;                  // 1: further down than it, -1: further up
      int half = kSList / 5;         // entries either side of the goal
      for (int attempt = 0; attempt < 6; ++attempt) {
        // the ends' bins: a search a warp
        const int warp = tid >> 5;
        if (by_k) {
          if (warp == 0) shi[0] = first(cum_c, (uint32_t)k);
        } else if (warp < 3) {
          shi[warp] = first(cum_m, warp == 0 ? goal : warp == 1 ? fmaxf(goal - slack, 0.f) : goal + slack);
        }
        __syncthreads();
        int ja = 0, jb = shi[0];
        if (by_k) {
          headed = cum_c[jb] >= (uint32_t)k && k <= kSList;
        } else {
          const int jg = shi[0], at = (int)cum_c[jg];
          if (warp < 4)  // so many entries up and down; the bins next to the goal's that hold any
            shi[4 + warp] = first(cum_c, warp == 0 ? (uint32_t)max(at - half, 1) : warp == 1 ? (uint32_t)(at + half)
                                         : warp == 2 ? (uint32_t)(at + 1) : jg > 0 ? cum_c[jg - 1] : 0u);
          __syncthreads();
          auto entries = [&](int a, int b) { return (int)cum_c[b] - (a > 0 ? (int)cum_c[a - 1] : 0); };
          // within the slack, and well within what the list holds; but a bin on either side if it can (one bf16 value
          // may stand for thousands of entries)
          ja = max(shi[1], min(shi[4], jg));
          jb = min(shi[2], max(shi[5] - 1, jg));
          if (entries(min(ja, shi[7]), jb) <= kSList * 6 / 7) ja = min(ja, shi[7]);
          if (entries(ja, max(jb, shi[6])) <= kSList * 6 / 7) jb = max(jb, shi[6]);
          headed = move == 0 && cum_c[jb] <= kSList / 2;
        }
        float x_lo = logit_at((float)(jb + 1)), x_hi = headed ? INFINITY : logit_at((float)ja);
        // no entry of the range before is in this one, and it reaches a bin further (more at a later attempt)
        const float reach = 1.5f * (float)attempt / bins.c;
        if (move > 0) {
          x_hi = fminf(x_hi, logit_below(r_lo));
          x_lo = fminf(x_lo, r_lo - reach);
        } else if (move < 0) {
          x_lo = fmaxf(x_lo, key_logit(logit_key(r_hi) + 1));
          x_hi = fmaxf(x_hi, r_hi + reach);
        }
        if (by_k && !headed) break;
        const float nan = __uint_as_float(0x7fc00000u);  // in no range
        const uint32_t nan_w = Row::E == 8 ? 0x7fc07fc0u : __float_as_uint(nan);
        const uint4 none = make_uint4(nan_w, nan_w, nan_w, nan_w);
        n_part = 0;
        const uint32_t below = (1u << (tid & 31)) - 1u;
        // the indices of the entries in range, by whole warps: an entry a step of the lane that has most among four
        // pieces (bits 0..15: their float32 entries or low halves, four a piece; above: the high halves)
        uint32_t in4 = 0;
        auto collect_piece = [&](const uint4& q) {
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
          uint32_t in = 0;
          if (Row::E == 8) {  // two compares at a time, against the ends rounded inwards to bf16
            const __nv_bfloat16 a = __float2bfloat16_ru(x_lo), b = __float2bfloat16_rd(x_hi);
            const __nv_bfloat162 a2 = __halves2bfloat162(a, a), b2 = __halves2bfloat162(b, b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
              in |= __hge2_mask(x, a2) & __hle2_mask(x, b2) & (0x10001u << i);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) in |= __uint_as_float(w[i]) >= x_lo && __uint_as_float(w[i]) <= x_hi ? 1u << i : 0u;
          }
          in4 = (in4 >> 4) & 0x0fff0fffu | in << 12;  // (each piece moves the ones before it down)
        };
        auto skip_piece = [&]() { in4 = (in4 >> 4) & 0x0fff0fffu; };
        auto collect = [&](int g, int gap) {
          const int v = row.a0 + g * Row::E;
          for (uint32_t all; (all = __ballot_sync(0xffffffffu, in4 != 0)) != 0; in4 &= in4 - 1) {
            const int bit = __ffs(in4) - 1, i = bit & 3, at = n_part + __popc(all & below);
            if (in4 != 0 && at < kPart)
              part[at].y = (uint32_t)(v + ((bit >> 2) & 3) * gap * Row::E + (Row::E == 4 ? i : 2 * i + (bit >> 4)));
            n_part += __popc(all);
          }
        };
        auto collect_loose = [&]() {  // at most 2 E entries: the first warp takes them
          if (tid >= 32) return;
          const int n = V - row.nv * Row::E, v = tid < row.a0 ? tid : tid + row.nv * Row::E;
          const float x = tid < n ? row.at(v) : nan;
          const bool in = x >= x_lo && x <= x_hi;
          const uint32_t all = __ballot_sync(0xffffffffu, in);
          const int at = n_part + __popc(all & below);
          if (in && at < kPart) part[at].y = (uint32_t)v;
          n_part += __popc(all);
        };
        unsigned long long gap_mass = 0;
        if (by_k) {
          row.pieces(0, row.nv, tid, nt, [&](const uint4& q, int v, bool ok) {
            if (__any_sync(0xffffffffu, ok && Row::largest(q) >= x_lo)) collect_piece(ok ? q : none);
            else skip_piece();
          }, [&](int g) { collect(g, nt); });
          collect_loose();
        } else if (move == 0) {  // the row's mass, and what lies above the range
          MassSum sum, over;
          bool ups = false;
          row.template pieces<kDraw>(0, row.nv, tid, nt, [&](const uint4& q, int, bool ok) {
            float x[Row::E];
            Row::split(q, x);
            const float g = Row::largest(q);
            const bool some = __any_sync(0xffffffffu, g > x_hi);
            ups |= some;
#pragma unroll
            for (int e = 0; e < Row::E; e += 2) {
              const MassPair m = weights(x[e], x[e + 1]);
              sum.add(m);
              if (some) over.add_if(m, x[e] > x_hi, x[e + 1] > x_hi);
            }
            if (__any_sync(0xffffffffu, ok && g >= x_lo)) collect_piece(ok ? q : none);
            else skip_piece();
          }, [&](int g) {
            collect(g, kDraw ? 32 : nt);
            if (!by_run) return;
            unsigned long long m = 0;
            if (ups) {  // (32 lanes' 4 E masses: the halves' sums fit 32 bits)
              const uint32_t hi = __reduce_add_sync(0xffffffffu, over.hi), lo = __reduce_add_sync(0xffffffffu, over.lo);
              m = ((unsigned long long)hi << 20) + lo;
            }
            if ((tid & 31) == 0 && g < row.nv) run_mass[g / kRun] = MassBin{(uint32_t)m, (uint32_t)(m >> 32)};
            over = MassSum();
            ups = false;
          });
          __syncthreads();
          row.loose(tid, nt, [&](float x, int v) {
            const MassPair m = weights(x, x);
            sum.add_if(m, true, false);
            if (!by_run) over.add_if(m, x > x_hi, false);
            else if (x > x_hi) add_mass(run_mass + run_of(v), mass_of(logit_key(x)));
          });
          collect_loose();
          S = block_sum_u64(sum.total(), sh);
          unsigned long long up = over.total();
          if (by_run)
            for (int i = tid; i < n_runs; i += nt) up += run_mass[i].value();
          above = headed ? 0ull : block_sum_u64(up, sh);
          run_hi = by_run && !headed ? x_hi : -INFINITY;
          want = max(1ull, scale_mass((double)fminf(tp, 1.f - 0x1p-24f), S));
        } else {  // another range: only what lies between the two counts
          run_hi = -INFINITY;
          MassSum gap;
          const float g_lo = move > 0 ? x_hi : r_hi, g_hi = move > 0 ? r_lo : x_lo, least = move > 0 ? x_lo : r_hi;
          row.pieces(0, row.nv, tid, nt, [&](const uint4& q, int v, bool ok) {
            if (!__any_sync(0xffffffffu, ok && Row::largest(q) >= least)) {
              skip_piece();
              return;
            }
            const uint4 p = ok ? q : none;
            float x[Row::E];
            Row::split(p, x);
            bool some = false;
#pragma unroll
            for (int e = 0; e < Row::E; ++e) some |= x[e] > g_lo && x[e] < g_hi;
            if (__any_sync(0xffffffffu, some)) {
#pragma unroll
              for (int e = 0; e < Row::E; e += 2)
                gap.add_if(weights(x[e], x[e + 1]), x[e] > g_lo && x[e] < g_hi, x[e + 1] > g_lo && x[e + 1] < g_hi);
            }
            collect_piece(p);
          }, [&](int g) { collect(g, nt); });
          row.loose(tid, nt, [&](float x, int) { gap.add_if(weights(x, x), x > g_lo && x < g_hi, false); });
          collect_loose();
          gap_mass = block_sum_u64(gap.total(), sh);
        }
        __syncthreads();
        if ((tid & 31) == 0) s_range[tid >> 5] = make_uint2((uint32_t)n_part, 0u);
        __syncthreads();
        n_list = 0;
        for (int i = 0; i < NT / 32; ++i) {
          const int n = (int)s_range[i].x;
          n_list = n > kPart || n_list > kSList ? kSList + 1 : n_list + n;
        }
        if (n_list <= kSList) {
#pragma unroll 4
          for (int i = tid & 31; i < n_part; i += 32) part[i].x = logit_key(row.at((int)part[i].y));
          __syncwarp();
        }
        // does the rule end among the list's entries?
        if (n_list > kSList) {  // a smaller range, from the upper end of this one on
          if (by_k || move < 0) break;
          if (move > 0) above = below_before + gap_mass;
          below_before = above;
          r_lo = x_hi < INFINITY ? key_logit(logit_key(x_hi) + 1) : INFINITY;
          move = 1;
          half /= 4;
          goal = est_at(x_hi) + ((float)want - (float)above) * 0x1p-40f;
          headed = false;
          __syncthreads();
          continue;
        }
        if (by_k) {
          found = n_list >= k;
          break;
        }
        unsigned long long in = 0;
        for (int i = tid & 31; i < n_part; i += 32) in += mass_of(part[i].x);
        in = block_sum_u64(in, sh);
        if (move > 0) above = below_before + gap_mass;
        else if (move < 0) above = above - gap_mass - in;
        below_before = above + in;
        found = above < want && want <= above + in;
        if (found) break;
        // the estimate holds between two logits near one another: from what is now known at the nearer end on
        move = want > above ? 1 : -1;
        const unsigned long long known = move > 0 ? above + in : above;
        r_lo = x_lo;
        r_hi = x_hi;
        if (headed && move < 0) break;
        goal = est_at(move > 0 ? x_lo : x_hi) + ((float)want - (float)known) * 0x1p-40f;
        slack = est * 0.004f;
        __syncthreads();
      }
      if (found) {
        // ---- 3: selection on the list ----
        auto from_list = [&](auto f) {
          for (int i = tid & 31; i < n_part; i += 32) f(part[i].x);
        };
        if (n_list <= kRanked) {  // few entries: each one's place by comparing it with all
          int at = 0;
          for (int i = 0; i < (tid >> 5); ++i) at += (int)s_range[i].x;
          __syncthreads();  // (the short list lies over the weight bins)
          for (int i = tid & 31; i < n_part; i += 32) few_list[at + i] = part[i];
          const Ranked e = rank_entries(few_list, n_list, mass_of, [](const uint2& a, const uint2& b) {
            return a.x > b.x | (a.x == b.x & a.y < b.y);
          }, few);
          const int most = by_k ? min(k, n_list) : n_list;
          if (by_k && by_p) {
            if (tid < n_list && e.rank == most - 1) s_pick[2] = e.before + e.mass;
            __syncthreads();
            want = max(1ull, scale_mass((double)fminf(tp, 1.f - 0x1p-24f), s_pick[2]));
          }
          const unsigned long long start = above + e.before, end = start + e.mass;
          if (tid < n_list && e.rank < most && (!by_p || start < want) && !(e.rank + 1 < most && (!by_p || end < want))) {
            s_pick[0] = few_list[tid].x;  // the last entry that both rules keep
            s_pick[1] = few_list[tid].y;
          }
          __syncthreads();
          th = Threshold{(uint32_t)s_pick[0], 0, 0};
          cut = (int)s_pick[1] + 1;
        } else {
          uint32_t k_lo = 0xffffffffu, k_hi = 0u;
          for (int i = tid & 31; i < n_part; i += 32) {
            k_lo = min(k_lo, part[i].x);
            k_hi = max(k_hi, part[i].x);
          }
          k_lo = __reduce_min_sync(0xffffffffu, k_lo);
          k_hi = __reduce_max_sync(0xffffffffu, k_hi);
          __syncthreads();
          if ((tid & 31) == 0) s_range[tid >> 5] = make_uint2(k_lo, k_hi);
          __syncthreads();
          for (int i = 0; i < (nt >> 5); ++i) {
            k_lo = min(k_lo, s_range[i].x);
            k_hi = max(k_hi, s_range[i].y);
          }
          if (by_k) {
            th = select_key<false, kUnit>(from_list, no_mass, (unsigned long long)k, 0ull, k_lo, k_hi, scratch);
            if (by_p) {
              S = top_mass(from_list);
              want = max(1ull, scale_mass((double)fminf(tp, 1.f - 0x1p-24f), S));
              th = select_key<true, kUnit>(from_list, mass_of, want, 0ull, th.key, k_hi, scratch);
            }
          } else {
            th = select_key<true, kUnit>(from_list, mass_of, want, above, k_lo, k_hi, scratch);
          }
        }
        if (th.ties < th.count) {  // the index of the last tie that is kept: the ties-th smallest
          if (th.count <= (uint32_t)kRanked) {
            __syncthreads();
            if (tid == 0) shi[0] = 0;
            __syncthreads();
            for (int i = tid & 31; i < n_part; i += 32)
              if (part[i].x == th.key) few_list[atomicAdd(&shi[0], 1)] = part[i];  // in any order: a rank does not depend on it
            const Ranked e = rank_entries(few_list, (int)th.count, no_mass, [](const uint2& a, const uint2& b) { return a.y < b.y; }, few);
            if (tid < (int)th.count && e.rank == (int)th.ties - 1) s_pick[0] = few_list[tid].y;
            __syncthreads();
            cut = (int)s_pick[0] + 1;
          } else {
            auto tie_index = [&](auto f) {
              for (int i = tid & 31; i < n_part; i += 32)
                if (part[i].x == th.key) f(~part[i].y);
            };
            const Threshold at = select_key<false, 0>(tie_index, no_mass, th.ties, 0ull, ~(uint32_t)(V - 1), 0xffffffffu, scratch);
            cut = (int)~at.key + 1;
          }
        }
      }
    }
    if (!found) {  // the same selection on the row
      headed = false;
      cut = V;
      uint32_t lo = lowest;
      if (by_k) {
        th = select_key<false, kUnit>(from_row, no_mass, (unsigned long long)k, 0ull, lo, hi, scratch);
        lo = th.key;
        if (by_p) S = top_mass(from_row);
      } else {
        MassSum sum;
        row.all([&](float x, int) { sum.add(MassPair(rule_weight(x, M, rate), 0.f)); });
        S = block_sum_u64(sum.total(), sh);
      }
      if (by_p) {
        want = max(1ull, scale_mass((double)fminf(tp, 1.f - 0x1p-24f), S));
        th = select_key<true, kUnit>(from_row, mass_of, want, 0ull, lo, hi, scratch);
      }
      if (th.ties < th.count) {
        const float xs = key_logit(th.key);
        auto tie_index = [&](auto f) {
          row.all([&](float x, int v) {
            if (x == xs) f(~(uint32_t)v);
          });
        };
        const Threshold at = select_key<false, 0>(tie_index, no_mass, th.ties, 0ull, ~(uint32_t)(V - 1), 0xffffffffu, scratch);
        cut = (int)~at.key + 1;
      }
    }
    if (th.key >= key) key = th.key;
    else cut = V;  // the threshold fell on entries of -inf: all others are kept
  }
  // the smallest key whose weight reaches min_p, by 32-way search (exp2f has weights below 2^-126 too; above, it and
  // ex2.approx have given the same bits for every float32 argument)
  if (!greedy && min_w > 0.f) {
    uint32_t lo = key, hi = logit_key(M);  // the weight of hi is 1
    for (int round = 0; lo < hi && round < 32; ++round) {
      const uint32_t step = (hi - lo) / 32 + 1;
      const uint32_t at = (uint32_t)min((unsigned long long)hi, lo + (unsigned long long)step * (tid & 31));
      const uint32_t ok = __ballot_sync(0xffffffffu, exp2f(rule_exponent(key_logit(at), M, rate)) >= min_w);
      const int first = ok ? __ffs(ok) - 1 : 32;  // lanes before it lie below
      hi = (uint32_t)min((unsigned long long)hi, lo + (unsigned long long)step * first);
      if (first > 0) lo = (uint32_t)min((unsigned long long)hi, lo + (unsigned long long)step * (first - 1) + 1);
      else hi = lo;
    }
    if (lo > key) { key = lo; cut = V; }
  }
  const float xs = key_logit(key);
  auto kept = [&](float x, int v) { return x > xs || (x == xs && v < cut); };

  if (!kDraw) {
    Tin* out = static_cast<Tin*>(p.out) + r * V;
    const bool aligned = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row.row)) & 15) == 0;
    const uint32_t low = sizeof(Tin) == 2 ? 0xff7fu : 0xff7fffffu;  // the lowest finite value
    if (aligned) {
      // two compares at a time against the threshold rounded up to bf16: it is a bf16 value unless min-p set
      // it, and then x >= xs (cut = V) holds for the same bf16 values x
      const __nv_bfloat16 t16 = __float2bfloat16_ru(xs);
      const __nv_bfloat162 t2 = __halves2bfloat162(t16, t16);
      row.pieces(0, row.nv, tid, nt, [&](const uint4& q, int v, bool ok) {
        if (!ok) return;
        uint32_t w[4] = {q.x, q.y, q.z, q.w};
        const bool whole = v + Row::E <= cut;  // ties of the whole piece are kept
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (Row::E == 8) {
            const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
            uint32_t keep = __hge2_mask(x, t2);
            if (!whole) keep = (kept(__low2float(x), v + 2 * i) ? 0xffffu : 0u) | (kept(__high2float(x), v + 2 * i + 1) ? 0xffff0000u : 0u);
            w[i] = (w[i] & keep) | ((low | low << 16) & ~keep);
          } else {
            w[i] = kept(__uint_as_float(w[i]), v + i) ? w[i] : low;
          }
        }
        __stcs(reinterpret_cast<uint4*>(out + v), make_uint4(w[0], w[1], w[2], w[3]));
      });
    }
    const int loose = aligned ? V - row.nv * Row::E : V;
    for (int i = tid; i < loose; i += nt) {
      const int v = aligned && i >= row.a0 ? i + row.nv * Row::E : i;
      const Tin raw = row.row[v];
      if (kept(row.at(v), v)) out[v] = raw;
      else if (sizeof(Tin) == 2) *reinterpret_cast<uint16_t*>(out + v) = (uint16_t)low;
      else *reinterpret_cast<uint32_t*>(out + v) = low;
    }
  }
  if (!kDraw) return;
  if (greedy) {
    if (tid == 0) {
      p.tokens[r] = cut - 1;
      if (p.prob) p.prob[r] = 1.f;
    }
    return;
  }
  if (headed && n_list <= kRanked) {  // every kept entry is on a short list: places by index
    auto kept_mass = [&](const uint2& a) { return kept(key_logit(a.x), (int)a.y) ? mass_of(a.x) : 0ull; };
    unsigned long long m = tid < n_list ? kept_mass(few_list[tid]) : 0ull;
    const unsigned long long Z = block_sum_u64(m, sh), t = scale_mass(p.u[r], Z);
    const Ranked e = rank_entries(few_list, n_list, mass_of, [&](const uint2& a, const uint2& b) {
      return a.y < b.y & kept(key_logit(a.x), (int)a.y);
    }, few);
    if (m > 0 && e.before <= t && e.before + m > t) {
      p.tokens[r] = (int)few_list[tid].y;
      if (p.prob) p.prob[r] = (float)((double)m / (double)Z);
    }
    return;
  }
  if (headed) {  // every kept entry is on the list: the draw selects an index by mass
    unsigned long long Z = 0;
    for (int i = tid & 31; i < n_part; i += 32)
      if (kept(key_logit(part[i].x), (int)part[i].y)) Z += mass_of(part[i].x);
    Z = block_sum_u64(Z, sh);
    const unsigned long long t = scale_mass(p.u[r], Z);
    unsigned long long c_above = 0, lo_i = 0, hi_i = (unsigned long long)V - 1;  // index range that holds the token
    for (int round = 0; lo_i < hi_i && round < 32; ++round) {
      const int bits = 32 - __clz((uint32_t)(hi_i - lo_i)), shift = bits > kSBits ? bits - kSBits : 0;
      __syncthreads();
      for (int b = tid; b < kSBins; b += nt) scratch.mass[b] = MassBin{0, 0};
      __syncthreads();
      for (int i = tid & 31; i < n_part; i += 32) {
        const uint2 e = part[i];
        if (e.y >= lo_i && e.y <= hi_i && kept(key_logit(e.x), (int)e.y)) add_mass(&scratch.mass[(e.y - lo_i) >> shift], mass_of(e.x));
      }
      __syncthreads();
      find_bin([&](int b) { return scratch.mass[b].value(); }, t + 1, c_above, sh, s_pick);
      const unsigned long long b = s_pick[0];
      c_above = s_pick[1];
      lo_i += b << shift;
      hi_i = min(hi_i, lo_i + ((1ull << shift) - 1));
    }
    if (tid == 0) {
      p.tokens[r] = (int)lo_i;
      if (p.prob) p.prob[r] = (float)((double)mass_of(logit_key(row.at((int)lo_i))) / (double)Z);
    }
    return;
  }
  // the draw on the row: where the token's piece is, then the masses of a few pieces a thread
  MassSum sum;
  auto weigh = [&](int v) {
    const float x = row.at(v);
    sum.add(MassPair(kept(x, v) ? rule_weight(x, M, rate) : 0.f, 0.f));
  };
  auto weigh_piece = [&](const uint4& q, int v) {
    if (tiny) {
#pragma unroll 1
      for (int e = 0; e < Row::E; ++e) weigh(v + e);
      return;
    }
    float x[Row::E];
    Row::split(q, x);
    const bool plain = v + Row::E <= cut;  // ties of the whole piece are kept
#pragma unroll
    for (int e = 0; e < Row::E; e += 2)
      sum.add_if(weights(x[e], x[e + 1]), plain ? x[e] >= xs : kept(x[e], v + e), plain ? x[e + 1] >= xs : kept(x[e + 1], v + e + 1));
  };
  unsigned long long Z, t, start;
  int g0, g1;
  bool at_first, at_last;
  if (run_hi >= xs) {  // the runs' masses are known but for the list's entries
    __syncthreads();
    for (int i = tid & 31; i < n_part; i += 32)
      if (kept(key_logit(part[i].x), (int)part[i].y)) add_mass(run_mass + run_of((int)part[i].y), mass_of(part[i].x));
    __syncthreads();
    Z = 0;
    for (int i = tid; i < n_runs; i += nt) Z += run_mass[i].value();
    Z = block_sum_u64(Z, sh);
    t = scale_mass(p.u[r], Z);
    __syncthreads();
    find_bin([&](int b) { return b < n_runs ? run_mass[b].value() : 0ull; }, t + 1, 0ull, sh, s_pick);
    const int c = (int)s_pick[0];
    g0 = c * kRun;
    g1 = min(g0 + kRun, row.nv);
    at_first = c == 0;
    at_last = c == n_runs - 1;
  } else {  // a stretch of pieces a warp; the loose entries go with the first and the last
    const int warp = tid >> 5, nw = nt >> 5, stretch = (row.nv + nw - 1) / nw;
    row.pieces(min(warp * stretch, row.nv), min((warp + 1) * stretch, row.nv), tid & 31, 32, [&](const uint4& q, int v, bool ok) {
      if (ok && Row::largest(q) >= xs) weigh_piece(q, v);
    });
    if (warp == 0)
      for (int v = tid; v < row.a0; v += 32) weigh(v);
    if (warp == nw - 1)
      for (int v = row.a0 + row.nv * Row::E + (tid & 31); v < V; v += 32) weigh(v);
    const unsigned long long m = sum.total();
    const unsigned long long end = block_scan_u64(m, sh);
    Z = block_sum_u64(m, sh);
    t = scale_mass(p.u[r], Z);
    start = __shfl_sync(0xffffffffu, end - m, 0);
    const unsigned long long stop = __shfl_sync(0xffffffffu, end, 31);
    if (start <= t && stop > t && (tid & 31) == 0) { s_pick[0] = warp; s_pick[1] = start; }
    __syncthreads();
    g0 = min((int)s_pick[0] * stretch, row.nv);
    g1 = min(g0 + stretch, row.nv);
    at_first = s_pick[0] == 0;
    at_last = (int)s_pick[0] == nw - 1;
  }
  start = s_pick[1];
  const int each = (g1 - g0 + nt - 1) / nt;
  const int ga = min(g0 + tid * each, g1), ge = min(ga + each, g1);
  const int p0 = row.a0 + ga * Row::E, p1 = row.a0 + ge * Row::E;
  const int a = at_first && tid == 0 ? 0 : p0, e = at_last && tid == nt - 1 ? V : p1;
  sum = MassSum();
  for (int v = a; v < p0; ++v) weigh(v);
#pragma unroll 2
  for (int g = ga; g < ge; ++g) weigh_piece(row.piece(g), row.a0 + g * Row::E);
  for (int v = p1; v < e; ++v) weigh(v);
  const unsigned long long m = sum.total();
  unsigned long long c = block_scan_u64(m, sh) - m + start;
  if (c <= t && c + m > t) {
    for (int v = a; v < e; ++v) {
      const float x = row.at(v);
      if (!kept(x, v)) continue;
      const unsigned long long w = fx40(rule_weight(x, M, rate));
      c += w;
      if (c > t) {
        p.tokens[r] = v;
        if (p.prob) p.prob[r] = (float)((double)w / (double)Z);
        break;
      }
    }
  }
}

template <class Tin, int NT, int kBlocks, bool kDraw>
static cudaError_t launch_rule(const SampleParams& p, int N, cudaStream_t s) {
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = set_smem_limit_once((const void*)sampling_rule_kernel<Tin, NT, kBlocks, kDraw>, (int)kSSmem, attr);
  if (e != cudaSuccess) return e;
  sampling_rule_kernel<Tin, NT, kBlocks, kDraw><<<N, NT, kSSmem, s>>>(p);
  return cudaGetLastError();
}

template <class Tin, bool kDraw>
static cudaError_t launch_rule(const SampleParams& p, int N, bool alone, cudaStream_t s) {
  return alone ? launch_rule<Tin, 512, 1, kDraw>(p, N, s) : launch_rule<Tin, 512, 2, kDraw>(p, N, s);
}

template <bool kDraw>
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
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSPARK_ERR_CUDA;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const cudaError_t e = dtype == DSPARK_BF16 ? launch_rule<__nv_bfloat16, kDraw>(p, N, N <= sms, (cudaStream_t)stream)
                                             : launch_rule<float, kDraw>(p, N, N <= sms, (cudaStream_t)stream);
  note_launches(1);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

}  // namespace dspark

using namespace dspark;

extern "C" dspark_status dspark_sample(int32_t N, int32_t V, int32_t dtype, const void* logits, const float* temperature,
                                       const int32_t* top_k, const float* top_p, const float* min_p, const double* u,
                                       int32_t* tokens, float* prob, void* workspace, size_t workspace_bytes,
                                       dspark_stream_t stream) {
  note_launches(0);
  if (N > 0 && (!u || !tokens)) return DSPARK_ERR_INVALID_ARG;
  return sampling_entry<true>(N, V, dtype, logits, temperature, top_k, top_p, min_p, u, tokens, prob, nullptr, workspace,
                        workspace_bytes, stream);
}

extern "C" dspark_status dspark_truncate(int32_t N, int32_t V, int32_t dtype, const void* logits,
                                         const float* temperature, const int32_t* top_k, const float* top_p,
                                         const float* min_p, void* out, void* workspace, size_t workspace_bytes,
                                         dspark_stream_t stream) {
  note_launches(0);
  if (N > 0 && !out) return DSPARK_ERR_INVALID_ARG;
  return sampling_entry<false>(N, V, dtype, logits, temperature, top_k, top_p, min_p, nullptr, nullptr, nullptr, out, workspace,
                        workspace_bytes, stream);
}
