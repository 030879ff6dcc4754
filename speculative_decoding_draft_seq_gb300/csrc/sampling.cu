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
// of the top-k set; min-p keeps the entries with w >= min_p. All three are
// prefixes of that order, so the kept set is "logit above x*, or equal to it
// and index below cut": one threshold, found in three steps.
//   1  the row streams in once from memory: maximum, and counts in 4096 bins of
//      1/32 octave of weight (relative to an entry of the row, so that the
//      maximum need not be known yet);
//   2  the bins give the count, and within a few per mille the mass, at which
//      top-k or top-p ends; a second pass (from L2) collects the entries of the
//      bins in question, or of all bins from the top where they fit, in shared
//      memory, and adds up the exact masses that the answer needs;
//   3  radix selection on the collected entries' order-preserving integer keys
//      (2048-bin histograms of counts and masses over a shrinking key range).
// Where step 2 finds no set of bins that fits (thousands of equal entries, or
// logits hundreds of octaves apart), the selection runs on the row itself.
// One block a row: a row of 129,280 bf16 is 258 KB, and the rows in flight stay
// in L2 between the passes.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "verify_common.cuh"

namespace dspark {

constexpr int kSBins = 2048;    // bins of a selection round
constexpr int kWBins = 4096;    // weight bins, 32 an octave
constexpr int kSList = 6144;    // collected entries
constexpr uint32_t kSSmem = kWBins * 4 + kWBins * 8 + kSList * 8;

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
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Sum of floor(w 2^40) over weights in [0, 1], as two sums of 20-bit halves: adding 8 with rounding
// towards zero leaves floor(w 2^20) in the low mantissa bits, and what it cut off gives the other half.
// Up to 2^11 weights fit.
struct MassSum {
  uint32_t hi = 0, lo = 0, n = 0;
  __device__ __forceinline__ void add(float w) {
    const float a = __fadd_rz(w, 8.f);
    const float b = __fmaf_rz(__fsub_rn(w, __fsub_rn(a, 8.f)), 0x1p20f, 8.f);
    hi += __float_as_uint(a);
    lo += __float_as_uint(b);
    ++n;
  }
  __device__ __forceinline__ unsigned long long total() const {
    const uint32_t base = n * 0x41000000u;
    return ((unsigned long long)(hi - base) << 20) + (lo - base);
  }
};

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
// Plain loads: dspark_truncate may write the row in place.
template <class Tin>
struct RowView {
  static constexpr int E = 16 / (int)sizeof(Tin);
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
  // f(x, v) for the entries of pieces g0 <= g < g1 (tid-th of nt threads) and, with `ends`, the loose ones
  template <class F>
  __device__ __forceinline__ void each(int g0, int g1, int tid, int nt, bool ends, F f) const {
    constexpr int U = 4;
    for (int g = g0 + tid; g < g1; g += U * nt) {
      uint4 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (g + u * nt < g1) q[u] = piece(g + u * nt);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (g + u * nt >= g1) break;
        float x[E];
        split(q[u], x);
        const int v = a0 + (g + u * nt) * E;
#pragma unroll
        for (int e = 0; e < E; ++e) f(x[e], v + e);
      }
    }
    if (ends) {
      const int loose = V - nv * E;
      for (int i = tid; i < loose; i += nt) {
        const int v = i < a0 ? i : i + nv * E;
        f(at(v), v);
      }
    }
  }
  template <class F>
  __device__ __forceinline__ void all(F f) const { each(0, nv, threadIdx.x, blockDim.x, true, f); }
};

struct Threshold {
  uint32_t key;             // the last kept key
  unsigned long long ties;  // entries of this key that are kept, in index order
  unsigned long long count, above;  // entries of this key; the mass of the larger keys
};

struct SelectScratch {
  uint32_t* cnt;              // [kSBins]
  unsigned long long* mass;   // [kSBins]
  unsigned long long* sh;     // [32]
  unsigned long long* pick;   // [4]
};

// The key at which the running count (by_mass = false) or mass in descending order first reaches
// `target`, among the keys lo..hi of the entries that `source` enumerates; `above` is the mass of the
// larger keys that it leaves out.
template <class Source, class Mass>
__device__ Threshold select_key(Source source, Mass mass_of, bool by_mass, unsigned long long target, unsigned long long c_above,
                                unsigned long long m_above, uint32_t lo, uint32_t hi, const SelectScratch& s) {
  const int tid = threadIdx.x, nt = blockDim.x, per = kSBins / nt;
  for (;;) {
    const uint32_t span = hi - lo;
    const int bits = 32 - __clz(span), shift = bits > 11 ? bits - 11 : 0;
    __syncthreads();
    for (int b = tid; b < kSBins; b += nt) { s.cnt[b] = 0; s.mass[b] = 0; }
    __syncthreads();
    source([&](uint32_t k) {
      if (k < lo || k > hi) return;
      const uint32_t b = (hi - k) >> shift;
      atomicAdd(&s.cnt[b], 1u);
      atomicAdd(&s.mass[b], mass_of(k));
    });
    __syncthreads();
    unsigned long long c = 0, m = 0;
    for (int i = 0; i < per; ++i) { c += s.cnt[per * tid + i]; m += s.mass[per * tid + i]; }
    unsigned long long ci = block_scan_u64(c, s.sh) - c + c_above, mi = block_scan_u64(m, s.sh) - m + m_above;
    for (int i = 0; i < per; ++i) {
      const unsigned long long cb = s.cnt[per * tid + i], mb = s.mass[per * tid + i];
      const unsigned long long start = by_mass ? mi : ci, end = by_mass ? mi + mb : ci + cb;
      if (start < target && end >= target) {
        s.pick[0] = per * tid + i;
        s.pick[1] = ci;
        s.pick[2] = mi;
        s.pick[3] = cb;
      }
      ci += cb;
      mi += mb;
    }
    __syncthreads();
    const uint32_t b = (uint32_t)s.pick[0];
    c_above = s.pick[1];
    m_above = s.pick[2];
    const unsigned long long cnt = s.pick[3];
    if (shift == 0) {
      Threshold t;
      t.key = hi - b;
      t.count = cnt;
      t.above = m_above;
      const unsigned long long w = mass_of(t.key);
      t.ties = by_mass ? (target - m_above + w - 1) / w : target - c_above;
      if (t.ties > cnt) t.ties = cnt;
      __syncthreads();
      return t;
    }
    const uint32_t top = hi - (b << shift);
    lo = max(lo, top - ((1u << shift) - 1));
    hi = top;
  }
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

template <class Tin>
__global__ void __launch_bounds__(1024, 1) sampling_rule_kernel(SampleParams p) {
  extern __shared__ __align__(16) unsigned char s_raw[];
  __shared__ unsigned long long sh[32], s_pick[4];
  __shared__ float shf[32];
  __shared__ int shi[32], s_n;
  uint32_t* cum_c = reinterpret_cast<uint32_t*>(s_raw);                               // [kWBins] from the top bin down
  unsigned long long* cum_m = reinterpret_cast<unsigned long long*>(cum_c + kWBins);  // [kWBins] the same, estimated mass
  uint2* list = reinterpret_cast<uint2*>(cum_m + kWBins);                             // [kSList] (key, index)
  const SelectScratch scratch{reinterpret_cast<uint32_t*>(cum_m + kSBins), cum_m, sh, s_pick};
  const int tid = threadIdx.x, nt = blockDim.x, V = p.V;
  const size_t r = blockIdx.x;
  const RowView<Tin> row(static_cast<const Tin*>(p.logits) + r * V, V);
  const float T = __ldg(p.temperature + r), tp = __ldg(p.top_p + r);
  const float min_w = fminf(fmaxf(__ldg(p.min_p + r), 0.f), 1.f);
  const int k = __ldg(p.top_k + r);
  const bool greedy = !(T > 0.f), by_k = !greedy && k > 0 && k < V, by_p = !greedy && tp < 1.f;
  const float rate = fminf(__fdiv_rn(1.4426950408889634f, T), 1e30f);

  // ---- 1: maximum and weight bins ----
  WeightBins bins{32.f * rate, 0.f};
  bool binned = by_k || by_p;
  if (binned) {  // the bins' origin: the largest of the first entries
    float m0 = -INFINITY;
    for (int v = tid & 31; v < min(V, 256); v += 32) m0 = fmaxf(m0, row.at(v));
    m0 = warp_max(m0);
    if (!(fabsf(m0) < INFINITY)) m0 = 0.f;
    const float o = rintf(m0 * bins.c);
    binned = fabsf(o) <= 524288.f && rate > 0.f;  // else too far for bins of 1/32 octave in float32
    bins.off = 8388608.f + (kWBins / 2) - o;
    for (int b = tid; b < kWBins; b += nt) cum_c[b] = 0;
    __syncthreads();
  }
  float M = -INFINITY;
  if (binned)
    row.all([&](float x, int) {
      M = max_nan(M, x);
      atomicAdd(&cum_c[kWBins - 1 - WeightBins::index(bins.pos(x))], 1u);
    });
  else
    row.all([&](float x, int) { M = max_nan(M, x); });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
  if ((tid & 31) == 0) shf[tid >> 5] = M;
  __syncthreads();
  for (int i = 0; i < (nt >> 5); ++i) M = max_nan(M, shf[i]);
  if (!(M < INFINITY) || M == -INFINITY) {  // a NaN or +inf, or nothing finite: no distribution
    if (tid == 0) {
      set_status(p.status, DSPARK_ERR_NONFINITE);
      if (p.tokens) p.tokens[r] = -1;
      if (p.prob) p.prob[r] = 0.f;
    }
    if (p.out) {
      Tin* out = static_cast<Tin*>(p.out) + r * V;
      for (int v = tid; v < V; v += nt) out[v] = row.row[v];
    }
    return;
  }
  M = __fadd_rn(M, 0.f);
  auto mass_of = [&](uint32_t key) { return fx40(rule_weight(key_logit(key), M, rate)); };
  auto from_row = [&](auto f) { row.all([&](float x, int) { f(logit_key(x)); }); };

  // the kept set: logits above key_logit(key), and those equal to it up to index `cut`
  uint32_t key = logit_key(-INFINITY) + 1;
  int cut = V;
  bool headed = false;  // the list holds every kept entry
  int n_list = 0;
  if (greedy) {
    int at = V;
    row.all([&](float x, int v) { at = x == M ? min(at, v) : at; });
    at = block_min_i(at, shi);
    key = logit_key(M);
    cut = at + 1;
  } else if (by_k || by_p) {
    const uint32_t hi = logit_key(M), lowest = logit_key(-INFINITY);
    const float tm = __fmaf_rn(M, bins.c, bins.off - 8388608.f);  // the maximum's place on the bins' axis
    binned = binned && tm > 0.f && tm < kWBins - 1;
    Threshold th;
    bool found = false;
    unsigned long long S = 0;
    // ---- 2: the bins in question ----
    if (binned) {
      const int per = kWBins / nt;
      unsigned long long c = 0, m = 0;
      for (int i = 0; i < per; ++i) {
        const int j = per * tid + i;
        const unsigned long long n = cum_c[j];
        c += n;
        if (by_p && !by_k) m += n * fx40(ex2_approx(fminf(((float)(kWBins - 1 - j) - tm) * 0.03125f, 0.f)));
        cum_c[j] = (uint32_t)c;
        cum_m[j] = m;
      }
      const unsigned long long c0 = block_scan_u64(c, sh) - c;
      const unsigned long long m0 = by_p && !by_k ? block_scan_u64(m, sh) - m : 0ull;
      for (int i = 0; i < per; ++i) {
        cum_c[per * tid + i] += (uint32_t)c0;
        cum_m[per * tid + i] += m0;
      }
      __syncthreads();
      auto first_c = [&](unsigned long long want) {  // the first bin (from the top) where the count reaches `want`
        int a = 0, b = kWBins - 1;
        while (a < b) {
          const int mid = (a + b) >> 1;
          if (cum_c[mid] >= want) b = mid;
          else a = mid + 1;
        }
        return a;
      };
      auto first_m = [&](unsigned long long want) {
        int a = 0, b = kWBins - 1;
        while (a < b) {
          const int mid = (a + b) >> 1;
          if (cum_m[mid] >= want) b = mid;
          else a = mid + 1;
        }
        return a;
      };
      auto count_in = [&](int a, int b) { return (int)(cum_c[b] - (a > 0 ? cum_c[a - 1] : 0u)); };
      unsigned long long est = cum_m[kWBins - 1], want = 0;
      long long shift = 0;  // exact minus estimated mass at the bins looked at
      if (by_p && !by_k) want = scale_mass((double)fminf(tp, 1.f - 0x1p-24f), est);
      for (int attempt = 0; attempt < 4 && !found; ++attempt) {
        int ja, jb;  // bins, counted from the top
        if (by_k) {
          ja = jb = first_c((unsigned long long)k);
        } else {
          for (unsigned long long d = est >> (attempt == 0 ? 8 : 10);; d >>= 1) {
            const long long w = (long long)want - shift;
            ja = first_m(w > (long long)d ? (unsigned long long)(w - (long long)d) : 1ull);
            jb = first_m(w + (long long)d > 0 ? (unsigned long long)(w + (long long)d) : 1ull);
            if (d == 0 || count_in(ja, jb) <= kSList) break;
          }
        }
        headed = cum_c[jb] <= kSList;
        if (headed) ja = 0;
        n_list = count_in(ja, jb);
        if (n_list > kSList) break;
        const float f_lo = WeightBins::edge(kWBins - 1 - jb), f_hi = WeightBins::edge(kWBins - 1 - ja);
        __syncthreads();
        if (tid == 0) s_n = 0;
        __syncthreads();
        auto collect = [&](float t, float x, int v) {
          if (t >= f_lo && t <= f_hi) list[atomicAdd(&s_n, 1)] = make_uint2(logit_key(x), (uint32_t)v);
        };
        unsigned long long above = 0;
        if (by_p && !by_k) {
          MassSum sum, over;
          if (S == 0 && headed) {
            row.all([&](float x, int v) {
              sum.add(ex2_approx(__fmul_rn(__fsub_rn(x, M), rate)));
              collect(bins.pos(x), x, v);
            });
          } else {
            row.all([&](float x, int v) {
              const float w = ex2_approx(__fmul_rn(__fsub_rn(x, M), rate)), t = bins.pos(x);
              sum.add(w);
              over.add(t > f_hi ? w : 0.f);
              collect(t, x, v);
            });
          }
          S = block_sum_u64(sum.total(), sh);
          above = headed ? 0ull : block_sum_u64(over.total(), sh);
          want = max(1ull, scale_mass((double)fminf(tp, 1.f - 0x1p-24f), S));
        } else {
          if (by_p && !headed) break;  // the top-k set's mass would not be known
          row.all([&](float x, int v) { collect(bins.pos(x), x, v); });
        }
        __syncthreads();
        if (!by_k) {  // does the mass end among the list's entries?
          unsigned long long in = 0;
          for (int i = tid; i < n_list; i += nt) in += mass_of(list[i].x);
          in = block_sum_u64(in, sh);
          if (!(above < want && want <= above + in)) {
            if (want > above) shift = (long long)(above + in) - (long long)cum_m[jb];
            else shift = (long long)above - (long long)(ja > 0 ? cum_m[ja - 1] : 0ull);
            continue;
          }
        }
        found = true;
        // ---- 3: selection on the list ----
        auto from_list = [&](auto f) {
          for (int i = tid; i < n_list; i += nt) f(list[i].x);
        };
        if (by_k) {
          const unsigned long long before = ja > 0 ? cum_c[ja - 1] : 0u;
          __syncthreads();
          th = select_key(from_list, mass_of, false, (unsigned long long)k, before, 0ull, lowest, hi, scratch);
          if (by_p) {
            S = th.above + th.ties * mass_of(th.key);
            want = max(1ull, scale_mass((double)fminf(tp, 1.f - 0x1p-24f), S));
            th = select_key(from_list, mass_of, true, want, 0ull, 0ull, th.key, hi, scratch);
          }
        } else {
          th = select_key(from_list, mass_of, true, want, 0ull, above, lowest, hi, scratch);
        }
        if (th.ties < th.count) {  // the index of the last tie that is kept: the ties-th smallest
          auto tie_index = [&](auto f) {
            for (int i = tid; i < n_list; i += nt)
              if (list[i].x == th.key) f(~list[i].y);
          };
          const Threshold at = select_key(tie_index, [](uint32_t) { return 1ull; }, false, th.ties, 0ull, 0ull,
                                          ~(uint32_t)(V - 1), 0xffffffffu, scratch);
          cut = (int)~at.key + 1;
        }
      }
    }
    if (!found) {  // the same selection on the row
      headed = false;
      uint32_t lo = lowest;
      if (by_k) {
        th = select_key(from_row, mass_of, false, (unsigned long long)k, 0ull, 0ull, lo, hi, scratch);
        lo = th.key;
        S = th.above + th.ties * mass_of(th.key);
      } else {
        MassSum sum;
        row.all([&](float x, int) { sum.add(rule_weight(x, M, rate)); });
        S = block_sum_u64(sum.total(), sh);
      }
      if (by_p) {
        const unsigned long long want = max(1ull, scale_mass((double)fminf(tp, 1.f - 0x1p-24f), S));
        th = select_key(from_row, mass_of, true, want, 0ull, 0ull, lo, hi, scratch);
      }
      if (th.ties < th.count) {
        const float xs = key_logit(th.key);
        auto tie_index = [&](auto f) {
          row.all([&](float x, int v) {
            if (x == xs) f(~(uint32_t)v);
          });
        };
        const Threshold at = select_key(tie_index, [](uint32_t) { return 1ull; }, false, th.ties, 0ull, 0ull,
                                        ~(uint32_t)(V - 1), 0xffffffffu, scratch);
        cut = (int)~at.key + 1;
      }
    }
    if (th.key >= key) key = th.key;
    else cut = V;  // the threshold fell on entries of -inf: all others are kept
  }
  if (!greedy && min_w > 0.f) {  // the smallest key whose weight reaches min_p, by 32-way search
    uint32_t lo = key, hi = logit_key(M);  // the weight of hi is 1
    while (lo < hi) {
      const uint32_t step = (hi - lo) / 32 + 1;
      const uint32_t at = (uint32_t)min((unsigned long long)hi, lo + (unsigned long long)step * (tid & 31));
      const uint32_t ok = __ballot_sync(0xffffffffu, rule_weight(key_logit(at), M, rate) >= min_w);
      const int first = ok ? __ffs(ok) - 1 : 32;  // lanes before it lie below
      hi = (uint32_t)min((unsigned long long)hi, lo + (unsigned long long)step * first);
      if (first > 0) lo = (uint32_t)min((unsigned long long)hi, lo + (unsigned long long)step * (first - 1) + 1);
      else hi = lo;
    }
    if (lo > key) { key = lo; cut = V; }
  }
  const float xs = key_logit(key);
  auto kept = [&](float x, int v) { return x > xs || (x == xs && v < cut); };

  if (p.out) {
    Tin* out = static_cast<Tin*>(p.out) + r * V;
    const bool aligned = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row.row)) & 15) == 0;
    const uint32_t low = sizeof(Tin) == 2 ? 0xff7fu : 0xff7fffffu;  // the lowest finite value
    if (aligned) {
      constexpr int E = RowView<Tin>::E, U = 4;
      for (int g = tid; g < row.nv; g += U * nt) {
        uint4 q[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (g + u * nt < row.nv) q[u] = row.piece(g + u * nt);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (g + u * nt >= row.nv) break;
          float x[E];
          RowView<Tin>::split(q[u], x);
          const int v = row.a0 + (g + u * nt) * E;
          uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (E == 8) {
              const uint32_t keep = (kept(x[(2 * i) % E], v + 2 * i) ? 0xffffu : 0u) | (kept(x[(2 * i + 1) % E], v + 2 * i + 1) ? 0xffff0000u : 0u);
              w[i] = (w[i] & keep) | ((low | low << 16) & ~keep);
            } else {
              w[i] = kept(x[i % E], v + i) ? w[i] : low;
            }
          }
          __stcs(reinterpret_cast<uint4*>(out + v), make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
    }
    const int loose = aligned ? V - row.nv * RowView<Tin>::E : V;
    for (int i = tid; i < loose; i += nt) {
      const int v = aligned && i >= row.a0 ? i + row.nv * RowView<Tin>::E : i;
      const Tin raw = row.row[v];
      if (kept(row.at(v), v)) out[v] = raw;
      else if (sizeof(Tin) == 2) *reinterpret_cast<uint16_t*>(out + v) = (uint16_t)low;
      else *reinterpret_cast<uint32_t*>(out + v) = low;
    }
  }
  if (!p.tokens) return;
  if (greedy) {
    if (tid == 0) {
      p.tokens[r] = cut - 1;
      if (p.prob) p.prob[r] = 1.f;
    }
    return;
  }
  if (headed) {  // every kept entry is on the list: the draw selects an index by mass
    unsigned long long Z = 0;
    for (int i = tid; i < n_list; i += nt)
      if (kept(key_logit(list[i].x), (int)list[i].y)) Z += mass_of(list[i].x);
    Z = block_sum_u64(Z, sh);
    const unsigned long long t = scale_mass(p.u[r], Z);
    unsigned long long c_above = 0, lo_i = 0, hi_i = (unsigned long long)V - 1;  // index range that holds the token
    while (lo_i < hi_i) {
      const int bits = 32 - __clz((uint32_t)(hi_i - lo_i)), shift = bits > 11 ? bits - 11 : 0;
      __syncthreads();
      for (int b = tid; b < kSBins; b += nt) scratch.mass[b] = 0;
      __syncthreads();
      for (int i = tid; i < n_list; i += nt) {
        const uint2 e = list[i];
        if (e.y >= lo_i && e.y <= hi_i && kept(key_logit(e.x), (int)e.y)) atomicAdd(&scratch.mass[(e.y - lo_i) >> shift], mass_of(e.x));
      }
      __syncthreads();
      const int per = kSBins / nt;
      unsigned long long m = 0;
      for (int i = 0; i < per; ++i) m += scratch.mass[per * tid + i];
      unsigned long long at = block_scan_u64(m, sh) - m + c_above;
      for (int i = 0; i < per; ++i) {
        const unsigned long long mb = scratch.mass[per * tid + i];
        if (at <= t && at + mb > t) { s_pick[0] = per * tid + i; s_pick[1] = at; }
        at += mb;
      }
      __syncthreads();
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
  // the draw on the row: masses of one stretch of entries a warp, then the entries of the stretch
  const int warp = tid >> 5, lane = tid & 31, nw = nt >> 5;
  const int len = ((V + nw - 1) / nw + 31) & ~31, b0 = min(warp * len, V), b1 = min(b0 + len, V);
  unsigned long long m = 0;
  for (int v = b0 + lane; v < b1; v += 32) {
    const float x = row.at(v);
    if (kept(x, v)) m += fx40(rule_weight(x, M, rate));
  }
  const unsigned long long end = block_scan_u64(m, sh), Z = block_sum_u64(m, sh);
  const unsigned long long t = scale_mass(p.u[r], Z);
  unsigned long long start = __shfl_sync(0xffffffffu, end - m, 0);
  const unsigned long long stop = __shfl_sync(0xffffffffu, end, 31);
  if (start <= t && stop > t && lane == 0) { s_pick[0] = b0; s_pick[1] = start; }
  __syncthreads();
  const int s0 = (int)s_pick[0], s1 = min(s0 + len, V);
  start = s_pick[1];
  const int each = (len + nt - 1) / nt, a = min(s0 + tid * each, s1), e = min(a + each, s1);
  m = 0;
  for (int v = a; v < e; ++v) {
    const float x = row.at(v);
    if (kept(x, v)) m += fx40(rule_weight(x, M, rate));
  }
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
  static std::atomic<unsigned long long> attr_bf16{0}, attr_f32{0};
  const bool bf16 = dtype == DSPARK_BF16;
  const void* fn = bf16 ? (const void*)sampling_rule_kernel<__nv_bfloat16> : (const void*)sampling_rule_kernel<float>;
  if (set_smem_limit_once(fn, (int)kSSmem, bf16 ? attr_bf16 : attr_f32) != cudaSuccess) return DSPARK_ERR_CUDA;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSPARK_ERR_CUDA;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int threads = N <= sms ? 1024 : 512;  // a block an SM for few rows, two for many (their phases overlap)
  if (bf16) sampling_rule_kernel<__nv_bfloat16><<<N, threads, kSSmem, (cudaStream_t)stream>>>(p);
  else sampling_rule_kernel<float><<<N, threads, kSSmem, (cudaStream_t)stream>>>(p);
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
