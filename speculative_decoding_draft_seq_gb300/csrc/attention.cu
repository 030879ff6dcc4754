// Attention of a round's tokens over a shared prefix and each request's own
// pages of a paged key/value cache: for query token i of request r and head h,
//   x_j = scale q . k_j over the prefix's keys and the request's keys up to the
//   token's own position, out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),
//   lse = m + ln sum_j e^(x_j - m), m = max_j x_j.
//
// The softmax of a row is joined from parts over disjoint key ranges: a part
// gives (m, z = sum 2^(x log2(e) - m), o = sum 2^(x log2(e) - m) v), and parts
// add up after scaling by 2^(m - max m). The prefix is one key range for the
// rows of all requests (its keys are read once for 256 rows of the whole batch
// instead of once a request), a request's own pages are another, and either is
// split further when that makes enough work for every SM.
//
// Launches:
//   attn_plan_kernel   one CTA: cuts the work into items (a key head, a block of
//                      query tokens, a range of 128-key tiles), equal shares of
//                      about 1/kPlanShare of an SM's work;
//   attn_tiles_kernel  persistent, one CTA an SM; a CTA takes the next item when it
//                      is done with one. Prefix items (bound by the tensor cores)
//                      and page items (bound by memory) alternate in their
//                      numbers' ratio, so that both run at any time;
//   attn_join_kernel   adds a row's parts up.
//
// attn_tiles_kernel: rows are (token, query head of the key head), packed
// floor(128 / group) tokens a 128-row half. Per step of 64 keys: S = Q K^T into
// one of two 64-column buffers of TMEM, four warps turn S into bf16 weights in
// place (one thread a row; S is in registers for the maximum and the weights),
// O += P V with P read from TMEM. S of the next step is formed meanwhile. Two such
// groups of warps, each with its buffers and an O, work side by side: an item with
// more tokens than a half holds gives each one a half of the rows (K and V tiles are
// read once for both); an item with fewer gives them the even and the odd 128-key
// tiles of the same rows (two parts).
//   Roundings: the weights that multiply v, and out, to bf16; scores, maxima, sums and O
// are float32 (the sum is of the unrounded weights). The tensor cores take both operands
// of a product in one type, and v is bf16; weights in two halves, value and rest, would take
// a second P V, half of a step's MMA cycles again. out's error against 64 bits is 0.0023
// relative; rounding out alone leaves 0.0017.
//   The weights use a reference maximum that is moved, and O rescaled, only when
// the row's maximum has risen by more than 8 (2^8 fits every type on the way), so O is
// rarely rescaled.
//   warps 0..3, 4..7  softmax and epilogue of group 0, 1
//   warp 8            takes the items; TMA loads: Q once an item, a ring of K and V
//                     tiles, one box a page (or 128 rows of a longer one), 64
//                     columns wide
//   warps 9, 10       MMA issue of group 0, 1 (and TMEM allocation): the waits and
//                     commits for both groups would take one warp longer than the
//                     MMAs. The V rows of the last 16-key group that lie past the
//                     keys are zeroed here (a weight of 0 times a NaN is a NaN).
//
// What bounds it. A step of both groups (256 rows, 64 keys) at D = 128 is 1,040
// cycles of MMAs issued back to back and 1,000 of softmax, which overlap; it takes
// about 1,750, in which each issuing warp is held for 740 cycles by an S's eight MMAs (33
// cycles each alone) and 410 by a product's four (64 each): the tensor pipe is 42% busy, the
// warps issue in 32% of the cycles, L2 and DRAM under 20%. Steps of 128 keys, one buffer, wait
// for the softmax instead: 294 us for a prefix of 65,553 (316 tokens, 28 heads on
// 4, D = 64; 149 GFLOP) instead of 271 (0.29 of the measured tensor rate), 304 instead of
// 299 for 128 requests, 1,144 tokens, with a prefix of 8,192 and up to 2,048 own keys
// (32 heads on 8, D = 128; 173 GFLOP, 0.59 GB; 0.31). TMEM's 512 columns are all taken at
// D = 128 (two O, four S), so that wider steps with two buffers have no room.
// 128 requests of one token, up to 4,096 own keys: 234 us, 4.7 TB/s (0.69 of the
// measured copy bandwidth): the warps wait for tiles, which are 256-byte rows 2 KB
// apart, five tiles of 32 KB in flight an SM.
// One token over 1,333 keys: 22.5 to 24 us, three dependent launches.
// A prompt chunk of one request (32 heads on 8, D = 128): 1,024 tokens 105 us (8.6 GFLOP), 2,048 over a
// prefix of 8,192 411 us (309 GFLOP; 0.40 of the tensor rate), 8,192 811 us (550; 0.36). One token over 65,536
// keys, own 183 us, prefix 153 (268 MB; floor 40): the plan forms a request's items, and the token's map, in one
// thread, and the join adds up a row's parts in one warp.
//
// Every wait is bounded: one that runs out records DSPARK_ERR_TIMEOUT, the
// roles wind down, issued copies and MMAs land, and the TMEM is freed.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"
#include "verify_common.cuh"

namespace dspark {

constexpr int kATile = 128;        // keys a tile of the ring
constexpr int kAChunk = 64;        // keys a step
constexpr int kASoftmaxWarps = 8;    // four a group: one thread a row
constexpr int kAThreads = 32 * (kASoftmaxWarps + 3);
constexpr int kPlanShare = 6;      // items are at most about 1/6 of an SM's share of the work
constexpr int kExtraSlots = 8192;  // token slots beyond one part for the prefix and two for the pages
constexpr int kMaxSms = 256;

struct AttnItem {
  int head;    // key head, and kAlternate
  int req;     // request, or -1: the prefix
  int tok0;    // first query token
  int n_tok;   // query tokens (at most two halves)
  int key0;    // first key, a multiple of kATile
  int n_keys;  // keys from key0 on that any row sees
  int slot0;   // part slot of the first token; -1: the only part of its rows, written to out
  int pos0;    // keys from key0 on that the first token sees (one more for each further token)
};
// An item of a block with at most one half's tokens: its warpgroups take the even and the odd tiles, and with two
// tiles or more it has two parts, the second one n_tok slots on.
constexpr int kAlternate = 1 << 30;

struct AttnHead {  // written by the plan
  int n_items, prefix_items, prefix_parts, n_tokens;
  unsigned int next;  // items taken
};

struct AttnParams {
  int R, T, Hq, Hkv, G, TB, page, page_log2, n_pages, max_pages, prefix_len, sms;
  long long cap_slots;
  const int32_t* prefix_pages;
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* kv_len;
  float rate;  // scale log2(e)
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
  AttnHead* head;
  AttnItem* items;
  int4* tokens;   // [T]: first page part slot, slots between parts, page parts (-1: nothing to join), unused
  float2* stat;   // [slot][Hq]: (m, z)
  float* acc;     // [slot][Hq][D]
};

struct AttnLayout {
  size_t head, tokens, items, stat, acc, total;
  long long slots;
};

inline int attn_tokens_per_half(int G) { return 128 / G; }

inline AttnLayout attn_layout(int R, int T, int Hq, int Hkv, int D) {
  AttnLayout L;
  const int TB = attn_tokens_per_half(Hq / Hkv);
  const long long blocks = 2ll * ceil_div(T, 2 * TB) + R + 1;
  const long long items = blocks * Hkv + (long long)kMaxSms * kPlanShare;
  L.slots = 3ll * T + kExtraSlots;
  size_t o = 256;
  L.head = o;   o = align256(o + sizeof(AttnHead));
  L.tokens = o; o = align256(o + (size_t)T * sizeof(int4));
  L.items = o;  o = align256(o + (size_t)items * sizeof(AttnItem));
  L.stat = o;   o = align256(o + (size_t)L.slots * Hq * sizeof(float2));
  L.acc = o;    o = align256(o + (size_t)L.slots * Hq * D * sizeof(float));
  L.total = o;
  return L;
}

// Waits until the launch before this one in the stream is complete and its writes are visible; lets the launch
// after this one be set up (it waits in turn).
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------------------
// The plan. Request r's queries are cut into blocks of two halves; block b of
// n tokens sees the first kv_len - n + (its last token) + 1 private keys.
constexpr int kAPlanThreads = 1024;  // at most; a thread a request, in turns of so many

__device__ __forceinline__ long long plan_sum(long long v, long long* sh) {  // over the block
  const int nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < nw; ++i) v += sh[i];
  return v;
}
__device__ __forceinline__ longlong2 plan_scan(longlong2 v, longlong2* sh, longlong2& total) {  // exclusive, over the block
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  longlong2 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) { x.x += a; x.y += b; }
  }
  __syncthreads();
  if (lane == 31) sh[w] = x;
  __syncthreads();
  longlong2 before = make_longlong2(0, 0);
  total = before;
  for (int i = 0; i < nw; ++i) {
    const longlong2 s = sh[i];
    if (i < w) { before.x += s.x; before.y += s.y; }
    total.x += s.x;
    total.y += s.y;
  }
  return make_longlong2(before.x + x.x - v.x, before.y + x.y - v.y);
}

__global__ void __launch_bounds__(kAPlanThreads, 1) attn_plan_kernel(AttnParams p) {
  __shared__ long long sh[32];
  __shared__ longlong2 sh2[32];
  const int tid = threadIdx.x, nthr = blockDim.x;
  let_next_launch();
  const int step = 2 * p.TB;  // tokens a block
  bool bad = false;
  auto request = [&](int r, int& start, int& n, int& len) {
    const int a = __ldg(p.q_start + r), b = __ldg(p.q_start + r + 1), l = __ldg(p.kv_len + r);
    const long long most = min((long long)p.max_pages * p.page, 0x7fffff00ll);
    bad |= l < 0 || l > most;
    start = a;
    n = b - a;
    len = (int)max(0ll, min((long long)l, most));
  };
  auto tiles_of = [&](int n, int len, int t0) {  // key tiles that the block of tokens t0.. of n sees
    return ceil_div(max(0ll, (long long)len - n + min(t0 + step, n)), kATile);
  };
  // starts that fall or leave [0, T]: their blocks would not be bounded by T, so nothing is computed
  bool broken = tid == 0 && __ldg(p.q_start) != 0;
  for (int r = tid; r < p.R; r += nthr) {
    const int a = __ldg(p.q_start + r), b = __ldg(p.q_start + r + 1);
    broken |= a < 0 || b < a || b > p.T;
  }
  if (__syncthreads_or(broken)) {
    if (tid == 0) {
      *p.head = AttnHead{0, 0, 0, 0, 0u};
      set_status(p.status, DSPARK_ERR_RANGE);
    }
    return;
  }
  const int n_tokens = __ldg(p.q_start + p.R);
  // how `tiles` key tiles of a block of `nt` tokens are split into items, and the parts that they leave
  auto splits_of = [&](int tiles, int nt, long long share) {
    const int ns = ceil_div(tiles, share);
    return nt <= p.TB ? max(min(ns, tiles / 2), min(tiles, 1)) : ns;  // two tiles at least for the two groups
  };
  auto parts_of = [&](int tiles, int nt, int ns) { return nt <= p.TB && tiles > 1 ? 2 * ns : ns; };
  const int p_tiles = ceil_div(p.prefix_len, kATile), p_blocks = ceil_div(n_tokens, step);
  long long units = 0;
  for (int r = tid; r < p.R; r += nthr) {
    int start, n, len;
    request(r, start, n, len);
    for (int t0 = 0; t0 < n; t0 += step) units += tiles_of(n, len, t0);
  }
  const long long total = (plan_sum(units, sh) + (long long)p_blocks * p_tiles) * p.Hkv;
  long long share = max(1ll, (total + (long long)p.sms * kPlanShare - 1) / ((long long)p.sms * kPlanShare));
  // page items of at least half a share come first, then the smaller ones
  auto small = [&](int tiles, int ns) { return 2ll * tiles < share * ns; };
  int p_splits, p_parts;
  long long all_large;
  for (;;) {  // tiles an item: more where the parts would not fit
    p_splits = splits_of(p_tiles, n_tokens, share);
    p_parts = parts_of(p_tiles, n_tokens, p_splits);
    long long slots = 0, larges = 0;
    for (int r = tid; r < p.R; r += nthr) {
      int start, n, len;
      request(r, start, n, len);
      for (int t0 = 0; t0 < n; t0 += step) {
        const int tiles = tiles_of(n, len, t0), nt = min(step, n - t0), ns = splits_of(tiles, nt, share);
        slots += (long long)parts_of(tiles, nt, ns) * nt;
        if (!small(tiles, ns)) larges += (long long)ns * p.Hkv;
      }
    }
    slots = plan_sum(slots, sh);
    all_large = plan_sum(larges, sh);
    if (slots + (long long)p_parts * n_tokens <= p.cap_slots || share > (1 << 30)) break;
    share *= 2;
  }
  const long long p_items = (long long)p_blocks * p.Hkv * p_splits;
  for (long long i = tid; i < p_items; i += nthr) {  // blocks that read the same keys next to one another
    const int b = (int)(i % p_blocks), s = (int)((i / p_blocks) % p_splits), h = (int)(i / p_blocks / p_splits);
    const int a = (int)((long long)s * p_tiles / p_splits), e = (int)((long long)(s + 1) * p_tiles / p_splits);
    AttnItem it;
    it.head = h | (n_tokens <= p.TB ? kAlternate : 0);
    it.req = -1;
    it.tok0 = b * step;
    it.n_tok = min(step, n_tokens - it.tok0);
    it.key0 = a * kATile;
    it.n_keys = min(p.prefix_len, e * kATile) - it.key0;
    it.slot0 = (p_parts > p_splits ? 2 * s : s) * n_tokens + it.tok0;
    it.pos0 = it.n_keys;
    p.items[i] = it;
  }
  long long large0 = p_items, small0 = p_items + all_large, slot0 = (long long)p_parts * n_tokens;
  for (int r0 = 0; r0 < p.R; r0 += nthr) {
    const int r = r0 + tid;
    int start = 0, n = 0, len = 0;
    if (r < p.R) request(r, start, n, len);
    long long larges = 0, smalls = 0, slots = 0;
    for (int t0 = 0; t0 < n; t0 += step) {
      const int tiles = tiles_of(n, len, t0), nt = min(step, n - t0), ns = splits_of(tiles, nt, share);
      (small(tiles, ns) ? smalls : larges) += (long long)ns * p.Hkv;
      slots += (long long)parts_of(tiles, nt, ns) * nt;
    }
    longlong2 all;
    const longlong2 at = plan_scan(make_longlong2(larges | smalls << 32, slots), sh2, all);
    long long large_at = large0 + (at.x & 0xffffffffll), small_at = small0 + (at.x >> 32), slot = slot0 + at.y;
    large0 += all.x & 0xffffffffll;
    small0 += all.x >> 32;
    slot0 += all.y;
    for (int t0 = 0; t0 < n; t0 += step) {
      const int tiles = tiles_of(n, len, t0), nt = min(step, n - t0), ns = splits_of(tiles, nt, share);
      const int parts = parts_of(tiles, nt, ns);
      const bool direct = p_splits == 0 && parts == 1;
      for (int i = 0; i < nt; ++i)
        p.tokens[start + t0 + i] = make_int4((int)slot + i, nt, direct ? -1 : parts, 0);
      const int seen = max(0, min(len, len - n + t0 + nt));  // keys that the block's last token sees
      long long& item = small(tiles, ns) ? small_at : large_at;
      for (int s = 0; s < ns; ++s) {
        const int a = (int)((long long)s * tiles / ns), e = (int)((long long)(s + 1) * tiles / ns);
        for (int h = 0; h < p.Hkv; ++h, ++item) {
          AttnItem it;
          it.head = h | (nt <= p.TB ? kAlternate : 0);
          it.req = r;
          it.tok0 = start + t0;
          it.n_tok = nt;
          it.key0 = a * kATile;
          it.n_keys = min(seen, e * kATile) - it.key0;
          it.slot0 = direct ? -1 : (int)slot + (parts > ns ? 2 * s : s) * nt;
          it.pos0 = len - n + t0 + 1 - it.key0;
          p.items[item] = it;
        }
      }
      slot += (long long)parts * nt;
    }
  }
  if (tid == 0) {
    p.head->n_items = (int)small0;
    p.head->prefix_items = (int)p_items;
    p.head->prefix_parts = p_parts;
    p.head->n_tokens = n_tokens;
    p.head->next = 0;
  }
  if (bad) set_status(p.status, DSPARK_ERR_RANGE);
}

// ---------------------------------------------------------------------------
template <int D>
struct AttnSmem {
  static constexpr int kHalves = D / 64;               // 64-column boxes of a head
  static constexpr uint32_t kBox = kATile * 128;       // 128 rows of 64 bf16
  static constexpr uint32_t kTileBytes = kHalves * kBox;
  static constexpr int kSlots = D == 128 ? 5 : 10;     // K and V tiles in the ring
  static constexpr uint32_t kQ = 2 * kTileBytes;
  static constexpr uint32_t kTotal = kQ + kSlots * kTileBytes + 512;
  static_assert(kTotal <= 227 * 1024, "shared memory of a CTA");
};

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// 32 bytes in one store (32-byte aligned).
__device__ __forceinline__ void store32(float* to, const float* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(__float_as_uint(v[0])),
               "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
               "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])),
               "r"(__float_as_uint(v[7]))
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kAThreads, 1)
    attn_tiles_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                      const __grid_constant__ CUtensorMap mapV, AttnParams p, int q_rows, int box_rows) {
  using S = AttnSmem<D>;
  constexpr int kHalves = S::kHalves, kSlots = S::kSlots;
  // (no room to align by hand: the swizzled tiles need 1024 bytes, which the base has without static shared memory)
  extern __shared__ __align__(1024) unsigned char smem[];
  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) set_status(p.status, DSPARK_ERR_CUDA);
    return;
  }
  unsigned char* sQ = smem;
  unsigned char* sKV = smem + S::kQ;
  uint64_t* full = reinterpret_cast<uint64_t*>(sKV + kSlots * S::kTileBytes);
  uint64_t* empty = full + kSlots;
  uint64_t* qFull = empty + kSlots;  // [2] Q of a half
  uint64_t* qEmpty = qFull + 2;      // [2]
  uint64_t* sFull = qEmpty + 2;   // [2][2] S of a group and buffer is in TMEM
  uint64_t* pFull = sFull + 4;    // [2][2] P is, in its place
  uint64_t* oDone = pFull + 4;    // [2][2] P V has been added to O
  uint64_t* oEmpty = oDone + 4;   // [2] the epilogue has read O
  uint64_t* drain = oEmpty + 2;
  uint64_t* iFull = drain + 1;    // [2] an item is there
  uint64_t* iEmpty = iFull + 2;   // [2] every role has read it
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(iEmpty + 2);
  volatile int* sAbort = reinterpret_cast<volatile int*>(sTmem + 1);
  int4* sItem = reinterpret_cast<int4*>((reinterpret_cast<uintptr_t>(sTmem) + 31) & ~uintptr_t(15));  // [2][2] an AttnItem

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    // both issuing warps pass every phase of every tile and Q, in order, and sign every release: a warp that skipped
    // some could get more than one phase apart from the other, where the parity of a wait means nothing
    for (int i = 0; i < kSlots; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 2); }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&qFull[g], 1);
      mbar_init(&qEmpty[g], 2);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sFull[2 * g + b], 1);
        mbar_init(&pFull[2 * g + b], kASoftmaxWarps / 2);
        mbar_init(&oDone[2 * g + b], 1);
      }
      mbar_init(&oEmpty[g], kASoftmaxWarps / 2);
      mbar_init(&iFull[g], 1);
      mbar_init(&iEmpty[g], kASoftmaxWarps + 2);
    }
    mbar_init(drain, 2);
    *sAbort = 0;
    mbar_fence_init();
  }
  if (warp == kASoftmaxWarps + 1) {
    __syncwarp();
    tmem_alloc(sTmem, 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sTmem;  // 0: all 512 columns are this CTA's
  wait_for_launch_before();      // (the set-up above runs under the plan)
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, sAbort, p.status)) != 0;
  };
  // the k-th item of this CTA (n_keys 0: there is none); by whole warps
  auto take = [&](int k) {
    const int slot = k & 1;
    AttnItem it;
    it.n_keys = 0;
    const bool ok = warp_wait(&iFull[slot], (k >> 1) & 1);
    const int4 a = sItem[2 * slot], b = sItem[2 * slot + 1];
    if (ok) {
      it.head = a.x; it.req = a.y; it.tok0 = a.z; it.n_tok = a.w;
      it.key0 = b.x; it.n_keys = b.y; it.slot0 = b.z; it.pos0 = b.w;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&iEmpty[slot]);
    return it;
  };

  if (warp == kASoftmaxWarps) {
    // ---- loads ----
    if (lane == 0) {
      prefetch_tensormap(&mapQ);
      prefetch_tensormap(&mapK);
      prefetch_tensormap(&mapV);
    }
    const uint64_t pol = l2_policy_evict_normal();
    int n = 0, q_turn = 0;        // ring tiles issued; the Q buffer of the next item that needs one
    uint32_t qPhase[2] = {1, 1};
    bool stop = false;
    const int n_items = p.head->n_items, n_prefix = p.head->prefix_items;
    for (int k = 0; !stop; ++k) {
      // the next item: prefix items and page items in their numbers' ratio
      int item = 0;
      if (lane == 0) {
        const long long t = atomicAdd(&p.head->next, 1u);
        const long long a = t * n_prefix / max(n_items, 1), b = (t + 1) * n_prefix / max(n_items, 1);
        item = t >= n_items ? -1 : (int)(b > a ? a : n_prefix + t - a);
      }
      item = __shfl_sync(0xffffffffu, item, 0);
      int4 half = make_int4(0, 0, 0, 0);  // lanes 0 and 1: the item's two halves
      if (item >= 0 && lane < 2) half = __ldcg(reinterpret_cast<const int4*>(p.items + item) + lane);
      if (!warp_wait(&iEmpty[k & 1], ((k >> 1) & 1) ^ 1)) break;
      if (lane < 2) sItem[2 * (k & 1) + lane] = half;
      __syncwarp();
      if (lane == 0) mbar_arrive(&iFull[k & 1]);
      if (item < 0) break;
      AttnItem it;
      it.head = __shfl_sync(0xffffffffu, half.x, 0);
      it.req = __shfl_sync(0xffffffffu, half.y, 0);
      it.tok0 = __shfl_sync(0xffffffffu, half.z, 0);
      it.key0 = __shfl_sync(0xffffffffu, half.x, 1);
      it.n_keys = __shfl_sync(0xffffffffu, half.y, 1);
      const int nt = ceil_div(it.n_keys, kATile);
      const int32_t* pages = it.req < 0 ? p.prefix_pages : p.table + (size_t)it.req * p.max_pages;
      const int boxes = kATile / box_rows;
      auto page_at = [&](int j) {  // lane i: the page of box i of tile j
        const int pos = j * kATile + lane * box_rows;
        return lane < boxes && pos < it.n_keys ? __ldg(pages + ((it.key0 + pos) >> p.page_log2)) : 0;
      };
      const int head = it.head & ~kAlternate, groups = it.head & kAlternate ? 1 : 2, ahead = groups == 2 ? 1 : 2;
      // one K (kv = 0) or V tile into the ring
      auto load = [&](int j, int kv, int pg) {
        const int live = min(boxes, ceil_div(it.n_keys - j * kATile, box_rows));
        const int row = (it.key0 + j * kATile + lane * box_rows) & (p.page - 1);
        const int slot = n % kSlots;
        if (lane < live && (pg < 0 || pg >= p.n_pages)) set_status(p.status, DSPARK_ERR_RANGE);
        if (!warp_wait(&empty[slot], ((n / kSlots) & 1) ^ 1)) {
          stop = true;
          return;
        }
        if (lane == 0) mbar_expect_tx(&full[slot], (uint32_t)(live * box_rows * 128 * kHalves));
        __syncwarp();
        if (lane < live) {
          unsigned char* dst = sKV + slot * S::kTileBytes + lane * box_rows * 128;
#pragma unroll
          for (int c = 0; c < kHalves; ++c)
            tma_load_4d(dst + c * S::kBox, kv ? &mapV : &mapK, 64 * c, head, row, pg, &full[slot], pol);
        }
        ++n;
      };
      // in the order of use: K of the first tiles, then V of a tile and K of the tile `ahead` on
      int pgs[3] = {page_at(0), nt > 1 ? page_at(1) : 0, 0};  // pages of tiles j, j + 1, j + 2
      load(0, 0, pgs[0]);
      // Q behind the first K tile: both halves, or one of the two buffers in turn, each free once the item that
      // it held has no S left to form
      for (int i = 0; i < groups && !stop; ++i) {
        const int buf = groups == 2 ? i : q_turn;
        if (!warp_wait(&qEmpty[buf], qPhase[buf])) { stop = true; break; }
        qPhase[buf] ^= 1;
        if (lane == 0) {
          mbar_expect_tx(&qFull[buf], (uint32_t)(q_rows * 128 * kHalves));
          for (int c = 0; c < kHalves; ++c)
            tma_load_4d(sQ + buf * S::kTileBytes + c * S::kBox, &mapQ, 64 * c, 0, head, it.tok0 + i * p.TB, &qFull[buf], pol);
        }
      }
      if (groups == 1) q_turn ^= 1;
      if (stop) break;
      if (ahead == 2 && nt > 1) load(1, 0, pgs[1]);
      for (int j = 0; j < nt && !stop; ++j) {
        pgs[2] = j + 2 < nt ? page_at(j + 2) : 0;
        load(j, 1, pgs[0]);
        if (!stop && j + ahead < nt) load(j + ahead, 0, pgs[ahead]);
        pgs[0] = pgs[1];
        pgs[1] = pgs[2];
      }
    }
    let_next_launch();
    // no copy outlives the CTA: the last kSlots ring tiles and the last Q
    for (int i = 0; i < 2; ++i) mbar_wait_drain(&qFull[i], qPhase[i] & 1, p.status);
    for (int i = 1; i <= kSlots && n - i >= 0; ++i)
      mbar_wait_drain(&full[(n - i) % kSlots], ((n - i) / kSlots) & 1, p.status);
  } else if (warp > kASoftmaxWarps) {
    // ---- MMA issue, a warp for each group: the whole warp goes through the waits, one elected lane issues ----
    const uint32_t g = warp - (kASoftmaxWarps + 1);
    const uint32_t idesc_qk = idesc_bf16_f32(128, kAChunk, 0), idesc_pv = idesc_bf16_f32(128, D, 1);
    uint32_t pPhase = 0, oPhase = 1, qPhase = 0, q_turn = 0;  // (pPhase, qPhase: a bit a buffer)
    uint32_t ring = 0, passed = 0;  // ring tiles of the items before; tiles whose arrival this warp has seen
    bool stop = false;
    // descriptor words: start addresses in 16-byte units, the rest constant
    const uint32_t q_lo = smem_u32(sQ) >> 4, kv_lo = smem_u32(sKV) >> 4;
    constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride 1024 B, version 1, 128-byte swizzle
    constexpr uint32_t kTileUnits = S::kTileBytes >> 4, kBoxUnits = S::kBox >> 4;
    // passes the tiles before n, which are not this warp's: waits for each and signs it off
    auto pass = [&](uint32_t n) {
      for (; passed < n && !stop; ++passed) {
        const uint32_t slot = passed % kSlots;
        if (!warp_wait(&full[slot], (passed / kSlots) & 1)) stop = true;
        else if (elect_one()) mbar_arrive(&empty[slot]);
      }
    };
    // waits for ring tile n; its slot
    auto tile = [&](uint32_t n) {
      pass(n);
      const uint32_t slot = n % kSlots;
      if (!stop && !warp_wait(&full[slot], (n / kSlots) & 1)) stop = true;
      ++passed;
      tc_fence_after();
      return slot;
    };
    constexpr uint32_t kChunkUnits = kAChunk * 128 / 16;
    // S of the group, in buffer h, from Q buffer qb and chunk h of the K tile in slot s0; signed off: the tile if `done`,
    // Q if `end`
    auto qk = [&](uint32_t qb, uint32_t s0, uint32_t h, bool done, bool end) {
      const uint32_t q = q_lo + qb * kTileUnits, kk = kv_lo + s0 * kTileUnits + h * kChunkUnits;
      if (elect_one()) {
#pragma unroll 1
        for (uint32_t c = 0; c < kHalves; ++c)  // (four a turn: 75 cycles an issued step fell to those of the products)
#pragma unroll
          for (uint32_t s = 0; s < 4; ++s)
            tc_mma_bf16_lo(128u * g + kAChunk * h, q + c * kBoxUnits + 2 * s, kHi, kk + c * kBoxUnits + 2 * s, kHi, idesc_qk,
                           s > 0 ? 1u : c);
        tc_commit(&sFull[2 * g + h]);
        if (done) tc_commit(&empty[s0]);
        if (end) tc_commit(&qEmpty[qb]);
      }
    };
    // O += P V with chunk h of `keys` keys of the V tile in slot s0, once P is there (at the group's first chunk of an item,
    // once the epilogue before has read O); the tile is signed off if `done`
    auto pv = [&](uint32_t s0, uint32_t h, uint32_t keys, bool first, bool done) {
      const uint32_t steps = (keys + 15) >> 4;
      if (keys & 15) {  // V rows past the keys: their weights are 0, but the rows may hold anything
        unsigned char* v = sKV + s0 * S::kTileBytes + (kAChunk * h + keys) * 128;
        const uint32_t rows = 16 - (keys & 15);
        for (uint32_t i = lane; i < rows * 8 * kHalves; i += 32) {
          const uint32_t c = i / (rows * 8), rest = i - c * rows * 8;
          *reinterpret_cast<uint4*>(v + c * S::kBox + rest * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (!warp_wait(&pFull[2 * g + h], (pPhase >> h) & 1u)) return false;
      pPhase ^= 1u << h;
      if (first) {
        if (!warp_wait(&oEmpty[g], oPhase)) return false;
        oPhase ^= 1;
      }
      tc_fence_after();
      const uint32_t v = (kv_lo + s0 * kTileUnits + h * kChunkUnits) | (kBoxUnits << 16);  // MN-major: the leading offset is a box
      const uint32_t d = 256u + 128u * g, a = 128u * g + kAChunk * h;
      if (elect_one()) {
#pragma unroll
        for (uint32_t s = 0; s < kAChunk / 16; ++s)
          if (s < steps) tc_mma_bf16_ts_lo(d, a + 8u * s, v + 128u * s, kHi, idesc_pv, s > 0 || !first);
        tc_commit(&oDone[2 * g + h]);
        if (done) tc_commit(&empty[s0]);
      }
      return true;
    };
    for (int k = 0; !stop; ++k) {
      const AttnItem it = take(k);
      // (through a warp-wide reduction: the result is in a uniform register)
      const uint32_t n_keys = __reduce_max_sync(0xffffffffu, (uint32_t)it.n_keys);
      const uint32_t halves = __reduce_max_sync(0xffffffffu, it.head & kAlternate ? 0u : 1u);
      if (n_keys == 0) break;
      const uint32_t nt = (n_keys + kATile - 1) / kATile;
      // half g of the rows over every tile (K0 V0 K1 V1 ... in the ring), or tiles g, g + 2, ... of all rows
      // (K0 K1 V0 K2 V1 K3 ...)
      const uint32_t first = halves ? 0u : g, step = halves ? 1u : 2u, qb = halves ? g : q_turn;
      for (uint32_t b = 0; b < 2 && !stop; ++b) {
        if (!halves && b != q_turn) continue;
        if (!warp_wait(&qFull[b], (qPhase >> b) & 1u)) stop = true;
        qPhase ^= 1u << b;
      }
      if (stop) break;
      if (halves) {
        if (elect_one()) mbar_arrive(&qEmpty[g ^ 1]);
      } else {
        q_turn ^= 1;
      }
      auto chunks = [&](uint32_t j) { return n_keys - j * kATile > kAChunk ? 2u : 1u; };
      if (first < nt) {
        // two chunks ahead: S of a chunk is formed while the softmax of the one before runs
        const uint32_t s0 = tile(ring + first), n0 = chunks(first);
        if (stop) break;
        qk(qb, s0, 0, n0 == 1, n0 == 1);
        if (n0 > 1) qk(qb, s0, 1, true, first + step >= nt);
        for (uint32_t j = first; j < nt; j += step) {
          const uint32_t next = j + step, n = chunks(j), n1 = next < nt ? chunks(next) : 0u;
          const uint32_t sv = tile(halves ? ring + 2 * j + 1 : j + 1 < nt ? ring + 2 + 2 * j : ring + 2 * nt - 1);
          const uint32_t sk = n1 ? tile(ring + 2 * j + 1 + step) : 0;  // (seen before P is, not between its MMAs)
          const bool end = next + step >= nt;
          if (stop || !pv(sv, 0, min(n_keys - j * kATile, (uint32_t)kAChunk), j == first, n == 1)) { stop = true; break; }
          if (n1) qk(qb, sk, 0, n1 == 1, end && n1 == 1);
          if (n > 1 && !pv(sv, 1, min(n_keys - j * kATile - kAChunk, (uint32_t)kAChunk), false, true)) { stop = true; break; }
          if (n1 > 1) qk(qb, sk, 1, true, end);
        }
      } else if (elect_one()) {
        mbar_arrive(&qEmpty[qb]);
      }
      ring += 2 * nt;
      pass(ring);
    }
    if (elect_one()) tc_commit(drain);  // every MMA issued so far by either warp has completed
    __syncwarp();
    mbar_wait_drain(drain, 0, p.status);
  } else {
    // ---- softmax and epilogue: group g, one thread a row ----
    const int g = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + 128u * g, tO = tmem + lane_base + 256u + 128u * g;
    const unsigned long long rate2 = f32x2_pack(p.rate, p.rate), one2 = f32x2_pack(1.f, 1.f);
    uint32_t sPhase = 0, pCount = 0;  // of each buffer: S's phase, the parity of its P's (a bit a buffer)
    bool stop = false;
    for (int k = 0; !stop; ++k) {
      const AttnItem it = take(k);
      if (it.n_keys == 0) break;
      const int nt = ceil_div(it.n_keys, kATile);
      const bool halves = !(it.head & kAlternate);  // else the even tiles of all rows, or the odd ones
      if (!halves && g >= nt) continue;
      const int tok = (halves ? g * p.TB : 0) + row / p.G;
      const bool valid = row < p.TB * p.G && tok < it.n_tok;
      const int limit = !valid ? 0 : it.req < 0 ? it.n_keys : min(it.n_keys, it.pos0 + tok);  // keys the row sees
      int clear = valid ? limit : 0x7fffffff;  // keys that every row of the warp sees
      clear = warp_min_i(clear);
      const bool any = clear != 0x7fffffff;
      float m = -INFINITY, z = 0.f;
      bool first = true;
      uint32_t last = 0;  // the last chunk's buffer
      for (int key = halves ? 0 : g * kATile; key < it.n_keys;) {
        const uint32_t h = (key / kAChunk) & 1;
        if (!warp_wait(&sFull[2 * g + h], (sPhase >> h) & 1u)) { stop = true; break; }
        sPhase ^= 1u << h;
        tc_fence_after();
        const uint32_t tC = tS + kAChunk * h;
        if (any) {
          if (key + kAChunk > clear) {  // scores of keys that the row does not see: -inf, in TMEM
            const int left = limit - key;
#pragma unroll 1
            for (int c = 0; c < kAChunk; c += 8) {
              uint32_t u[8];
              tmem_ld8(tC + c, u);
#pragma unroll
              for (int i = 0; i < 8; ++i) u[i] = c + i < left ? u[i] : 0xff800000u;
              tmem_st8(tC + c, u);
            }
            tmem_st_wait();
          }
          uint32_t s[kAChunk], w[kAChunk / 2];
          tmem_ld64_nowait(tC, s);
          tmem_ld_wait64(s);
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = fmaxf(__uint_as_float(s[e]), __uint_as_float(s[4 + e]));
#pragma unroll
          for (int i = 8; i < kAChunk; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = max3(x[e], __uint_as_float(s[i + e]), __uint_as_float(s[i + 4 + e]));
          const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * p.rate;
          const bool rise = top > m + 8.f || (m == -INFINITY && top > m);
          if (__any_sync(0xffffffffu, rise)) {
            const float mn = rise ? top : m;
            const float f = m == -INFINITY ? 0.f : ex2_approx(m - mn);  // mn >= m; 1 where m stays
            m = mn;
            z *= f;
            if (!first) {  // (the chunk before may still be being added; this S says that those before it are)
              if (!warp_wait(&oDone[2 * g + (h ^ 1)], ((pCount >> (h ^ 1)) & 1u) ^ 1u)) { stop = true; break; }
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 8) {
                uint32_t u[8];
                tmem_ld8(tO + c, u);
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * f);
                tmem_st8(tO + c, u);
              }
            }
          }
          const float neg = m == -INFINITY ? 0.f : -m;  // a row that has seen no key yet: 2^(-inf) = 0
          const unsigned long long neg2 = f32x2_pack(neg, neg);
          unsigned long long z2[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 0; c < kAChunk; c += 2) {
            float e0, e1;
            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), rate2, neg2), e0, e1);
            e0 = ex2_approx(e0);
            e1 = ex2_approx(e1);
            z2[(c >> 1) & 1] = f32x2_fma(f32x2_pack(e0, e1), one2, z2[(c >> 1) & 1]);
            w[c >> 1] = pack_bf16x2(e0, e1);
          }
          tmem_st32(tC, w);
          float s0, s1, s2, s3;
          f32x2_unpack(z2[0], s0, s1);
          f32x2_unpack(z2[1], s2, s3);
          z += (s0 + s1) + (s2 + s3);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pFull[2 * g + h]);
        pCount ^= 1u << h;
        last = h;
        first = false;
        key += kAChunk;
        if (!halves && h) key += kATile;  // the other group's tile
      }
      if (stop) break;
      if (!warp_wait(&oDone[2 * g + last], ((pCount >> last) & 1u) ^ 1u)) break;
      tc_fence_after();
      if (any) {
        const int hq = (it.head & ~kAlternate) * p.G + row % p.G;
        const size_t t = it.slot0 < 0 ? (size_t)it.tok0 + tok : (size_t)it.slot0 + tok + (!halves && g ? it.n_tok : 0);
        const size_t at = valid ? t * p.Hq + hq : 0;
        if (it.slot0 < 0) {
          const float inv = z != 0.f ? 1.f / z : 0.f;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            __syncwarp();
            tmem_ld32(tO + c, o);
            if (valid) {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= inv;
#pragma unroll
              for (int i = 0; i < 32; i += 8) *reinterpret_cast<uint4*>(p.out + at * D + c + i) = pack_bf16x8(o + i);
            }
          }
        } else {
          // Four lanes trade 32-byte pieces of their rows, so that each store of theirs covers 128 bytes of one row: a
          // lane that wrote its own row took a cache line a store (8,000 cycles an item of 256 rows)
          const int i4 = lane & 3;
          size_t to[4];
          uint32_t have = 0;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            to[r] = __shfl_sync(0xffffffffu, (unsigned long long)at, (lane & ~3) + r);
            have |= (__shfl_sync(0xffffffffu, valid, (lane & ~3) + r) ? 1u : 0u) << r;
          }
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            __syncwarp();
            tmem_ld32(tO + c, o);
#pragma unroll
            for (int step = 1; step <= 2; step <<= 1) {
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                if (u & step) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) {  // pieces u and u + step of lanes that differ in `step`
                  float& lo = o[8 * u + e];
                  float& hi = o[8 * (u | step) + e];
                  const float got = __shfl_xor_sync(0xffffffffu, i4 & step ? lo : hi, step);
                  if (i4 & step) lo = got;
                  else hi = got;
                }
              }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if ((have >> r) & 1u) store32(p.acc + to[r] * D + c + 8 * i4, o + 8 * r);
          }
        }
        if (valid) {
          if (it.slot0 >= 0) p.stat[at] = make_float2(m, z);
          else if (p.lse) p.lse[at] = z != 0.f ? (m + log2f(z)) * 0.6931471805599453f : -INFINITY;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&oEmpty[g]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kASoftmaxWarps + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// One warp a (token, query head): the parts of the prefix, then those of the pages, in that order.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(AttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  wait_for_launch_before();
  const int np = p.head->prefix_parts;
  if (row >= (long long)p.head->n_tokens * p.Hq) return;
  const int t = (int)(row / p.Hq), hq = (int)(row % p.Hq);
  const int4 map = __ldcg(p.tokens + t);
  if (map.z < 0) return;
  const int n = np + map.z, n_tokens = p.head->n_tokens;
  auto slot = [&](int i) {
    return ((size_t)(i < np ? (long long)i * n_tokens + t : (long long)map.x + (long long)(i - np) * map.y)) * p.Hq + hq;
  };
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) {
    const float2 s = __ldcg(p.stat + slot(i));
    if (s.y != 0.f) M = fmaxf(M, s.y == s.y ? s.x : 0.f);  // (a sum that is NaN: the row's, whatever the maximum)
  }
  M = warp_max(M);
  float o[E] = {}, Z = 0.f;
  if (M > -INFINITY) {
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const size_t at = slot(i);
      const float2 s = __ldcg(p.stat + at);
      float a[E];
      if (E == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p.acc + at * D) + lane);
        a[0] = v.x; a[1] = v.y; a[2 % E] = v.z; a[3 % E] = v.w;
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(p.acc + at * D) + lane);
        a[0] = v.x; a[1] = v.y;
      }
      const float f = s.y == 0.f ? 0.f : ex2_approx(s.x - M);  // (a part without keys has z = 0 and o = 0)
      Z = fmaf(s.y, f, Z);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(a[e], f, o[e]);
    }
  }
  const float inv = Z != 0.f ? 1.f / Z : 0.f;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(p.out + row * D + lane * E + e) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  if (p.lse && lane == 0) p.lse[row] = Z != 0.f ? (M + log2f(Z)) * 0.6931471805599453f : -INFINITY;
}

template <int D>
static cudaError_t launch_attention(const AttnParams& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                    int q_rows, int box_rows, cudaStream_t s) {
  static std::atomic<unsigned long long> attr{0};
  cudaError_t e = set_smem_limit_once((const void*)attn_tiles_kernel<D>, (int)AttnSmem<D>::kTotal, attr);
  if (e != cudaSuccess) return e;
  attn_plan_kernel<<<1, std::min(kAPlanThreads, std::max(128, (p.R + 31) & ~31)), 0, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // the next two may be set up before the one before has ended
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(p.sms);
  cfg.blockDim = dim3(kAThreads);
  cfg.dynamicSmemBytes = AttnSmem<D>::kTotal;
  if ((e = cudaLaunchKernelEx(&cfg, attn_tiles_kernel<D>, mq, mk, mv, p, q_rows, box_rows)) != cudaSuccess) return e;
  cfg.gridDim = dim3(ceil_div((long long)p.T * p.Hq, 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  if ((e = cudaLaunchKernelEx(&cfg, attn_join_kernel<D>, p)) != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace dspark

using namespace dspark;

static bool attn_heads_ok(int n_heads, int n_kv_heads, int head_dim) {
  return n_heads >= 1 && n_kv_heads >= 1 && n_heads % n_kv_heads == 0 && n_heads / n_kv_heads <= 128 &&
         (head_dim == 64 || head_dim == 128);
}

extern "C" size_t dspark_attention_workspace_bytes(int32_t R, int32_t T, int32_t n_heads, int32_t n_kv_heads,
                                                   int32_t head_dim) {
  if (R < 1 || T < 0 || !attn_heads_ok(n_heads, n_kv_heads, head_dim)) return 0;
  return attn_layout(R, T, n_heads, n_kv_heads, head_dim).total;
}

extern "C" dspark_status dspark_prefix_attention(int32_t R, int32_t T, int32_t n_heads, int32_t n_kv_heads,
                                                 int32_t head_dim, int32_t page_size, int32_t n_pages,
                                                 int32_t max_pages, int32_t prefix_len, const void* q,
                                                 const void* k_cache, const void* v_cache, const int32_t* prefix_pages,
                                                 const int32_t* block_table, const int32_t* q_start,
                                                 const int32_t* kv_len, float scale, void* out, float* lse,
                                                 void* workspace, size_t workspace_bytes, dspark_stream_t stream) {
  note_launches(0);
  if (R < 1 || T < 0 || !attn_heads_ok(n_heads, n_kv_heads, head_dim) || page_size < 16 || page_size > 4096 ||
      (page_size & (page_size - 1)) != 0 || n_pages < 1 || max_pages < 1 || prefix_len < 0 || prefix_len > 0x7fffff00 ||
      (long long)T * n_heads > (1ll << 30) || !(scale > 0.f) || !isfinite(scale))
    return DSPARK_ERR_INVALID_ARG;
  if (T > 0 && (!q || !k_cache || !v_cache || (prefix_len > 0 && !prefix_pages) || !block_table || !q_start || !kv_len || !out))
    return DSPARK_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
       reinterpret_cast<uintptr_t>(out)) & 15)
    return DSPARK_ERR_INVALID_ARG;
  const AttnLayout L = attn_layout(R, T, n_heads, n_kv_heads, head_dim);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < L.total)
    return DSPARK_ERR_WORKSPACE;
  if (T == 0) return DSPARK_OK;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSPARK_ERR_CUDA;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (sms <= 0) return DSPARK_ERR_CUDA;
  AttnParams p{};
  p.R = R; p.T = T; p.Hq = n_heads; p.Hkv = n_kv_heads;
  p.G = n_heads / n_kv_heads;
  p.TB = attn_tokens_per_half(p.G);
  p.page = page_size;
  while ((1 << p.page_log2) < page_size) ++p.page_log2;
  p.n_pages = n_pages; p.max_pages = max_pages; p.prefix_len = prefix_len;
  p.sms = std::min(sms, kMaxSms);
  p.cap_slots = L.slots;
  p.prefix_pages = prefix_pages; p.table = block_table; p.q_start = q_start; p.kv_len = kv_len;
  p.rate = scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.status = static_cast<uint32_t*>(workspace);
  p.head = ws_at<AttnHead>(workspace, L.head);
  p.tokens = ws_at<int4>(workspace, L.tokens);
  p.items = ws_at<AttnItem>(workspace, L.items);
  p.stat = ws_at<float2>(workspace, L.stat);
  p.acc = ws_at<float>(workspace, L.acc);
  const uint64_t D = head_dim, e = 2;
  CUtensorMap mq, mk, mv;
  const int box_tokens = std::min(p.TB, T), box_rows = std::min(page_size, kATile);
  {
    const uint64_t dims[4] = {D, (uint64_t)p.G, (uint64_t)n_kv_heads, (uint64_t)T};
    const uint64_t strides[3] = {D * e, D * e * p.G, D * e * n_heads};
    const uint32_t box[4] = {64, (uint32_t)p.G, 1, (uint32_t)box_tokens};
    if (!make_tmap_bf16(&mq, q, 4, dims, strides, box)) return DSPARK_ERR_CUDA;
  }
  const uint64_t dims[4] = {D, (uint64_t)n_kv_heads, (uint64_t)page_size, (uint64_t)n_pages};
  const uint64_t strides[3] = {D * e, D * e * n_kv_heads, D * e * n_kv_heads * page_size};
  const uint32_t box[4] = {64, 1, (uint32_t)box_rows, 1};
  if (!make_tmap_bf16(&mk, k_cache, 4, dims, strides, box) || !make_tmap_bf16(&mv, v_cache, 4, dims, strides, box))
    return DSPARK_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  const int q_rows = box_tokens * p.G;
  const cudaError_t err = head_dim == 128 ? launch_attention<128>(p, mq, mk, mv, q_rows, box_rows, s)
                                          : launch_attention<64>(p, mq, mk, mv, q_rows, box_rows, s);
  note_launches(3);
  return err == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
