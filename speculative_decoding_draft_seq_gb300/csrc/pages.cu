// Upkeep of the paged cache's pages: which are held and which are free, rows that
// continue other rows and share their pages, live pages moved to the front, and the copies that
// follow from both.
//
// The block table is the only record of who holds a page: counts and lists are formed from
// it anew, so that nothing can drift from it. Each call is a few phases over the table's entries and over the
// pages, every phase done by all CTAs before the next begins: in one cluster of CTAs, which meet at the
// hardware's barrier, or, where there is more to read than one cluster reads in the time that saves, in a cooperative launch
// over the GPU, whose CTAs meet at a counter. Both run the same code with another number of CTAs. Integers
// only, and every list in ascending order: results do not depend on which.
//
// Bound by the chain of phases: collecting the holders of 128 rows of up to 64 pages takes 7 us in one cluster (1.9 of them the
// launch and its barriers) and 8.4 over the GPU; 256 rows of 128 pages 9.6 either way, 1,024 19 and 9.6, 8,192 (5.8 MB)
// 104 and 17. (A launch for each phase: 15 for the last, but 20 with the host's four launches.) page_copy_kernel is bound by
// bytes: 1,180 pages of 32 KB, four times (keys and values of two layers, 308 MB read and written), in 54 us (5.7 TB/s); 4
// units a thread in flight instead of 8: 64.
#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"

namespace dspark {

constexpr int kPgThreads = 1024;
constexpr int kPgWarps = kPgThreads / 32;
constexpr int kPgCluster = 8;
constexpr int kPgGrid = 128;      // a power of two, at most the SMs
constexpr int kPgMeetWord = 40;   // of the status block: the CTAs' meetings so far

// Workspace: status block, counts a CTA, and two words a page.
constexpr size_t kPgCounts = 256;
constexpr int kPgListEnd = kPgGrid;  // word behind the counts: where a fork's list of free pages ends
constexpr size_t kPgMarks = 256 + 4 * 256;
static size_t page_workspace(int n_pages) { return align256(kPgMarks + (size_t)n_pages * 8); }

struct PageParams {
  int R, page, max_pages, n_pages, n_pinned, from;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* pinned;
  // collect
  int32_t* refs;
  int32_t* free_pages;
  int32_t* n_free;
  // fork: R new rows from `from` rows; compact
  const int32_t* parent;
  const int32_t* length;
  int free_count;
  const int32_t* free_list;
  int32_t* new_table;
  int32_t* new_len;
  int32_t* src;
  int32_t* dst;
  int32_t* tokens;
  int32_t* used;
  int32_t* new_pinned;
  int32_t* n_live;
  // workspace
  uint32_t* status;
  int32_t* counts;
  int32_t* mark0;
  int32_t* mark1;
};

// One CTA's view of a phase: CTA `rank` of n.
struct Team {
  int rank, n;
  __device__ __forceinline__ long long first() const { return (long long)rank * kPgThreads + threadIdx.x; }
  __device__ __forceinline__ long long step() const { return (long long)n * kPgThreads; }
  // the contiguous share of `total` things that this CTA looks after
  __device__ __forceinline__ void share(int total, int& lo, int& hi) const {
    const int each = ceil_div(total, n);
    lo = (int)min((long long)rank * each, (long long)total);
    hi = (int)min((long long)lo + each, (long long)total);
  }
};

__device__ __forceinline__ int block_sum_int(int v, int* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Number of set flags in the block's threads before this one; `total` of all.
__device__ __forceinline__ int block_rank(bool flag, int* sh, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t b = __ballot_sync(0xffffffffu, flag);
  __syncthreads();
  if (lane == 0) sh[warp] = __popc(b);
  __syncthreads();
  const int w = sh[lane];
  int c = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) c += y;
  }
  total = __shfl_sync(0xffffffffu, c, 31);
  return __shfl_sync(0xffffffffu, c - w, warp) + __popc(b & ((1u << lane) - 1u));
}

// Pages of a row's tokens; a length outside the row's columns is clamped.
__device__ __forceinline__ int row_pages(const PageParams& p, int len, bool& bad) {
  const long long most = (long long)p.max_pages * p.page;
  bad |= len < 0 || len > most;
  const uint32_t l = (uint32_t)min((long long)max(len, 0), most);
  return (int)(l / (uint32_t)p.page + (l % (uint32_t)p.page != 0 ? 1 : 0));
}

// f(row, first column, last + 1) for every stretch of at most 256 columns of the R rows, a warp each.
template <class F>
__device__ __forceinline__ void for_stretches(const PageParams& p, const Team& t, F f) {
  const int per_row = ceil_div(p.max_pages, 256);
  const long long units = (long long)p.R * per_row, warps = (long long)t.n * kPgWarps;
  for (long long u = (long long)(threadIdx.x >> 5) * t.n + t.rank; u < units; u += warps) {
    const long long r = u / per_row;
    const int c = (int)(u - r * per_row) * 256;
    f((int)r, c, min(c + 256, p.max_pages));
  }
}
// f(page id) for every entry within its row's length.
template <class Need, class F>
__device__ __forceinline__ void for_entries(const PageParams& p, const Team& t, Need need, F f) {
  for_stretches(p, t, [&](int r, int lo, int hi) {
    const int n = min(hi, need(r));
    for (int c = lo + ((int)threadIdx.x & 31); c < n; c += 32) f(__ldg(p.table + (size_t)r * p.max_pages + c));
  });
}

// ---- collect: 0 clear, 1 count, 2 free pages a share, 3 the list
__device__ __forceinline__ void collect_phase(const PageParams& p, const Team& t, int phase, int* sh) {
  if (phase == 0) {
    for (long long i = t.first(); i < p.n_pages; i += t.step()) p.refs[i] = 0;
    return;
  }
  if (phase == 1) {
    bool bad = false;
    for_entries(p, t, [&](int r) { return row_pages(p, __ldg(p.kv_len + r), bad); }, [&](int x) {
      if (x >= 0 && x < p.n_pages) atomicAdd(p.refs + x, 1);
      else bad = true;
    });
    for (long long i = t.first(); i < p.n_pinned; i += t.step()) {
      const int x = __ldg(p.pinned + i);
      if (x >= 0 && x < p.n_pages) atomicAdd(p.refs + x, 1);
      else bad = true;
    }
    if (bad) set_status(p.status, DSPARK_ERR_RANGE);
    return;
  }
  int lo, hi;
  t.share(p.n_pages, lo, hi);
  if (phase == 2) {
    int n = 0;
    for (int i = lo + (int)threadIdx.x; i < hi; i += kPgThreads) n += __ldcg(p.refs + i) == 0;
    n = block_sum_int(n, sh);
    if (threadIdx.x == 0) p.counts[t.rank] = n;
    return;
  }
  int before = 0, all = 0;
  for (int i = threadIdx.x; i < t.n; i += kPgThreads) {
    const int n = __ldcg(p.counts + i);
    all += n;
    if (i < t.rank) before += n;
  }
  before = block_sum_int(before, sh);
  all = block_sum_int(all, sh);
  for (int i0 = lo; i0 < hi; i0 += kPgThreads) {
    const int i = i0 + (int)threadIdx.x;
    const bool is_free = i < hi && __ldcg(p.refs + i) == 0;
    int n;
    const int k = block_rank(is_free, sh, n);
    if (is_free) p.free_pages[before + k] = i;
    before += n;
  }
  for (int i = max(lo, all) + (int)threadIdx.x; i < hi; i += kPgThreads) p.free_pages[i] = -1;
  if (t.rank == 0 && threadIdx.x == 0) p.n_free[0] = all;
}

// ---- fork: 0 clear, 1 mark, 2 copies a share of the rows, 3 lists and rows
// mark0: the page is held in full by a new row, or pinned; mark1: the first new row that ends inside it. The list of free pages
// ends at its first negative id: phase 1 looks for it among the R entries that could be asked for.
struct Fork {
  int parent, whole, rest;  // full pages, tokens of the last one
};
__device__ __forceinline__ Fork fork_of(const PageParams& p, int i, bool& bad) {
  Fork f{__ldg(p.parent + i), 0, 0};
  if (f.parent < 0 || f.parent >= p.from) {
    bad |= f.parent < -1 || f.parent >= p.from;
    f.parent = -1;
    return f;
  }
  const int have = __ldg(p.kv_len + f.parent);
  const long long most = min((long long)have, (long long)p.max_pages * p.page);
  bad |= have != most;
  const int want = p.length ? __ldg(p.length + i) : (int)max(most, 0ll);
  bad |= want < 0 || want > most || most < 0;
  const uint32_t l = (uint32_t)max(0ll, min((long long)want, most));
  f.whole = (int)(l / (uint32_t)p.page);
  f.rest = (int)(l % (uint32_t)p.page);
  return f;
}
// whether new row i must write its last tokens elsewhere than in the page it ends in
__device__ __forceinline__ bool fork_copies(const PageParams& p, const Fork& f, int i) {
  if (f.rest == 0) return false;
  const int x = __ldg(p.table + (size_t)f.parent * p.max_pages + f.whole);
  return x >= 0 && x < p.n_pages && (__ldcg(p.mark0 + x) != 0 || __ldcg(p.mark1 + x) < i);
}
__device__ __forceinline__ void fork_phase(const PageParams& p, const Team& t, int phase, int* sh) {
  if (phase == 0) {
    for (long long i = t.first(); i < p.n_pages; i += t.step()) {
      p.mark0[i] = 0;
      p.mark1[i] = INT_MAX;
    }
    if (t.first() == 0) p.counts[kPgListEnd] = INT_MAX;
    return;
  }
  bool bad = false;
  const int lane = threadIdx.x & 31;
  if (phase == 1) {
    const int listed = min(p.R, p.free_count);
    for_stretches(p, t, [&](int i, int lo, int hi) {
      const Fork f = fork_of(p, i, bad);
      for (int c = lo + lane; c < hi; c += 32) {
        int x = -1;
        if (c < f.whole || (c == f.whole && f.rest)) {
          x = __ldg(p.table + (size_t)f.parent * p.max_pages + c);
          if (x < 0 || x >= p.n_pages) bad = true;
          else if (c < f.whole) p.mark0[x] = 1;
          else atomicMin(p.mark1 + x, i);
        }
        p.new_table[(size_t)i * p.max_pages + c] = x;
      }
      if (lo == 0 && lane == 0) p.new_len[i] = f.whole * p.page + f.rest;
    });
    for (long long i = t.first(); i < p.n_pinned; i += t.step()) {
      const int x = __ldg(p.pinned + i);
      if (x >= 0 && x < p.n_pages) p.mark0[x] = 1;
      else bad = true;
    }
    for (long long i = t.first(); i < listed; i += t.step()) {
      // (the first of a run of negative ids is enough)
      if (__ldg(p.free_list + i) < 0 && (i == 0 || __ldg(p.free_list + i - 1) >= 0)) atomicMin(p.counts + kPgListEnd, (int)i);
    }
    if (bad) set_status(p.status, DSPARK_ERR_RANGE);
    return;
  }
  int lo, hi;
  t.share(p.R, lo, hi);
  if (phase == 2) {
    int n = 0;
    for (int i = lo + (int)threadIdx.x; i < hi; i += kPgThreads) n += fork_copies(p, fork_of(p, i, bad), i);
    n = block_sum_int(n, sh);
    if (threadIdx.x == 0) p.counts[t.rank] = n;
    return;
  }
  const int list_end = min(p.free_count, __ldcg(p.counts + kPgListEnd));
  int before = 0, all = 0;
  for (int i = threadIdx.x; i < t.n; i += kPgThreads) {
    const int n = __ldcg(p.counts + i);
    all += n;
    if (i < t.rank) before += n;
  }
  before = block_sum_int(before, sh);
  all = block_sum_int(all, sh);
  for (int i0 = lo; i0 < hi; i0 += kPgThreads) {
    const int i = i0 + (int)threadIdx.x;
    Fork f{};
    bool copies = false;
    if (i < hi) {
      f = fork_of(p, i, bad);
      copies = fork_copies(p, f, i);
    }
    int n;
    const int k = before + block_rank(copies, sh, n);
    before += n;
    if (i >= hi) continue;
    int from = -1, to = -1;
    if (copies) {
      if (k < list_end) to = __ldg(p.free_list + k);
      if (to < 0 || to >= p.n_pages) {
        set_status(p.status, to < p.n_pages ? DSPARK_ERR_CAPACITY : DSPARK_ERR_RANGE);
        to = -1;
      } else {
        from = __ldg(p.table + (size_t)f.parent * p.max_pages + f.whole);
      }
      p.new_table[(size_t)i * p.max_pages + f.whole] = to;
    }
    p.src[i] = from;
    p.dst[i] = to;
    p.tokens[i] = to >= 0 ? f.rest : 0;
  }
  if (t.rank == 0 && threadIdx.x == 0) p.used[0] = min(all, list_end);
}

// ---- compact: 0 clear, 1 mark, 2 live pages a share, 3 names and lists, 4 rows
// mark0: the page is held; mark1: of a held page past the front, the number of its move.
__device__ __forceinline__ int renamed(const PageParams& p, int x, int m) {
  return x >= m ? __ldcg(p.dst + __ldcg(p.mark1 + x)) : x;
}
__device__ __forceinline__ void compact_phase(const PageParams& p, const Team& t, int phase, int* sh) {
  if (phase == 0) {
    for (long long i = t.first(); i < p.n_pages; i += t.step()) p.mark0[i] = 0;
    for (long long i = t.first(); i < p.n_pages / 2; i += t.step()) p.src[i] = p.dst[i] = -1;
    return;
  }
  bool bad = false;
  const auto need = [&](int r) { return row_pages(p, __ldg(p.kv_len + r), bad); };
  if (phase == 1) {
    for_entries(p, t, need, [&](int x) {
      if (x >= 0 && x < p.n_pages) p.mark0[x] = 1;
      else bad = true;
    });
    for (long long i = t.first(); i < p.n_pinned; i += t.step()) {
      const int x = __ldg(p.pinned + i);
      if (x >= 0 && x < p.n_pages) p.mark0[x] = 1;
      else bad = true;
    }
    if (bad) set_status(p.status, DSPARK_ERR_RANGE);
    return;
  }
  int lo, hi;
  t.share(p.n_pages, lo, hi);
  if (phase == 2) {
    int n = 0;
    for (int i = lo + (int)threadIdx.x; i < hi; i += kPgThreads) n += __ldcg(p.mark0 + i);
    n = block_sum_int(n, sh);
    if (threadIdx.x == 0) p.counts[t.rank] = n;
    return;
  }
  // live pages before this share, in all, and before page m = their number
  int before = 0, m = 0;
  for (int i = threadIdx.x; i < t.n; i += kPgThreads) {
    const int n = __ldcg(p.counts + i);
    m += n;
    if (i < t.rank) before += n;
  }
  before = block_sum_int(before, sh);
  m = block_sum_int(m, sh);
  if (phase == 3) {
    const int each = ceil_div(p.n_pages, t.n);
    int front = 0;
    for (int i = threadIdx.x; i < m / each; i += kPgThreads) front += __ldcg(p.counts + i);
    for (int i = m / each * each + (int)threadIdx.x; i < m; i += kPgThreads) front += __ldcg(p.mark0 + i);
    front = block_sum_int(front, sh);
    for (int i0 = lo; i0 < hi; i0 += kPgThreads) {
      const int i = i0 + (int)threadIdx.x;
      const bool live = i < hi && __ldcg(p.mark0 + i) != 0;
      int n;
      const int k = before + block_rank(live, sh, n);  // live pages before page i
      before += n;
      if (i >= hi) continue;
      if (live && i >= m) {
        p.mark1[i] = k - front;
        p.src[k - front] = i;
      } else if (!live && i < m) {
        p.dst[i - k] = i;
      }
    }
    if (t.rank == 0 && threadIdx.x == 0) p.n_live[0] = m;
    return;
  }
  for_stretches(p, t, [&](int r, int c0, int c1) {
    const int n = need(r);
    for (int c = c0 + ((int)threadIdx.x & 31); c < c1; c += 32) {
      int x = -1;
      if (c < n) {
        x = __ldg(p.table + (size_t)r * p.max_pages + c);
        if (x >= 0 && x < p.n_pages) x = renamed(p, x, m);
      }
      p.new_table[(size_t)r * p.max_pages + c] = x;
    }
  });
  for (long long i = t.first(); i < p.n_pinned; i += t.step()) {
    const int x = __ldg(p.pinned + i);
    p.new_pinned[i] = x >= 0 && x < p.n_pages ? renamed(p, x, m) : x;
  }
}

enum { kCollect, kFork, kCompact };
constexpr int phases_of(int op) { return op == kCompact ? 5 : 4; }
template <int kOp>
__device__ __forceinline__ void run_phase(const PageParams& p, const Team& t, int phase, int* sh) {
  if constexpr (kOp == kCollect) collect_phase(p, t, phase, sh);
  else if constexpr (kOp == kFork) fork_phase(p, t, phase, sh);
  else compact_phase(p, t, phase, sh);
}
// All phases in one cluster.
template <int kOp>
__global__ void __launch_bounds__(kPgThreads) pages_cluster_kernel(PageParams p) {
  __shared__ int sh[32];
  const Team t{(int)cluster_rank(), kPgCluster};
#pragma unroll
  for (int phase = 0; phase < phases_of(kOp); ++phase) {
    if (phase > 0) {
      cluster_arrive();
      cluster_wait();
    }
    run_phase<kOp>(p, t, phase, sh);
    __syncwarp();
  }
}
// All phases over the GPU: the CTAs of a cooperative launch (all resident) meet between two. The word counts on from call
// to call: its number of CTAs divides 2^32, so a meeting is over when it reaches the next multiple. Bounded: a wait that runs
// out records DSPARK_ERR_TIMEOUT, and its CTA returns (the workspace has to be cleared then).
constexpr uint32_t kMeetLimit = 1u << 20;  // about 1 s of polls
__device__ __forceinline__ bool meet(uint32_t* word, uint32_t* status, int* ok) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const uint32_t goal = (atomicAdd(word, 1u) / kPgGrid + 1u) * kPgGrid;
    int there = 0;
    for (uint32_t i = 0; i < kMeetLimit && !there; ++i) {
      uint32_t v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(word) : "memory");
      there = (int32_t)(v - goal) >= 0;
      if (!there && i > 64) __nanosleep(32);
    }
    if (!there) set_status(status, DSPARK_ERR_TIMEOUT);
    *ok = there;
  }
  __syncthreads();
  return *ok != 0;
}
template <int kOp>
__global__ void __launch_bounds__(kPgThreads) pages_grid_kernel(PageParams p) {
  __shared__ int sh[32];
  __shared__ int ok;
  const Team t{(int)blockIdx.x, kPgGrid};
#pragma unroll
  for (int phase = 0; phase < phases_of(kOp); ++phase) {
    if (phase > 0 && !meet(p.status + kPgMeetWord, p.status, &ok)) return;
    run_phase<kOp>(p, t, phase, sh);
  }
}

template <int kOp>
static dspark_status launch_pages(const PageParams& p, cudaStream_t s) {
  const long long reads = (long long)p.R * p.max_pages + p.n_pages;
  cudaError_t e;
  if (reads <= 65536) {
    e = launch_clusters(pages_cluster_kernel<kOp>, p, kPgCluster, kPgCluster, kPgThreads, 0, s);
    note_launches(1);
  } else {
    PageParams q = p;
    void* args[] = {&q};
    e = cudaLaunchCooperativeKernel((const void*)pages_grid_kernel<kOp>, dim3(kPgGrid), dim3(kPgThreads), args, 0, s);
    note_launches(1);
  }
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

// ---------------------------------------------------------------------------
struct CopyParams {
  int n, layers, n_pages, page, per_token, chunks, chunk;  // per_token: units of a token's row; chunk: units of a piece of a page
  const int32_t* src;
  const int32_t* dst;
  const int32_t* tokens;
  void* k;
  void* v;
  uint32_t* status;
};
constexpr int kCopyAhead = 8;  // units of a page that a thread has in flight
// A CTA takes a piece of one page of one layer's keys or values at a time, and has the page numbers of the next one
// ready when it is done.
template <class Tv>
__global__ void __launch_bounds__(256) page_copy_kernel(CopyParams p) {
  const long long page_units = (long long)p.page * p.per_token;
  const int per_entry = 2 * p.layers * p.chunks;
  const long long items = (long long)p.n * per_entry;
  struct Item {
    int from, to, tokens, side, piece;
  };
  const auto item = [&](long long it) {
    Item x{-1, -1, p.page, 0, 0};
    if (it < items) {
      const int i = (int)(it / per_entry), rest = (int)(it - (long long)i * per_entry);
      x.side = rest / p.chunks;
      x.piece = rest - x.side * p.chunks;
      x.from = __ldg(p.src + i);
      x.to = __ldg(p.dst + i);
      if (p.tokens) x.tokens = __ldg(p.tokens + i);
    }
    return x;
  };
  Item next = item(blockIdx.x);
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const Item x = next;
    next = item(it + gridDim.x);
    if (x.from < 0 || x.to < 0) continue;
    if (x.from >= p.n_pages || x.to >= p.n_pages) {
      if (threadIdx.x == 0) set_status(p.status, DSPARK_ERR_RANGE);
      continue;
    }
    const long long lo = (long long)x.piece * p.chunk;
    const long long hi = min(lo + p.chunk, (long long)min(max(x.tokens, 0), p.page) * p.per_token);
    Tv* cache = static_cast<Tv*>(x.side & 1 ? p.v : p.k) + (long long)(x.side >> 1) * p.n_pages * page_units;
    const Tv* a = cache + x.from * page_units;
    Tv* b = cache + x.to * page_units;
    for (long long u = lo + threadIdx.x; u < hi; u += 256 * kCopyAhead) {
      Tv q[kCopyAhead];
#pragma unroll
      for (int i = 0; i < kCopyAhead; ++i)
        if (u + 256 * i < hi) q[i] = a[u + 256 * i];
#pragma unroll
      for (int i = 0; i < kCopyAhead; ++i)
        if (u + 256 * i < hi) b[u + 256 * i] = q[i];
    }
  }
}

static bool page_args(int R, int page, int max_pages, int n_pages, int n_pinned, const void* pinned) {
  return R >= 1 && page >= 1 && max_pages >= 1 && n_pages >= 1 && n_pinned >= 0 && (n_pinned == 0 || pinned);
}
static bool page_workspace_ok(const void* ws, size_t bytes, int n_pages) {
  return ws && (reinterpret_cast<uintptr_t>(ws) & 255) == 0 && bytes >= page_workspace(n_pages);
}
static void use_workspace(PageParams& p, void* ws) {
  p.status = static_cast<uint32_t*>(ws);
  p.counts = ws_at<int32_t>(ws, kPgCounts);
  p.mark0 = ws_at<int32_t>(ws, kPgMarks);
  p.mark1 = p.mark0 + p.n_pages;
}

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_page_workspace_bytes(int32_t n_pages) { return n_pages < 1 ? 0 : page_workspace(n_pages); }

extern "C" dspark_status dspark_page_collect(int32_t R, int32_t page_size, int32_t max_pages, int32_t n_pages,
                                             int32_t n_pinned, const int32_t* block_table, const int32_t* kv_len,
                                             const int32_t* pinned, int32_t* refs, int32_t* free_pages, int32_t* n_free,
                                             void* workspace, size_t workspace_bytes, dspark_stream_t stream) {
  note_launches(0);
  if (!page_args(R, page_size, max_pages, n_pages, n_pinned, pinned) || !block_table || !kv_len || !refs || !free_pages ||
      !n_free)
    return DSPARK_ERR_INVALID_ARG;
  if (!page_workspace_ok(workspace, workspace_bytes, n_pages)) return DSPARK_ERR_WORKSPACE;
  const long long entries = (long long)R * max_pages;
  if (!separate({span(block_table, entries), span(kv_len, R), span(pinned, n_pinned)},
                {span(refs, n_pages), span(free_pages, n_pages), span(n_free, 1)}))
    return DSPARK_ERR_INVALID_ARG;
  PageParams p{};
  p.R = R; p.page = page_size; p.max_pages = max_pages; p.n_pages = n_pages; p.n_pinned = n_pinned;
  p.table = block_table; p.kv_len = kv_len; p.pinned = pinned;
  p.refs = refs; p.free_pages = free_pages; p.n_free = n_free;
  use_workspace(p, workspace);
  return launch_pages<kCollect>(p, (cudaStream_t)stream);
}

extern "C" dspark_status dspark_page_fork(int32_t R_from, int32_t R, int32_t page_size, int32_t max_pages, int32_t n_pages,
                                          int32_t n_free, int32_t n_pinned, const int32_t* block_table,
                                          const int32_t* kv_len, const int32_t* parent, const int32_t* fork_len,
                                          const int32_t* free_pages, const int32_t* pinned, int32_t* new_table,
                                          int32_t* new_len, int32_t* src, int32_t* dst, int32_t* tokens, int32_t* used,
                                          void* workspace, size_t workspace_bytes, dspark_stream_t stream) {
  note_launches(0);
  if (!page_args(R, page_size, max_pages, n_pages, n_pinned, pinned) || R_from < 1 || n_free < 0 ||
      (n_free > 0 && !free_pages) || !block_table || !kv_len || !parent || !new_table || !new_len || !src || !dst ||
      !tokens || !used || (long long)max_pages * page_size > 0x7fffffffll || new_table == block_table)
    return DSPARK_ERR_INVALID_ARG;
  if (!page_workspace_ok(workspace, workspace_bytes, n_pages)) return DSPARK_ERR_WORKSPACE;
  if (!separate({span(block_table, (long long)R_from * max_pages), span(kv_len, R_from), span(parent, R), span(fork_len, R),
                 span(free_pages, n_free), span(pinned, n_pinned)},
                {span(new_table, (long long)R * max_pages), span(new_len, R), span(src, R), span(dst, R), span(tokens, R), span(used, 1)}))
    return DSPARK_ERR_INVALID_ARG;
  PageParams p{};
  p.R = R; p.from = R_from; p.page = page_size; p.max_pages = max_pages; p.n_pages = n_pages; p.n_pinned = n_pinned;
  p.table = block_table; p.kv_len = kv_len; p.pinned = pinned; p.parent = parent; p.length = fork_len;
  p.free_count = n_free; p.free_list = free_pages;
  p.new_table = new_table; p.new_len = new_len; p.src = src; p.dst = dst; p.tokens = tokens; p.used = used;
  use_workspace(p, workspace);
  return launch_pages<kFork>(p, (cudaStream_t)stream);
}

extern "C" dspark_status dspark_page_compact(int32_t R, int32_t page_size, int32_t max_pages, int32_t n_pages,
                                             int32_t n_pinned, const int32_t* block_table, const int32_t* kv_len,
                                             const int32_t* pinned, int32_t* new_table, int32_t* new_pinned,
                                             int32_t* src, int32_t* dst, int32_t* n_live, void* workspace,
                                             size_t workspace_bytes, dspark_stream_t stream) {
  note_launches(0);
  if (!page_args(R, page_size, max_pages, n_pages, n_pinned, pinned) || !block_table || !kv_len || !new_table ||
      (n_pinned > 0 && !new_pinned) || (n_pages > 1 && (!src || !dst)) || !n_live)
    return DSPARK_ERR_INVALID_ARG;
  if (!page_workspace_ok(workspace, workspace_bytes, n_pages)) return DSPARK_ERR_WORKSPACE;
  const long long entries = (long long)R * max_pages;
  const Span table = span(block_table, new_table == block_table ? 0 : entries), pins = span(pinned, new_pinned == pinned ? 0 : n_pinned);
  if (!separate({table, span(kv_len, R), pins},  // (those may be written in place)
                {span(new_table, entries), span(new_pinned, n_pinned), span(src, n_pages / 2), span(dst, n_pages / 2), span(n_live, 1)}))
    return DSPARK_ERR_INVALID_ARG;
  PageParams p{};
  p.R = R; p.page = page_size; p.max_pages = max_pages; p.n_pages = n_pages; p.n_pinned = n_pinned;
  p.table = block_table; p.kv_len = kv_len; p.pinned = pinned;
  p.new_table = new_table; p.new_pinned = new_pinned; p.src = src; p.dst = dst; p.n_live = n_live;
  use_workspace(p, workspace);
  return launch_pages<kCompact>(p, (cudaStream_t)stream);
}

extern "C" dspark_status dspark_page_copy(int32_t n, int32_t n_layers, int32_t n_pages, int32_t page_size,
                                          int32_t n_kv_heads, int32_t head_dim, int32_t dtype, const int32_t* src,
                                          const int32_t* dst, const int32_t* tokens, void* k_cache, void* v_cache,
                                          void* workspace, size_t workspace_bytes, dspark_stream_t stream) {
  note_launches(0);
  if (n < 0 || n_layers < 1 || n_pages < 1 || page_size < 1 || n_kv_heads < 1 || head_dim < 1 ||
      (long long)n_kv_heads * head_dim > (1 << 24) || (dtype != DSPARK_FP32 && dtype != DSPARK_BF16) ||
      (long long)page_size * n_kv_heads * head_dim > (1ll << 30) || n_layers > (1 << 20))
    return DSPARK_ERR_INVALID_ARG;
  if (n > 0 && (!src || !dst || !k_cache || !v_cache)) return DSPARK_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < 256)
    return DSPARK_ERR_WORKSPACE;
  if (n == 0) return DSPARK_OK;
  const int elem = dtype == DSPARK_BF16 ? 2 : 4;
  const long long row = (long long)n_kv_heads * head_dim * elem;
  const uintptr_t at = reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache);
  const int unit = ((at | (uintptr_t)row) & 15) == 0 ? 16 : elem;  // bytes a thread copies at a time
  CopyParams p{n, n_layers, n_pages, page_size, (int)(row / unit), 0, 256 * kCopyAhead, src, dst, tokens, k_cache, v_cache,
               static_cast<uint32_t*>(workspace)};
  p.chunks = ceil_div((long long)page_size * p.per_token, p.chunk);
  if (2ll * n_layers * p.chunks > 0x7fffffff) return DSPARK_ERR_INVALID_ARG;
  const long long items = (long long)n * n_layers * 2 * p.chunks;
  const int grid = (int)std::min<long long>(items, 152 * 16);
  cudaStream_t s = (cudaStream_t)stream;
  if (unit == 16) page_copy_kernel<uint4><<<grid, 256, 0, s>>>(p);
  else if (unit == 4) page_copy_kernel<uint32_t><<<grid, 256, 0, s>>>(p);
  else page_copy_kernel<uint16_t><<<grid, 256, 0, s>>>(p);
  note_launches(1);
  return cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
