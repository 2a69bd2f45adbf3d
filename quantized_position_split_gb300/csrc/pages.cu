// The page tables of a paged cache on the device: pages for the next positions of its sequences
// (and those behind a window or a trimmed end given back), sequences that continue others, and the
// live pages of a pool moved to its front; pages copied where that needs it.
//
// All three are integer work on a few hundred KB, in steps of which each needs all of the one
// before: reference counts changed, free pages counted, the lowest ones given out.  One cluster of
// CTAs takes them with a cluster barrier between (a grid per step would cost a launch each); its
// size is chosen by how much there is to scan (pages_ctas).  Every CTA keeps the sequences' state
// in shared memory and scans it for itself, so that a step waits for what it needs of the others
// alone: with state in global memory, scanned by one CTA, five to seven barriers with loads behind
// each took 23 us for a decode step of 64 sequences over 65536 pages.  A free page's rank is found
// by a scan in order and leads the CTA that finds it to the entry that it is for, so results do not
// depend on the order of threads.  What a step reads of another CTA's is read past L1 (__ldcg).
//
// The copies that follow are a second launch, over a list of (from, to, rows) in the workspace:
// every plane of every cache in chunks of kChunk bytes, one a CTA at a time.  They are bound by
// HBM.
//
// Measured (captured): that decode step 12 us, seven beams 12 us, 60 forks of up to 257 pages each 18 us
// (copies 9), 4096 pages of which half are moved (1.07 GB) 338 us, 6.4 TB/s.
#include <algorithm>
#include <exception>
#include <string>
#include <vector>

#include "paged.h"

namespace qps {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kClusterMost = 8;
constexpr int kMostSeqs = 4096;  // their state lies in shared memory

struct SeqsP {
  int32_t* table;
  int64_t stride;
  int width, batch;
  int32_t* lens;
  int32_t* refs;
  int n_pages, page_shift;
  unsigned int* err;
};

// Workspace of a call.
struct PagesWs {
  int* counts;   // [kClusterMost] pages found by each CTA
  int* copies;   // [1] jobs
  int* list;     // (compact) free pages before the live count, in order
  int* list2;    // (compact) pages in use from it on, in order
  int* rows;     // (fork) [items][width] source rows as they were
  int4* jobs;    // (from, to, rows, whether `from` has a use less then)
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// f(item, part, parts) for every item, by whole warps; an item's work is cut into `parts`.
template <class F>
__device__ __forceinline__ void for_items(int n, F f) {
  const int gw = blockIdx.x * kWarps + (threadIdx.x >> 5), all = gridDim.x * kWarps;
  if (n <= 0) return;
  if (n >= all) {
    for (int i = gw; i < n; i += all) f(i, 0, 1);
  } else {
    const int parts = all / n, i = gw % n, part = gw / n;
    if (part < parts) f(i, part, parts);
  }
}

// Inclusive sum over the block; the total in *all.  `tmp`: kWarps values of shared memory.
template <class T>
__device__ __forceinline__ T block_scan(T v, T* tmp, T* all) {
  static_assert(kWarps == 32, "a lane for each warp");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) tmp[warp] = v;
  __syncthreads();
  const T mine = tmp[lane];
  T w = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *all = __shfl_sync(0xffffffffu, w, 31);
  const T before = __shfl_sync(0xffffffffu, w - mine, warp);
  __syncthreads();
  return v + before;
}

// This CTA's share [x, y) of the pages: whole groups of 4.
__device__ __forceinline__ int2 page_share(int n_pages) {
  const int64_t each = ((n_pages + 4 * (int64_t)gridDim.x - 1) / (4 * gridDim.x)) * 4, p0 = each * blockIdx.x;
  return make_int2((int)min((int64_t)n_pages, p0), (int)min((int64_t)n_pages, p0 + each));
}
// Reference counts of the pages p .. p + 3 (behind `end`: -1).
__device__ __forceinline__ int4 refs4(const SeqsP& s, int p, int end) {
  if (p + 3 < end && (reinterpret_cast<uintptr_t>(s.refs) & 15) == 0) return __ldcg(reinterpret_cast<const int4*>(s.refs + p));
  return make_int4(p < end ? __ldcg(s.refs + p) : -1, p + 1 < end ? __ldcg(s.refs + p + 1) : -1,
                   p + 2 < end ? __ldcg(s.refs + p + 2) : -1, p + 3 < end ? __ldcg(s.refs + p + 3) : -1);
}

// Pages of [p0, p1) for which f(page, refs): how many.  Every thread has the count.
template <class F>
__device__ __forceinline__ int count_pages(const SeqsP& s, int p0, int p1, int* tmp, F f) {
  int n = 0;
#pragma unroll 4
  for (int p = p0 + 4 * (int)threadIdx.x; p < p1; p += 4 * kThreads) {
    const int4 r = refs4(s, p, p1);
    n += f(p, r.x) + (p + 1 < p1 && f(p + 1, r.y)) + (p + 2 < p1 && f(p + 2, r.z)) + (p + 3 < p1 && f(p + 3, r.w));
  }
  int all;
  block_scan(n, tmp, &all);
  return all;
}
// The same pages in order as take(rank, page), rank from `rank` on and below `most`, by whole warps:
// take is called by all lanes, with page -1 where a lane has none.
template <class F, class T>
__device__ __forceinline__ void take_pages(const SeqsP& s, int p0, int p1, int rank, int most, int* tmp, F f, T take) {
  for (int at = p0; at < p1 && rank < most; at += 4 * kThreads) {
    const int p = at + 4 * (int)threadIdx.x;
    const int4 r = refs4(s, p, p1);
    const bool is[4] = {p < p1 && f(p, r.x), p + 1 < p1 && f(p + 1, r.y), p + 2 < p1 && f(p + 2, r.z), p + 3 < p1 && f(p + 3, r.w)};
    const int n = is[0] + is[1] + is[2] + is[3];
    int all;
    int to = rank + block_scan(n, tmp, &all) - n;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool mine = is[k] && to < most;
      if (__any_sync(0xffffffffu, mine)) take(to, mine ? p + k : -1);
      to += is[k];
    }
    rank += all;
  }
}

__device__ __forceinline__ bool page_ok(const SeqsP& s, int pg) { return (uint32_t)pg < (uint32_t)s.n_pages; }
__device__ __forceinline__ int seq_len(const SeqsP& s, int b) {
  const int n = __ldcg(s.lens + b), cut = min(max(n, 0), s.width << s.page_shift);
  if (cut != n) atomicOr(s.err, kErrIndex);
  return cut;
}
__device__ __forceinline__ int pages_of(const SeqsP& s, int64_t n) { return (int)((n + (1 << s.page_shift) - 1) >> s.page_shift); }
// One use of a page less.  A page that nothing used stays at zero, and the status says so.
__device__ __forceinline__ void drop_ref(const SeqsP& s, int pg) {
  if (!page_ok(s, pg)) return;
  if (atomicSub(s.refs + pg, 1) <= 0) {
    atomicAdd(s.refs + pg, 1);
    atomicOr(s.err, kErrIndex);
  }
}
// Free pages: counted by every CTA (each its share) before a barrier, the counts of the first pages
// of the share kept in registers; behind it, the first of them given out in order, `most` in all.
constexpr int kKept = 2;
struct Share {
  int2 at;
  int4 kept[kKept];
};
__device__ __forceinline__ Share count_free(const SeqsP& s, const PagesWs& w, int* tmp) {
  Share sh;
  sh.at = page_share(s.n_pages);
  auto free4 = [](int4 r) { return (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0); };
  int n = 0;
#pragma unroll
  for (int k = 0; k < kKept; ++k) {
    sh.kept[k] = refs4(s, sh.at.x + 4 * ((int)threadIdx.x + k * kThreads), sh.at.y);
    n += free4(sh.kept[k]);
  }
#pragma unroll 4
  for (int p = sh.at.x + 4 * ((int)threadIdx.x + kKept * kThreads); p < sh.at.y; p += 4 * kThreads) n += free4(refs4(s, p, sh.at.y));
  int all;
  block_scan(n, tmp, &all);
  if (threadIdx.x == 0) w.counts[blockIdx.x] = all;
  return sh;
}
struct Found {
  int before, all;  // by the CTAs before this one, by all
};
__device__ __forceinline__ Found found(const int* counts) {
  int n = 0;
  const int lane = threadIdx.x & 31;
  if (lane < (int)gridDim.x) n = __ldcg(counts + lane);
  return {__reduce_add_sync(0xffffffffu, lane < (int)blockIdx.x ? n : 0), __reduce_add_sync(0xffffffffu, n)};
}
// list[0 .. n) are pages in order, the first of rank `rank`: take(rank, list, n) is called by the whole
// block, between barriers, for at most 4 kThreads pages at a time.
template <class T>
__device__ __forceinline__ void give_free(const SeqsP& s, const Share& sh, Found n, int most, int* tmp, int* list, T take) {
  int rank = n.before;
  most = min(most, n.all);
  int k = 0;
  for (int at = sh.at.x; at < sh.at.y && rank < most; at += 4 * kThreads, ++k) {
    const int p = at + 4 * (int)threadIdx.x;
    const int4 r = k == 0 ? sh.kept[0] : k == 1 ? sh.kept[1] : refs4(s, p, sh.at.y);
    const int is[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
    const int mine = is[0] + is[1] + is[2] + is[3];
    int all;
    int to = block_scan(mine, tmp, &all) - mine;
    const int got = min(all, most - rank);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (is[i] && to < got) list[to] = p + i;
      to += is[i];
    }
    __syncthreads();
    if (got > 0) take(rank, list, got);
    __syncthreads();
    rank += all;
  }
}

// f(j, entry) for the entries [j0, j1) of a row, by the warps part, part + parts, ..: four neighbours
// a lane (16 bytes, where they lie so), kGroups such under way.
template <class F>
__device__ __forceinline__ void for_entries(const SeqsP& s, const int32_t* row, int j0, int j1, int part, int parts, F f) {
  constexpr int kGroups = 4;
  if (j0 >= j1) return;
  const int lane = threadIdx.x & 31, off = (int)(reinterpret_cast<uintptr_t>(row) >> 2 & 3);
  // group g: entries 4 g - off .. 4 g - off + 3
  const int g0 = (j0 + off) >> 2, g1 = (j1 + off + 3) >> 2;
  for (int g = g0 + part * 32 + lane; __any_sync(0xffffffffu, g < g1); g += parts * 32 * kGroups) {
    int4 v[kGroups];
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      const int j = 4 * (g + u * parts * 32) - off;
      v[u] = make_int4(-1, -1, -1, -1);
      if (j >= j0 && j + 3 < j1) {
        v[u] = __ldcg(reinterpret_cast<const int4*>(row + j));
      } else if (j + 3 >= j0 && j < j1) {
        if (j >= j0) v[u].x = __ldcg(row + j);
        if (j + 1 >= j0 && j + 1 < j1) v[u].y = __ldcg(row + j + 1);
        if (j + 2 >= j0 && j + 2 < j1) v[u].z = __ldcg(row + j + 2);
        if (j + 3 >= j0 && j + 3 < j1) v[u].w = __ldcg(row + j + 3);
      }
    }
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      const int j = 4 * (g + u * parts * 32) - off;
      if (page_ok(s, v[u].x)) f(j, v[u].x);
      if (page_ok(s, v[u].y)) f(j + 1, v[u].y);
      if (page_ok(s, v[u].z)) f(j + 2, v[u].z);
      if (page_ok(s, v[u].w)) f(j + 3, v[u].w);
    }
  }
}

// ---- extend -----------------------------------------------------------------------------------
struct ExtendP {
  SeqsP s;
  PagesWs w;
  const int32_t* n_new;
  int window, sinks;
  int64_t max_tokens;
  int32_t* starts;
  int64_t* slots;
  int64_t* positions;
};

// A sequence's state in shared memory.
struct ExtendSeq {
  int len;     // before the call
  int grow;    // n_new
  int start;   // first row of its new tokens
  int base;    // rank of its first page
  int part;    // (growing) the page that its first new position lies in, if it holds one; else -1
  int rank;    // place of its copy, -1: none; -2: it does not fit its row or the rows of slots
};

__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const __grid_constant__ ExtendP p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int tmp[kWarps];
  __shared__ int64_t tmp64[kWarps];
  int4* const rows = reinterpret_cast<int4*>(smem);                 // [4 kThreads]
  int* const list = reinterpret_cast<int*>(rows + 4 * kThreads);    // [4 kThreads]
  ExtendSeq* const seq = reinterpret_cast<ExtendSeq*>(list + 4 * kThreads);
  const SeqsP& s = p.s;
  const int lane = threadIdx.x & 31, page = 1 << s.page_shift;
  const int64_t held = (int64_t)s.width << s.page_shift;
  asm volatile("griddepcontrol.launch_dependents;" :::);  // (the copies: they wait for this grid's end)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- every sequence, and where its tokens' rows start ----------------------------------------
  int64_t tokens = 0;
  for (int b0 = 0; b0 < s.batch; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    ExtendSeq q = {0, 0, 0, 0, -1, -1};
    if (b < s.batch) {
      q.grow = p.n_new[b];
      q.len = seq_len(s, b);
      if (q.grow > 0 && (q.len & (page - 1))) {  // (no step of this call gives it back)
        const int pg = __ldcg(s.table + b * s.stride + (q.len >> s.page_shift));
        if (page_ok(s, pg)) q.part = pg;
      }
    }
    const int64_t more = max(0, q.grow);
    int64_t all;
    const int64_t upto = tokens + block_scan(more, tmp64, &all);
    tokens += all;
    q.start = (int)min(upto - more, p.max_tokens);
    if (more > 0 && (q.len + more > held || upto > p.max_tokens)) q.rank = -2;
    if (b < s.batch) {
      seq[b] = q;
      if (blockIdx.x == 0) p.starts[b] = q.start;
    }
  }
  const int total = (int)min(tokens, p.max_tokens);
  if (blockIdx.x == 0 && threadIdx.x == 0) p.starts[s.batch] = total;
  __syncthreads();
  auto end_of = [&](const ExtendSeq& q) { return max((int64_t)0, (int64_t)q.len + q.grow); };
  // ---- pages behind a trimmed end, and those that no later token's window reaches; the tokens'
  // positions -----------------------------------------------------------------------------------
  for_items(s.batch, [&](int b, int part, int parts) {
    const ExtendSeq q = seq[b];
    int32_t* row = s.table + b * s.stride;
    auto give = [&](int j, int pg) {
      drop_ref(s, pg);
      row[j] = -1;
    };
    const int had = pages_of(s, q.len), keep = min(had, pages_of(s, min((int64_t)q.len, end_of(q))));
    for_entries(s, row, keep, had, part, parts, give);
    if (p.window) {
      const int64_t low = (q.grow > 0 ? (int64_t)q.len : end_of(q)) - p.window + 1;
      if (low > 0) for_entries(s, row, pages_of(s, p.sinks), min(keep, (int)(low >> s.page_shift)), part, parts, give);
    }
    const int n = (b + 1 < s.batch ? seq[b + 1].start : total) - q.start;
    for (int i = part * 32 + lane; i < n; i += parts * 32) p.positions[q.start + i] = (int64_t)q.len + i;
  });
  for (int64_t i = total + blockIdx.x * kThreads + threadIdx.x; i < p.max_tokens; i += (int64_t)gridDim.x * kThreads) {
    p.slots[i] = -1;
    p.positions[i] = 0;
  }
  cluster_sync();
  // ---- free pages; what each sequence needs, in order ------------------------------------------
  const Share share = count_free(s, p.w, tmp);
  int need = 0, copies = 0;
  for (int b0 = 0; b0 < s.batch; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int n = 0, copy = 0;
    if (b < s.batch && seq[b].grow > 0 && seq[b].rank != -2) {
      // (a last page that others name too is copied before it is written)
      copy = seq[b].part >= 0 && __ldcg(s.refs + seq[b].part) > 1;
      n = pages_of(s, end_of(seq[b])) - pages_of(s, seq[b].len) + copy;
    }
    int64_t all;  // (pages below, copies above)
    const int64_t upto = block_scan((int64_t)copy << 32 | n, tmp64, &all);
    if (b < s.batch) {
      seq[b].base = need + (int)(uint32_t)upto - n;
      if (copy) seq[b].rank = copies + (int)(upto >> 32) - 1;
    }
    need += (int)(uint32_t)all;
    copies += (int)(all >> 32);
  }
  cluster_sync();
  // ---- a free page finds its entry by its rank ---------------------------------------------------
  const Found free = found(p.w.counts);
  auto next_base = [&](int b) { return b + 1 < s.batch ? seq[b + 1].base : need; };
  // of a sequence that grows: whether it gets its pages
  auto served = [&](int b) { return seq[b].rank != -2 && (next_base(b) <= free.all || next_base(b) == seq[b].base); };
  give_free(s, share, free, need, tmp, list, [&](int rank0, const int* pages, int n) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int rank = rank0 + i, pg = pages[i];
      int lo = 0, hi = s.batch;  // the last sequence with base <= rank
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq[mid].base <= rank) lo = mid;
        else hi = mid;
      }
      int4 r = make_int4(0, 0, 0, 0);  // the first row of slots on the page, how many, the first slot
      if (served(lo)) {
        const ExtendSeq& q = seq[lo];
        const int j = pages_of(s, q.len) + rank - q.base - (q.rank >= 0);  // (the copy first, in the place before)
        if (q.rank >= 0 && rank == q.base) p.w.jobs[q.rank] = make_int4(q.part, pg, q.len & (page - 1), 1);
        s.table[lo * s.stride + j] = pg;
        s.refs[pg] = 1;
        const int64_t t0 = max((int64_t)j << s.page_shift, (int64_t)q.len), t1 = min((int64_t)(j + 1) << s.page_shift, end_of(q));
        r = make_int4(q.start + (int)(t0 - q.len), (int)(t1 - t0), pg * page + (int)(t0 & (page - 1)), 0);
      }
      rows[i] = r;
    }
    __syncthreads();
    for (int i = threadIdx.x >> 5; i < n; i += kWarps) {
      const int4 r = rows[i];
      for (int t = lane; t < r.y; t += 32) p.slots[r.x + t] = r.z + t;
    }
  });
  for_items(s.batch, [&](int b, int part, int) {
    const ExtendSeq& q = seq[b];
    if (part != 0) return;
    const bool ok = q.grow <= 0 || served(b);
    if (lane == 0) {
      if (!ok) atomicOr(s.err, kErrIndex);
      else s.lens[b] = (int32_t)end_of(q);
      if (q.rank >= 0 && !ok) p.w.jobs[q.rank] = make_int4(0, 0, 0, 0);
    }
    if (q.grow <= 0) return;
    const int n = (b + 1 < s.batch ? seq[b + 1].start : total) - q.start;
    if (!ok) {  // (its rows as far as there are any)
      for (int i = lane; i < n; i += 32) p.slots[q.start + i] = -1;
    } else if ((q.len & (page - 1)) && q.rank < 0) {  // rows on the page that it has
      const int m = min(n, page - (q.len & (page - 1)));
      for (int i = lane; i < m; i += 32)
        p.slots[q.start + i] = q.part < 0 ? -1 : (int64_t)q.part * page + (q.len & (page - 1)) + i;
    }
  });
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.w.copies = copies;
}

// ---- fork -------------------------------------------------------------------------------------
struct ForkP {
  SeqsP s;
  PagesWs w;
  const int32_t* src;
  const int32_t* dst;
  int n;
};

// One of the n in shared memory.
struct ForkItem {
  int src, dst;  // dst -1: nothing to do
  int len;       // of the source
  int part;      // its last page, if that is not full; else -1
  int rank;      // place of its copy, -1: none
};

__global__ void __launch_bounds__(kThreads, 1) fork_kernel(const __grid_constant__ ForkP p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int tmp[kWarps];
  ForkItem* const item = reinterpret_cast<ForkItem*>(smem);
  int* const of_rank = reinterpret_cast<int*>(item + p.n);  // [n] the item of a copy
  int* const owner = of_rank + p.n;                          // [batch]
  int* const list = owner + p.s.batch;                       // [4 kThreads]
  const SeqsP& s = p.s;
  const int lane = threadIdx.x & 31, page = 1 << s.page_shift;
  asm volatile("griddepcontrol.launch_dependents;" :::);  // (the copies: they wait for this grid's end)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- the items; a row that is named twice goes to the first ------------------------------------
  for (int b = threadIdx.x; b < s.batch; b += kThreads) owner[b] = 0x7fffffff;
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += kThreads) {
    const int a = p.src[i], b = p.dst[i];
    const bool valid = a < s.batch && (uint32_t)b < (uint32_t)s.batch;
    item[i] = ForkItem{a, valid ? b : -1, 0, -1, -1};
    if (valid) atomicMin(owner + b, i);
    else atomicOr(s.err, kErrIndex);
  }
  __syncthreads();
  int copies = 0;
  for (int i0 = 0; i0 < p.n; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    ForkItem q = {-1, -1, 0, -1, -1};
    if (i < p.n) {
      q = item[i];
      if (q.dst >= 0 && owner[q.dst] != i) {
        atomicOr(s.err, kErrIndex);
        q.dst = -1;
      }
      if (q.src == q.dst) q.dst = -1;
      if (q.dst >= 0 && q.src >= 0) {
        q.len = seq_len(s, q.src);
        if (q.len & (page - 1)) {
          const int pg = __ldcg(s.table + q.src * s.stride + (q.len >> s.page_shift));
          if (page_ok(s, pg)) q.part = pg;
        }
      }
    }
    int all;
    const int upto = copies + block_scan(q.part >= 0 ? 1 : 0, tmp, &all);
    copies += all;
    if (q.part >= 0) {
      q.rank = upto - 1;
      of_rank[q.rank] = i;
    }
    if (i < p.n) item[i] = q;
  }
  __syncthreads();
  // ---- the sources' rows as they are, each of their pages held once more; what the destinations
  // held is given back (no count falls to zero that is used again) ---------------------------------
  for_items(p.n, [&](int i, int part, int parts) {
    const ForkItem q = item[i];
    if (q.dst < 0) return;
    int* to = p.w.rows + (int64_t)i * s.width;
    const int n = pages_of(s, q.len);
    const int32_t* row = s.table + max(q.src, 0) * s.stride;
#pragma unroll 4
    for (int j = part * 32 + lane; j < n; j += parts * 32) {
      const int pg = __ldcg(row + j);
      const bool ok = page_ok(s, pg);
      to[j] = ok ? pg : -1;
      if (ok) atomicAdd(s.refs + pg, 1);
    }
    for_entries(s, s.table + q.dst * s.stride, 0, pages_of(s, seq_len(s, q.dst)), part, parts, [&](int, int pg) { drop_ref(s, pg); });
  });
  cluster_sync();
  // ---- free pages; the rows, but for the pages that are copied -----------------------------------
  const Share share = count_free(s, p.w, tmp);
  for_items(p.n, [&](int i, int part, int parts) {
    const ForkItem q = item[i];
    if (q.dst < 0) return;
    const int n = pages_of(s, q.len), last = q.part >= 0 ? n - 1 : -1;
    const int* from = p.w.rows + (int64_t)i * s.width;
    int32_t* row = s.table + q.dst * s.stride;
#pragma unroll 4
    for (int j = part * 32 + lane; j < s.width; j += parts * 32)
      if (j != last) row[j] = j < n ? __ldcg(from + j) : -1;
  });
  cluster_sync();
  // ---- a page for each last one that is not full -------------------------------------------------
  const Found free = found(p.w.counts);
  give_free(s, share, free, copies, tmp, list, [&](int rank0, const int* pages, int n) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const ForkItem q = item[of_rank[rank0 + i]];
      s.table[q.dst * s.stride + (q.len >> s.page_shift)] = pages[i];
      s.refs[pages[i]] = 1;
      p.w.jobs[rank0 + i] = make_int4(q.part, pages[i], q.len & (page - 1), 1);
    }
  });
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < p.n; i += gridDim.x * kThreads) {
    const ForkItem q = item[i];
    if (q.dst < 0) continue;
    const bool short_of = q.rank >= free.all;  // (no page for the last positions: they are left out)
    s.lens[q.dst] = short_of ? q.len & ~(page - 1) : q.len;
    if (short_of) {
      atomicOr(s.err, kErrIndex);
      s.table[q.dst * s.stride + (q.len >> s.page_shift)] = -1;
      p.w.jobs[q.rank] = make_int4(q.part, 0, 0, 1);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.w.copies = copies;
}

// ---- compact ----------------------------------------------------------------------------------
struct CompactP {
  SeqsP s;
  PagesWs w;
  int32_t* new_ids;
  int32_t* live;
};

__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const __grid_constant__ CompactP p) {
  __shared__ int tmp[kWarps];
  const SeqsP& s = p.s;
  asm volatile("griddepcontrol.launch_dependents;" :::);  // (the copies: they wait for this grid's end)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 sh = page_share(s.n_pages);
  const int n = count_pages(s, sh.x, sh.y, tmp, [](int, int r) { return r > 0; });
  if (threadIdx.x == 0) p.w.counts[blockIdx.x] = n;
  cluster_sync();
  const Found in_use = found(p.w.counts);
  const int live = in_use.all;
  // holes before `live`, pages in use from it on: as many of the one as of the other.  The pages in
  // use before `live` are those of the shares that lie before it, and of the part of the share that
  // it lies in, which every CTA counts for itself.
  auto hole = [&](int pg, int r) { return pg < live && r <= 0; };
  auto far = [&](int pg, int r) { return pg >= live && r > 0; };
  const int each = max(4, (int)(((s.n_pages + 4 * (int64_t)gridDim.x - 1) / (4 * gridDim.x)) * 4)), mid = min(live / each, (int)gridDim.x - 1);
  int near = count_pages(s, min(s.n_pages, mid * each), live, tmp, [](int, int r) { return r > 0; });
  for (int c = 0; c < mid; ++c) near += __ldcg(p.w.counts + c);
  const int moves = live - near;
  // ranks of this share's first hole and first far page
  const int h0 = sh.x < live ? sh.x - in_use.before : moves, f0 = sh.x < live ? 0 : in_use.before - near;
  if (sh.x < live)
    take_pages(s, sh.x, min(sh.y, live), h0, moves, tmp, hole, [&](int rank, int pg) {
      if (pg >= 0) p.w.list[rank] = pg;
    });
  if (sh.y > live)
    take_pages(s, sh.x, sh.y, f0, moves, tmp, far, [&](int rank, int pg) {
      if (pg >= 0) p.w.list2[rank] = pg;
    });
  for (int pg = sh.x + threadIdx.x; pg < sh.y; pg += kThreads)
    if (const int r = __ldcg(s.refs + pg); !far(pg, r)) p.new_ids[pg] = r > 0 ? pg : -1;
  cluster_sync();
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < moves; i += gridDim.x * kThreads) {
    const int from = __ldcg(p.w.list2 + i), to = __ldcg(p.w.list + i);
    p.new_ids[from] = to;
    s.refs[to] = __ldcg(s.refs + from);
    s.refs[from] = 0;
    p.w.jobs[i] = make_int4(from, to, 1 << s.page_shift, 0);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *p.w.copies = moves;
    p.live[0] = live;
  }
  cluster_sync();
  for_items(s.batch, [&](int b, int part, int parts) {
    int32_t* row = s.table + b * s.stride;
    for_entries(s, row, 0, pages_of(s, seq_len(s, b)), part, parts, [&](int j, int pg) { row[j] = __ldcg(p.new_ids + pg); });
  });
}

// ---- copies -----------------------------------------------------------------------------------
constexpr int kChunk = 16 * 1024, kCopyThreads = 256, kMostPlanes = 96;

struct Plane {
  uint8_t* data;
  uint32_t head_bytes;  // of a page and head: page_size rows (a power of two)
  uint32_t bytes;       // of a page
};
struct CopyP {
  Plane planes[kMostPlanes];
  int first[kMostPlanes + 1];  // chunks of a page before the plane's
  int n, drops;
  const int4* jobs;
  const int* count;
  int most;                    // jobs there can be
  SeqsP s;
};

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyP p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int jobs = min(*p.count, p.most), chunks = p.first[p.n];
  // (of the uses that the tables' kernel has left to drop: while it gave pages out, what is copied
  // must not count as free, and here it need not wait for all of its CTAs once more)
  if (p.drops)
    for (int i = blockIdx.x * kCopyThreads + threadIdx.x; i < jobs; i += gridDim.x * kCopyThreads)
      if (p.jobs[i].w) drop_ref(p.s, p.jobs[i].x);
  for (int64_t u = blockIdx.x; u < (int64_t)jobs * chunks; u += gridDim.x) {
    const int4 job = p.jobs[u / chunks];
    const int ch = (int)(u % chunks);
    int lo = 0, hi = p.n;  // the plane: first[lo] <= ch < first[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.first[mid] <= ch) lo = mid;
      else hi = mid;
    }
    const Plane pl = p.planes[lo];
    const uint32_t at = (uint32_t)(ch - p.first[lo]) * kChunk, end = min(pl.bytes, at + kChunk);
    const uint32_t used = (uint32_t)(((uint64_t)pl.head_bytes * job.z) >> p.s.page_shift);  // bytes of a head that are copied
    if (used == 0 || !in_bounds(page_ok(p.s, job.x) && page_ok(p.s, job.y), p.s.err)) continue;
    const uint8_t* src = pl.data + (int64_t)job.x * pl.bytes;
    uint8_t* dst = pl.data + (int64_t)job.y * pl.bytes;
    constexpr int U = kChunk / (16 * kCopyThreads);
    uint4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const uint32_t x = at + (k * kCopyThreads + threadIdx.x) * 16, y = x & (pl.head_bytes - 1);
      if (x < end && y + 16 <= used) v[k] = __ldcs(reinterpret_cast<const uint4*>(src + x));
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const uint32_t x = at + (k * kCopyThreads + threadIdx.x) * 16, y = x & (pl.head_bytes - 1);
      if (x >= end || y >= used) continue;
      if (y + 16 <= used) {
        __stcs(reinterpret_cast<uint4*>(dst + x), v[k]);
      } else {  // (a row is 2 bytes at least)
        for (uint32_t i = 0; y + i < used; i += 2) *reinterpret_cast<uint16_t*>(dst + x + i) = *reinterpret_cast<const uint16_t*>(src + x + i);
      }
    }
  }
}

// ---- host -------------------------------------------------------------------------------------
qps_status bad(const char* call, const char* what, qps_status st = QPS_ERR_INVALID_ARG) {
  return fail(st, std::string(call) + ": " + what);
}

struct Seqs {
  SeqsP p;
  std::vector<Plane> planes;
};

qps_status check_seqs(const qps_paged_seqs& a, const char* call, Seqs* out) {
  if (a.reserved0 != 0) return bad(call, "reserved fields must be 0");
  if (!a.caches || a.n_caches < 1 || a.n_caches > 65535) return bad(call, "caches is NULL, or n_caches not in [1, 65535]");
  if (a.batch < 1 || a.batch > kMostSeqs) return bad(call, "batch must be in [1, 4096]");
  if (!a.page_table || !a.kv_lens || !a.refs || !aligned_to(a.page_table, 4) || !aligned_to(a.kv_lens, 4) || !aligned_to(a.refs, 4))
    return bad(call, "page_table / kv_lens / refs are NULL or misaligned");
  SeqsP& p = out->p;
  p = SeqsP{};
  for (int i = 0; i < a.n_caches; ++i) {
    PagedKv kv;
    const qps_status st = check_paged_kv(a.caches[i], call, &kv);
    if (st != QPS_OK) return st;
    if (i > 0 && (kv.n_pages != p.n_pages || kv.page_shift != p.page_shift))
      return bad(call, "the caches must have one page size and one number of pages");
    p.n_pages = (int)kv.n_pages;
    p.page_shift = kv.page_shift;
    for (int side = 0; side < 2; ++side)
      for (int k = 0; k < plane_count(side ? kv.vfmt : kv.kfmt); ++k) {
        const int64_t head = plane_row_bytes(side ? kv.vfmt : kv.kfmt, k, kv.d) << kv.page_shift, all = head * kv.hkv;
        if (all >= (int64_t)1 << 31) return bad(call, "a page of a plane must be below 2^31 bytes", QPS_ERR_UNSUPPORTED);
        out->planes.push_back(Plane{side ? kv.v[k] : kv.k[k], (uint32_t)head, (uint32_t)all});
      }
  }
  if (a.table_width < 1 || ((int64_t)a.table_width << p.page_shift) >= ((int64_t)1 << 31) - 1024)
    return bad(call, "need table_width >= 1 and table_width * page_size < 2^31 - 1024");
  if (a.batch > 1 && a.table_stride < a.table_width) return bad(call, "table_stride must be >= table_width");
  p.table = a.page_table;
  p.stride = a.batch > 1 ? a.table_stride : a.table_width;
  p.width = a.table_width;
  p.batch = a.batch;
  p.lens = a.kv_lens;
  p.refs = a.refs;
  return QPS_OK;
}

struct Range {
  const void* at;
  int64_t bytes;
};
bool apart(const std::vector<Range>& written, const std::vector<Range>& read) {
  auto meet = [](const Range& a, const Range& b) {
    const char *pa = (const char*)a.at, *pb = (const char*)b.at;
    return a.bytes > 0 && b.bytes > 0 && pa < pb + b.bytes && pb < pa + a.bytes;
  };
  for (size_t i = 0; i < written.size(); ++i) {
    for (size_t j = 0; j < i; ++j)
      if (meet(written[i], written[j])) return false;
    for (const Range& r : read)
      if (meet(written[i], r)) return false;
  }
  return true;
}
std::vector<Range> tables(const SeqsP& s) {
  return {{s.table, ((s.batch - 1) * s.stride + s.width) * 4}, {s.lens, (int64_t)s.batch * 4}, {s.refs, (int64_t)s.n_pages * 4}};
}

// The workspace, cut up; `bytes` after it.
struct Cut {
  char* at;
  size_t bytes = 0;
  template <class T>
  T* take(size_t n) {
    T* r = reinterpret_cast<T*>(at + bytes);
    bytes += (n * sizeof(T) + 255) & ~(size_t)255;
    return r;
  }
};
size_t lay_out(PagesWs* w, void* base, int64_t list, int64_t rows, int64_t jobs) {
  Cut c{reinterpret_cast<char*>(base)};
  w->counts = c.take<int>(kClusterMost);
  w->copies = c.take<int>(1);
  w->list = c.take<int>(list);
  w->list2 = c.take<int>(list);
  w->rows = c.take<int>(rows);
  w->jobs = c.take<int4>(jobs);
  return c.bytes;
}

int pages_ctas(const SeqsP& s) { return s.n_pages > 4096 || s.batch > kWarps ? kClusterMost : 1; }

// `smem`: bytes of the state.
template <class P>
qps_status launch_pages(void (*kernel)(P), const P& p, size_t smem, cudaStream_t s) {
  if (smem > 32 * 1024) QPS_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  cudaLaunchConfig_t cfg = {};
  const int ctas = pages_ctas(p.s);
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  QPS_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, p));
  count_launch();
  QPS_CUDA_TRY(cudaGetLastError());
  return QPS_OK;
}

qps_status launch_copies(const Seqs& q, const PagesWs& w, int64_t most, cudaStream_t s) {
  const int sms = sm_count_current();
  for (size_t at = 0; at < q.planes.size(); at += kMostPlanes) {
    CopyP p;
    p.n = (int)std::min<size_t>(kMostPlanes, q.planes.size() - at);
    int64_t chunks = 0;
    for (int i = 0; i < p.n; ++i) {
      p.planes[i] = q.planes[at + i];
      p.first[i] = (int)chunks;
      chunks += (p.planes[i].bytes + kChunk - 1) / kChunk;
    }
    p.first[p.n] = (int)chunks;  // (96 planes of 2^31 bytes: below 2^24)
    p.drops = at == 0;
    p.jobs = w.jobs;
    p.count = w.copies;
    p.most = (int)most;
    p.s = q.p;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(most * chunks, (int64_t)sms * 8)));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    QPS_CUDA_TRY(cudaLaunchKernelEx(&cfg, copy_pages_kernel, p));
    count_launch();
    QPS_CUDA_TRY(cudaGetLastError());
  }
  return QPS_OK;
}

qps_status check_workspace(const char* call, void* ws, size_t have, size_t need) {
  if (!ws || have < need) return bad(call, "workspace missing or smaller than its plan reports");
  if (!aligned_to(ws, 256)) return bad(call, "workspace must be 256-byte aligned");
  return QPS_OK;
}

const char* const kExtend = "kv_extend_paged";
qps_status plan_extend(const qps_paged_extend_args* a, Seqs* q, PagesWs* w, size_t* bytes, int64_t* jobs) {
  if (!a) return bad(kExtend, "args is NULL");
  const qps_status st = check_seqs(a->seqs, kExtend, q);
  if (st != QPS_OK) return st;
  if (!a->n_new || !aligned_to(a->n_new, 4)) return bad(kExtend, "n_new is NULL or misaligned");
  if (a->window < 0 || a->sinks < 0) return bad(kExtend, "window and sinks must be >= 0");
  if (a->max_tokens < 0 || a->max_tokens >= (int64_t)1 << 31) return bad(kExtend, "max_tokens must be in [0, 2^31)");
  *jobs = std::min<int64_t>(a->seqs.batch, a->max_tokens);
  *bytes = lay_out(w, a->workspace, 0, 0, *jobs);
  return QPS_OK;
}

qps_status kv_extend_paged(const qps_paged_extend_args* a, cudaStream_t s) {
  Seqs q;
  ExtendP p{};
  size_t bytes;
  int64_t jobs;
  qps_status st = plan_extend(a, &q, &p.w, &bytes, &jobs);
  if (st != QPS_OK) return st;
  if (!a->q_starts || !aligned_to(a->q_starts, 4)) return bad(kExtend, "q_starts is NULL or misaligned");
  if (a->max_tokens > 0 && (!a->slots || !aligned_to(a->slots, 8) || !a->positions || !aligned_to(a->positions, 8)))
    return bad(kExtend, "slots / positions are NULL or misaligned");
  st = check_workspace(kExtend, a->workspace, a->workspace_bytes, bytes);
  if (st != QPS_OK) return st;
  std::vector<Range> written = tables(q.p);
  written.insert(written.end(), {{a->q_starts, (a->seqs.batch + 1) * (int64_t)4}, {a->slots, a->max_tokens * 8},
                                 {a->positions, a->max_tokens * 8}, {a->workspace, (int64_t)bytes}});
  if (!apart(written, {{a->n_new, a->seqs.batch * (int64_t)4}})) return bad(kExtend, "what is written overlaps itself or n_new");
  q.p.err = device_error_word();
  if (!q.p.err) return bad(kExtend, "cannot allocate the device error word", QPS_ERR_CUDA);
  p.s = q.p;
  p.n_new = a->n_new;
  // (as in the attention: a window that no sequence outgrows is none)
  const int64_t held = (int64_t)p.s.width << p.s.page_shift;
  p.window = a->window > 0 && a->window < held && a->sinks < held ? a->window : 0;
  p.sinks = p.window ? a->sinks : 0;
  p.max_tokens = a->max_tokens;
  p.starts = a->q_starts;
  p.slots = a->slots;
  p.positions = a->positions;
  st = launch_pages(extend_kernel, p, p.s.batch * sizeof(ExtendSeq) + 4 * kThreads * (sizeof(int) + sizeof(int4)), s);
  return st != QPS_OK || jobs == 0 ? st : launch_copies(q, p.w, jobs, s);
}

const char* const kFork = "kv_fork_paged";
qps_status plan_fork(const qps_paged_fork_args* a, Seqs* q, PagesWs* w, size_t* bytes) {
  if (!a) return bad(kFork, "args is NULL");
  const qps_status st = check_seqs(a->seqs, kFork, q);
  if (st != QPS_OK) return st;
  if (a->reserved0 != 0) return bad(kFork, "reserved fields must be 0");
  if (a->n < 0 || a->n > kMostSeqs) return bad(kFork, "n must be in [0, 4096]");
  if (a->n > 0 && (!a->src || !a->dst || !aligned_to(a->src, 4) || !aligned_to(a->dst, 4)))
    return bad(kFork, "src / dst are NULL or misaligned");
  *bytes = lay_out(w, a->workspace, 0, (int64_t)a->n * a->seqs.table_width, a->n);
  return QPS_OK;
}

qps_status kv_fork_paged(const qps_paged_fork_args* a, cudaStream_t s) {
  Seqs q;
  ForkP p{};
  size_t bytes;
  qps_status st = plan_fork(a, &q, &p.w, &bytes);
  if (st != QPS_OK || a->n == 0) return st;
  st = check_workspace(kFork, a->workspace, a->workspace_bytes, bytes);
  if (st != QPS_OK) return st;
  std::vector<Range> written = tables(q.p);
  written.push_back({a->workspace, (int64_t)bytes});
  if (!apart(written, {{a->src, a->n * (int64_t)4}, {a->dst, a->n * (int64_t)4}}))
    return bad(kFork, "what is written overlaps itself, src or dst");
  q.p.err = device_error_word();
  if (!q.p.err) return bad(kFork, "cannot allocate the device error word", QPS_ERR_CUDA);
  p.s = q.p;
  p.src = a->src;
  p.dst = a->dst;
  p.n = a->n;
  st = launch_pages(fork_kernel, p, p.n * (sizeof(ForkItem) + sizeof(int)) + (p.s.batch + 4 * kThreads) * sizeof(int), s);
  return st != QPS_OK ? st : launch_copies(q, p.w, a->n, s);
}

const char* const kCompact = "kv_compact_paged";
qps_status plan_compact(const qps_paged_compact_args* a, Seqs* q, PagesWs* w, size_t* bytes) {
  if (!a) return bad(kCompact, "args is NULL");
  const qps_status st = check_seqs(a->seqs, kCompact, q);
  if (st != QPS_OK) return st;
  const int64_t moves = q->p.n_pages / 2;  // (a hole for each)
  *bytes = lay_out(w, a->workspace, moves, 0, moves);
  return QPS_OK;
}

qps_status kv_compact_paged(const qps_paged_compact_args* a, cudaStream_t s) {
  Seqs q;
  CompactP p{};
  size_t bytes;
  qps_status st = plan_compact(a, &q, &p.w, &bytes);
  if (st != QPS_OK) return st;
  if (!a->new_ids || !aligned_to(a->new_ids, 4) || !a->live || !aligned_to(a->live, 4))
    return bad(kCompact, "new_ids / live are NULL or misaligned");
  st = check_workspace(kCompact, a->workspace, a->workspace_bytes, bytes);
  if (st != QPS_OK) return st;
  std::vector<Range> written = tables(q.p);
  written.insert(written.end(), {{a->workspace, (int64_t)bytes}, {a->new_ids, q.p.n_pages * (int64_t)4}, {a->live, 4}});
  if (!apart(written, {})) return bad(kCompact, "what is written overlaps itself");
  q.p.err = device_error_word();
  if (!q.p.err) return bad(kCompact, "cannot allocate the device error word", QPS_ERR_CUDA);
  p.s = q.p;
  p.new_ids = a->new_ids;
  p.live = a->live;
  st = launch_pages(compact_kernel, p, 0, s);
  return st != QPS_OK ? st : launch_copies(q, p.w, q.p.n_pages / 2, s);
}

template <class A, class F>
qps_status guarded(const A* a, F f) {
  try {
    return f(a);
  } catch (const std::exception&) {
    return QPS_ERR_INTERNAL;
  }
}

}  // namespace
}  // namespace qps

using namespace qps;

extern "C" {

qps_status qps_kv_extend_plan(const qps_paged_extend_args* a, size_t* workspace_bytes) {
  return guarded(a, [&](auto* x) {
    Seqs q;
    PagesWs w;
    size_t bytes = 0;
    int64_t jobs;
    const qps_status st = plan_extend(x, &q, &w, &bytes, &jobs);
    if (st == QPS_OK && workspace_bytes) *workspace_bytes = bytes;
    return st;
  });
}
qps_status qps_kv_extend_paged(const qps_paged_extend_args* a, void* stream) {
  return guarded(a, [&](auto* x) { return kv_extend_paged(x, reinterpret_cast<cudaStream_t>(stream)); });
}
qps_status qps_kv_fork_plan(const qps_paged_fork_args* a, size_t* workspace_bytes) {
  return guarded(a, [&](auto* x) {
    Seqs q;
    PagesWs w;
    size_t bytes = 0;
    const qps_status st = plan_fork(x, &q, &w, &bytes);
    if (st == QPS_OK && workspace_bytes) *workspace_bytes = bytes;
    return st;
  });
}
qps_status qps_kv_fork_paged(const qps_paged_fork_args* a, void* stream) {
  return guarded(a, [&](auto* x) { return kv_fork_paged(x, reinterpret_cast<cudaStream_t>(stream)); });
}
qps_status qps_kv_compact_plan(const qps_paged_compact_args* a, size_t* workspace_bytes) {
  return guarded(a, [&](auto* x) {
    Seqs q;
    PagesWs w;
    size_t bytes = 0;
    const qps_status st = plan_compact(x, &q, &w, &bytes);
    if (st == QPS_OK && workspace_bytes) *workspace_bytes = bytes;
    return st;
  });
}
qps_status qps_kv_compact_paged(const qps_paged_compact_args* a, void* stream) {
  return guarded(a, [&](auto* x) { return kv_compact_paged(x, reinterpret_cast<cudaStream_t>(stream)); });
}

}  // extern "C"
