// The page tables of a paged cache on the device: pages for the next positions of its sequences
// (and those behind a window or a trimmed end given back), sequences that continue others, and the
// live pages of a pool moved to its front; pages copied where that needs it.
//
// All three are integer work on a few hundred KB, in steps of which each needs all of the one
// before: reference counts changed, free pages counted, the lowest ones listed, entries written.
// One cluster of CTAs takes them with a cluster barrier between (a grid per step would cost a
// launch each): its size is chosen by how much there is to scan (pages_ctas).  Free pages are
// ranked by a scan in order, so results do not depend on the order of threads.  What the steps
// share lies in global memory and is read past L1 (__ldcg).
//
// The copies that follow are a second launch, over a list of (from, to, rows) in the workspace:
// every plane of every cache in chunks of kChunk bytes, one a CTA at a time.  They are bound by
// HBM.
#include <algorithm>
#include <exception>
#include <string>
#include <vector>

#include "paged.h"

namespace qps {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kClusterMost = 8;

struct SeqsP {
  int32_t* table;
  int64_t stride;
  int width, batch;
  int32_t* lens;
  int32_t* refs;
  int n_pages, page_shift;
  unsigned int* err;
};

// Workspace of a call: counts of each CTA, totals, lists.
struct PagesWs {
  int* counts;     // [2][kClusterMost]
  int* totals;     // [2 + kClusterMost]: pages needed, copies; (compact) far pages of each CTA
  int* list;       // free pages, in order (compact: holes)
  int* list2;      // (compact) pages behind the live count, in order
  int* base;       // [items] rank of the item's first page
  int* need;       // [items] pages it needs; -1: it cannot be served
  int* copy_rank;  // [items] place of its copy, -1: none
  int* rows;       // (fork) [items][width] source rows as they were
  int* len;        // (fork) [items] source lengths
  int* owner;      // (fork) [batch]
  int4* jobs;      // (from, to, rows, 0)
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
// The same pages in order, to list[rank ..), as far as `most` of them.
template <class F>
__device__ __forceinline__ void list_pages(const SeqsP& s, int p0, int p1, int rank, int most, int* list, int* tmp, F f) {
  for (int at = p0; at < p1 && rank < most; at += 4 * kThreads) {
    const int p = at + 4 * (int)threadIdx.x;
    const int4 r = refs4(s, p, p1);
    const bool a = p < p1 && f(p, r.x), b = p + 1 < p1 && f(p + 1, r.y), c = p + 2 < p1 && f(p + 2, r.z), d = p + 3 < p1 && f(p + 3, r.w);
    const int n = a + b + c + d;
    int all;
    int to = rank + block_scan(n, tmp, &all) - n;
    if (a && to < most) list[to] = p;
    to += a;
    if (b && to < most) list[to] = p + 1;
    to += b;
    if (c && to < most) list[to] = p + 2;
    to += c;
    if (d && to < most) list[to] = p + 3;
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
__device__ __forceinline__ bool is_free(int, int refs) { return refs == 0; }

// The free pages' numbers: counted by every CTA (each its share), then listed, the lowest `need`
// of them; `need` is known to all after the barrier between.
__device__ __forceinline__ void count_free(const SeqsP& s, const PagesWs& w, int* tmp) {
  const int2 sh = page_share(s.n_pages);
  const int n = count_pages(s, sh.x, sh.y, tmp, is_free);
  if (threadIdx.x == 0) w.counts[blockIdx.x] = n;
}
__device__ __forceinline__ int list_free(const SeqsP& s, const PagesWs& w, int need, int* tmp) {
  int before = 0, all = 0;
  for (int c = 0; c < (int)gridDim.x; ++c) {
    const int n = __ldcg(w.counts + c);
    if (c < (int)blockIdx.x) before += n;
    all += n;
  }
  const int2 sh = page_share(s.n_pages);
  list_pages(s, sh.x, sh.y, before, min(need, all), w.list, tmp, is_free);
  return all;
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

struct Growth {
  int len;        // before
  int64_t more;   // new positions asked for
  int64_t end;    // after, if it can be served
};
__device__ __forceinline__ Growth growth(const ExtendP& p, int b) {
  Growth g;
  g.len = seq_len(p.s, b);
  const int n = p.n_new[b];
  g.more = n > 0 ? n : 0;
  g.end = max((int64_t)0, (int64_t)g.len + n);
  return g;
}

__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const __grid_constant__ ExtendP p) {
  __shared__ int tmp[kWarps];
  __shared__ int64_t tmp64[kWarps];
  const SeqsP& s = p.s;
  const int lane = threadIdx.x & 31, page = 1 << s.page_shift;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- pages behind a trimmed end, and those that no later token's window reaches -----------
  for_items(s.batch, [&](int b, int part, int parts) {
    const Growth g = growth(p, b);
    int32_t* row = s.table + b * s.stride;
    const int had = pages_of(s, g.len);
    auto give = [&](int j0, int j1) {
#pragma unroll 4
      for (int j = j0 + part * 32 + lane; j < j1; j += parts * 32) {
        const int pg = row[j];
        if (page_ok(s, pg)) {
          drop_ref(s, pg);
          row[j] = -1;
        }
      }
    };
    const int keep = min(had, pages_of(s, min((int64_t)g.len, g.end)));
    give(keep, had);
    if (p.window) {
      const int64_t low = (g.more ? (int64_t)g.len : g.end) - p.window + 1;
      if (low > 0) give(pages_of(s, p.sinks), min(keep, (int)(low >> s.page_shift)));
    }
  });
  cluster_sync();
  // ---- free pages; what each sequence needs, in order ------------------------------------------
  count_free(s, p.w, tmp);
  if (blockIdx.x == 0) {
    int64_t tokens = 0, pages = 0;
    int copies = 0;
    for (int b0 = 0; b0 < s.batch; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      Growth g = {0, 0, 0};
      if (b < s.batch) g = growth(p, b);
      int64_t all;
      const int64_t upto = tokens + block_scan(g.more, tmp64, &all);
      if (b < s.batch) p.starts[b] = (int32_t)min(upto - g.more, p.max_tokens);
      tokens += all;
      const bool grows = g.more > 0, fits = g.end <= (int64_t)s.width << s.page_shift && upto <= p.max_tokens;
      bool copy = false;
      int need = 0;
      if (grows && fits) {
        if (g.len & (page - 1)) {  // (a last page that others name too is copied before it is written)
          const int pg = __ldcg(s.table + b * s.stride + (g.len >> s.page_shift));
          copy = page_ok(s, pg) && __ldcg(s.refs + pg) > 1;
        }
        need = pages_of(s, g.end) - pages_of(s, g.len) + copy;
      }
      const int64_t upto_pages = pages + block_scan((int64_t)need, tmp64, &all);
      pages += all;
      int all_copies;
      const int upto_copies = copies + block_scan((int)copy, tmp, &all_copies);
      copies += all_copies;
      if (b < s.batch) {
        p.w.base[b] = (int)min(upto_pages - need, (int64_t)0x7fffffff);
        p.w.need[b] = grows && !fits ? -1 : need;
        p.w.copy_rank[b] = copy ? upto_copies - 1 : -1;
      }
    }
    if (threadIdx.x == 0) {
      p.starts[s.batch] = (int32_t)min(tokens, p.max_tokens);
      p.w.totals[0] = (int)min(pages, (int64_t)s.n_pages);
      p.w.totals[1] = copies;
    }
  }
  cluster_sync();
  const int free = list_free(s, p.w, __ldcg(p.w.totals), tmp);
  cluster_sync();
  // ---- the new tokens' rows and the new entries ---------------------------------------------------
  for_items(s.batch, [&](int b, int part, int parts) {
    const Growth g = growth(p, b);  // (lengths, and the entries of pages that are copied, change behind the next barrier)
    const int need = __ldcg(p.w.need + b), base = __ldcg(p.w.base + b), rank = __ldcg(p.w.copy_rank + b);
    const bool served = need == 0 || (need > 0 && base <= free - need);
    const int copy = rank >= 0, had = pages_of(s, g.len);
    int32_t* row = s.table + b * s.stride;
    int32_t old = -1;  // the page of the rows behind the last position
    if (g.more && (g.len & (page - 1))) old = copy ? -1 : __ldcg(row + (g.len >> s.page_shift));
    if (!served) atomicOr(s.err, kErrIndex);
    const int64_t s0 = __ldcg(p.starts + b), s1 = __ldcg(p.starts + b + 1);
    for (int64_t i = s0 + part * 32 + lane; i < s1; i += parts * 32) {
      const int64_t at = g.len + (i - s0);
      const int j = (int)(at >> s.page_shift);
      int pg = -1;
      if (served) pg = j >= had ? __ldcg(p.w.list + base + copy + (j - had)) : copy ? __ldcg(p.w.list + base) : old;
      p.slots[i] = page_ok(s, pg) ? (int64_t)pg * page + (at & (page - 1)) : -1;
      p.positions[i] = at;
    }
    if (served && need > 0) {
      for (int k = part * 32 + lane; k < need - copy; k += parts * 32) {
        const int pg = __ldcg(p.w.list + base + copy + k);
        row[had + k] = pg;
        s.refs[pg] = 1;
      }
    }
  });
  const int64_t total = __ldcg(p.starts + s.batch);
  for (int64_t i = total + blockIdx.x * kThreads + threadIdx.x; i < p.max_tokens; i += (int64_t)gridDim.x * kThreads) {
    p.slots[i] = -1;
    p.positions[i] = 0;
  }
  cluster_sync();
  // ---- copies and lengths -------------------------------------------------------------------------
  for (int b = blockIdx.x * kThreads + threadIdx.x; b < s.batch; b += gridDim.x * kThreads) {
    const Growth g = growth(p, b);
    const int need = __ldcg(p.w.need + b), base = __ldcg(p.w.base + b), rank = __ldcg(p.w.copy_rank + b);
    const bool served = need == 0 || (need > 0 && base <= free - need);
    if (rank >= 0) {
      int4 job = make_int4(0, 0, 0, 0);
      if (served) {
        int32_t* at = s.table + b * s.stride + (g.len >> s.page_shift);
        const int from = __ldcg(at), to = __ldcg(p.w.list + base);
        job = make_int4(from, to, g.len & (page - 1), 0);
        *at = to;
        s.refs[to] = 1;
        drop_ref(s, from);
      }
      p.w.jobs[rank] = job;
    }
    if (served) s.lens[b] = (int32_t)g.end;
  }
}

// ---- fork -------------------------------------------------------------------------------------
struct ForkP {
  SeqsP s;
  PagesWs w;
  const int32_t* src;
  const int32_t* dst;
  int n;
};

__global__ void __launch_bounds__(kThreads, 1) fork_kernel(const __grid_constant__ ForkP p) {
  __shared__ int tmp[kWarps];
  const SeqsP& s = p.s;
  const int lane = threadIdx.x & 31, page = 1 << s.page_shift;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto each = [&](int n, auto f) {
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads) f(i);
  };
  // ---- a row that is named twice goes to the first ----------------------------------------------
  each(s.batch, [&](int b) { p.w.owner[b] = 0x7fffffff; });
  cluster_sync();
  auto valid = [&](int i) { return p.src[i] < s.batch && (uint32_t)p.dst[i] < (uint32_t)s.batch; };
  each(p.n, [&](int i) {
    if (valid(i)) atomicMin(p.w.owner + p.dst[i], i);
    else atomicOr(s.err, kErrIndex);
  });
  cluster_sync();
  auto active = [&](int i) { return valid(i) && __ldcg(p.w.owner + p.dst[i]) == i && p.src[i] != p.dst[i]; };
  // ---- the sources as they are, each of their pages held once more ------------------------------
  for_items(p.n, [&](int i, int part, int parts) {
    if (!active(i)) {
      if (valid(i) && __ldcg(p.w.owner + p.dst[i]) != i) atomicOr(s.err, kErrIndex);
      return;
    }
    const int b = p.src[i], n = b < 0 ? 0 : seq_len(s, b);
    if (part == 0 && lane == 0) p.w.len[i] = n;
    int* row = p.w.rows + (int64_t)i * s.width;
#pragma unroll 4
    for (int j = part * 32 + lane; j < s.width; j += parts * 32) {
      int pg = j < pages_of(s, n) ? __ldcg(s.table + b * s.stride + j) : -1;
      if (!page_ok(s, pg)) pg = -1;
      row[j] = pg;
      if (pg >= 0) atomicAdd(s.refs + pg, 1);
    }
  });
  cluster_sync();
  for_items(p.n, [&](int i, int part, int parts) {
    if (!active(i)) return;
    const int b = p.dst[i], n = pages_of(s, seq_len(s, b));
#pragma unroll 4
    for (int j = part * 32 + lane; j < n; j += parts * 32) drop_ref(s, __ldcg(s.table + b * s.stride + j));
  });
  cluster_sync();
  // ---- a page for each last one that is not full -------------------------------------------------
  auto part_of = [&](int i) -> int {  // the page that is copied, or -1
    const int n = __ldcg(p.w.len + i);
    return n & (page - 1) ? __ldcg(p.w.rows + (int64_t)i * s.width + (n >> s.page_shift)) : -1;
  };
  count_free(s, p.w, tmp);
  if (blockIdx.x == 0) {
    int copies = 0;
    for (int i0 = 0; i0 < p.n; i0 += kThreads) {
      const int i = i0 + threadIdx.x;
      const int copy = i < p.n && active(i) && part_of(i) >= 0;
      int all;
      const int upto = copies + block_scan(copy, tmp, &all);
      copies += all;
      if (i < p.n) p.w.copy_rank[i] = copy ? upto - 1 : -1;
    }
    if (threadIdx.x == 0) p.w.totals[0] = p.w.totals[1] = copies;
  }
  cluster_sync();
  const int free = list_free(s, p.w, __ldcg(p.w.totals), tmp);
  cluster_sync();
  // ---- the new rows ------------------------------------------------------------------------------
  for_items(p.n, [&](int i, int part, int parts) {
    if (!active(i)) return;
    const int b = p.dst[i], n = __ldcg(p.w.len + i), rank = __ldcg(p.w.copy_rank + i);
    const int last = rank >= 0 ? n >> s.page_shift : -1;
    const bool served = rank < free;
    int32_t* row = s.table + b * s.stride;
    for (int j = part * 32 + lane; j < s.width; j += parts * 32) {
      int pg = __ldcg(p.w.rows + (int64_t)i * s.width + j);
      if (j == last) {
        const int from = pg;
        pg = served ? __ldcg(p.w.list + rank) : -1;
        p.w.jobs[rank] = served ? make_int4(from, pg, n & (page - 1), 0) : make_int4(0, 0, 0, 0);
        if (served) s.refs[pg] = 1;
        drop_ref(s, from);
      }
      row[j] = pg;
    }
    if (part == 0 && lane == 0) {
      if (!served) atomicOr(s.err, kErrIndex);
      s.lens[b] = served ? n : n & ~(page - 1);  // (no page for the last positions: they are left out)
    }
  });
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
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 sh = page_share(s.n_pages);
  const int n = count_pages(s, sh.x, sh.y, tmp, [](int, int r) { return r > 0; });
  if (threadIdx.x == 0) p.w.counts[blockIdx.x] = n;
  cluster_sync();
  int live = 0;
  for (int c = 0; c < (int)gridDim.x; ++c) live += __ldcg(p.w.counts + c);
  // holes before `live`, pages in use from it on: as many of the one as of the other
  auto hole = [&](int pg, int r) { return pg < live && r <= 0; };
  auto far = [&](int pg, int r) { return pg >= live && r > 0; };
  const int holes = sh.x >= live ? 0 : sh.y <= live ? sh.y - sh.x - n : count_pages(s, sh.x, sh.y, tmp, hole);
  const int fars = sh.x >= live ? n : sh.y <= live ? 0 : n - (live - sh.x - holes);
  if (threadIdx.x == 0) {
    p.w.counts[kClusterMost + blockIdx.x] = holes;
    p.w.totals[2 + blockIdx.x] = fars;
  }
  cluster_sync();
  int h0 = 0, f0 = 0, moves = 0;
  for (int c = 0; c < (int)gridDim.x; ++c) {
    const int h = __ldcg(p.w.counts + kClusterMost + c), f = __ldcg(p.w.totals + 2 + c);
    if (c < (int)blockIdx.x) {
      h0 += h;
      f0 += f;
    }
    moves += h;
  }
  if (holes > 0) list_pages(s, sh.x, sh.y, h0, moves, p.w.list, tmp, hole);
  if (fars > 0) list_pages(s, sh.x, sh.y, f0, moves, p.w.list2, tmp, far);
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
    p.w.totals[1] = moves;
    p.live[0] = live;
  }
  cluster_sync();
  for_items(s.batch, [&](int b, int part, int parts) {
    const int m = pages_of(s, seq_len(s, b));
    int32_t* row = s.table + b * s.stride;
#pragma unroll 4
    for (int j = part * 32 + lane; j < m; j += parts * 32) {
      const int pg = row[j];
      if (page_ok(s, pg)) row[j] = __ldcg(p.new_ids + pg);
    }
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
  int n, page_shift, n_pages;
  const int4* jobs;
  const int* count;
  int most;                    // jobs there can be
  unsigned int* err;
};

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyP p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int jobs = min(*p.count, p.most), chunks = p.first[p.n];
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
    const uint32_t used = (uint32_t)(((uint64_t)pl.head_bytes * job.z) >> p.page_shift);  // bytes of a head that are copied
    if (used == 0 || !in_bounds((uint32_t)job.x < (uint32_t)p.n_pages && (uint32_t)job.y < (uint32_t)p.n_pages, p.err)) continue;
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
  if (a.batch < 1 || a.batch > 65535) return bad(call, "batch must be in [1, 65535]");
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
size_t lay_out(PagesWs* w, void* base, int64_t items, int64_t list, int64_t list2, int64_t jobs, int64_t rows, int64_t batch) {
  Cut c{reinterpret_cast<char*>(base)};
  w->counts = c.take<int>(2 * kClusterMost);
  w->totals = c.take<int>(2 + kClusterMost);
  w->list = c.take<int>(list);
  w->list2 = c.take<int>(list2);
  w->base = c.take<int>(items);
  w->need = c.take<int>(items);
  w->copy_rank = c.take<int>(items);
  w->len = c.take<int>(items);
  w->rows = c.take<int>(rows);
  w->owner = c.take<int>(batch);
  w->jobs = c.take<int4>(jobs);
  return c.bytes;
}

int pages_ctas(const SeqsP& s) { return s.n_pages > 4096 || s.batch > kWarps ? kClusterMost : 1; }

template <class P>
qps_status launch_pages(void (*kernel)(P), const P& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int ctas = pages_ctas(p.s);
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
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
    p.page_shift = q.p.page_shift;
    p.n_pages = q.p.n_pages;
    p.jobs = w.jobs;
    p.count = w.totals + 1;
    p.most = (int)most;
    p.err = q.p.err;
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
  // (a sequence's share of the tokens takes one page more than its full ones, and a copy)
  const int64_t list = std::min<int64_t>(q->p.n_pages, (a->max_tokens >> q->p.page_shift) + 2 * (int64_t)a->seqs.batch);
  *jobs = std::min<int64_t>(a->seqs.batch, a->max_tokens);
  *bytes = lay_out(w, a->workspace, a->seqs.batch, list, 0, *jobs, 0, 0);
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
  st = launch_pages(extend_kernel, p, s);
  return st != QPS_OK || jobs == 0 ? st : launch_copies(q, p.w, jobs, s);
}

const char* const kFork = "kv_fork_paged";
qps_status plan_fork(const qps_paged_fork_args* a, Seqs* q, PagesWs* w, size_t* bytes) {
  if (!a) return bad(kFork, "args is NULL");
  const qps_status st = check_seqs(a->seqs, kFork, q);
  if (st != QPS_OK) return st;
  if (a->reserved0 != 0) return bad(kFork, "reserved fields must be 0");
  if (a->n < 0 || a->n > 65535) return bad(kFork, "n must be in [0, 65535]");
  if (a->n > 0 && (!a->src || !a->dst || !aligned_to(a->src, 4) || !aligned_to(a->dst, 4)))
    return bad(kFork, "src / dst are NULL or misaligned");
  *bytes = lay_out(w, a->workspace, a->n, a->n, 0, a->n, (int64_t)a->n * a->seqs.table_width, a->seqs.batch);
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
  st = launch_pages(fork_kernel, p, s);
  return st != QPS_OK ? st : launch_copies(q, p.w, a->n, s);
}

const char* const kCompact = "kv_compact_paged";
qps_status plan_compact(const qps_paged_compact_args* a, Seqs* q, PagesWs* w, size_t* bytes) {
  if (!a) return bad(kCompact, "args is NULL");
  const qps_status st = check_seqs(a->seqs, kCompact, q);
  if (st != QPS_OK) return st;
  const int64_t moves = q->p.n_pages / 2;  // (a hole for each)
  *bytes = lay_out(w, a->workspace, 0, moves, moves, moves, 0, 0);
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
  st = launch_pages(compact_kernel, p, s);
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
