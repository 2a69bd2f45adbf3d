// Decode attention of many query rows per KV head on the fifth-generation tensor cores:
// a shared prefix (the rows of a whole batch) or a verify batch, over fp16 pages.
//
// A CTA holds 128 query rows of one KV head (M of the products) and walks its chunk in
// tiles of 128 positions:
//     S = Q K^T          tcgen05.mma, Q and K in shared memory (K-major), S in TMEM (f32)
//     P = 2^(S' - m)     4 warps, one query row a thread: no reduction crosses lanes
//     O += P V           tcgen05.mma, P (fp16) in TMEM over the S it came from, V in shared
//                        memory as it lies in the page (MN-major), O in TMEM (f32)
// Even and odd tiles are two streams with an S, an O and softmax state of their own (TMEM:
// 128 + 128 + 2 D <= 512 columns), so that one stream's exponentials run beside the other's
// products; the two states are merged once at the end, as two parts would be.
//
// The running reference m of a row is set kRefShift (log2) below a tile's maximum, and again
// only when one exceeds what it was set for by more than kRefLazy: P stays within fp16 and
// the rescale of O is rare.  P is rounded once to fp16 (the operand type); sums, m and O are
// float32.
//
// Measured: 256 rows per KV head, 8 heads of 128, 32768 shared positions: 40 us, of which
// the first three tiles take 9 (every CTA's first tiles at once, and the queries behind
// them) and the other 26 of a CTA 0.9 us each: 0.6 of the products' rate.  Two row tiles
// a CTA, so that K and V pass from L2 once, took 45 us: the stages left beside the second
// tile's queries hold too few bytes under way.
//
// Roles: warp 0 brings the tiles (tensor-map boxes of one page each, kStages ahead), warp 1
// issues the products, warps 4-7 and 8-11 are the streams' softmax.  Every wait is bounded
// (see mma::mbar_wait); one that gives up stops the CTA's roles, the copies and products in
// flight are waited for, the TMEM is freed, and the error word is set.
#pragma once

#include <cuda_bf16.h>

#include <atomic>
#include <cstring>

#include "attn_mma.cuh"

namespace qps {
namespace tm {

using mma::global_ns;
using mma::mbar_expect_tx;
using mma::mbar_init;
using mma::mbar_try_wait;
using mma::smem_addr;
using mma::tma_load_4d;
using mma::TmaSet;

constexpr int kRows = 128, kTok = 128, kThreads = 384;

template <int D>
struct Geo {
  static constexpr int CG = D / 64;                // 128-byte column groups of a row
  static constexpr int TILE = kTok * D * 2;        // bytes of a K or V tile (and of Q)
  static constexpr int STAGES = D == 64 ? 5 : 3;
  static constexpr int K_OFF = TILE;               // Q first
  static constexpr int V_OFF = K_OFF + STAGES * TILE;
  static constexpr int BAR = V_OFF + STAGES * TILE;
  static constexpr int SMEM = BAR + 256 + 1024;    // + slack for the 1024-byte base alignment
  // TMEM columns
  static constexpr int S_COL = 0, O_COL = 256;
};

// ---- tcgen05 -------------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, int cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, int cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// One value for the warp's lanes, which the compiler can keep in a uniform register.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
// The products and commits below are issued by one lane, chosen by a predicate on the
// instruction instead of a branch: the warp stays converged, so descriptors are computed in
// uniform registers (under a branch each product took 100 cycles to issue, more than it
// takes to run).
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}
__device__ __forceinline__ void commit(uint32_t bar, uint32_t one) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.u32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(one)
      : "memory");
}
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(one)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add), "r"(one)
      : "memory");
}
// 32 columns of the warp's 32 lanes
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand descriptor, 128-byte swizzle: rows (K-major) or k steps (MN-major)
// of 128 bytes in groups of 8 (1024 bytes apart); `lead` is the distance of the next 64
// columns of an MN-major operand (K-major: unused).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// f16 x f16 -> f32, M = 128; b_mn: B is MN-major
__device__ __forceinline__ constexpr uint32_t instr_desc(int n, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The CTA's word for a wait that has run out: its tile and warp; not 0, which lets the others go on.
__device__ __forceinline__ int gave_up(int tile, int warp) { return (tile << 5 | warp) + 1; }
// At the end of a CTA in which one has (the waits themselves stay short: this in each of them
// cost 2 us of 24 in instruction fetches), one lane: the report, and the record if it is the
// launch's first (internal.h), which is then finished by the drain.
static __device__ __noinline__ bool report_give_up(unsigned int* err, int word, int issued, int tiles, int positions) {
  atomicOr(err, kErrTimeout);
  if (atomicAdd(err + 1, 1u) != 0) return false;
  unsigned int* r = err + 2;
  r[0] = blockIdx.x;
  r[1] = blockIdx.y;
  r[2] = blockIdx.z;
  r[3] = (word - 1) & 31;
  r[4] = (word - 1) >> 5;
  r[5] = issued;
  r[6] = tiles;
  r[7] = positions;
  return true;
}

// ---- the kernel ------------------------------------------------------------------------------
// P: PagedAttnParams, or WindowAttnParams.
template <int D, class P>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tm_kernel(const __grid_constant__ P p, const __grid_constant__ TmaSet maps) {
  using G = Geo<D>;
  constexpr int ST = G::STAGES;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(smem);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- this CTA's rows and positions ------------------------------------------------------
  const int rtiles = (p.rows_per_cta + kRows - 1) / kRows;
  const int split = blockIdx.x / rtiles, row0 = (blockIdx.x % rtiles) * kRows;
  const int head = blockIdx.y;
  int bz, t0, t1;  // the sequence (of a shared prefix: whose page entries it is read through)
  bool whole = false;
  if (p.shared) {
    t0 = split * (int)p.chunk;
    const PagedPrefix pre = paged_prefix(p, lane);
    bz = pre.b;
    t1 = (int)min((int64_t)pre.len, t0 + p.chunk);  // (at or before t0: an empty part)
  } else {
    const PagedChunk ch = paged_find(p, split, lane);
    if (ch.b < 0) return;  // more CTAs than chunks (every warp finds the same)
    if (ch.first && head == 0 && row0 == 0 && threadIdx.x == 0 && in_bounds(ch.b < p.batch, p.err))
      p.chunks[ch.b] = make_int2(split, ch.count);
    bz = ch.b;
    t0 = ch.t0;
    t1 = ch.t1;
    whole = ch.whole;
  }
  const int ntiles = uniform(t1 > t0 ? (t1 - t0 + kTok - 1) / kTok : 0);  // 0: no own positions
  const PagedWindow win = paged_window(p, bz);

  // ---- barriers, TMEM, queries ---------------------------------------------------------------
  const uint32_t bars = sbase + G::BAR;
  auto k_full = [&](int s) { return bars + 8 * s; };
  auto k_empty = [&](int s) { return bars + 8 * (ST + s); };
  auto v_full = [&](int s) { return bars + 8 * (2 * ST + s); };
  auto v_empty = [&](int s) { return bars + 8 * (3 * ST + s); };
  auto s_full = [&](int w) { return bars + 8 * (4 * ST + w); };
  auto p_ready = [&](int w) { return bars + 8 * (4 * ST + 2 + w); };
  const uint32_t all_done = bars + 8 * (4 * ST + 4), q_full = bars + 8 * (4 * ST + 5);
  static_assert(8 * (4 * ST + 6) <= 240, "barriers fit their region");
  uint32_t* tmem_word = reinterpret_cast<uint32_t*>(smem + G::BAR + 240);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + G::BAR + 244);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4 * ST + 6; ++i)
      mbar_init(bars + 8 * i, i == 4 * ST + 5 ? 8 : i >= 4 * ST + 2 && i < 4 * ST + 4 ? 4 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    *abort_flag = 0;
  }
  if (warp == 2) tmem_alloc(smem_addr(tmem_word), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = uniform(*tmem_word);

  int issued = 0;  // (warp 0) copies of K and V under way or landed, two a tile
  // Bounded wait of a whole warp (at `tile`), with one answer for all of its lanes; gives up at
  // once when another role has.
  auto wait = [&](uint32_t bar, uint32_t parity, int tile) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t since = global_ns();
    for (;;) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      int over = 0;
      if (lane == 0) {
        over = *abort_flag;
        if (!over && global_ns() - since >= p.wait_ns) *abort_flag = over = gave_up(tile, warp);
      }
      if (__shfl_sync(0xffffffffu, over, 0)) return false;
    }
  };
  // Q [128][D], K-major: row r's 16-byte chunk c of a column group at r * 128 + (c ^ r % 8) *
  // 16; by the softmax warps, every load first, while the first tiles are under way.
  auto load_q = [&]() {
    constexpr int N = kRows * D / 8 / 256;
    uint4 v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x - 128 + k * 256, r = i / (D / 8), c = i % (D / 8), rr = row0 + r;
      v[k] = make_uint4(0, 0, 0, 0);
      if (rr < p.rows_per_cta) {
        const int e = rr / p.group, h = head * p.group + rr % p.group;
        const int b = p.shared ? e / p.n_q : bz, qi = p.shared ? e % p.n_q : e;
        const int64_t at = (int64_t)b * p.q_bstride + ((int64_t)qi * p.hq + h) * D + c * 8;
        if (q_in_bounds(p, at)) v[k] = *reinterpret_cast<const uint4*>(p.q + at);
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x - 128 + k * 256, r = i / (D / 8), c = i % (D / 8);
      *reinterpret_cast<uint4*>(smem + (c >> 3) * (kRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v[k];
    }
    mma::fence_proxy_async();
    __syncwarp();
    if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(q_full) : "memory");
  };

  if (warp == 0) {
    // ---- tiles: each box is min(page, 128) positions of one page and 64 columns, at most 16 of
    // them a tile, one a lane.  A lane reads its page a tile ahead (read when the box is due, the
    // table's latency kept the copies 1800 cycles a tile apart, twice the products' time). ------
    const int br = min(1 << p.page_shift, kTok), nb = kTok / br;
    const int32_t* row = p.table + (int64_t)bz * p.table_stride;
    const int cg = lane % G::CG, r = lane / G::CG;
    auto has = [&](int j) {
      const int t = t0 + j * kTok + r * br;
      return r < nb && t < t1 && !paged_unseen(p, win, t, br);
    };
    auto at = [&](int j) { return paged_true(p, win, t0 + j * kTok + r * br); };
    auto entry = [&](int j) {
      const int i = at(j) >> p.page_shift;
      return has(j) && entry_in_bounds(p, bz * p.table_stride + i) ? row[i] : 0;
    };
    auto load = [&](const TensorMap* map, uint32_t dst, uint32_t bar, int j, int page) {
      if (lane == 0) mbar_expect_tx(bar, G::TILE);
      __syncwarp();
      if (r < nb && (map != &maps.k || j != p.drop_tile) &&
          in_bounds(cg * (kTok * 128) + (r + 1) * br * 128 <= G::TILE && dst - sbase + G::TILE <= G::BAR && page <= p.n_pages &&
                        head < p.hkv && (at(j) & ((1 << p.page_shift) - 1)) + br <= 1 << p.page_shift,
                    p.err))
        tma_load_4d(dst + cg * (kTok * 128) + r * br * 128, map, cg * 128,
                    at(j) & ((1 << p.page_shift) - 1), head, page, bar);
    };
    int next = entry(0);
    for (int j = 0; j < ntiles; ++j) {
      const int s = j % ST;
      const uint32_t par = ((j / ST) & 1) ^ 1;
      int page = (int)p.n_pages;  // behind the last position, or out of range: zeros
      if (has(j)) {
        if ((uint64_t)(int64_t)next < (uint64_t)p.n_pages) page = next;
        else atomicOr(p.err, kErrIndex);
      }
      next = entry(j + 1);
      if (j >= ST && !wait(k_empty(s), par, j)) break;
      __syncwarp();
      load(&maps.k, sbase + G::K_OFF + s * G::TILE, k_full(s), j, page);
      issued = 2 * j + 1;
      if (j >= ST && !wait(v_empty(s), par, j)) break;
      __syncwarp();
      load(&maps.v, sbase + G::V_OFF + s * G::TILE, v_full(s), j, page);
      issued = 2 * j + 2;
    }
  } else if (warp == 1) {
    // ---- products --------------------------------------------------------------------------------
    constexpr uint32_t ID_S = instr_desc(kTok, 0), ID_O = instr_desc(D, 1);
    const uint32_t one = elect_lane();
    auto s_product = [&](int j) -> bool {  // S of tile j
      const int s = j % ST;
      if (!wait(k_full(s), (j / ST) & 1, j)) return false;
      fence_after();
      const uint32_t d = tmem + G::S_COL + (j & 1) * kTok;
      const uint64_t a = smem_desc(sbase, 16), b = smem_desc(sbase + G::K_OFF + s * G::TILE, 16);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = ((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4;
        mma_ss(d, a + off, b + off, ID_S, kk > 0, one);
      }
      commit(k_empty(s), one);
      commit(s_full(j & 1), one);
      return true;
    };
    bool ok = ntiles == 0 || wait(q_full, 0, 0);
    for (int j = 0; j < min(2, ntiles) && ok; ++j) ok = s_product(j);
    for (int j = 0; j < ntiles && ok; ++j) {
      const int s = j % ST, w = j & 1;
      if (!(ok = wait(v_full(s), (j / ST) & 1, j))) break;
      const int left = t1 - (t0 + j * kTok);
      const uint32_t vb = G::V_OFF + s * G::TILE;
      if (left < kTok) {
        // rows of the last page behind the end hold whatever was there, and 0 x NaN is NaN
        for (int i = left * 8 + lane; i < kTok * 8; i += 32)
#pragma unroll
          for (int cg = 0; cg < G::CG; ++cg)
            if (in_bounds(left >= 0 && cg * (kTok * 128) + i * 16 + 16 <= G::TILE, p.err))
              *reinterpret_cast<uint4*>(smem + vb + cg * (kTok * 128) + i * 16) = make_uint4(0, 0, 0, 0);
        mma::fence_proxy_async();
        __syncwarp();
      }
      if constexpr (has_window<P>) {
        const int tb = t0 + j * kTok;
        if (tb < win.none_lo && tb + kTok > p.sinks) {  // nor do rows that no window reaches
          for (int i = max(0, p.sinks - tb) * 8 + lane; i < min(kTok, win.none_lo - tb) * 8; i += 32)
#pragma unroll
            for (int cg = 0; cg < G::CG; ++cg)
              if (in_bounds(cg * (kTok * 128) + i * 16 + 16 <= G::TILE, p.err))
                *reinterpret_cast<uint4*>(smem + vb + cg * (kTok * 128) + i * 16) = make_uint4(0, 0, 0, 0);
          mma::fence_proxy_async();
          __syncwarp();
        }
      }
      if (!(ok = wait(p_ready(w), (j >> 1) & 1, j))) break;
      fence_after();
      const uint32_t d = tmem + G::O_COL + w * D, a = tmem + G::S_COL + w * kTok;
      const uint64_t b = smem_desc(sbase + vb, kTok * 128);
#pragma unroll
      for (int kk = 0; kk < kTok / 16; ++kk)
        mma_ts(d, a + kk * 8, b + (uint64_t)((kk * 2048) >> 4), ID_O, j >= 2 || kk > 0, one);
      commit(v_empty(s), one);
      if (j + 2 < ntiles) ok = s_product(j + 2);
    }
    commit(all_done, one);  // completes when everything issued above has
  } else if (warp >= 4) {
    // ---- softmax: stream w, one row a thread --------------------------------------------------
    const int w = (warp - 4) >> 2, r = (warp & 3) * 32 + lane, rr = row0 + r;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const uint32_t s_at = tmem + lanes + G::S_COL + w * kTok, o_at = tmem + lanes + G::O_COL + w * D;
    load_q();
    int lim = 0, low = 0;  // positions below lim are visible to the row, but for [sinks, low)
    if (rr < p.rows_per_cta) {
      const int e = rr / p.group, b = p.shared ? e / p.n_q : bz, qi = p.shared ? e % p.n_q : e;
      lim = paged_len(p, b);
      if (p.causal) lim += qi + 1 - p.n_q;
      if constexpr (has_window<P>) low = lim - p.window;
      lim = min(lim, t1);
    }
    constexpr float LOG2E = 1.4426950408889634f;
    const float qs = p.scale * LOG2E, cap = p.softcap, cap_k = cap > 0.f ? 2.f * LOG2E / cap : 0.f;
    auto logit = [&](uint32_t v) -> float {
      const float s = __uint_as_float(v);
      return cap > 0.f ? mma::softcap_tanh(s * p.scale, cap, cap_k) * LOG2E : s * qs;
    };
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = w; j < ntiles; j += 2) {
      if (!(ok = wait(s_full(w), (j >> 1) & 1, j))) break;
      fence_after();
      const int first = t0 + j * kTok;
      // Whole tiles of plain logits, the common case, have a body of their own: maxima and
      // exponentials straight from S (a positive scale keeps the order), four chains each,
      // the next 32 columns read beside the present ones' arithmetic.
      const bool fast = __all_sync(0xffffffffu, (first + kTok <= lim && (!has_window<P> || first >= low)) || rr >= p.rows_per_cta) &&
                        cap <= 0.f && qs >= 0.f;
      auto hidden = [&](int t) {
        if constexpr (has_window<P>)
          if (t < low && t >= p.sinks) return true;
        return t >= lim;
      };
      uint32_t va[32], vb[32];
      float mx = -INFINITY;
      if (fast) {
        float mm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto most = [&](const uint32_t (&v)[32]) {
#pragma unroll
          for (int i = 0; i < 32; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mm[k] = fmaxf(fmaxf(mm[k], __uint_as_float(v[i + k])), __uint_as_float(v[i + 4 + k]));
        };
        tmem_ld32(va, s_at);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kTok / 32; c += 2) {
          tmem_ld32(vb, s_at + 32 * (c + 1));
          most(va);
          tmem_wait_ld();
          if (c + 2 < kTok / 32) tmem_ld32(va, s_at + 32 * (c + 2));
          most(vb);
          if (c + 2 < kTok / 32) tmem_wait_ld();
        }
        mx = fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3])) * qs;
      } else {
#pragma unroll 1
        for (int c = 0; c < kTok / 32; ++c) {
          __syncwarp();
          tmem_ld32(va, s_at + 32 * c);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!hidden(first + 32 * c + i)) mx = fmaxf(mx, logit(va[i]));
        }
        __syncwarp();
      }
      mx -= kRefShift;
      const bool raise = mx - m > kRefLazy;  // (false when both are -inf)
      const float cr = raise ? ex2(m - mx) : 1.f;  // (0 from -inf)
      if (raise) {
        m = mx;
        l *= cr;
      }
      // S of this tile is complete, so every product before it is: this stream's O is at rest
      if (j >= 2 && __any_sync(0xffffffffu, raise)) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          __syncwarp();
          tmem_ld32(va, o_at + 32 * c);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) va[i] = __float_as_uint(__uint_as_float(va[i]) * cr);
          tmem_st32(o_at + 32 * c, va);
        }
      }
      const float ms = m == -INFINITY ? 0.f : m;
      float sum = 0.f;
      if (fast) {
        float ss[4] = {0.f, 0.f, 0.f, 0.f};
        auto weigh = [&](const uint32_t (&v)[32], int c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float a = ex2(fmaf(__uint_as_float(v[2 * i]), qs, -ms));
            const float b = ex2(fmaf(__uint_as_float(v[2 * i + 1]), qs, -ms));
            ss[(2 * i) & 3] += a;
            ss[(2 * i + 1) & 3] += b;
            pk[i] = mma::pack_h2(a, b);
          }
          tmem_st16(s_at + 16 * c, pk);  // (over columns of S that are already read, none under way)
        };
        tmem_ld32(va, s_at);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kTok / 32; c += 2) {
          tmem_ld32(vb, s_at + 32 * (c + 1));
          weigh(va, c);
          tmem_wait_ld();
          if (c + 2 < kTok / 32) tmem_ld32(va, s_at + 32 * (c + 2));
          weigh(vb, c + 1);
          if (c + 2 < kTok / 32) tmem_wait_ld();
        }
        sum = (ss[0] + ss[1]) + (ss[2] + ss[3]);
      } else {
#pragma unroll 1
        for (int c = 0; c < kTok / 32; ++c) {
          __syncwarp();
          tmem_ld32(va, s_at + 32 * c);
          tmem_wait_ld();
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a = ex2(logit(va[2 * i]) - ms), b = ex2(logit(va[2 * i + 1]) - ms);
            if (hidden(first + 32 * c + 2 * i)) a = 0.f;
            if (hidden(first + 32 * c + 2 * i + 1)) b = 0.f;
            sum += a + b;
            pk[i] = mma::pack_h2(a, b);
          }
          __syncwarp();
          tmem_st16(s_at + 16 * c, pk);
        }
        __syncwarp();
      }
      l += sum;
      tmem_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(p_ready(w)) : "memory");
    }
    // ---- merge the streams, write the chunk's part --------------------------------------------
    if (ok) ok = wait(all_done, 0, ntiles);
    fence_after();
    // The streams exchange halves of O through the stages (every tile has been consumed), and
    // their states: stream w finishes the columns [w D/2, (w + 1) D/2).  Column-major, so that
    // a warp's rows are neighbours.
    constexpr int H = D / 2;
    float* hand = reinterpret_cast<float*>(smem + G::K_OFF);   // [2][D / 2][128]
    float* state = reinterpret_cast<float*>(smem);              // [2][2][128] (over Q)
    const bool two = ntiles > 1;
    if (ok) {
      state[w * 2 * kRows + r] = m;
      state[w * 2 * kRows + kRows + r] = l;
      if (two) {
#pragma unroll
        for (int c = 0; c < H / 32; ++c) {
          uint32_t v[32];
          __syncwarp();
          tmem_ld32(v, o_at + (1 - w) * H + 32 * c);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) hand[w * H * kRows + (32 * c + i) * kRows + r] = __uint_as_float(v[i]);
        }
      }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (ok && !__any_sync(0xffffffffu, *abort_flag)) {
      const float m0 = m, l0 = l, m1 = state[(1 - w) * 2 * kRows + r], l1 = state[(1 - w) * 2 * kRows + kRows + r];
      const float mx = fmaxf(m0, m1);
      const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - mx), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - mx);
      const float den = l0 * f0 + l1 * f1;
      const bool empty = den == 0.f;
      const float inv = empty ? 0.f : 1.f / den;
      const float w0 = f0 * inv, w1 = f1 * inv;  // of this stream's columns, and of the other's
      const bool has0 = ntiles > w, has1 = ntiles > 1 - w;
      int64_t at = 0;
      bool mine = rr < p.rows_per_cta;
      if (mine) {
        const int h = head * p.group + rr % p.group;
        const int64_t local = (int64_t)(rr / p.group) * p.hq + h;  // of the batch, or of the sequence
        at = p.shared ? (int64_t)split * p.rows_total + local
             : whole  ? (int64_t)bz * (p.n_q * p.hq) + local
                      : (int64_t)split * (p.n_q * p.hq) + local;
        mine = out_in_bounds(p, whole, split, whole ? at : local);
        if (mine && w == 0)
          (whole ? p.out_lse : p.shared ? p.pre_lse : p.own_lse)[at] =
              empty ? -INFINITY : (mx + log2f(den)) * 0.6931471805599453f;
      }
      float* parts = p.shared ? p.pre_o : p.own_o;
      // stream 1 wrote nothing where there is one tile: stream 0's half is then read from TMEM
      const uint32_t o_own = (two || w == 0) ? o_at + w * H : tmem + lanes + G::O_COL + H;
#pragma unroll
      for (int c = 0; c < H / 32; ++c) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(v, o_own + 32 * c);
        tmem_wait_ld();
        const float wv = two || w == 0 ? w0 : w1;  // the weight of what was read
        const bool hv = two || w == 0 ? has0 : has1;
        float o[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          o[i] = hv && wv != 0.f ? __uint_as_float(v[i]) * wv : 0.f;
          if (two && w1 != 0.f) o[i] = fmaf(hand[(1 - w) * H * kRows + (32 * c + i) * kRows + r], w1, o[i]);
        }
        const int64_t to = at * D + w * H + 32 * c;
        if (!mine) {
          // (no row: nothing to store)
        } else if (!whole || p.out_dtype == QPS_DT_F32) {
          float4* dst = reinterpret_cast<float4*>((whole ? reinterpret_cast<float*>(p.out) : parts) + to);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + to);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t x[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float a = o[8 * i + 2 * q], b = o[8 * i + 2 * q + 1];
              if (p.out_dtype == QPS_DT_F16) {
                x[q] = mma::pack_h2(a, b);
              } else {
                const __nv_bfloat162 hb = __floats2bfloat162_rn(a, b);
                x[q] = *reinterpret_cast<const uint32_t*>(&hb);
              }
            }
            dst[i] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      }
    }
    fence_before();
  }

  // ---- end: nothing may be in flight when the CTA leaves -----------------------------------------
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (*abort_flag) {  // (uniform: the flag is only set before the barrier above)
    // (one more bounded wait for each copy still under way: none may land after the CTA has gone)
    if (warp == 0) {
      const bool first = lane == 0 && report_give_up(p.err, *abort_flag, issued, ntiles, t1 - t0);
      const uint64_t since = global_ns();
      bool done = true;
#pragma unroll 1
      for (int i = max(0, issued - 2 * ST); i < issued; ++i) {  // K and V of a tile in turn
        const int j = i >> 1;
        done &= mma::mbar_wait(i & 1 ? v_full(j % ST) : k_full(j % ST), (j / ST) & 1, p.wait_ns);
      }
      if (first) {
        p.err[10] = (unsigned)min((uint64_t)0xffffffffu, global_ns() - since);
        p.err[11] = done ? 1u : 0u;
      }
    }
    if (warp == 1) mma::mbar_wait(all_done, 0, p.wait_ns);
    __syncthreads();
  }
  fence_after();
  if (warp == 2) tmem_free(tmem, 512);
}

template <int D, class P>
qps_status launch_tm(const P& p, cudaStream_t s) {
  using G = Geo<D>;
  static_assert(G::SMEM <= 227 * 1024, "the stages exceed the shared memory of one CTA");
  static_assert(G::O_COL + 2 * D <= 512, "S and O exceed TMEM");
  TmaSet maps;
  std::memset(&maps, 0, sizeof(maps));
  const int page = 1 << p.page_shift, rows = page < kTok ? page : kTok;
  for (int i = 0; i < 2; ++i)
    if (!encode_plane_map(i ? &maps.v : &maps.k, i ? p.v.data : p.k.data, 2 * D, page, p.hkv, page, (int)p.n_pages,
                          (int64_t)p.hkv * page, 128, 128, rows))
      return QPS_ERR_CUDA;
  auto kern = attn_tm_kernel<D, P>;
  static std::atomic<uint64_t> sized{0};
  int dev = 0;
  QPS_CUDA_TRY(cudaGetDevice(&dev));
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(sized.load(std::memory_order_relaxed) & bit) || !bit) {
    QPS_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM));
    sized.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.shared ? p.n_split : p.max_chunks) * ((p.rows_per_cta + kRows - 1) / kRows), p.hkv, 1);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = G::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  QPS_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, p, maps));
  count_launch();
  QPS_CUDA_TRY(cudaGetLastError());
  return QPS_OK;
}

}  // namespace tm
}  // namespace qps
