// Attention of prompt chunks over fp16 pages (or compressed rows decoded to fp16) on the
// fifth-generation tensor cores, causal, with or without a sliding window:
//     S = Q K^T          tcgen05.mma, Q and K in shared memory (K-major), S in TMEM (f32)
//     P = 2^(S' - m)     4 warps, one query row a thread: no reduction crosses lanes
//     O += P V           tcgen05.mma, P (fp16) in TMEM over the S it came from, V in shared
//                        memory as it lies in the page (MN-major), O in TMEM (f32)
// The rows of a CTA are the query tokens of one sequence times the heads of one KV head's group.
// At head_dim 64 and 128 there are two tiles of 128 rows (streams), each with an S, an O and
// softmax state of its own, so that one's exponentials run beside the other's products and every
// tile of K and V that is brought serves both.  At 256 and 512 O takes half of TMEM: one tile of
// rows, two buffers of S, so that S of the next tile is ready when P of this one is; at 512 two
// CTAs share a row, each computing all of S and half of O's columns.
//
// K and V pass through one ring of slots, [128 positions][SD columns] each, in the order of their
// first use; one stream gives a slot back when its products have run, two when the second's have
// (K and V of a tile are then held together: at most 4 of 5 slots).  A K that was compressed comes in two parts, the fp16 value and what its rounding
// left, whose products are summed: logits keep float32 accuracy.  So does a compressed V, but for
// a bf16 output: one part's rounding beside that of P made an fp16 output's error 1.7 times the
// one its type has (3.6e-4 against 2.1e-4), and is lost in bf16's.
//
// The running reference m of a row is set kRefShift (log2) below a tile's maximum, and again only
// when one exceeds what it was set for by more than kRefLazy (paged.h): P stays within fp16, and
// the rescale of O is rare.  P is rounded once to fp16 (the operand type); sums, m and O are
// float32.
//
// Roles: warp 0 brings the slots, warp 1 issues the products, warp 3 asks for the next CTA's queries,
// warps 4.. are the streams' softmax.  Waits are bounded as in attn_tm.cuh.
//
// Measured, 40 / 8 heads of 128, fp16: 16384 tokens 1757 to 1797 us by the device (1.53 to 1.56 PFLOP/s
// of useful products, 0.79 to 0.81 of the measured rate), 4096 tokens 142 to 153 us, behind a window of
// 1024 95 us; 4096 tokens of heads of 64 120 us, of 256 271 to 278 us; 2048 tokens behind 8192, 16 / 2
// heads of 512 with keys and values in two parts 1333 to 1345 us.  A tile of two streams takes 2614 cycles where its products take 2048; a CTA's start
// and end take 12000 to 13000.  Heads of 512: the products of queries and keys read 128 bytes a cycle
// of shared memory, its rate, beside the boxes that are written.
#pragma once

#include <atomic>
#include <cstring>

#include "attn_prompt.h"
#include "attn_tm.cuh"

namespace qps {
namespace prompt {

using namespace tm;

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 16 columns of the warp's 32 lanes
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}

template <int D, int KP, int VP>
struct GeoP {
  static constexpr int NQ = D <= 128 ? 2 : 1;      // tiles of rows
  // columns of a slot (64 at head_dim 512 too, in twice as many slots: 4096 tokens of q8_0 555 us for
  // 520, 2048 behind 8192 of q8_0 / tq3 1298 for 1337, so they gain in the one and lose more in the
  // other; at 256: 331 for 271; means of two runs a side)
  static constexpr int SD = D < 128 ? D : 128;
  static constexpr int VD = D <= 256 ? D : 256;    // columns of O
  static constexpr int CG = SD / 64;               // 128-byte column groups of a slot
  static constexpr int SLOT = kTok * SD * 2;
  static constexpr int KS = KP * D / SD, VC = VD / SD, VS = VP * VC;  // slots of a tile
  static constexpr int Q_TILE = kRows * D * 2;
  static constexpr int STAGES = D == 64 ? 10 : D == 512 ? 3 : 5;
  static constexpr int RING = NQ * Q_TILE;
  static constexpr int BAR = RING + STAGES * SLOT;
  static constexpr int SMEM = BAR + 256 + 1024;    // + slack for the 1024-byte base alignment
  static constexpr int THREADS = 128 + 128 * NQ;
  // two streams: registers a thread of the first warps and of the softmax (3 x 168 at launch)
  static constexpr int FEW = 72, MANY = 216;
  static constexpr int S_COL = 0, O_COL = 256;     // TMEM columns
};

template <int D, int KP, int VP>
__global__ void __launch_bounds__(GeoP<D, KP, VP>::THREADS, 1)
    attn_prompt_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ TmaSet maps) {
  using G = GeoP<D, KP, VP>;
  constexpr int ST = G::STAGES, NQ = G::NQ;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(smem);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  // ---- barriers, TMEM --------------------------------------------------------------------------
  const uint32_t bars = sbase + G::BAR;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (ST + s); };
  auto s_full = [&](int w) { return bars + 8 * (2 * ST + w); };
  auto p_ready = [&](int w, int h) { return bars + 8 * (2 * ST + 2 + 2 * w + h); };  // (half a tile's positions)
  const uint32_t q_full = bars + 8 * (2 * ST + 6), all_done = bars + 8 * (2 * ST + 7), pv_done = bars + 8 * (2 * ST + 8);
  static_assert(8 * (2 * ST + 9) <= 240, "barriers fit their region");
  uint32_t* tmem_word = reinterpret_cast<uint32_t*>(smem + G::BAR + 240);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + G::BAR + 244);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * ST + 9; ++i)
      mbar_init(bars + 8 * i, i == 2 * ST + 6 ? 4 * NQ : i >= 2 * ST + 2 && i < 2 * ST + 6 ? 4 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    *abort_flag = 0;
  }
  if (warp == 2) tmem_alloc(smem_addr(tmem_word), 512);
  // (Before the wait for the grid ahead: a CTA that starts early may hold TMEM, as a grid is let in only
  // when every CTA ahead of it has started, and those that use TMEM let it in behind their allocation.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- this CTA's rows and tiles -------------------------------------------------------------
  // CTA `idx` of the grid: KV head, half of O's columns, split, row tile (sequences in order, the last
  // rows of each first: they see the most).  Sequence -1: there are fewer row tiles.
  struct Work {
    int head, half, split, bz, row0, dense0;  // dense0: the sequence's first decoded tile
    PromptSeq sq;
  };
  auto find = [&](int idx) {
    Work k = {};
    k.head = idx % p.hkv;
    idx /= p.hkv;
    k.half = idx % (D / G::VD);
    idx /= D / G::VD;
    k.split = idx % p.n_split;
    idx /= p.n_split;
    k.bz = -1;
    int before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      PromptSeq mine = {0, 0, 0};
      if (b0 + lane < p.batch) mine = prompt_seq(p, b0 + lane);
      const int cnt = (int)(((int64_t)mine.n * p.group + NQ * kRows - 1) / (NQ * kRows));
      int sum = cnt;  // inclusive scan over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + sum > idx);
      const int src = hit ? __ffs(hit) - 1 : 32;
      if (p.dense_k || p.dense_v) {
        const int tiles = lane < src && mine.n > 0 ? prompt_tiles(p, mine.len - mine.n, mine.len - 1).count : 0;
        k.dense0 += __reduce_add_sync(0xffffffffu, tiles);
      }
      if (hit) {
        k.bz = b0 + src;
        k.sq.first = __shfl_sync(0xffffffffu, mine.first, src);
        k.sq.n = __shfl_sync(0xffffffffu, mine.n, src);
        k.sq.len = __shfl_sync(0xffffffffu, mine.len, src);
        k.row0 = (before + __shfl_sync(0xffffffffu, sum, src) - 1 - idx) * NQ * kRows;
        break;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    return k;
  };
  const Work work = find(blockIdx.x);
  const int head = work.head, half = work.half, split = work.split, bz = work.bz, row0 = work.row0, dense0 = work.dense0;
  const PromptSeq sq = work.sq;
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = uniform(*tmem_word);
  if (bz < 0) {  // more CTAs than row tiles (every warp finds the same)
    if (warp == 2) tmem_free(tmem, 512);
    return;
  }
  const int rows = min(NQ * kRows, (int)min((int64_t)sq.n * p.group - row0, (int64_t)NQ * kRows));
  const int pos0 = sq.len - sq.n;  // position of the sequence's first query token
  const int q_lo = pos0 + row0 / p.group, q_hi = pos0 + (row0 + rows - 1) / p.group;
  const PromptTiles all = prompt_tiles(p, q_lo, q_hi);
  const PromptTiles dense = prompt_tiles(p, pos0, sq.len - 1);
  const int i0 = (int)((int64_t)all.count * split / p.n_split), i1 = (int)((int64_t)all.count * (split + 1) / p.n_split);
  const int ntiles = uniform(i1 - i0);
  const int end = q_hi + 1;                                       // no row sees a position from here on
  const int none_lo = p.window ? max(0, q_lo - p.window + 1) : 0; // nor any of [sinks, none_lo)
  const int live = uniform(NQ == 1 || rows > kRows ? NQ : 1);     // streams that have rows
  auto first_of = [&](int j) { return prompt_tile(all, i0 + j) * kPromptTile; };

  int issued = 0;  // (warp 0) slots under way or landed
  auto wait = [&](uint32_t bar, uint32_t parity, int tile) -> bool {  // (as in attn_tm.cuh)
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
  // Places of the tiles' slots in the ring's order: K(0), V(0), K(1), V(1), .. where a tile of K
  // serves two streams before V(j) does, else K(0), K(1), V(0), K(2), V(1), .. (S of the next
  // tile is issued before O of this one).
  constexpr int KV = G::KS + G::VS;
  auto k_at = [&](int j) { return NQ == 2 || j == 0 ? j * KV : G::KS + (j - 1) * KV; };
  auto v_at = [&](int j) { return NQ == 2 ? j * KV + G::KS : G::KS + j * KV + (j + 1 < ntiles ? G::KS : 0); };

  if (warp < 4) {
    if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::FEW));
    if (warp == 0) {
      // ---- slots: boxes of min(page, 128) positions of one page and 64 columns, one a lane; a
      // lane's page of the next tile is read a tile ahead.  Decoded rows: boxes of 128 positions. ----
      const int br = min(1 << p.page_shift, kTok), nb = kTok / br;
      const int cg = lane % G::CG, r = lane / G::CG;
      const int32_t* row = p.table + (int64_t)bz * p.table_stride;
      const bool paged = !p.dense_k || !p.dense_v;
      auto entry = [&](int j) -> int {  // the lane's page of tile j (n_pages: none, zeros)
        if (!paged || j >= ntiles || r >= nb) return (int)p.n_pages;
        const int t = first_of(j) + r * br;
        if (t >= end || (t >= p.sinks && t + br <= none_lo)) return (int)p.n_pages;
        const int at = t >> p.page_shift;
        if (!in_bounds(at < p.table_width, p.err)) return (int)p.n_pages;
        const int pg = row[at];
        if ((uint64_t)(int64_t)pg < (uint64_t)p.n_pages) return pg;
        atomicOr(p.err, kErrIndex);
        return (int)p.n_pages;
      };
      int f = 0;
      auto put = [&](const TensorMap* map, bool dec, int col, int j, int page) -> bool {
        const int s = f % ST;
        if (f >= ST && !wait(empty(s), ((f / ST) & 1) ^ 1, j)) return false;
        __syncwarp();
        if (lane == 0) mbar_expect_tx(full(s), G::SLOT);
        __syncwarp();
        const uint32_t dst = sbase + G::RING + s * G::SLOT + cg * (kTok * 128);
        const int x = (col + cg * 64) * 2, t = first_of(j);
        const bool drop = map == &maps.k && j == p.drop_tile;
        if (dec) {  // (behind the room: zeros)
          const int at = prompt_dense(dense, t / kPromptTile);
          if (r == 0 && !drop && in_bounds(at >= 0 && G::RING + (s + 1) * G::SLOT <= G::BAR, p.err))
            tma_load_4d(dst, map, x, 0, head, min(dense0 + at, p.dense_tiles), full(s));
        } else if (r < nb && !drop) {
          const int y = (t + r * br) & ((1 << p.page_shift) - 1);
          if (in_bounds(page <= p.n_pages && y + br <= 1 << p.page_shift && head < p.hkv && G::RING + (s + 1) * G::SLOT <= G::BAR, p.err))
            tma_load_4d(dst + r * br * 128, map, x, y, head, page, full(s));
        }
        issued = ++f;
        return true;
      };
      auto put_k = [&](int j, int page) -> bool {
        for (int s = 0; s < G::KS; ++s)
          if (!put(&maps.k, p.dense_k != nullptr, s * G::SD, j, page)) return false;
        return true;
      };
      auto put_v = [&](int j, int page) -> bool {
        for (int s = 0; s < G::VS; ++s)
          if (!put(&maps.v, p.dense_v != nullptr, s / G::VC * D + half * G::VD + s % G::VC * G::SD, j, page)) return false;
        return true;
      };
      int page = entry(0), next = entry(1);
      // (the first tile, then the queries: the whole ring before them kept them 1500 cycles longer)
      bool ok = ntiles == 0 || (put_k(0, page) && (NQ == 1 || put_v(0, page)) && wait(q_full, 0, 0));
      for (int j = 0; j < ntiles && ok; ++j) {
        const int after = entry(j + 2);
        if constexpr (NQ == 2) ok = j == 0 || (put_k(j, page) && put_v(j, page));
        else ok = (j + 1 >= ntiles || put_k(j + 1, next)) && put_v(j, page);
        page = next;
        next = after;
      }
    } else if (warp == 1) {
      // ---- products: step i is tile i / NQ of stream i % NQ, S(i) in buffer i % 2.  S(0), S(1),
      // then O(i) and S(i + 2) in turn. ------------------------------------------------------------
      constexpr uint32_t ID_S = instr_desc(kTok, 0), ID_O = instr_desc(G::SD, 1);
      const uint32_t one = elect_lane();
      const int steps = ntiles * NQ;
      auto qk = [&](int i) -> bool {
        const int j = i / NQ, w = i % NQ, at = k_at(j);
        const uint32_t d = tmem + G::S_COL + (i & 1) * kTok;
#pragma unroll 1
        for (int s = 0; s < G::KS; ++s) {
          const int st = (at + s) % ST;
          if (w == 0 && !wait(full(st), ((at + s) / ST) & 1, j)) return false;
          fence_after();
          if (w < live) {
            const uint64_t a = smem_desc(sbase + w * G::Q_TILE + (s * G::CG % (D / 64)) * (kRows * 128), 16);
            const uint64_t b = smem_desc(sbase + G::RING + st * G::SLOT, 16);
#pragma unroll
            for (int kk = 0; kk < G::SD / 16; ++kk) {
              const uint64_t off = ((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4;
              mma_ss(d, a + off, b + off, ID_S, s > 0 || kk > 0, one);
            }
          }
          if (w == NQ - 1) commit(empty(st), one);
        }
        commit(s_full(i & 1), one);
        return true;
      };
      bool ok = steps == 0 || wait(q_full, 0, 0);
      for (int i = 0; i < min(2, steps) && ok; ++i) ok = qk(i);
      for (int i = 0; i < steps && ok; ++i) {
        const int j = i / NQ, w = i % NQ, at = v_at(j);
        // (rows that no query sees hold whatever was there, and 0 x NaN is NaN)
        const int t = first_of(j), a0 = max(0, p.sinks - t), a1 = min(kTok, none_lo - t), b0 = end - t;
#pragma unroll 1
        for (int s = 0; s < G::VS && ok; ++s) {
          const int st = (at + s) % ST;
          if (w == 0) {
            if (!(ok = wait(full(st), ((at + s) / ST) & 1, j))) break;
            if (b0 < kTok || a0 < a1) {
              for (int r = lane >> 3; r < kTok; r += 4)
                if (r >= b0 || (r >= a0 && r < a1))
#pragma unroll
                  for (int g = 0; g < G::CG; ++g)
                    *reinterpret_cast<uint4*>(smem + G::RING + st * G::SLOT + g * (kTok * 128) + r * 128 + (lane & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
              mma::fence_proxy_async();
              __syncwarp();
            }
          }
          const uint32_t d = tmem + G::O_COL + w * D + s % G::VC * G::SD, a = tmem + G::S_COL + (i & 1) * kTok;
          const uint64_t b = smem_desc(sbase + G::RING + st * G::SLOT, kTok * 128);
          const uint32_t more = j > 0 || s >= G::VC;  // (0: a stream's first product starts its O)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (w >= live) continue;
            if (s == 0 && !(ok = wait(p_ready(i & 1, h), NQ == 2 ? j & 1 : (j >> 1) & 1, j))) break;
            fence_after();
#pragma unroll
            for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
              mma_ts(d, a + kk * 8, b + (uint64_t)((kk * 2048) >> 4), ID_O, more | (kk > 0), one);
          }
          if (ok && w == NQ - 1) commit(empty(st), one);
        }
        if (!ok) break;
        if constexpr (NQ == 1) commit(pv_done, one);
        if (i + 2 < steps) ok = qk(i + 2);
      }
      commit(all_done, one);  // completes when everything issued above has
    } else if (warp == 3) {
      // ---- the queries of the CTA that follows on this SM, about, into L2 (from HBM they took 5200
      // cycles of a CTA's start) -------------------------------------------------------------------
      const int next = blockIdx.x + p.resident;
      const Work k = next < (int)gridDim.x && p.group <= NQ * kRows ? find(next) : Work{0, 0, 0, -1, 0, 0, {0, 0, 0}};
      if (k.bz >= 0) {
        const int t0 = k.row0 / p.group, t1 = (int)min((int64_t)k.sq.n - 1, ((int64_t)k.row0 + NQ * kRows - 1) / p.group);
        const int lines = (p.group * D * 2 + 127) / 128;
        for (int i = lane; i < (t1 - t0 + 1) * lines; i += 32) {
          const int64_t at = (int64_t)(k.sq.first + t0 + i / lines) * p.q_tok + (int64_t)k.head * p.group * D + min(i % lines * 64, p.group * D - 8);
          if (in_bounds(k.sq.first + t0 + i / lines < p.tokens, p.err)) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + at));
        }
      }
    }
  } else {
    if constexpr (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::MANY));
    // ---- softmax: stream w, one row a thread --------------------------------------------------
    const int w = (warp - 4) >> 2, r = (warp & 3) * 32 + lane, rr = w * kRows + r;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const uint32_t o_at = tmem + lanes + G::O_COL + w * D;
    const bool mine = rr < rows;
    // the row's query token, counted from the CTA's first, and head
    const int t_first = row0 / p.group, tok = (row0 + rr) / p.group - t_first, h = head * p.group + (row0 + rr) % p.group;
    {
      // Q [128][D] of the stream, K-major: row r's 16-byte chunk c of a column group at r * 128 +
      // (c ^ r % 8) * 16; each warp its own 32 rows, the loads of one round together
      constexpr int N = D / 8, U = N < 16 ? N : 16;
#pragma unroll 1
      for (int k0 = 0; k0 < N; k0 += U) {
        uint4 v[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int i = (k0 + k) * 32 + lane, qr = i / (D / 8), c = i % (D / 8);
          const int qt = __shfl_sync(0xffffffffu, tok, qr), qh = __shfl_sync(0xffffffffu, h, qr);
          v[k] = make_uint4(0, 0, 0, 0);
          if (w * kRows + (warp & 3) * 32 + qr < rows) {
            const int64_t t = (int64_t)sq.first + t_first + qt;
            if (in_bounds(t < p.tokens && qh < p.hq, p.err)) v[k] = *reinterpret_cast<const uint4*>(p.q + t * p.q_tok + qh * D + c * 8);
          }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int i = (k0 + k) * 32 + lane, qr = (warp & 3) * 32 + i / (D / 8), c = i % (D / 8);
          *reinterpret_cast<uint4*>(smem + w * G::Q_TILE + (c >> 3) * (kRows * 128) + qr * 128 + (((c & 7) ^ (qr & 7)) << 4)) = v[k];
        }
      }
      mma::fence_proxy_async();
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(q_full) : "memory");
    }
    // positions below lim are visible to the row, but for [sinks, low)
    const int lim = mine ? pos0 + t_first + tok + 1 : 0, low = p.window ? lim - p.window : 0;
    constexpr float LOG2E = 1.4426950408889634f;
    const float qs = p.scale * LOG2E, cap = p.softcap, cap_k = cap > 0.f ? 2.f * LOG2E / cap * p.scale : 0.f;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < ntiles && w < live; ++j) {
      const int buf = NQ == 2 ? w : j & 1, par = NQ == 2 ? j & 1 : (j >> 1) & 1;
      const uint32_t s_at = tmem + lanes + G::S_COL + buf * kTok;
      if (!(ok = wait(s_full(buf), par, j))) break;
      fence_after();
      // the row's 128 logits, in registers
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(v[c], s_at + 32 * c);
      tmem_wait_ld();
      float f = qs;  // from here on logits, in units of log2, are f v
      if (cap > 0.f) {  // c tanh(x / c) = c - 2 c / (1 + e^(2 x / c))
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(__uint_as_float(v[c][i]) * cap_k)));
            v[c][i] = __float_as_uint(fmaf(-2.f * LOG2E * cap, r, LOG2E * cap));
          }
        f = 1.f;
      } else if (!(qs > 0.f)) {  // (the maximum below is of v)
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) v[c][i] = __float_as_uint(__uint_as_float(v[c][i]) * qs);
        f = 1.f;
      }
      const int first = first_of(j);
      if (__any_sync(0xffffffffu, first + kTok > lim)) {
        const int b0 = lim - first;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i >= b0) v[c][i] = 0xff800000u;
      }
      if (__any_sync(0xffffffffu, first < low && first + kTok > p.sinks)) {
        const int b1 = low - first, b2 = p.sinks - first;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i < b1 && 32 * c + i >= b2) v[c][i] = 0xff800000u;
      }
      // Exponentials of the first half against the present reference, before the maximum is known:
      // it is rarely raised, and the two then run beside each other (in turn, the products waited
      // 360 cycles a tile for them).
      float ms = m == -INFINITY ? 0.f : m;
      uint64_t sum[2];
      uint32_t pk[2][16];
      auto weigh = [&](const uint32_t (&x)[32], uint32_t (&o)[16]) {
        const uint64_t f2 = pack2(f, f), m2 = pack2(-ms, -ms);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 y = unpack2(fma2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), f2, m2));
          const float a = ex2(y.x), b = ex2(y.y);
          sum[i & 1] = add2(sum[i & 1], pack2(a, b));
          o[i] = mma::pack_h2(a, b);
        }
      };
      sum[0] = sum[1] = 0;
      weigh(v[0], pk[0]);
      weigh(v[1], pk[1]);
      float mm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // (a NaN is no maximum)
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) mm[k] = max3(mm[k], __uint_as_float(v[c][i + k]), __uint_as_float(v[c][i + 4 + k]));
      const float mx = fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3])) * f - kRefShift;
      const bool raise = mx - m > kRefLazy;  // (false when both are -inf)
      if (__any_sync(0xffffffffu, raise)) {
        const float cr = raise ? ex2(m - mx) : 1.f;  // (0 from -inf)
        if (raise) {
          m = mx;
          l *= cr;
        }
        if (j > 0) {
          // two streams: S of this tile was issued behind this stream's last product, so O is at
          // rest; one: the last product may still run
          if constexpr (NQ == 1) {
            if (!(ok = wait(pv_done, (j - 1) & 1, j))) break;
            fence_after();
          }
#pragma unroll 1
          for (int c = 0; c < G::VD / 16; ++c) {
            uint32_t o[16];
            __syncwarp();
            tmem_ld16(o, o_at + 16 * c);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * cr);
            tmem_st16(o_at + 16 * c, o);
          }
        }
        ms = m == -INFINITY ? 0.f : m;
        sum[0] = sum[1] = 0;
        weigh(v[0], pk[0]);
        weigh(v[1], pk[1]);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (hf) {
          weigh(v[2], pk[0]);
          weigh(v[3], pk[1]);
        }
        tmem_st16(s_at + 32 * hf, pk[0]);
        tmem_st16(s_at + 32 * hf + 16, pk[1]);
        tmem_wait_st();  // half of the positions: the product with their values may start
        fence_before();
        __syncwarp();
        if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(p_ready(buf, hf)) : "memory");
      }
      const float2 s2 = unpack2(add2(sum[0], sum[1]));
      l += s2.x + s2.y;
    }
    // ---- the rows' output, or their part of it: through shared memory (the ring, all of whose slots
    // have been used), each warp its own rows, and out as whole lines (from the registers, a row a lane,
    // 7200 cycles; as a bulk copy a row 3900) ---------------------------------------------------------
    if (ok) ok = wait(all_done, 0, ntiles);
    fence_after();
    if (ok && !__any_sync(0xffffffffu, *abort_flag)) {
      constexpr int PC = G::VD < 128 ? G::VD : 128;  // columns at a time
      const bool none = l == 0.f;  // (a NaN stays one)
      const float inv = none ? 0.f : 1.f / l;
      const bool whole = p.n_split == 1, wide = !whole || p.out_dtype == QPS_DT_F32;
      const int64_t at = ((int64_t)sq.first + t_first + tok) * p.hq + h;
      const bool store = mine && in_bounds(at < p.tokens * p.hq, p.err);
      const int64_t to = whole ? at : (int64_t)split * p.tokens * p.hq + at;
      if (store && half == 0) (whole ? p.out_lse : p.part_lse)[to] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      // (16 bytes between rows: the 32 rows' chunks fall on all banks)
      const uint32_t bytes = PC * (wide ? 4 : 2);
      uint8_t* row = smem + G::RING + (uint32_t)(w * kRows + r) * (bytes + 16);
      static_assert(NQ * kRows * (PC * 4 + 16) <= ST * G::SLOT, "the rows fit the ring");
#pragma unroll 1
      for (int x = 0; x < G::VD; x += PC) {
#pragma unroll
        for (int c = 0; c < PC / 32; ++c) {
          uint32_t v[32];
          __syncwarp();
          if (ntiles > 0 && w < live) {
            tmem_ld32(v, o_at + x + 32 * c);
            tmem_wait_ld();
          }
          float o[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : __uint_as_float(v[i]) * inv;
          if (wide) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(row + 128 * c + 16 * i) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t y[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float a = o[8 * i + 2 * q], b = o[8 * i + 2 * q + 1];
                if (p.out_dtype == QPS_DT_F16) {
                  y[q] = mma::pack_h2(a, b);
                } else {
                  const __nv_bfloat162 hb = __floats2bfloat162_rn(a, b);
                  y[q] = *reinterpret_cast<const uint32_t*>(&hb);
                }
              }
              *reinterpret_cast<uint4*>(row + 64 * c + 16 * i) = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
        }
        __syncwarp();
        const uint32_t to32 = (uint32_t)(store ? to : 0);
        const uint8_t* rows32 = row - lane * (bytes + 16);
        auto copy_out = [&](auto size) {  // 32 rows of PC values of `size` bytes
          constexpr int S = decltype(size)::value, CHUNKS = PC * S / 16;
          uint8_t* const out = reinterpret_cast<uint8_t*>(whole ? p.out : p.part_o) + (half * G::VD + x) * S;
#pragma unroll 8
          for (int k = 0; k < CHUNKS; ++k) {
            const int i = k * 32 + lane, rr = i / CHUNKS, c = i % CHUNKS;
            const int64_t dst = __shfl_sync(0xffffffffu, to32, rr);
            if (__shfl_sync(0xffffffffu, (int)store, rr))
              *reinterpret_cast<uint4*>(out + dst * (D * S) + 16 * c) = *reinterpret_cast<const uint4*>(rows32 + rr * (PC * S + 16) + 16 * c);
          }
        };
        if (wide) copy_out(std::integral_constant<int, 4>{});
        else copy_out(std::integral_constant<int, 2>{});
        __syncwarp();
      }
    }
    fence_before();
  }

  // ---- end: nothing may be in flight when the CTA leaves -----------------------------------------
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (*abort_flag) {  // (uniform: the flag is only set before the barrier above)
    if (warp == 0) {
      const bool first = lane == 0 && report_give_up(p.err, *abort_flag, issued, ntiles, ntiles * kTok);
      const uint64_t since = global_ns();
      bool done = true;
#pragma unroll 1
      for (int f = max(0, issued - ST); f < issued; ++f) done &= mma::mbar_wait(full(f % ST), (f / ST) & 1, p.wait_ns);
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

template <int D, int KP, int VP>
qps_status launch_prompt(const PromptParams& p, cudaStream_t s) {
  using G = GeoP<D, KP, VP>;
  static_assert(G::NQ == 1 || G::FEW + 2 * G::MANY <= 3 * 168, "the registers of three warpgroups at launch");
  static_assert(G::SMEM <= 227 * 1024, "the slots exceed the shared memory of one CTA");
  static_assert(G::O_COL + G::NQ * G::VD <= 512, "S and O exceed TMEM");
  TmaSet maps;
  std::memset(&maps, 0, sizeof(maps));
  const int page = 1 << p.page_shift, rows = page < kTok ? page : kTok;
  for (int i = 0; i < 2; ++i) {
    const __half* dense = i ? p.dense_v : p.dense_k;
    const int cols = (i ? VP : KP) * D;
    const bool ok = dense ? encode_plane_map(i ? &maps.v : &maps.k, dense, 2 * cols, kTok, p.hkv, kTok, p.dense_tiles,
                                             (int64_t)p.hkv * kTok, 128, 128, kTok)
                          : encode_plane_map(i ? &maps.v : &maps.k, i ? p.v[0] : p.k[0], 2 * D, page, p.hkv, page, (int)p.n_pages,
                                             (int64_t)p.hkv * page, 128, 128, rows);
    if (!ok) return QPS_ERR_CUDA;
  }
  auto kern = attn_prompt_kernel<D, KP, VP>;
  static std::atomic<uint64_t> sized{0};
  int dev = 0;
  QPS_CUDA_TRY(cudaGetDevice(&dev));
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(sized.load(std::memory_order_relaxed) & bit) || !bit) {
    QPS_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM));
    // (the split draws on the registers of the launch: with fewer, the softmax warps would wait for ever)
    cudaFuncAttributes fa;
    QPS_CUDA_TRY(cudaFuncGetAttributes(&fa, kern));
    if (G::NQ == 2 && 3 * fa.numRegs < G::FEW + 2 * G::MANY)
      return fail(QPS_ERR_INTERNAL, "attn_prompt_paged: the kernel was built with too few registers for its split");
    sized.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.tiles * p.n_split * (D / G::VD) * p.hkv));
  cfg.blockDim = dim3(G::THREADS);
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

}  // namespace prompt
}  // namespace qps
