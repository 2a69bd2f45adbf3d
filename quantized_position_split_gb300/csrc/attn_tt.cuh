// Decode attention of many query rows, up to 64 a CTA, on the fifth-generation tensor cores,
// over pages of head_dim 128, 256 and 512 with K F16 / Q8_0 and V F16 / Q8_0 / TQ3 / TQ2 (but
// F16 / F16 at 128, which is attn_tm.cuh's): verify batches and shared prefixes of compressed
// caches, where the products on the older path (mma.sync, 8 rows a warp) decode the same
// positions again for every 8 to 24 rows, as they still do for a TurboQuant K, a TQ4 V and
// compressed rows of head_dim 64.
//
// The products run with the positions and the head dimension on the wide side (M = 128)
// and the query rows on the narrow one (N = 16 .. 64), so their time follows the number of
// rows:
//     S^T [128 positions][N] = K Q^T      A = K (TMEM), B = Q (shared, K-major), per 64 dims
//     P   = 2^(S' - m)                    one position and 32 rows a thread
//     O^T [128 dims][N]     += V^T P^T    A = V (shared, MN-major, as stored), B = P (MN-major)
// S^T (two buffers), O^T (D / 128 blocks) and two slots of K live in TMEM; S^T of the next
// tile and O^T of the last one are issued in turn, as their slots are decoded.
//
// The stored rows arrive by tensor-map boxes in small raw stages; four warps decode K, one
// position a thread, from there into TMEM (64 dims a slot), four more V into 32 KB slots of
// fp16 operands (128 dims; fp16 values are boxed there as they are).  K by way of shared
// memory slots too, a tile took 17000 cycles at head_dim 512: 8600 of shared-memory traffic
// and most of the rest in the decoding warps' waits.  Numerics: a q8_0 key (code x scale)
// is its hi + lo fp16 parts, two products, so logits keep float32 accuracy (where a
// position's scales reach 2^8 they are halved until its products fit fp16, and its logits
// doubled back: a key of fp16's largest value is stored as 127 x 516 = 65532); a TurboQuant V
// is its exact fp16 levels in the rotated domain with the norm folded into P before P's one
// rounding (and into the reference that P x norm is held against), the output being rotated
// back once; a q8_0 V is rounded once to fp16; sums,
// maxima and O are float32.
//
// A row's maximum over the positions would cross all threads, so the running reference m
// (in shared memory) is raised only when some operand would leave the room above it (paged.h):
// one vote a tile, and on a raise the maxima are taken, O and the sums rescaled.
//
// Measured: four sequences of five tokens and 30000 to 32768 positions, two KV heads of 512,
// q8_0 / tq3 (40 rows): 87 us, 2.1 TB/s.  57% of the issue slots are used and the tensor pipe
// runs 20% of the time: no unit is at its limit, the roles wait for one another (each tile's
// softmax behind its page and norm loads and two readings of S).
//
// Roles: warp 0 issues the products, warps 2 and 3 the boxes of K and V, warps 4-11 are the
// softmax (two groups of rows), 12-15 decode K and 16-19 V.  Waits are bounded as in
// attn_tm.cuh.
#pragma once

#include "attn_tm.cuh"

namespace qps {
namespace tt {

using namespace tm;

constexpr int kN = 64;             // query rows per CTA
constexpr int kTile = 128;         // positions per tile
constexpr int kThreadsTt = 640;
constexpr int kSlot = 32 * 1024;  // a slot of V's fp16 operands
constexpr int kPBytes = kTile * kN * 2;  // a buffer of P
// -m of a row without a reference: any finite logit is far above it, and 2^(-inf + it) is 0
constexpr float kNone = 0x1p126f;

template <int D, int KF, int VF>
struct GeoTt {
  static constexpr int KC = D / 64, VC = D / 128;   // slots of a tile: K's and V's
  static constexpr int Q_BYTES = kN * D * 2;
  // P: two buffers [128][64] fp16, for a q8_0 V with what the rounding left beside them (V's
  // values are rounded already, and a second rounding of the same size would make the
  // output's error 1.7 times the one its type has)
  static constexpr int PLO = VF == QPS_FMT_Q8_0 ? 1 : 0;
  static constexpr int P_OFF = Q_BYTES, P_STEP = (1 + PLO) * kPBytes;
  static constexpr int RING = P_OFF + 2 * P_STEP;
  static constexpr int SLOTS = PLO ? 2 : 3;         // of V
  // raw stages: [128 positions] of 64 dims of K (codes, or fp16), of 128 of V (codes, or the
  // 2-bit plane and behind it the signs)
  static constexpr int RAW_BYTES = (D == 128 ? 32 : 16) * 1024;  // of each side
  static constexpr int KSTAGE = (KF == QPS_FMT_F16 ? 16 : 8) * 1024, KN = RAW_BYTES / KSTAGE;
  static constexpr int VSTAGE = (VF == QPS_FMT_Q8_0 ? 16 : 8) * 1024, VN = RAW_BYTES / VSTAGE;
  static constexpr int KRAW = RING + SLOTS * kSlot, VRAW = KRAW + RAW_BYTES;
  static constexpr int MISC = VRAW + RAW_BYTES;
  static constexpr int EXPS = D == 128 ? 4 : 2;     // buffers of the positions' exponents
  static constexpr int MISC_BYTES = D == 128 ? 2560 : 2048;
  static constexpr int SMEM = MISC + MISC_BYTES + 1024;  // + slack for the 1024-byte base alignment
};

// Position in a 16-column word of a TurboQuant V -> column: the decode yields the columns
// j, j + 4, j + 8, j + 12 of step j.
__device__ __forceinline__ int tq_unswap(int pos) { return (pos >> 2) + 4 * (pos & 3); }

template <int D, int KF, int VF>
__global__ void __launch_bounds__(kThreadsTt, 1)
    attn_tt_kernel(const __grid_constant__ PagedAttnParams p, const __grid_constant__ TmaSet maps) {
  using G = GeoTt<D, KF, VF>;
  constexpr bool VDEC = VF != QPS_FMT_F16;  // V is decoded, or boxed into the slots
  constexpr float LOG2E = 1.4426950408889634f;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(smem);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- this CTA's rows and positions ------------------------------------------------------
  const int rtiles = (p.rows_per_cta + kN - 1) / kN;
  const int split = blockIdx.x / rtiles, row0 = (blockIdx.x % rtiles) * kN;
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
  const int ntiles = uniform(t1 > t0 ? (t1 - t0 + kTile - 1) / kTile : 0);  // 0: no own positions
  const int nrows = min(kN, p.rows_per_cta - row0);
  const int n16 = uniform((nrows + 15) & ~15);  // N of the products
  // TMEM columns: S (two buffers), K (two slots of 32 hi and 32 lo), O
  const int k_col = 2 * n16, o_col = k_col + 128;

  // ---- barriers, TMEM, queries, row state ----------------------------------------------------
  uint8_t* misc = smem + G::MISC;
  float* mneg = reinterpret_cast<float*>(misc);           // [64] -m (kNone: no reference yet)
  int* lim = reinterpret_cast<int*>(misc + 256);          // [64] positions below it are visible
  int* red = reinterpret_cast<int*>(misc + 512);          // [4][64] maxima, then sums
  // [EXPS][128] how often a position's q8_0 scales were halved.  A tile's are written when its
  // buffer's last reader is known to be done: S of two tiles ago (four buffers, the tile's first
  // slot), or a slot of S of the same tile (two buffers, its third slot) has been issued, and
  // each S waits for P of two tiles before it.
  uint8_t* kexp = misc + 1536;
  constexpr int TAIL = 1536 + G::EXPS * kTile;
  uint32_t* tmem_word = reinterpret_cast<uint32_t*>(misc + TAIL);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + TAIL + 4);
  const uint32_t bars = sbase + G::MISC + TAIL + 8;
  constexpr int KN = G::KN, VN = G::VN, kSlots = G::SLOTS;
  auto bar_at = [&](int i) { return bars + 8 * i; };
  auto s_full = [&](int w) { return bar_at(w); };
  auto p_free = [&](int w) { return bar_at(2 + w); };
  const uint32_t all_done = bar_at(4);
  auto k_empty = [&](int s) { return bar_at(5 + s); };           // TMEM slots of K
  auto v_empty = [&](int s) { return bar_at(7 + s); };           // slots of V
  auto kraw_full = [&](int s) { return bar_at(7 + kSlots + s); };
  auto vraw_full = [&](int s) { return bar_at(7 + kSlots + KN + s); };
  constexpr int ONES = 7 + kSlots + KN + VN;                      // the barriers above count one, those below four
  auto p_ready = [&](int w) { return bar_at(ONES + w); };         // (p_ready, q_full: eight)
  const uint32_t q_full = bar_at(ONES + 2);
  auto k_full = [&](int s) { return bar_at(ONES + 3 + s); };
  auto v_full = [&](int s) { return bar_at(ONES + 5 + s); };
  auto kraw_empty = [&](int s) { return bar_at(ONES + 5 + kSlots + s); };
  auto vraw_empty = [&](int s) { return bar_at(ONES + 5 + kSlots + KN + s); };
  constexpr int NBARS = ONES + 5 + kSlots + KN + VN;
  static_assert(TAIL + 8 + 8 * NBARS <= G::MISC_BYTES, "the row state and barriers fit their region");
  if (threadIdx.x == 0) {
    for (int i = 0; i < NBARS; ++i) mbar_init(bar_at(i), i < ONES ? 1 : i < ONES + 3 ? 8 : 4);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    *abort_flag = 0;
  }
  if (warp == 1) tmem_alloc(smem_addr(tmem_word), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = uniform(*tmem_word);

  int issued = 0;  // (warps 2, 3) stages or slots boxed
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
  auto arrive = [&](uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
  };

  if (warp == 0) {
    // ---- products: S(0), S(1), then S(j + 1) beside O(j - 1), while the softmax of tile j runs:
    // two slots of K, then one of V.  (S(j + 1), then O(j), each waiting for its decoders in
    // turn, took 4% longer at head_dim 512; four slots, then two, 2%.) ----
    const uint32_t id_s = instr_desc(n16, 0), id_o = instr_desc(n16, 1) | (1u << 15), one = elect_lane();
    int fk = 0, fv = 0;  // slots used
    bool ok = ntiles == 0 || wait(q_full, 0, 0);
    for (int j = -1; j <= ntiles && ntiles > 0 && ok; ++j) {
      const bool qk = j + 1 < ntiles, pv = j >= 1;
      // (P of tile j - 1 is there: its S, whose buffer S(j + 1) takes, has been read)
      if (pv && !(ok = wait(p_ready((j - 1) & 1), ((j - 1) >> 1) & 1, j))) break;
      const uint32_t ds = tmem + ((j + 1) & 1) * n16;
      const uint64_t bp = smem_desc(sbase + G::P_OFF + ((j - 1) & 1) * G::P_STEP, 16);
#pragma unroll 1
      for (int u = 0; u < G::VC && ok; ++u) {
        if (qk) {
#pragma unroll 1
          for (int c = 2 * u; c < 2 * u + 2; ++c, ++fk) {
            const int s = fk & 1;
            if (!(ok = wait(k_full(s), (fk >> 1) & 1, j))) break;
            fence_after();
            const uint32_t a = tmem + k_col + s * 64;
            const uint64_t bq = smem_desc(sbase + c * (kN * 128), 16);
            const uint32_t fresh = c > 0;  // (0: a tile's first product starts its accumulator)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t b = bq + (uint64_t)(kk * 2);
              if constexpr (KF == QPS_FMT_Q8_0) {
                mma_ts(ds, a + kk * 8, b, id_s, fresh | (kk > 0), one);
                mma_ts(ds, a + 32 + kk * 8, b, id_s, 1, one);
              } else {
                mma_ts(ds, a + kk * 8, b, id_s, fresh | (kk > 0), one);
              }
            }
            commit(k_empty(s), one);
            if (c == G::KC - 1) commit(s_full((j + 1) & 1), one);
          }
        }
        if (pv && ok) {
          const int s = fv % kSlots;
          if (!(ok = wait(v_full(s), (fv / kSlots) & 1, j))) break;
          if constexpr (!VDEC) {
            // fp16 rows behind the end hold whatever was there, and 0 x NaN is NaN
            const int left = t1 - (t0 + (j - 1) * kTile);
            if (left < kTile) {
              for (int i = left * 8 + lane; i < kTile * 8; i += 32)
#pragma unroll
                for (int g = 0; g < 2; ++g)
                  *reinterpret_cast<uint4*>(smem + G::RING + s * kSlot + g * (kSlot / 2) + i * 16) = make_uint4(0, 0, 0, 0);
              mma::fence_proxy_async();
              __syncwarp();
            }
          }
          const uint64_t a = smem_desc(sbase + G::RING + s * kSlot, kSlot / 2);
          fence_after();
#pragma unroll
          for (int part = 0; part <= G::PLO; ++part)
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk) {
              const uint64_t o = (uint64_t)((kk * 2048) >> 4);
              mma_ss(tmem + o_col + u * n16, a + o, bp + o + (uint64_t)((part * kPBytes) >> 4), id_o, j > 1 || kk > 0 || part > 0,
                     one);
            }
          commit(v_empty(s), one);
          ++fv;
          if (u == G::VC - 1) commit(p_free((j - 1) & 1), one);
        }
      }
    }
    commit(all_done, one);
    wait(all_done, 0, ntiles);
  } else if (warp == 2 || warp == 3) {
    // ---- boxes of min(page, 128) positions, K's (warp 2) and V's (warp 3), each lane's page read
    // a tile ahead -------------------------------------------------------------------------------
    const bool v = warp == 3;
    const int br = min(1 << p.page_shift, kTile), nb = kTile / br;
    const int32_t* table = p.table + (int64_t)bz * p.table_stride;
    // bytes of a position's row in a box; V: column groups of a slot, signs behind the codes
    const int rb = v ? (VF == QPS_FMT_F16 || VF == QPS_FMT_Q8_0 ? 128 : 32) : (KF == QPS_FMT_F16 ? 128 : 64);
    const int groups = v && !VDEC ? 2 : 1;
    const bool signs = v && VF == QPS_FMT_TQ3;
    const int ring = !v ? KN : VDEC ? VN : kSlots, nc = v ? G::VC : G::KC, count = ntiles * nc;
    const int grp = lane / nb, r = lane % nb;  // (16 boxes at most, one a lane)
    auto has = [&](int j) { return grp < groups && t0 + j * kTile + r * br < t1; };
    auto entry = [&](int j) {
      const int i = (t0 + j * kTile + r * br) >> p.page_shift;
      return has(j) && entry_in_bounds(p, bz * p.table_stride + i) ? table[i] : 0;
    };
    int next = entry(0), page = 0;
    for (int f = 0; f < count; ++f) {
      const int s = f % ring, round = f / ring, j = f / nc, c = f % nc;
      if (c == 0) {
        page = (int)p.n_pages;  // behind the last position, or out of range: zeros
        if (has(j)) {
          if ((uint64_t)(int64_t)next < (uint64_t)p.n_pages) page = next;
          else atomicOr(p.err, kErrIndex);
        }
        next = entry(j + 1);
      }
      if (round > 0 && !wait(!v ? kraw_empty(s) : VDEC ? vraw_empty(s) : v_empty(s), (round & 1) ^ 1, j)) break;
      const uint32_t bar = !v ? kraw_full(s) : VDEC ? vraw_full(s) : v_full(s);
      const uint32_t dst = sbase + (!v ? G::KRAW + s * G::KSTAGE : VDEC ? G::VRAW + s * G::VSTAGE : G::RING + s * kSlot);
      if (lane == 0) {
        mbar_expect_tx(bar, kTile * (groups * rb + (signs ? 16 : 0)));
        if (v && !VDEC)
          for (int i = 1; i < 4; ++i) arrive(bar);  // (a slot's barrier counts four)
      }
      __syncwarp();
      const int y = (t0 + j * kTile + r * br) & ((1 << p.page_shift) - 1);
      // the box stays in its page and its stage (or slot), the stage in its ring
      const bool fits = in_bounds(
          grp >= groups || (y + br <= 1 << p.page_shift && page <= p.n_pages && head < p.hkv &&
                            grp * (kSlot / 2) + (r + 1) * br * rb <= (!v ? G::KSTAGE : VDEC ? G::VSTAGE : kSlot) &&
                            dst - sbase + (!v ? G::KSTAGE : VDEC ? G::VSTAGE : kSlot) <=
                                (!v ? G::VRAW : VDEC ? G::MISC : G::KRAW) &&
                            (!signs || kTile * 32 + (r + 1) * br * 16 <= G::VSTAGE)),
          p.err);
      if (grp < groups && (v || j != p.drop_tile) && fits) {
        tma_load_4d(dst + grp * (kSlot / 2) + r * br * rb, v ? &maps.v : &maps.k, (c * groups + grp) * rb, y, head, page, bar);
        if (signs) tma_load_4d(dst + kTile * 32 + r * br * 16, &maps.va, c * 16, y, head, page, bar);
      }
      issued = f + 1;
    }
  } else if (warp >= 12) {
    // ---- decode: one position a thread, K by warps 12-15, V by warps 16-19 ------------------------
    const bool v = warp >= 16;
    const int tok = threadIdx.x & 127;
    const int32_t* table = p.table + (int64_t)bz * p.table_stride;
    // the position's q8_0 scales (0: no position, or no page), loaded a tile ahead
    constexpr int W = D / 64;  // words of two
    auto load_scales = [&](int j, const void* aux, uint32_t (&w)[W]) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = 0u;
      const int at = t0 + j * kTile + tok;
      if (j >= ntiles || at >= t1) return;
      if (!entry_in_bounds(p, bz * p.table_stride + (at >> p.page_shift))) return;
      const int pg = table[at >> p.page_shift];
      if ((uint64_t)(int64_t)pg >= (uint64_t)p.n_pages) return;  // (reported by the boxes' warps)
      const int64_t row = (((int64_t)pg * p.hkv + head) << p.page_shift) + (at & ((1 << p.page_shift) - 1));
      if (!in_bounds(row < (v ? p.v_rows : p.k_rows), p.err)) return;
      const uint2* src = reinterpret_cast<const uint2*>(reinterpret_cast<const __half*>(aux) + row * (D / 32));
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const uint2 x = src[i];
        w[2 * i] = x.x;
        w[2 * i + 1] = x.y;
      }
    };
    auto scale_of = [](uint32_t w, int hi) { return __half2half2(__ushort_as_half((unsigned short)(hi ? w >> 16 : w))); };
    uint32_t next[W], w[W];
    if (!v) {
      const uint32_t lanes = (uint32_t)(warp & 3) << 21;
      if constexpr (KF == QPS_FMT_Q8_0) load_scales(0, p.k.aux, next);
      int f = 0;
      bool ok = true;
      for (int j = 0; j < ntiles && ok; ++j) {
        if constexpr (KF == QPS_FMT_Q8_0) {
#pragma unroll
          for (int i = 0; i < W; ++i) w[i] = next[i];
          load_scales(j + 1, p.k.aux, next);
        }
        int halved = 0;
        if constexpr (KF == QPS_FMT_Q8_0) {
          uint32_t most = 0u;  // (magnitudes of fp16 compare as integers)
#pragma unroll
          for (int i = 0; i < W; ++i) most = __vmaxu2(most, w[i] & 0x7fff7fffu);
          halved = max(0, (int)(max(most >> 16, most & 0xffffu) >> 10) - 22);  // 2^8: exponent field 23
          if (halved > 0) {
            const __half2 f2 = __half2half2(__ushort_as_half((unsigned short)((15 - halved) << 10)));
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = mma::hmul2_u(w[i], f2);
          }
          if constexpr (G::EXPS == 4) kexp[(j & 3) * kTile + tok] = (uint8_t)halved;
        }
#pragma unroll 1
        for (int c = 0; c < G::KC; ++c, ++f) {
          const int rs = f % KN, s = f & 1;
          if (!(ok = wait(kraw_full(rs), (f / KN) & 1, j))) break;
          const uint8_t* raw = smem + G::KRAW + rs * G::KSTAGE;
          const uint32_t dst = tmem + lanes + k_col + s * 64;
          if constexpr (KF == QPS_FMT_Q8_0) {
            uint4 q[4];  // 64 codes, chunk i of the 64-byte row at i ^ (row / 2) % 4
#pragma unroll
            for (int i = 0; i < 4; ++i)
              q[i] = *reinterpret_cast<const uint4*>(raw + tok * 64 + ((i ^ ((tok >> 1) & 3)) << 4));
            mma::fence_proxy_async();  // (the reads are done before the next box is written)
            __syncwarp();
            if (lane == 0) arrive(kraw_empty(rs));
            if (f >= 2 && !(ok = wait(k_empty(s), ((f >> 1) & 1) ^ 1, j))) break;
            fence_after();
            if (G::EXPS == 2 && c == 2) kexp[(j & 1) * kTile + tok] = (uint8_t)halved;
#pragma unroll
            for (int b = 0; b < 2; ++b) {  // a block of 32
              const __half2 sc = scale_of(w[0], b);
              uint32_t hi[16], lo[16];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint4 qq = q[2 * b + (i >> 2)];
                const uint32_t word = (i & 3) == 0 ? qq.x : (i & 3) == 1 ? qq.y : (i & 3) == 2 ? qq.z : qq.w;
                uint32_t code[2];
                mma::i8x4_to_h2x2(word, code[0], code[1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const __half2 c2 = *reinterpret_cast<const __half2*>(&code[k]);
                  const __half2 h = __hmul2(c2, sc), l = __hfma2(c2, sc, __hneg2(h));  // the product's rounding error
                  hi[2 * i + k] = *reinterpret_cast<const uint32_t*>(&h);
                  lo[2 * i + k] = *reinterpret_cast<const uint32_t*>(&l);
                }
              }
              tmem_st16(dst + 16 * b, hi);
              tmem_st16(dst + 32 + 16 * b, lo);
            }
#pragma unroll
            for (int i = 0; i + 1 < W; ++i) w[i] = w[i + 1];  // the next slot's scales
          } else {
            uint32_t x[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 q = *reinterpret_cast<const uint4*>(raw + tok * 128 + ((i ^ (tok & 7)) << 4));
              x[4 * i] = q.x;
              x[4 * i + 1] = q.y;
              x[4 * i + 2] = q.z;
              x[4 * i + 3] = q.w;
            }
            mma::fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive(kraw_empty(rs));
            if (f >= 2 && !(ok = wait(k_empty(s), ((f >> 1) & 1) ^ 1, j))) break;
            fence_after();
            tmem_st32(dst, x);
          }
          tmem_wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) arrive(k_full(s));
        }
      }
    } else if constexpr (VDEC) {
      // levels as fp16 (see attn_mma.cuh): TQ3 magnitudes m in bytes 2m, 2m + 1; TQ2 fields
      uint32_t tq_lo = 0u, tq_hi = 0u;
      if constexpr (VF == QPS_FMT_TQ3) {
        tq_lo = mma::pack_h2(p.tq_levels[4], p.tq_levels[5]);
        tq_hi = mma::pack_h2(p.tq_levels[6], p.tq_levels[7]);
      } else if constexpr (VF == QPS_FMT_TQ2) {
        tq_lo = mma::pack_h2(p.tq_levels[1], p.tq_levels[0]);
        tq_hi = mma::pack_h2(p.tq_levels[2], p.tq_levels[3]);
      }
      if constexpr (VF == QPS_FMT_Q8_0) load_scales(0, p.v.aux, next);
      // 16-byte chunk c of the position's row in a slot's column group g
      auto put = [&](uint8_t* slot, int g, int c, const uint32_t* o) {
        if (in_bounds(g < 2 && c < 8 && slot - smem + kSlot <= G::KRAW, p.err))
          *reinterpret_cast<uint4*>(slot + g * (kSlot / 2) + tok * 128 + ((c ^ (tok & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
      };
      int f = 0;
      bool ok = true;
      for (int j = 0; j < ntiles && ok; ++j) {
        if constexpr (VF == QPS_FMT_Q8_0) {
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const __half2 x = mma::cut_v_scale(*reinterpret_cast<const __half2*>(&next[i]));
            w[i] = *reinterpret_cast<const uint32_t*>(&x);
          }
          load_scales(j + 1, p.v.aux, next);
        }
#pragma unroll 1
        for (int c = 0; c < G::VC; ++c, ++f) {
          const int rs = f % VN, s = f % kSlots;
          if (!(ok = wait(vraw_full(rs), (f / VN) & 1, j))) break;
          const uint8_t* raw = smem + G::VRAW + rs * G::VSTAGE;
          uint8_t* slot = smem + G::RING + s * kSlot;
          if constexpr (VF == QPS_FMT_Q8_0) {
            uint4 q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = *reinterpret_cast<const uint4*>(raw + tok * 128 + ((i ^ (tok & 7)) << 4));
            mma::fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive(vraw_empty(rs));
            if (f >= kSlots && !(ok = wait(v_empty(s), ((f / kSlots) & 1) ^ 1, j))) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // 16 dims
              const __half2 sc = scale_of(w[i >> 2], (i >> 1) & 1);
              const uint32_t word[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
              uint32_t o[8];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                mma::i8x4_to_h2x2(word[k], o[2 * k], o[2 * k + 1]);
                o[2 * k] = mma::hmul2_u(o[2 * k], sc);
                o[2 * k + 1] = mma::hmul2_u(o[2 * k + 1], sc);
              }
              put(slot, i >> 2, (2 * i) & 7, o);
              put(slot, i >> 2, (2 * i + 1) & 7, o + 4);
            }
#pragma unroll
            for (int i = 0; i + 2 < W; ++i) w[i] = w[i + 2];  // the next slot's scales
          } else {
            uint4 q[2], sg = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 2; ++i) q[i] = *reinterpret_cast<const uint4*>(raw + tok * 32 + ((i ^ ((tok >> 2) & 1)) << 4));
            if constexpr (VF == QPS_FMT_TQ3) sg = *reinterpret_cast<const uint4*>(raw + kTile * 32 + tok * 16);
            mma::fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive(vraw_empty(rs));
            if (f >= kSlots && !(ok = wait(v_empty(s), ((f / kSlots) & 1) ^ 1, j))) break;
            const uint32_t words[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
            const uint32_t sgw[4] = {sg.x, sg.y, sg.z, sg.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {  // a word: 16 dims, two chunks
              const uint32_t word = words[k], g16 = k & 1 ? sgw[k >> 1] >> 16 : sgw[k >> 1] & 0xffffu;
              // signs of columns j, j + 4 | j + 8, j + 12 at bits j, 16 + j
              const uint32_t s1 = g16 | (g16 << 12), s2 = (g16 >> 8) | (g16 << 4);
              uint32_t o[8];
#pragma unroll
              for (int jj = 0; jj < 4; ++jj) {
                const uint32_t sel = ((word >> (2 * jj)) & 0x03030303u) * 0x22u + 0x10101010u;
                uint32_t m0 = __byte_perm(tq_lo, tq_hi, sel), m1 = __byte_perm(tq_lo, tq_hi, sel >> 16);
                if constexpr (VF == QPS_FMT_TQ3) {  // a clear sign bit stores a negative level
                  m0 |= ~(s1 << (15 - jj)) & 0x80008000u;
                  m1 |= ~(s2 << (15 - jj)) & 0x80008000u;
                }
                o[2 * jj] = m0;
                o[2 * jj + 1] = m1;
              }
              put(slot, k >> 2, (2 * k) & 7, o);
              put(slot, k >> 2, (2 * k + 1) & 7, o + 4);
            }
          }
          mma::fence_proxy_async();
          __syncwarp();
          if (lane == 0) arrive(v_full(s));
        }
      }
    }
  } else if (warp >= 4) {
    // ---- softmax: one position a thread, rows [0, 32) by warps 4-7, [32, 64) by warps 8-11 ---------
    const int tl = (warp & 3) * 32 + lane, half = (warp - 4) >> 2, tid = threadIdx.x - 128;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    // Q [64][D], K-major, 128-byte swizzle, column groups of 64 dims: every load first, while
    // the first boxes are under way
    {
      constexpr int N = kN * D / 8 / 256;
      uint4 v[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int i = tid + k * 256, r = i / (D / 8), c = i % (D / 8), rr = row0 + r;
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
        const int i = tid + k * 256, r = i / (D / 8), c = i % (D / 8);
        *reinterpret_cast<uint4*>(smem + (c >> 3) * (kN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v[k];
      }
      mma::fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive(q_full);
    }
    if (tid < kN) {
      const int rr = row0 + tid;
      int n = 0;
      if (rr < p.rows_per_cta) {
        const int e = rr / p.group, b = p.shared ? e / p.n_q : bz, qi = p.shared ? e % p.n_q : e;
        n = paged_len(p, b);
        if (p.causal) n += qi + 1 - p.n_q;
        n = min(n, t1);
      }
      lim[tid] = n;
      mneg[tid] = kNone;
    }
    auto meet = [&]() { asm volatile("barrier.cta.sync 2, 256;" ::: "memory"); };
    meet();
    const float qs = p.scale * LOG2E, cap = p.softcap, cap_k = cap > 0.f ? 2.f * LOG2E / cap : 0.f;
    constexpr int CH = kN / 32;                          // 16-row chunks of a thread
    const int r0 = half * 32, nch = max(0, min(CH, n16 / 16 - half * CH));  // (in use)
    int least = 0x7fffffff;                              // positions below it are visible to every row
    for (int r = 0; r < nrows; ++r) least = min(least, lim[r]);
    const int32_t* table = p.table + (int64_t)bz * p.table_stride;
    const void* norms = VF == QPS_FMT_TQ3 ? p.v.aux2 : p.v.aux;
    auto ld16 = [&](uint32_t (&v)[16], uint32_t addr) {
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
          "%15}, [%16];"
          : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
            "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
          : "r"(addr)
          : "memory");
    };
    // Over the 32 lanes, of 16 rows at once by halving exchange: after the steps 16, 8, 4, 2 a
    // lane holds one row over 16 lanes, the last step joins the pairs; lane 2i ends with row i.
    auto over_lanes = [&](float (&y)[16], auto join) -> float {
#pragma unroll
      for (int h = 8; h >= 1; h /= 2) {
        const bool up = (lane & (2 * h)) != 0;
#pragma unroll
        for (int i = 0; i < h; ++i) {
          const float give = up ? y[i] : y[i + h], keep = up ? y[i + h] : y[i];
          y[i] = join(keep, __shfl_xor_sync(0xffffffffu, give, 2 * h));
        }
      }
      return join(y[0], __shfl_xor_sync(0xffffffffu, y[0], 1));
    };
    float* fred = reinterpret_cast<float*>(red);
    float l[CH][16];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) l[c][i] = 0.f;
    // (After a wait has given up the loop runs on, every further wait returning at once: the
    // eight warps meet at barriers that none of them may stay away from.)
    bool ok = true;
    for (int j = 0; j < ntiles; ++j) {
      const int at = t0 + j * kTile + tl;
      const bool cut = t0 + (j + 1) * kTile > least;  // (uniform) some row does not see the whole tile
      float norm = 1.f;
      if constexpr (is_tq(VF)) {  // (0 behind the end and for a bad page: nothing there is read)
        norm = 0.f;
        if (at < t1 && entry_in_bounds(p, bz * p.table_stride + (at >> p.page_shift))) {
          const int pg = table[at >> p.page_shift];
          if ((uint64_t)(int64_t)pg < (uint64_t)p.n_pages &&
              in_bounds((((int64_t)pg * p.hkv + head) << p.page_shift) + (at & ((1 << p.page_shift) - 1)) < p.v_rows, p.err))
            norm = __half2float(reinterpret_cast<const __half*>(norms)[(((int64_t)pg * p.hkv + head) << p.page_shift) +
                                                                      (at & ((1 << p.page_shift) - 1))]);
        }
      }
      // (a TurboQuant V: the reference bounds P x norm, the operand; see attn_mma.cuh)
      const float lift = is_tq(VF) ? mma::norm_log2(norm) : 0.f, room = kRefShift + kRefLazy - lift;
      ok &= wait(s_full(j & 1), (j >> 1) & 1, j);
      fence_after();
      float qt = qs, st = p.scale;
      if constexpr (KF == QPS_FMT_Q8_0) {
        const float twice = __uint_as_float((127u + kexp[(j & (G::EXPS - 1)) * kTile + tl]) << 23);
        qt *= twice;
        st *= twice;
      }
      // the logits, in units of log2, of 16 rows at this thread's position (read again for
      // each use: kept beside the sums they would not fit the registers)
      const uint32_t s_at = tmem + lanes + (j & 1) * n16 + r0;
      auto logits = [&](int c, float (&x)[16]) {
        uint32_t v[16];
        __syncwarp();
        ld16(v, s_at + 16 * c);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(v[i]);
        if (cap > 0.f) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = mma::softcap_tanh(x[i] * st, cap, cap_k) * LOG2E;
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= qt;
        }
        if (cut) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (at >= lim[r0 + 16 * c + i]) x[i] = -INFINITY;
        }
      };
      bool over = false;
#pragma unroll 1
      for (int c = 0; c < nch; ++c) {
        float x[16];
        logits(c, x);
        float d[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 mn = *reinterpret_cast<const float4*>(mneg + r0 + 16 * c + i);
          d[0] = fmaxf(d[0], x[i] + mn.x);  // (a NaN is no maximum)
          d[1] = fmaxf(d[1], x[i + 1] + mn.y);
          d[2] = fmaxf(d[2], x[i + 2] + mn.z);
          d[3] = fmaxf(d[3], x[i + 3] + mn.w);
        }
        over |= fmaxf(fmaxf(d[0], d[1]), fmaxf(d[2], d[3])) > room;
      }
      int any;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 2, 256, p;\n selp.s32 %0, 1, 0, q;\n}\n"
          : "=r"(any)
          : "r"((int)over)
          : "memory");
      if (any) {
        // raise every reference for its row's maximum so far (fmaxf drops a NaN); O and the
        // sums follow
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (c >= nch) break;
          float y[16];
          logits(c, y);
          if constexpr (is_tq(VF)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] += lift;
          }
          const float top = over_lanes(y, [](float a, float b) { return fmaxf(a, b); });
          if (!(lane & 1)) fred[(warp & 3) * kN + r0 + 16 * c + (lane >> 1)] = top;
        }
        meet();
        float cr = 1.f;
        if (tid < n16) {
          float top = fred[tid];
#pragma unroll
          for (int w = 1; w < 4; ++w) top = fmaxf(top, fred[w * kN + tid]);
          top -= kRefShift;
          const float old = mneg[tid];
          if (top > -old) {
            cr = old == kNone ? 0.f : ex2(-old - top);
            mneg[tid] = -top;
          }
        }
        meet();  // (every maximum has been read)
        if (tid < n16) fred[tid] = cr;
        meet();
        if (j > 0) {
          ok &= wait(p_free((j - 1) & 1), ((j - 1) >> 1) & 1, j);  // O is at rest
          fence_after();
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (c >= nch) break;
          const float* f = fred + r0 + 16 * c;
#pragma unroll
          for (int i = 0; i < 16; ++i) l[c][i] *= f[i];
          if (j > 0) {
#pragma unroll 1
            for (int b = 0; b < G::VC; ++b) {
              uint32_t v[16];
              const uint32_t o_at = tmem + lanes + o_col + b * n16 + r0 + 16 * c;
              __syncwarp();
              ld16(v, o_at);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f[i]);
              tmem_st16(o_at, v);
            }
          }
        }
        if (j > 0) {
          tmem_wait_st();
          fence_before();
        }
        meet();  // (every factor has been read)
      }
      if (j >= 2) ok &= wait(p_free(j & 1), ((j - 2) >> 1) & 1, j);  // the buffer's last reader
      uint8_t* pbuf = smem + G::P_OFF + (j & 1) * G::P_STEP + tl * 128;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (c >= nch) break;
        float x[16];
        logits(c, x);
        uint32_t pk[8], pl[G::PLO ? 8 : 1];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 mn = *reinterpret_cast<const float4*>(mneg + r0 + 16 * c + i);
          const float a = ex2(x[i] + mn.x), b = ex2(x[i + 1] + mn.y);
          const float d = ex2(x[i + 2] + mn.z), e = ex2(x[i + 3] + mn.w);
          l[c][i] += a;
          l[c][i + 1] += b;
          l[c][i + 2] += d;
          l[c][i + 3] += e;
          pk[i / 2] = mma::pack_h2(a * norm, b * norm);
          pk[i / 2 + 1] = mma::pack_h2(d * norm, e * norm);
          if constexpr (G::PLO) {
            const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&pk[i / 2]));
            const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&pk[i / 2 + 1]));
            pl[i / 2] = mma::pack_h2(a - f0.x, b - f0.y);
            pl[i / 2 + 1] = mma::pack_h2(d - f1.x, e - f1.y);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<uint4*>(pbuf + (((r0 / 8 + 2 * c + h) ^ (tl & 7)) << 4)) =
              make_uint4(pk[4 * h], pk[4 * h + 1], pk[4 * h + 2], pk[4 * h + 3]);
        if constexpr (G::PLO) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<uint4*>(pbuf + kPBytes + (((r0 / 8 + 2 * c + h) ^ (tl & 7)) << 4)) =
                make_uint4(pl[4 * h], pl[4 * h + 1], pl[4 * h + 2], pl[4 * h + 3]);
        }
      }
      mma::fence_proxy_async();
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(p_ready(j & 1));
    }
    if (ok) ok = wait(all_done, 0, ntiles);
    fence_after();
    // ---- sums over the positions, O to shared memory ---------------------------------------------
    if (ok) {
      float* fin = reinterpret_cast<float*>(smem + G::P_OFF);  // [row][D] over P, the slots and the stages
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (c >= nch) break;
        const float sum = over_lanes(l[c], [](float a, float b) { return a + b; });
        if (!(lane & 1)) fred[(warp & 3) * kN + r0 + 16 * c + (lane >> 1)] = sum;
#pragma unroll 1
        for (int b = 0; b < G::VC && ntiles > 0; ++b) {
          const int dim = b * 128 + (is_tq(VF) ? (tl & ~15) + tq_unswap(tl & 15) : tl);
          uint32_t v[16];
          __syncwarp();
          ld16(v, tmem + lanes + o_col + b * n16 + r0 + 16 * c);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (in_bounds(dim < D && ((r0 + 16 * c + i) * D + dim + 1) * 4 <= G::MISC - G::P_OFF, p.err))
              fin[(r0 + 16 * c + i) * D + dim] = __uint_as_float(v[i]);
        }
      }
    }
    fence_before();
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" :::);
  const bool good = !*abort_flag;
  if (good) {
    // ---- the rotation's inverse, the division, the part: a row a warp, element lane + 32 e
    // in register e (with the row's elements spread over the CTA, the butterflies' addresses
    // and barriers took as many instructions as seven tiles) ----
    constexpr int E = D / 32;
    const float* fin = reinterpret_cast<const float*>(smem + G::P_OFF);
    const float* sums = reinterpret_cast<const float*>(red);
    for (int r = warp; r < nrows; r += kThreadsTt / 32) {
      const int rr = row0 + r;
      const float den = ntiles > 0 ? (sums[r] + sums[kN + r]) + (sums[2 * kN + r] + sums[3 * kN + r]) : 0.f;
      const bool none = den == 0.f;
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = none ? 0.f : fin[r * D + lane + 32 * e];
      if constexpr (is_tq(VF)) {  // x = s1 .* blockdiag(H_G)(s2 .* y) / sqrt(D G)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if ((p.vsigns2[e] >> lane) & 1u) o[e] = -o[e];
#pragma unroll
        for (int h = 1; h < 32; h *= 2) {  // (every block is at least 32 wide)
          const bool upper = (lane & h) != 0;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float other = __shfl_xor_sync(0xffffffffu, o[e], h);
            o[e] = upper ? other - o[e] : o[e] + other;
          }
        }
#pragma unroll
        for (int H = 1; H < E; H *= 2) {
          if (32 * H >= p.vblock) break;
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (!(e & H)) {
              const float a = o[e], b = o[e + H];
              o[e] = a + b;
              o[e + H] = a - b;
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
          if ((p.vsigns[e] >> lane) & 1u) o[e] = -o[e];
      }
      const float scale = none ? 0.f : (is_tq(VF) ? p.v_out_scale : 1.f) / den;
      const int64_t local = (int64_t)(rr / p.group) * p.hq + head * p.group + rr % p.group;
      const int64_t at = p.shared ? (int64_t)split * p.rows_total + local
                         : whole  ? (int64_t)bz * (p.n_q * p.hq) + local
                                  : (int64_t)split * (p.n_q * p.hq) + local;
      if (!out_in_bounds(p, whole, split, whole ? at : local)) continue;
      if (lane == 0)
        (whole ? p.out_lse : p.shared ? p.pre_lse : p.own_lse)[at] =
            none ? -INFINITY : (log2f(den) - mneg[r]) * 0.6931471805599453f;
      float* dst = whole ? reinterpret_cast<float*>(p.out) : p.shared ? p.pre_o : p.own_o;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float v = o[e] * scale;
        const int64_t i = at * D + lane + 32 * e;
        if (!whole || p.out_dtype == QPS_DT_F32) dst[i] = v;
        else if (p.out_dtype == QPS_DT_F16) reinterpret_cast<__half*>(p.out)[i] = __float2half_rn(v);
        else reinterpret_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(v);
      }
    }
  } else {  // the products and boxes under way, before their operands and TMEM go
    if (warp == 0) mma::mbar_wait(all_done, 0, p.wait_ns);
    if (warp == 2 || warp == 3) {
      const bool v = warp == 3, first = !v && lane == 0 && report_give_up(p.err, *abort_flag, issued, ntiles, t1 - t0);
      const int ring = !v ? KN : VDEC ? VN : kSlots;
      const uint64_t since = global_ns();
      bool done = true;
#pragma unroll 1
      for (int i = max(0, issued - ring); i < issued; ++i) {
        const int s = i % ring;
        done &= mma::mbar_wait(!v ? kraw_full(s) : VDEC ? vraw_full(s) : v_full(s), (i / ring) & 1, p.wait_ns);
      }
      if (first) {
        p.err[10] = (unsigned)min((uint64_t)0xffffffffu, global_ns() - since);
        p.err[11] = done ? 1u : 0u;
      }
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1) tmem_free(tmem, 512);
}

template <int D, int KF, int VF>
qps_status launch_tt(const PagedAttnParams& p, cudaStream_t s) {
  using G = GeoTt<D, KF, VF>;
  static_assert(G::SMEM <= 227 * 1024, "the slots exceed the shared memory of one CTA");
  static_assert((2 + G::VC) * kN + 128 <= 512, "S, K and O exceed TMEM");
  static_assert(kN * D * 4 <= G::MISC - G::P_OFF, "the output rows fit P, the slots and the raw stages");
  TmaSet maps;
  std::memset(&maps, 0, sizeof(maps));
  const int page = 1 << p.page_shift, rows = page < kTile ? page : kTile;
  auto map = [&](TensorMap* m, const void* plane, int row_bytes, int box, int swizzle) {
    return encode_plane_map(m, plane, row_bytes, page, p.hkv, page, (int)p.n_pages, (int64_t)p.hkv * page, box, swizzle, rows);
  };
  if (!(KF == QPS_FMT_F16 ? map(&maps.k, p.k.data, 2 * D, 128, 128) : map(&maps.k, p.k.data, D, 64, 64)) ||
      !(VF == QPS_FMT_F16    ? map(&maps.v, p.v.data, 2 * D, 128, 128)
        : VF == QPS_FMT_Q8_0 ? map(&maps.v, p.v.data, D, 128, 128)
                             : map(&maps.v, p.v.data, D / 4, 32, 32)) ||
      (VF == QPS_FMT_TQ3 && !map(&maps.va, p.v.aux, D / 8, 16, 0)))
    return QPS_ERR_CUDA;
  auto kern = attn_tt_kernel<D, KF, VF>;
  static std::atomic<uint64_t> sized{0};
  int dev = 0;
  QPS_CUDA_TRY(cudaGetDevice(&dev));
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(sized.load(std::memory_order_relaxed) & bit) || !bit) {
    QPS_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM));
    sized.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.shared ? p.n_split : p.max_chunks) * ((p.rows_per_cta + kN - 1) / kN), p.hkv, 1);
  cfg.blockDim = dim3(kThreadsTt);
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

// The format pairings of one head_dim.
template <int D>
qps_status launch_tt_d(const PagedAttnParams& p, cudaStream_t s) {
#define QPS_TT_CASE(KF, VF) \
  if (p.kfmt == KF && p.vfmt == VF) return launch_tt<D, KF, VF>(p, s);
  if constexpr (D > 128) {  // (128: attn_tm.cuh)
    QPS_TT_CASE(QPS_FMT_F16, QPS_FMT_F16)
  }
  QPS_TT_CASE(QPS_FMT_F16, QPS_FMT_Q8_0)
  QPS_TT_CASE(QPS_FMT_F16, QPS_FMT_TQ3)
  QPS_TT_CASE(QPS_FMT_F16, QPS_FMT_TQ2)
  QPS_TT_CASE(QPS_FMT_Q8_0, QPS_FMT_F16)
  QPS_TT_CASE(QPS_FMT_Q8_0, QPS_FMT_Q8_0)
  QPS_TT_CASE(QPS_FMT_Q8_0, QPS_FMT_TQ3)
  QPS_TT_CASE(QPS_FMT_Q8_0, QPS_FMT_TQ2)
#undef QPS_TT_CASE
  return fail(QPS_ERR_UNSUPPORTED, "attention: unsupported K/V format pairing");
}

}  // namespace tt
}  // namespace qps
