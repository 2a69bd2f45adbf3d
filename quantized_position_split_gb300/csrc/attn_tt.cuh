// Decode attention of up to 64 query rows per KV head on the fifth-generation tensor cores,
// over pages of any width and format: verify batches and shared prefixes of compressed
// caches, where the products on the older path (mma.sync, 8 rows a warp) decode the same
// positions again for every 8 to 24 rows.
//
// The products run with the positions and the head dimension on the wide side (M = 128)
// and the query rows on the narrow one (N = 16 .. 64), so their time follows the number of
// rows:
//     S^T [128 positions][N] = K Q^T      A = K (K-major), B = Q (K-major), per 64 dims
//     P   = 2^(S' - m)                    one position a thread, all rows in its registers
//     O^T [128 dims][N]     += V^T P^T    A = V (MN-major, as stored), B = P (MN-major)
// S^T (two buffers) and O^T (D / 128 blocks) live in TMEM: 128 + D / 2 columns.
//
// K and V are decoded once per tile by eight warps into 32 KB slots of fp16 operands (64
// dims of K, 128 of V), a ring that the products empty.  Numerics: a q8_0 key (code x
// scale) is stored as hi + lo fp16 parts, two products, so logits keep float32 accuracy; a
// TurboQuant V is its exact fp16 levels in the rotated domain with the norm folded into P
// before P's one rounding, the output being rotated back once; a q8_0 V is rounded once to
// fp16; sums, maxima and O are float32.
//
// A row's maximum over the positions would cross all threads, so the running reference m
// (in shared memory) is raised only when some position exceeds it by more than 8 (log2):
// one vote a tile, and on a raise the maxima are taken, O and the sums rescaled.
//
// Roles: warp 0 issues the products, warps 4-7 are the softmax, warps 8-15 decode.  Waits
// are bounded as in attn_tm.cuh.
#pragma once

#include "attn_tm.cuh"

namespace qps {
namespace tt {

using namespace tm;

constexpr int kN = 64;             // query rows per CTA
constexpr int kTile = 128;         // positions per tile
constexpr int kThreadsTt = 512;
constexpr int kSlot = 32 * 1024, kSlots = 4;

template <int D>
struct GeoTt {
  static constexpr int KC = D / 64, VC = D / 128;   // slots of a tile: K's and V's
  static constexpr int Q_BYTES = kN * D * 2;
  static constexpr int P_OFF = Q_BYTES;             // two buffers [128][64] fp16
  static constexpr int RING = P_OFF + 2 * kTile * kN * 2;
  static constexpr int MISC = RING + kSlots * kSlot;
  static constexpr int SMEM = MISC + 2048 + 1024;   // + slack for the 1024-byte base alignment
  static constexpr int S_COL = 0, O_COL = 128;
  static constexpr int COLS = O_COL + VC * kN <= 256 ? 256 : 512;
};

// Floats as integers of the same order, for integer maxima (-inf below all others; a NaN
// does not occur: it is not compared).
__device__ __forceinline__ int ordered(float f) {
  const int i = __float_as_int(f);
  return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff); }

// Position in a 16-column word of a TurboQuant V -> column: the decode yields the columns
// j, j + 4, j + 8, j + 12 of step j.
__device__ __forceinline__ int tq_unswap(int pos) { return (pos >> 2) + 4 * (pos & 3); }

template <int D, int KF, int VF>
__global__ void __launch_bounds__(kThreadsTt, 1)
    attn_tt_kernel(const __grid_constant__ PagedAttnParams p) {
  using G = GeoTt<D>;
  constexpr float LOG2E = 1.4426950408889634f;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- this CTA's rows and positions ------------------------------------------------------
  const int rtiles = (p.rows_per_cta + kN - 1) / kN;
  const int split = blockIdx.x / rtiles, row0 = (blockIdx.x % rtiles) * kN;
  const int head = blockIdx.y;
  int bz = 0, t0, t1;
  bool whole = false;
  if (p.shared) {
    t0 = split * (int)p.chunk;
    t1 = min((int)p.end, t0 + (int)p.chunk);
  } else {
    if (blockIdx.x == 0 && head == 0 && warp == 2) paged_publish(p, lane);
    const PagedChunk ch = paged_find(p, split, lane);
    if (ch.b < 0) return;  // more CTAs than chunks (every warp finds the same)
    bz = ch.b;
    t0 = ch.t0;
    t1 = ch.t1;
    whole = ch.whole;
  }
  const int ntiles = t1 > t0 ? (t1 - t0 + kTile - 1) / kTile : 0;  // 0: an empty sequence
  const int nrows = min(kN, p.rows_per_cta - row0);
  const int n16 = (nrows + 15) & ~15;  // N of the products

  // ---- barriers, TMEM, queries, row state ----------------------------------------------------
  uint8_t* misc = smem + G::MISC;
  float* thr = reinterpret_cast<float*>(misc);            // [64] m + 8 (-inf: no reference yet)
  float* mneg = reinterpret_cast<float*>(misc + 256);     // [64] -m (0: none)
  int* lim = reinterpret_cast<int*>(misc + 512);          // [64] positions below it are visible
  int* red = reinterpret_cast<int*>(misc + 768);          // [4][64] maxima, then sums
  uint32_t* tmem_word = reinterpret_cast<uint32_t*>(misc + 1792);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1796);
  const uint32_t bars = sbase + G::MISC + 1808;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kSlots + s); };
  auto s_full = [&](int w) { return bars + 8 * (2 * kSlots + w); };
  auto p_ready = [&](int w) { return bars + 8 * (2 * kSlots + 2 + w); };
  auto p_free = [&](int w) { return bars + 8 * (2 * kSlots + 4 + w); };
  const uint32_t all_done = bars + 8 * (2 * kSlots + 6);
  static_assert(1808 + 8 * (2 * kSlots + 7) <= 2048, "the row state and barriers fit their region");
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * kSlots + 7; ++i)
      mbar_init(bars + 8 * i, i < kSlots ? 8 : (i == 2 * kSlots + 2 || i == 2 * kSlots + 3) ? 4 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    *abort_flag = 0;
  }
  if (warp == 1) tmem_alloc(smem_addr(tmem_word), G::COLS);
  // Q [64][D], K-major, 128-byte swizzle, column groups of 64 dims
  for (int i = threadIdx.x; i < kN * D / 8; i += kThreadsTt) {
    const int r = i / (D / 8), c = i % (D / 8), rr = row0 + r;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (rr < p.rows_per_cta) {
      const int e = rr / p.group, h = head * p.group + rr % p.group;
      const int b = p.shared ? e / p.n_q : bz, qi = p.shared ? e % p.n_q : e;
      v = *reinterpret_cast<const uint4*>(p.q + (int64_t)b * p.q_bstride + ((int64_t)qi * p.hq + h) * D + c * 8);
    }
    *reinterpret_cast<uint4*>(smem + (c >> 3) * (kN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
  }
  if (threadIdx.x < kN) {
    const int rr = row0 + threadIdx.x;
    int n = 0;
    if (rr < p.rows_per_cta) {
      const int e = rr / p.group, b = p.shared ? e / p.n_q : bz, qi = p.shared ? e % p.n_q : e;
      n = paged_len(p, b);
      if (p.causal) n += qi + 1 - p.n_q;
      n = min(n, t1);
    }
    lim[threadIdx.x] = n;
    thr[threadIdx.x] = -INFINITY;
    mneg[threadIdx.x] = 0.f;
  }
  mma::fence_proxy_async();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_word;

  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {  // (as in attn_tm.cuh)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t since = global_ns();
    for (;;) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      int over = 0;
      if (lane == 0) {
        over = *abort_flag;
        if (!over && global_ns() - since >= mma::kWaitLimitNs) {
          atomicOr(p.err, kErrTimeout);
          atomicAdd(p.err + 1, 1u);
          *abort_flag = over = 1;
        }
      }
      if (__shfl_sync(0xffffffffu, over, 0)) return false;
    }
  };
  auto arrive = [&](uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
  };

  if (warp == 0) {
    // ---- products: K(0), then K(j + 1), V(j) for every tile, in the ring's order ----------------
    const uint32_t id_s = instr_desc(n16, 0), id_o = instr_desc(n16, 1) | (1u << 15);
    int f = 0;  // slots emptied
    auto s_product = [&](int j) -> bool {
      for (int c = 0; c < G::KC; ++c, ++f) {
        const int s = f % kSlots;
        if (!wait(full(s), (f / kSlots) & 1)) return false;
        fence_after();
        if (lane == 0) {
          const uint32_t d = tmem + G::S_COL + (j & 1) * kN, a = sbase + G::RING + s * kSlot, b = sbase + c * (kN * 128);
#pragma unroll
          for (int part = 0; part < (KF == QPS_FMT_Q8_0 ? 2 : 1); ++part)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss(d, smem_desc(a + part * (kSlot / 2) + kk * 32, 16), smem_desc(b + kk * 32, 16), id_s,
                     c > 0 || part > 0 || kk > 0);
          commit(empty(s));
          if (c == G::KC - 1) commit(s_full(j & 1));
        }
        __syncwarp();
      }
      return true;
    };
    bool ok = ntiles == 0 || s_product(0);
    for (int j = 0; j < ntiles && ok; ++j) {
      if (j + 1 < ntiles && !(ok = s_product(j + 1))) break;
      if (!(ok = wait(p_ready(j & 1), (j >> 1) & 1))) break;
      for (int c = 0; c < G::VC && ok; ++c, ++f) {
        const int s = f % kSlots;
        if (!(ok = wait(full(s), (f / kSlots) & 1))) break;
        fence_after();
        if (lane == 0) {
          const uint32_t d = tmem + G::O_COL + c * kN, a = sbase + G::RING + s * kSlot;
          const uint32_t b = sbase + G::P_OFF + (j & 1) * (kTile * kN * 2);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ss(d, smem_desc(a + kk * 2048, kSlot / 2), smem_desc(b + kk * 2048, 16), id_o, j > 0 || kk > 0);
          commit(empty(s));
          if (c == G::VC - 1) commit(p_free(j & 1));
        }
        __syncwarp();
      }
    }
    if (lane == 0) commit(all_done);
    __syncwarp();
    wait(all_done, 0);
  } else if (warp >= 8) {
    // ---- decode: one position and half a slot's columns a thread ------------------------------
    const int tid = threadIdx.x - 256, tok = tid >> 1, half = tid & 1;
    // levels as fp16 (see attn_mma.cuh): TQ3 magnitudes m in bytes 2m, 2m + 1; TQ2 fields
    uint32_t tq_lo = 0u, tq_hi = 0u;
    if constexpr (VF == QPS_FMT_TQ3) {
      tq_lo = mma::pack_h2(p.tq_levels[4], p.tq_levels[5]);
      tq_hi = mma::pack_h2(p.tq_levels[6], p.tq_levels[7]);
    } else if constexpr (VF == QPS_FMT_TQ2) {
      tq_lo = mma::pack_h2(p.tq_levels[1], p.tq_levels[0]);
      tq_hi = mma::pack_h2(p.tq_levels[2], p.tq_levels[3]);
    }
    const int32_t* table = p.table + (p.shared ? 0 : (int64_t)bz * p.table_stride);
    // A slot of the sequence K(0), K(1), V(0), K(2), V(1), ...: phase 0 is K(0), phase
    // 2i + 1 K(i + 1), phase 2i + 2 V(i).
    struct Task {
      int ph, c;
    };
    auto is_v = [](const Task& t) { return t.ph > 0 && !(t.ph & 1); };
    auto tile_of = [](const Task& t) { return t.ph == 0 ? 0 : (t.ph & 1) ? (t.ph + 1) >> 1 : (t.ph >> 1) - 1; };
    auto done = [&](const Task& t) { return t.ph > 0 && (t.ph >> 1) - ((t.ph & 1) ^ 1) >= ntiles; };
    auto advance = [&](Task& t) {
      if (++t.c < (is_v(t) ? G::VC : G::KC)) return;
      t.c = 0;
      ++t.ph;
      if ((t.ph & 1) && (t.ph + 1) >> 1 >= ntiles) ++t.ph;
    };
    constexpr int RAW = VF == QPS_FMT_F16 ? 8 : 4;
    struct Raw {
      uint4 d[RAW];
      uint32_t x[2];  // scales or signs
    };
    int64_t rows[2] = {-1, -1};  // this thread's row of tile j in rows[j & 1] (-1: none)
    auto load = [&](const Task& t, Raw& r) {
      const int j = tile_of(t);
#pragma unroll
      for (int i = 0; i < RAW; ++i) r.d[i] = make_uint4(0, 0, 0, 0);
      r.x[0] = r.x[1] = 0u;
      if (!is_v(t)) {
        if (t.c == 0) {
          const int at = t0 + j * kTile + tok;
          int64_t row = -1;
          if (at < t1) {
            const int pg = table[at >> p.page_shift];
            if ((uint64_t)(int64_t)pg < (uint64_t)p.n_pages)
              row = (((int64_t)pg * p.hkv + head) << p.page_shift) + (at & ((1 << p.page_shift) - 1));
            else
              atomicOr(p.err, kErrIndex);
          }
          if (j & 1) rows[1] = row;
          else rows[0] = row;
        }
        const int64_t row = (j & 1) ? rows[1] : rows[0];
        if (row < 0) return;
        const int e = t.c * 64 + half * 32;  // 32 dims
        if constexpr (KF == QPS_FMT_Q8_0) {
          const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p.k.data) + row * D + e);
          r.d[0] = src[0];
          r.d[1] = src[1];
          r.x[0] = reinterpret_cast<const uint16_t*>(p.k.aux)[row * (D / 32) + e / 32];
        } else {
          const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __half*>(p.k.data) + row * D + e);
#pragma unroll
          for (int i = 0; i < 4; ++i) r.d[i] = src[i];
        }
      } else {
        const int64_t row = (j & 1) ? rows[1] : rows[0];
        if (row < 0) return;
        const int e = t.c * 128 + half * 64;  // 64 dims
        if constexpr (VF == QPS_FMT_Q8_0) {
          const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p.v.data) + row * D + e);
#pragma unroll
          for (int i = 0; i < 4; ++i) r.d[i] = src[i];
          r.x[0] = reinterpret_cast<const uint32_t*>(p.v.aux)[(row * (D / 32) + e / 32) / 2];
        } else if constexpr (VF == QPS_FMT_F16) {
          const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __half*>(p.v.data) + row * D + e);
#pragma unroll
          for (int i = 0; i < 8; ++i) r.d[i] = src[i];
        } else {
          r.d[0] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p.v.data) + row * (D / 4) + e / 4);
          if constexpr (VF == QPS_FMT_TQ3) {
            const uint2 s = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(p.v.aux) + row * (D / 8) + e / 8);
            r.x[0] = s.x;
            r.x[1] = s.y;
          }
        }
      }
    };
    // 16-byte chunk c of the thread's row in a column group at `base`
    auto put = [&](uint8_t* base, int c, uint4 v) {
      *reinterpret_cast<uint4*>(base + tok * 128 + ((c ^ (tok & 7)) << 4)) = v;
    };
    auto convert = [&](const Task& t, const Raw& r, uint8_t* slot) {
      if (!is_v(t)) {
        if constexpr (KF == QPS_FMT_Q8_0) {
          const __half2 sc = __half2half2(__ushort_as_half((unsigned short)r.x[0]));
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 8 dims
            const uint32_t w[2] = {c & 1 ? r.d[c >> 1].z : r.d[c >> 1].x, c & 1 ? r.d[c >> 1].w : r.d[c >> 1].y};
            uint32_t code[4], hi[4], lo[4];
            mma::i8x4_to_h2x2(w[0], code[0], code[1]);
            mma::i8x4_to_h2x2(w[1], code[2], code[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __half2 x = *reinterpret_cast<const __half2*>(&code[i]);
              const __half2 h = __hmul2(x, sc), l = __hfma2(x, sc, __hneg2(h));  // the product's rounding error
              hi[i] = *reinterpret_cast<const uint32_t*>(&h);
              lo[i] = *reinterpret_cast<const uint32_t*>(&l);
            }
            put(slot, half * 4 + c, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            put(slot + kSlot / 2, half * 4 + c, make_uint4(lo[0], lo[1], lo[2], lo[3]));
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) put(slot, half * 4 + c, r.d[c]);
        }
      } else {
        uint8_t* base = slot + half * (kSlot / 2);  // the half's column group of 64 dims
        if constexpr (VF == QPS_FMT_Q8_0) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 q = r.d[c >> 1];
            const uint32_t w[2] = {c & 1 ? q.z : q.x, c & 1 ? q.w : q.y};
            const __half2 sc = __half2half2(__ushort_as_half((unsigned short)(c < 4 ? r.x[0] : r.x[0] >> 16)));
            uint32_t o[4];
            mma::i8x4_to_h2x2(w[0], o[0], o[1]);
            mma::i8x4_to_h2x2(w[1], o[2], o[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = mma::hmul2_u(o[i], sc);
            put(base, c, make_uint4(o[0], o[1], o[2], o[3]));
          }
        } else if constexpr (VF == QPS_FMT_F16) {
#pragma unroll
          for (int c = 0; c < 8; ++c) put(base, c, r.d[c]);
        } else {
          const uint32_t w[4] = {r.d[0].x, r.d[0].y, r.d[0].z, r.d[0].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // 16 dims: two chunks
            uint32_t s1 = 0u, s2 = 0u;
            if constexpr (VF == QPS_FMT_TQ3) {  // columns j, j + 4 | j + 8, j + 12 at bits j, 16 + j
              const uint32_t sg = k & 1 ? r.x[k >> 1] >> 16 : r.x[k >> 1] & 0xffffu;
              s1 = (sg & 0xfu) | ((sg & 0xf0u) << 12);
              s2 = ((sg >> 8) & 0xfu) | ((sg & 0xf000u) << 4);
            }
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t sel = ((w[k] >> (2 * j)) & 0x03030303u) * 0x22u + 0x10101010u;
              uint32_t m0 = __byte_perm(tq_lo, tq_hi, sel), m1 = __byte_perm(tq_lo, tq_hi, sel >> 16);
              if constexpr (VF == QPS_FMT_TQ3) {  // a clear sign bit stores a negative level
                m0 |= ~(s1 << (15 - j)) & 0x80008000u;
                m1 |= ~(s2 << (15 - j)) & 0x80008000u;
              }
              o[2 * j] = m0;
              o[2 * j + 1] = m1;
            }
            put(base, 2 * k, make_uint4(o[0], o[1], o[2], o[3]));
            put(base, 2 * k + 1, make_uint4(o[4], o[5], o[6], o[7]));
          }
        }
      }
    };
    Task next = {0, 0}, now = {0, 0};
    Raw ring[2];
    if (ntiles > 0) {
      load(next, ring[0]);
      advance(next);
      if (!done(next)) load(next, ring[1]);
      advance(next);
    }
    bool ok = true;
    auto turn = [&](int f, Raw& r) {  // fill slot f from r, then load two slots ahead into r
      const int s = f % kSlots;
      if (f >= kSlots && !wait(empty(s), ((f / kSlots) & 1) ^ 1)) {
        ok = false;
        return;
      }
      convert(now, r, smem + G::RING + s * kSlot);
      mma::fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive(full(s));
      advance(now);
      if (!done(next)) {
        load(next, r);
        advance(next);
      }
    };
    for (int f = 0; ntiles > 0 && ok && !done(now); f += 2) {
      turn(f, ring[0]);
      if (ok && !done(now)) turn(f + 1, ring[1]);
    }
  } else if (warp >= 4) {
    // ---- softmax: one position a thread ----------------------------------------------------------
    const int tl = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const float qs = p.scale * LOG2E, cap = p.softcap, cap_k = cap > 0.f ? 2.f * LOG2E / cap : 0.f;
    const int nch = n16 / 16;  // 16-row chunks in use
    int least = 0x7fffffff;    // positions below it are visible to every row
    for (int r = 0; r < nrows; ++r) least = min(least, lim[r]);
    const int32_t* table = p.table + (p.shared ? 0 : (int64_t)bz * p.table_stride);
    const void* norms = VF == QPS_FMT_TQ3 ? p.v.aux2 : p.v.aux;
    float l[kN];
#pragma unroll
    for (int r = 0; r < kN; ++r) l[r] = 0.f;
    // the logits (log2 domain) of 16 rows at this thread's position
    auto logits = [&](uint32_t addr, int c, int at, bool cut, float (&x)[16]) {
      uint32_t v[16];
      __syncwarp();
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
          "%15}, [%16];"
          : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
            "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
          : "r"(addr + 16 * c)
          : "memory");
      tmem_wait_ld();
      if (cap > 0.f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = mma::softcap_tanh(__uint_as_float(v[i]) * p.scale, cap, cap_k) * LOG2E;
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(v[i]) * qs;
      }
      if (cut) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (at >= lim[16 * c + i]) x[i] = -INFINITY;
      }
    };
    // (After a wait has given up the loop runs on, every further wait returning at once: the
    // four warps meet at barriers that none of them may stay away from.)
    bool ok = true;
    for (int j = 0; j < ntiles; ++j) {
      const int at = t0 + j * kTile + tl;
      const bool cut = t0 + (j + 1) * kTile > least;  // (uniform) some row does not see the whole tile
      float norm = 1.f;
      if constexpr (is_tq(VF)) {  // (0 behind the end and for a bad page: nothing there is read)
        norm = 0.f;
        if (at < t1) {
          const int pg = table[at >> p.page_shift];
          if ((uint64_t)(int64_t)pg < (uint64_t)p.n_pages)
            norm = __half2float(reinterpret_cast<const __half*>(norms)[(((int64_t)pg * p.hkv + head) << p.page_shift) +
                                                                      (at & ((1 << p.page_shift) - 1))]);
        }
      }
      // P x norm stays finite in fp16: the slack above the reference shrinks with a large norm
      const float slack = is_tq(VF) && fabsf(norm) > 255.f ? 8.f : 0.f;
      ok &= wait(s_full(j & 1), (j >> 1) & 1);
      fence_after();
      const uint32_t s_at = tmem + lanes + G::S_COL + (j & 1) * kN;
      bool over = false;
#pragma unroll 1
      for (int c = 0; c < nch; ++c) {
        float x[16];
        logits(s_at, c, at, cut, x);
        float d[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 th = *reinterpret_cast<const float2*>(thr + 16 * c + i);
          d[0] = fmaxf(d[0], x[i] - th.x);  // (+inf without a reference, NaN for -inf - -inf: no maximum)
          d[1] = fmaxf(d[1], x[i + 1] - th.y);
        }
        over |= fmaxf(d[0], d[1]) + slack > 0.f;
      }
      int any;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 2, 128, p;\n selp.s32 %0, 1, 0, q;\n}\n"
          : "=r"(any)
          : "r"((int)over)
          : "memory");
      if (any) {
        // raise every reference to its row's maximum so far; O and the sums follow
#pragma unroll 1
        for (int c = 0; c < nch; ++c) {
          float x[16];
          logits(s_at, c, at, cut, x);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int m = __reduce_max_sync(0xffffffffu, ordered(x[i] == x[i] ? x[i] : -INFINITY));
            if (lane == 0) red[(warp & 3) * kN + 16 * c + i] = m;
          }
        }
        asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
        float cr = 1.f;
        if (tl < 16 * nch) {
          int m = red[tl];
#pragma unroll
          for (int w = 1; w < 4; ++w) m = max(m, red[w * kN + tl]);
          const float top = unordered(m), old = thr[tl] - 8.f;
          if (top > old) {
            cr = old == -INFINITY ? 0.f : ex2(old - top);
            thr[tl] = top + 8.f;
            mneg[tl] = -top;
          }
        }
        asm volatile("barrier.cta.sync 2, 128;" ::: "memory");  // (every red has been read)
        if (tl < 16 * nch) red[tl] = __float_as_int(cr);
        asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
        const float* f = reinterpret_cast<const float*>(red);
#pragma unroll
        for (int r = 0; r < kN; ++r)
          if (r < 16 * nch) l[r] *= f[r];
        if (j > 0) {
          ok &= wait(p_free((j - 1) & 1), ((j - 1) >> 1) & 1);  // O is at rest
          fence_after();
#pragma unroll 1
          for (int b = 0; b < G::VC; ++b)
#pragma unroll 1
            for (int c = 0; c < nch; ++c) {
              uint32_t v[16];
              const uint32_t o_at = tmem + lanes + G::O_COL + b * kN + 16 * c;
              __syncwarp();
              asm volatile(
                  "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                  "%13, %14, %15}, [%16];"
                  : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                    "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                  : "r"(o_at)
                  : "memory");
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f[16 * c + i]);
              tmem_st16(o_at, v);
            }
          tmem_wait_st();
          fence_before();
        }
        asm volatile("barrier.cta.sync 2, 128;" ::: "memory");  // (every red has been read)
      }
      if (j >= 2) ok &= wait(p_free(j & 1), ((j - 2) >> 1) & 1);  // the buffer's last reader
      uint8_t* pbuf = smem + G::P_OFF + (j & 1) * (kTile * kN * 2) + tl * 128;
#pragma unroll
      for (int c = 0; c < kN / 16; ++c) {
        if (c >= nch) break;
        float x[16];
        logits(s_at, c, at, cut, x);
        uint32_t pk[8];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 mn = *reinterpret_cast<const float2*>(mneg + 16 * c + i);
          const float a = ex2(x[i] + mn.x), b = ex2(x[i + 1] + mn.y);
          l[16 * c + i] += a;
          l[16 * c + i + 1] += b;
          pk[i / 2] = mma::pack_h2(a * norm, b * norm);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<uint4*>(pbuf + (((2 * c + h) ^ (tl & 7)) << 4)) =
              make_uint4(pk[4 * h], pk[4 * h + 1], pk[4 * h + 2], pk[4 * h + 3]);
      }
      mma::fence_proxy_async();
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(p_ready(j & 1));
    }
    if (ok) ok = wait(all_done, 0);
    fence_after();
    // ---- sums over the positions, O to shared memory ---------------------------------------------
    if (ok) {
      float* sums = reinterpret_cast<float*>(red);
#pragma unroll
      for (int r = 0; r < kN; ++r) {
        float v = l[r];
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) sums[(warp & 3) * kN + r] = v;
      }
      float* fin = reinterpret_cast<float*>(smem + G::RING);  // [row][D] over the slots
      if (ntiles > 0) {
#pragma unroll 1
        for (int b = 0; b < G::VC; ++b) {
          const int dim = b * 128 + (is_tq(VF) ? (tl & ~15) + tq_unswap(tl & 15) : tl);
#pragma unroll 1
          for (int c = 0; c < nch; ++c) {
            uint32_t v[16];
            __syncwarp();
            asm volatile(
                "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                "%14, %15}, [%16];"
                : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                  "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                : "r"(tmem + lanes + G::O_COL + b * kN + 16 * c)
                : "memory");
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) fin[(16 * c + i) * D + dim] = __uint_as_float(v[i]);
          }
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
    const float* fin = reinterpret_cast<const float*>(smem + G::RING);
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
  } else if (warp == 0) {  // the products under way, before their operands and TMEM go
    const uint64_t since = global_ns();
    while (!mbar_try_wait(all_done, 0) && global_ns() - since < mma::kWaitLimitNs) {
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1) tmem_free(tmem, G::COLS);
}

template <int D, int KF, int VF>
qps_status launch_tt(const PagedAttnParams& p, cudaStream_t s) {
  using G = GeoTt<D>;
  static_assert(G::SMEM <= 227 * 1024, "the slots exceed the shared memory of one CTA");
  static_assert(G::O_COL + G::VC * kN <= G::COLS, "S and O exceed TMEM");
  static_assert(kN * D * 4 <= kSlots * kSlot, "the output rows fit the slots");
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
  QPS_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, p));
  count_launch();
  QPS_CUDA_TRY(cudaGetLastError());
  return QPS_OK;
}

// Every format pairing of one head_dim.
template <int D>
qps_status launch_tt_d(const PagedAttnParams& p, cudaStream_t s) {
#define QPS_TT_CASE(KF, VF) \
  if (p.kfmt == KF && p.vfmt == VF) return launch_tt<D, KF, VF>(p, s);
  QPS_TT_CASE(QPS_FMT_F16, QPS_FMT_F16)
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
