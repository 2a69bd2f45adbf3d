// Decode attention over a paged cache: argument checks, the split into chunks, and the
// merge of the chunks' parts.  The attention itself is attn_mma.cuh's kernel over page
// tables for few query rows, attn_tm.cuh's or attn_tt.cuh's for many (see shape_for).
//
// Measured over fp16 pages of 64 positions, 8 KV heads of 128, 4 rows each: 38 sequences of
// 8192 positions 6.6 TB/s of keys and values, one of 131072 87.5 us (6.1 TB/s); 33 ragged
// ones of 1 to 16384 positions on pages of 16: 62.5 us, 4.9 TB/s (bound by the start of each
// round of CTAs, several us until HBM is busy, and by the merge).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <exception>
#include <string>

#include "paged.h"

namespace qps {
namespace {

std::atomic<uint64_t> g_fault{0};

// ---- merge --------------------------------------------------------------------------------
// M = max lse, w = exp(lse - M), o = sum w o / sum w over the prefix's parts and the row's
// own chunks.  D / 4 threads read one part's row (16 bytes each); `groups` such sets share
// a row, kU parts of each in flight, so that a row takes about one round of loads; every
// thread keeps its maximum online and the sets meet in shared memory.  A row whose only
// part was written by the attention is skipped.
constexpr int kMergeThreads = 256;
constexpr int kU = 8;

__device__ __forceinline__ void store_out(void* o, int dtype, int64_t at, float4 v) {
  if (dtype == QPS_DT_F32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(o) + at) = v;
  } else {
    uint2 w;
    if (dtype == QPS_DT_F16) {
      const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
      w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
      w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(o) + at) = w;
  }
}

template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    paged_merge_kernel(const __grid_constant__ PagedAttnParams p, int groups) {
  constexpr int COLS = D / 4, SETS = kMergeThreads / COLS;
  __shared__ float wm[SETS], wd[SETS];
  __shared__ float4 wacc[SETS][COLS];
  const int rows = p.n_q * p.hq;
  const int set = threadIdx.x / COLS, grp = set % groups, col = (threadIdx.x % COLS) * 4;
  const int64_t row = (int64_t)blockIdx.x * (SETS / groups) + set / groups;
  const bool real = row < p.rows_total;
  const int b = real ? (int)(row / rows) : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 own = p.chunks[b];
  const int first = own.x, count = own.y;
  const bool mine = real && !(count == 1 && p.n_prefix == 0) &&  // (else written by the attention)
                    in_bounds(first >= 0 && count > 0 && first + count <= p.max_chunks, p.err);
  const int total = mine ? p.n_prefix + count : 0;
  float m = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t0 = grp; t0 < total; t0 += groups * kU) {
    float l[kU];
    float4 v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int t = t0 + u * groups;
      l[u] = -INFINITY;
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t < total) {
        const bool pre = t < p.n_prefix;
        const int64_t at = pre ? (int64_t)t * p.rows_total + row : (int64_t)(first + t - p.n_prefix) * rows + (row - (int64_t)b * rows);
        l[u] = (pre ? p.pre_lse : p.own_lse)[at];
        v[u] = *reinterpret_cast<const float4*>((pre ? p.pre_o : p.own_o) + at * D + col);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (l[u] == -INFINITY) continue;
      if (l[u] > m) {
        const float cr = __expf(m - l[u]);  // 0 when m == -inf
        den *= cr;
        acc = make_float4(acc.x * cr, acc.y * cr, acc.z * cr, acc.w * cr);
        m = l[u];
      }
      const float w = __expf(l[u] - m);
      den += w;
      acc.x = fmaf(w, v[u].x, acc.x);
      acc.y = fmaf(w, v[u].y, acc.y);
      acc.z = fmaf(w, v[u].z, acc.z);
      acc.w = fmaf(w, v[u].w, acc.w);
    }
  }
  float mx = m, dt = den;
  float4 s = acc;
  if (groups > 1) {
    if (col == 0) {
      wm[set] = m;
      wd[set] = den;
    }
    wacc[set][col / 4] = acc;
    __syncthreads();
    if (grp != 0) return;
    for (int g = 1; g < groups; ++g) mx = fmaxf(mx, wm[set + g]);
    dt = 0.f;
    s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = 0; g < groups; ++g) {
      const float f = wm[set + g] == -INFINITY ? 0.f : __expf(wm[set + g] - mx);
      dt += wd[set + g] * f;
      const float4 a = wacc[set + g][col / 4];
      s.x = fmaf(a.x, f, s.x);
      s.y = fmaf(a.y, f, s.y);
      s.z = fmaf(a.z, f, s.z);
      s.w = fmaf(a.w, f, s.w);
    }
  }
  if (!mine) return;
  // (a NaN logit makes its row's sums NaN: it stays one)
  const bool empty = mx == -INFINITY && dt == 0.f;
  const float inv = empty ? 0.f : 1.f / dt;
  store_out(p.out, p.out_dtype, row * D + col, make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv));
  if (col == 0) p.out_lse[row] = empty ? -INFINITY : mx + logf(dt);
}

template <int D>
qps_status launch_merge(const PagedAttnParams& p, int parts, cudaStream_t s) {
  constexpr int SETS = kMergeThreads / (D / 4);
  int groups = 1;
  while (groups < SETS && groups * kU < parts) groups *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.rows_total + SETS / groups - 1) / (SETS / groups)));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  QPS_CUDA_TRY(cudaLaunchKernelEx(&cfg, paged_merge_kernel<D>, p, groups));
  count_launch();
  QPS_CUDA_TRY(cudaGetLastError());
  return QPS_OK;
}

// ---- plan -----------------------------------------------------------------------------------
struct Plan {
  PagedAttnParams p;
  int window, sinks, win_round;  // (see WindowAttnParams; window 0: none)
  PagedKernel prefix_kernel, own_kernel;
  int parts;   // most parts a row can have; one: no merge
  size_t off_pre_lse, off_own_o, off_own_lse, off_chunks, bytes;
};

// Chunks of the sequences' own positions.  Few sequences: one round of the CTAs the GPU
// holds, less one for each sequence's short last chunk (a second round of a few CTAs costs
// as much as a full one).  More sequences than half a round: kWaves rounds, so that ragged
// lengths level out.  Each at least kMinPositions long, so that a part is worth its merge,
// or kMinMany where the sequences alone fill a round (64 suffixes of 1 to 512 positions
// behind a prefix, 8 KV heads: 23 us in chunks of 128).
constexpr int kWaves = 2;
constexpr int kMinPositions = 128, kMinMany = 512;

// The kernel for `rows` query rows per KV head, and the rows, positions and CTAs per SM
// that it works with.  The tcgen05 kernels cost the same for few rows as for many; the
// mma.sync kernel reads a chunk once for each 8, 16 or 24 rows.  16 sequences of 8192
// positions, us, tcgen05 against mma.sync:
//   f16 / f16, 8 heads of 128:    8 rows 99 / 96, 12 rows 101 / 113, 24 rows 107 / 131, 40 rows 116 / 202
//   f16 / f16, 8 heads of 64:     16 rows 68 / 65, 20 rows 70 / 79, 40 rows 76 / 123
//   q8_0 / q8_0, 8 heads of 128:  16 rows 109 / 114, 17 rows 137 / 148, 24 rows 143 / 151, 32 rows 147 / 225
//   f16 / q8_0, 8 heads of 128:   16 rows 108 / 103, 17 rows 116 / 132
//   q8_0 / f16, 8 heads of 128:   16 rows 100 / 94, 17 rows 111 / 115
//   q8_0 / tq3, 8 heads of 128:   24 rows 156 / 149, 32 rows 163 / 224
//   f16 / tq3, 8 heads of 128:    24 rows 135 / 136
//   q8_0 / tq3, 4 heads of 256:   8 rows 110 / 75, 9 rows 110 / 179
//   f16 / f16, 4 heads of 256:    8 rows 165 / 93, 9 rows 165 / 170
//   q8_0 / tq3, 2 heads of 512:   8 rows 85 / 63, 9 rows 86 / 120
// (A TurboQuant K, a TQ4 V and compressed rows at head_dim 64 have no tcgen05 instance, which
// is not a measured choice: any number of rows goes to the mma.sync kernel.)
struct Shape {
  PagedKernel kernel;
  int rows, tile, ctas_per_sm;
};
Shape shape_for(const PagedKv& kv, int rows, bool shared) {
  if (kv.kfmt == QPS_FMT_F16 && kv.vfmt == QPS_FMT_F16 && kv.d <= 128) {
    if (rows > (kv.d == 64 ? 16 : 8)) return {kTm, 128, 128, 1};
  } else if (kv.d >= 128 && !is_tq(kv.kfmt) && kv.vfmt != QPS_FMT_TQ4) {
    if (rows > (kv.d > 128 ? 8 : is_tq(kv.vfmt) ? 24 : 16)) return {kTt, 64, 128, 1};
  }
  const int n = mma_tile_rows(kv.d, rows, shared);
  return {kMma, n, 32, mma_ctas_per_sm(kv.d, n / 8, kv.vfmt)};
}

qps_status plan_paged(const qps_paged_attn_args* a, Plan* out) {
  if (!a) return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: args is NULL");
  PagedKv kv;
  qps_status st = check_paged_kv(a->kv, "attn_decode_paged", &kv);
  if (st != QPS_OK) return st;
  if (!a->q || !aligned_to(a->q, 16)) return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: q is NULL or not 16-byte aligned");
  if (a->batch < 1 || a->batch > 65535) return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: batch must be in [1, 65535]");
  if (a->n_q < 1 || a->n_q > 64) return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: n_q must be in [1, 64]");
  if (a->hq < 1 || a->hq % kv.hkv) return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: hq must be a multiple of hkv");
  const int group = a->hq / kv.hkv, rows = a->n_q * group;
  if (group > 1024 || rows > 1024) return fail(QPS_ERR_UNSUPPORTED, "attn_decode_paged: more than 1024 query rows per KV head and sequence");
  if (a->q_batch_stride % 8 || (a->batch > 1 && a->q_batch_stride < (int64_t)a->n_q * a->hq * kv.d))
    return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: q_batch_stride must be >= n_q*hq*d and a multiple of 8");
  if (!a->page_table || !aligned_to(a->page_table, 4) || !a->kv_lens || !aligned_to(a->kv_lens, 4))
    return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: page_table / kv_lens are NULL or misaligned");
  // (positions are 32-bit in the kernels, also those of the tile behind a sequence's last one;
  // so are the batch's units of 32 positions)
  if (a->table_width < 1 || ((int64_t)a->table_width << kv.page_shift) >= ((int64_t)1 << 31) - 1024)
    return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: need table_width >= 1 and table_width * page_size < 2^31 - 1024");
  if (a->batch * ((int64_t)a->table_width << kv.page_shift) >= (int64_t)1 << 35)
    return fail(QPS_ERR_UNSUPPORTED, "attn_decode_paged: batch * table_width * page_size must be below 2^35");
  if (a->batch > 1 && a->table_stride < a->table_width)
    return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: table_stride must be >= table_width");
  if (a->shared_len < 0 || a->shared_len & ((1 << kv.page_shift) - 1) ||
      a->shared_len > ((int64_t)a->table_width << kv.page_shift))
    return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: shared_len must be a multiple of page_size within the table");
  if (a->o_dtype != QPS_DT_F16 && a->o_dtype != QPS_DT_BF16 && a->o_dtype != QPS_DT_F32)
    return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: unknown o_dtype");
  if (!std::isfinite(a->scale) || !std::isfinite(a->softcap))
    return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: scale and softcap must be finite");
  if (a->window < 0 || a->sinks < 0 || (a->window > 0 && a->n_q > 1 && !a->causal))
    return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: window and sinks must be >= 0, and a window of several query tokens causal");
  const int64_t rows_total = (int64_t)a->batch * a->n_q * a->hq;
  if (rows_total > 0x7fffffffLL) return fail(QPS_ERR_UNSUPPORTED, "attn_decode_paged: too many rows");
  const int sms = sm_count_current();
  if (sms <= 0) return fail(QPS_ERR_CUDA, "attn_decode_paged: cannot query the current device's SM count");

  PagedAttnParams& p = out->p;
  p = PagedAttnParams{};
  p.q = reinterpret_cast<const __half*>(a->q);
  p.q_bstride = a->batch > 1 ? a->q_batch_stride : (int64_t)a->n_q * a->hq * kv.d;
  p.batch = a->batch;
  p.hq = a->hq;
  p.hkv = kv.hkv;
  p.d = kv.d;
  p.group = group;
  p.kfmt = kv.kfmt;
  p.vfmt = kv.vfmt;
  const int64_t page = (int64_t)1 << kv.page_shift;
  p.k = KvSide{kv.k[0], kv.k[1], kv.k[2], 1, page, kv.hkv * page};
  p.v = KvSide{kv.v[0], kv.v[1], kv.v[2], 1, page, kv.hkv * page};
  p.scale = a->scale;
  p.softcap = a->softcap > 0.f ? a->softcap : 0.f;
  p.n_q = a->n_q;
  p.causal = a->causal ? 1 : 0;
  p.rows_total = rows_total;
  p.q_elems = (int64_t)(a->batch - 1) * p.q_bstride + (int64_t)a->n_q * a->hq * kv.d;
  p.k_rows = p.v_rows = kv.n_pages * page * kv.hkv;
  const int g = a->kv.tq_block == 0 ? kv.d : a->kv.tq_block;
  p.vblock = g;
  p.v_out_scale = (float)(1.0 / std::sqrt((double)kv.d * g));
  p.k_rot_scale = (float)(1.0 / std::sqrt((double)g));
  p.k_norm_scale = (float)(1.0 / std::sqrt((double)kv.d));
  if (is_tq(kv.vfmt)) {
    for (int i = 0; i < kv.d / 32; ++i) {
      p.vsigns[i] = a->kv.signs1[i];
      p.vsigns2[i] = a->kv.signs2 ? a->kv.signs2[i] : 0u;
    }
    const Codebook* cb = tq_codebook(tq_bits(kv.vfmt));
    for (int i = 0; i < cb->n; ++i) p.tq_levels[i] = cb->levels[i];
  }
  p.table = a->page_table;
  p.table_stride = a->batch > 1 ? a->table_stride : a->table_width;
  p.lens = a->kv_lens;
  p.n_pages = kv.n_pages;
  p.page_shift = kv.page_shift;
  p.table_width = a->table_width;
  p.out_dtype = a->o_dtype;
  // (a window that no sequence outgrows is none; one that they do leaves no common prefix)
  const int held = a->table_width << kv.page_shift;
  out->window = a->window > 0 && a->window < held && a->sinks < held ? a->window : 0;
  out->sinks = out->window ? a->sinks : 0;

  // the prefix: whole tiles of the shared positions (what is left of them is read through
  // each sequence's own entries, which name the same pages)
  p.prefix_len = a->batch > 1 && out->window == 0 ? (int)(a->shared_len & ~(int64_t)31) : 0;
  if (p.prefix_len > 0) {
    const int all = a->batch * rows;
    const Shape sh = shape_for(kv, all, true);
    out->prefix_kernel = sh.kernel;
    const int ctas = kv.hkv * ((all + sh.rows - 1) / sh.rows), slots = sh.ctas_per_sm * sms;
    // one round of CTAs
    const int least = sh.kernel == kMma ? 512 : sh.tile;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(sh.kernel == kMma ? (slots + ctas - 1) / ctas : slots / ctas,
                                                                (p.prefix_len + least - 1) / least));
    const int64_t chunk = ((p.prefix_len + want - 1) / want + sh.tile - 1) / sh.tile * sh.tile;
    p.n_prefix = (int)((p.prefix_len + chunk - 1) / chunk);
    p.chunk = chunk;
  }
  {
    const Shape sh = shape_for(kv, rows, false);
    out->own_kernel = sh.kernel;
    const int ctas = kv.hkv * ((rows + sh.rows - 1) / sh.rows), slots = sh.ctas_per_sm * sms;
    const int round = slots / ctas;
    p.target = std::max(1, 2 * a->batch <= round ? round - a->batch + 1 : kWaves * slots / ctas);
    const int least = a->batch >= round ? kMinMany : kMinPositions;
    p.min_units = least / kPagedUnit;
    p.unit_round = sh.tile / kPagedUnit;
    out->win_round = sh.tile;
    // chunks of a sequence that fills its table (of what its window leaves), and of all of them
    int64_t most = ((int64_t)a->table_width << kv.page_shift) - p.prefix_len;
    if (out->window) most = std::min<int64_t>(most, (int64_t)out->window + a->n_q + out->sinks + 2 * sh.tile);
    const int64_t each = std::max<int64_t>(1, (most + least - 1) / least);
    p.max_chunks = (int)std::min<int64_t>((int64_t)p.target + a->batch, each * a->batch);
    out->parts = p.n_prefix + (int)std::min<int64_t>(each, p.target + 1);
  }
  const size_t own = (size_t)p.max_chunks * a->n_q * a->hq, pre = (size_t)p.n_prefix * rows_total;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  out->off_pre_lse = up(pre * kv.d * sizeof(float));
  out->off_own_o = out->off_pre_lse + up(pre * sizeof(float));
  out->off_own_lse = out->off_own_o + up(own * kv.d * sizeof(float));
  out->off_chunks = out->off_own_lse + up(own * sizeof(float));
  out->bytes = out->off_chunks + up((size_t)a->batch * sizeof(int2));
  return QPS_OK;
}

qps_status launch_paged(const PagedAttnParams& p, cudaStream_t s) {
  if (p.kernel == kTm) return p.d == 64 ? launch_paged_tm_d64(p, s) : launch_paged_tm_d128(p, s);
  if (p.kernel == kTt)
    return p.d == 128 ? launch_paged_tt_d128(p, s) : p.d == 256 ? launch_paged_tt_d256(p, s) : launch_paged_tt_d512(p, s);
  switch (p.d) {
    case 64: return launch_paged_mma_d64(p, s);
    case 128: return launch_paged_mma_d128(p, s);
    case 256: return launch_paged_mma_d256(p, s);
    default: return launch_paged_mma_d512(p, s);
  }
}

qps_status launch_window(const WindowAttnParams& p, cudaStream_t s) {
  if (p.kernel == kTm) return p.d == 64 ? launch_window_tm_d64(p, s) : launch_window_tm_d128(p, s);
  if (p.kernel == kTt)
    return p.d == 128 ? launch_window_tt_d128(p, s) : p.d == 256 ? launch_window_tt_d256(p, s) : launch_window_tt_d512(p, s);
  switch (p.d) {
    case 64: return launch_window_mma_d64(p, s);
    case 128: return launch_window_mma_d128(p, s);
    case 256: return launch_window_mma_d256(p, s);
    default: return launch_window_mma_d512(p, s);
  }
}

bool meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const char *pa = (const char*)a, *pb = (const char*)b;
  return pa < pb + nb && pb < pa + na;
}

qps_status attn_decode_paged(const qps_paged_attn_args* a, cudaStream_t s) {
  Plan pl;
  qps_status st = plan_paged(a, &pl);
  if (st != QPS_OK) return st;
  if (!a->o || !aligned_to(a->o, 16) || !a->lse || !aligned_to(a->lse, 4))
    return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: o / lse are NULL or misaligned (o: 16 bytes)");
  if (!a->workspace || a->workspace_bytes < pl.bytes)
    return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: workspace missing or smaller than qps_attn_paged_plan reports");
  if (!aligned_to(a->workspace, 256)) return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: workspace must be 256-byte aligned");
  PagedAttnParams& p = pl.p;
  // what is written lies apart from the queries (read until the last CTA) and from the rest
  const int64_t o_bytes = p.rows_total * p.d * dtype_bytes(a->o_dtype);
  const struct { const void* at; int64_t bytes; } out[3] = {
      {a->o, o_bytes}, {a->lse, p.rows_total * (int64_t)sizeof(float)}, {a->workspace, (int64_t)pl.bytes}};
  for (int i = 0; i < 3; ++i) {
    if (meet(out[i].at, out[i].bytes, a->q, p.q_elems * (int64_t)sizeof(__half)) ||
        meet(out[i].at, out[i].bytes, out[(i + 1) % 3].at, out[(i + 1) % 3].bytes))
      return fail(QPS_ERR_INVALID_ARG, "attn_decode_paged: o, lse and workspace overlap one another or q");
  }
  p.err = device_error_word();
  if (!p.err) return fail(QPS_ERR_CUDA, "attn_decode_paged: cannot allocate the device error word");
  char* ws = reinterpret_cast<char*>(a->workspace);
  p.pre_o = reinterpret_cast<float*>(ws);
  p.pre_lse = reinterpret_cast<float*>(ws + pl.off_pre_lse);
  p.own_o = reinterpret_cast<float*>(ws + pl.off_own_o);
  p.own_lse = reinterpret_cast<float*>(ws + pl.off_own_lse);
  p.chunks = reinterpret_cast<int2*>(ws + pl.off_chunks);
  p.out = a->o;
  p.out_lse = a->lse;
  const uint64_t fault = take_paged_fault();
  p.drop_tile = (int)(fault & 0xffffffffu) - 1;
  p.wait_ns = fault ? (uint32_t)(fault >> 32) * 1000000u : (uint32_t)kWaitLimitNs;
  const int rows = p.n_q * p.group;
  if (p.n_prefix > 0) {
    PagedAttnParams f = p;
    f.shared = 1;
    f.kernel = pl.prefix_kernel;
    f.rows_per_cta = p.batch * rows;
    f.n_split = p.n_prefix;
    f.begin = 0;
    f.end = p.prefix_len;
    st = launch_paged(f, s);
    if (st != QPS_OK) return st;
  }
  p.shared = 0;
  p.kernel = pl.own_kernel;
  p.rows_per_cta = rows;
  p.chunk = 0;
  if (pl.window) {
    WindowAttnParams w{};
    static_cast<PagedAttnParams&>(w) = p;
    w.window = pl.window;
    w.sinks = pl.sinks;
    w.win_round = pl.win_round;
    st = launch_window(w, s);
  } else {
    st = launch_paged(p, s);
  }
  if (st != QPS_OK || pl.parts <= 1) return st;
  switch (p.d) {
    case 64: return launch_merge<64>(p, pl.parts, s);
    case 128: return launch_merge<128>(p, pl.parts, s);
    case 256: return launch_merge<256>(p, pl.parts, s);
    default: return launch_merge<512>(p, pl.parts, s);
  }
}

}  // namespace

uint64_t take_paged_fault() { return g_fault.load(std::memory_order_relaxed) ? g_fault.exchange(0) : 0; }

}  // namespace qps

using namespace qps;

extern "C" {

qps_status qps_attn_paged_plan(const qps_paged_attn_args* a, size_t* workspace_bytes) {
  try {
    Plan pl;
    const qps_status st = plan_paged(a, &pl);
    if (st == QPS_OK && workspace_bytes) *workspace_bytes = pl.bytes;
    return st;
  } catch (const std::exception&) {
    return QPS_ERR_INTERNAL;
  }
}

qps_status qps_paged_inject_fault(int32_t tile, int32_t wait_ms) {
  if (tile < -1 || tile >= 1 << 30 || (tile >= 0 && (wait_ms < 1 || wait_ms > 1000)))
    return fail(QPS_ERR_INVALID_ARG, "paged_inject_fault: need tile >= -1 and wait_ms in [1, 1000]");
  g_fault.store(tile < 0 ? 0 : (uint64_t)(uint32_t)wait_ms << 32 | (uint32_t)(tile + 1));
  return QPS_OK;
}

qps_status qps_attn_decode_paged(const qps_paged_attn_args* a, void* stream) {
  try {
    return attn_decode_paged(a, reinterpret_cast<cudaStream_t>(stream));
  } catch (const std::exception&) {
    return QPS_ERR_INTERNAL;
  }
}

}  // extern "C"
