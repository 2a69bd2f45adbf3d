// Attention of prompt chunks over a paged cache: argument checks, the decoding of compressed rows,
// the merge of split positions.  The attention itself is attn_prompt.cuh's kernel.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <string>

#include "attn_prompt.h"

namespace qps {
namespace {

// ---- decoding -------------------------------------------------------------------------------
// The tiles that any query token of a sequence sees, once, to fp16 rows: the value, and behind it
// what its rounding left (V: where v_parts is 2).  The value is cut to fp16's range (a q8_0 code
// times its scale may pass it by a rounding: 127 x 516).  A warp takes a row: lane L holds the
// elements E L .. E L + E - 1 (E = D / 32).  A tile decoded here is read by many row tiles; over
// the row tiles themselves the decoding would be repeated for each.
constexpr int kDecodeWarps = 8, kDecodeRows = 32;  // rows per CTA

template <int D>
__device__ __forceinline__ void decode_row(const PromptParams& p, int fmt, const uint8_t* const (&plane)[3], int64_t row,
                                           int lane, float (&x)[D / 32]) {
  constexpr int E = D / 32;
  const int e0 = lane * E;
  if (fmt == QPS_FMT_F16) {
    const __half* src = reinterpret_cast<const __half*>(plane[0]) + row * D + e0;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(src + i));
      x[i] = f.x;
      x[i + 1] = f.y;
    }
  } else if (fmt == QPS_FMT_Q8_0) {
    const int8_t* src = reinterpret_cast<const int8_t*>(plane[0]) + row * D + e0;
    const float sc = __half2float(reinterpret_cast<const __half*>(plane[1])[row * (D / 32) + e0 / 32]);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const char2 c = *reinterpret_cast<const char2*>(src + i);
      x[i] = (float)c.x * sc;
      x[i + 1] = (float)c.y * sc;
    }
  } else {
    const int bits = tq_bits(fmt);
    const float norm = __half2float(reinterpret_cast<const __half*>(fmt == QPS_FMT_TQ3 ? plane[2] : plane[1])[row]);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = e0 + i;
      int k;
      if (bits == 4) {
        const int f = plane[0][row * (D / 2) + e / 2] >> (4 * (e & 1)) & 15;
        k = f & 8 ? 8 + (f & 7) : 7 - (f & 7);
      } else {
        const int f = plane[0][row * (D / 4) + e / 4] >> (2 * (e & 3)) & 3;
        if (bits == 3) k = plane[1][row * (D / 8) + e / 8] >> (e & 7) & 1 ? 4 + f : 3 - f;
        else k = f & 2 ? 2 + (f & 1) : 1 - (f & 1);
      }
      const float c = p.tq_levels[k];
      x[i] = (p.signs2[e >> 5] >> (e & 31)) & 1u ? -c : c;
    }
    // (a + b, a - b) over spans 1 .. G / 2: in the lane below E, between lanes from there
#pragma unroll
    for (int h = 1; h < E; h *= 2)
      if (h < p.tq_block)
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (!(i & h)) {
            const float a = x[i], b = x[i + h];
            x[i] = a + b;
            x[i + h] = a - b;
          }
#pragma unroll
    for (int o = 1; o < 32; o *= 2)
      if (o * E < p.tq_block)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float other = __shfl_xor_sync(0xffffffffu, x[i], o);
          x[i] = lane & o ? other - x[i] : x[i] + other;
        }
    const float f = norm * p.tq_scale;
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = (p.signs1[(e0 + i) >> 5] >> ((e0 + i) & 31)) & 1u ? -(x[i] * f) : x[i] * f;
  }
}

__device__ __forceinline__ float in_range(float x) { return fabsf(x) < INFINITY ? fminf(fmaxf(x, -65504.f), 65504.f) : x; }

template <int D>
__global__ void __launch_bounds__(32 * kDecodeWarps) prompt_decode_kernel(const __grid_constant__ PromptParams p) {
  constexpr int E = D / 32, PARTS = kPromptTile / kDecodeRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, head = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  const int b = blockIdx.x / PARTS / p.dense_tiles, at = blockIdx.x / PARTS % p.dense_tiles;
  const PromptSeq sq = prompt_seq(p, b);
  if (sq.n == 0) return;
  const PromptTiles t = prompt_tiles(p, sq.len - sq.n, sq.len - 1);
  if (at >= t.count) return;
  const int first = prompt_tile(t, at) * kPromptTile;
  const int low = p.window ? max(0, sq.len - sq.n - p.window + 1) : 0;
  for (int r = blockIdx.x % PARTS * kDecodeRows + warp; r < (blockIdx.x % PARTS + 1) * kDecodeRows; r += kDecodeWarps) {
    const int pos = first + r;
    // (what no query token sees is zeros, and its page is not looked up)
    int64_t row = -1;
    if (pos < sq.len && (pos >= low || pos < p.sinks) && in_bounds(pos >> p.page_shift < p.table_width, p.err)) {
      const int pg = p.table[b * p.table_stride + (pos >> p.page_shift)];
      if ((uint64_t)(int64_t)pg < (uint64_t)p.n_pages)
        row = (((int64_t)pg * p.hkv + head) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
      else
        atomicOr(p.err, kErrIndex);
    }
    const int64_t to = (((int64_t)b * p.dense_tiles + at) * p.hkv + head) * kPromptTile + r;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      __half* dst = side ? p.dense_v : p.dense_k;
      if (!dst) continue;
      float x[E];
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = 0.f;
      if (row >= 0) {
        if (side) decode_row<D>(p, p.vfmt, p.v, row, lane, x);
        else decode_row<D>(p, p.kfmt, p.k, row, lane, x);
      }
      __half hi[E], lo[E];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        hi[i] = __float2half_rn(in_range(x[i]));
        const float left = x[i] - __half2float(hi[i]);
        lo[i] = __float2half_rn(fabsf(left) <= 65504.f ? left : 0.f);
      }
      const bool two = !side || p.v_parts == 2;
      __half* out = dst + to * (two ? 2 * D : D) + lane * E;
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        *reinterpret_cast<__half2*>(out + i) = __halves2half2(hi[i], hi[i + 1]);
        if (two) *reinterpret_cast<__half2*>(out + D + i) = __halves2half2(lo[i], lo[i + 1]);
      }
    }
  }
}

template <int D>
qps_status launch_decode(const PromptParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * p.dense_tiles * (kPromptTile / kDecodeRows)), p.hkv);
  cfg.blockDim = dim3(32 * kDecodeWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  QPS_CUDA_TRY(cudaLaunchKernelEx(&cfg, prompt_decode_kernel<D>, p));
  count_launch();
  QPS_CUDA_TRY(cudaGetLastError());
  return QPS_OK;
}

// ---- merge ------------------------------------------------------------------------------------
// o = sum w o / sum w, w = exp(lse - max), over a row's parts; D / 4 threads a row, 16 bytes each.
constexpr int kMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) prompt_merge_kernel(const __grid_constant__ PromptParams p) {
  constexpr int COLS = D / 4;
  const int col = threadIdx.x % COLS * 4;
  const int64_t row = (int64_t)blockIdx.x * (kMergeThreads / COLS) + threadIdx.x / COLS, rows = p.tokens * p.hq;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= rows) return;
  const int64_t token = row / p.hq;  // (rows of no sequence are left as they are)
  if (token < p.starts[0] || token >= p.starts[p.batch]) return;
  float m = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int U = 8;
  for (int t0 = 0; t0 < p.n_split; t0 += U) {
    float l[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = (int64_t)(t0 + u) * rows + row;
      l[u] = t0 + u < p.n_split ? p.part_lse[at] : -INFINITY;
      v[u] = t0 + u < p.n_split ? *reinterpret_cast<const float4*>(p.part_o + at * D + col) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
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
  const bool none = m == -INFINITY && den == 0.f;  // (a NaN stays one)
  const float inv = none ? 0.f : 1.f / den;
  const float4 o = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  const int64_t to = row * D + col;
  if (p.out_dtype == QPS_DT_F32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + to) = o;
  } else if (p.out_dtype == QPS_DT_F16) {
    const __half2 a = __floats2half2_rn(o.x, o.y), b = __floats2half2_rn(o.z, o.w);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + to) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(o.x, o.y), b = __floats2bfloat162_rn(o.z, o.w);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + to) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  if (col == 0) p.out_lse[row] = none ? -INFINITY : m + logf(den);
}

template <int D>
qps_status launch_merge(const PromptParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.tokens * p.hq + kMergeThreads / (D / 4) - 1) / (kMergeThreads / (D / 4))));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  QPS_CUDA_TRY(cudaLaunchKernelEx(&cfg, prompt_merge_kernel<D>, p));
  count_launch();
  QPS_CUDA_TRY(cudaGetLastError());
  return QPS_OK;
}

// ---- plan -------------------------------------------------------------------------------------
struct Plan {
  PromptParams p;
  size_t off_lse, off_k, off_v, bytes;
};

qps_status bad(const char* what, qps_status st = QPS_ERR_INVALID_ARG) { return fail(st, std::string("attn_prompt_paged: ") + what); }

qps_status plan_prompt(const qps_paged_prompt_args* a, Plan* out) {
  if (!a) return bad("args is NULL");
  PagedKv kv;
  qps_status st = check_paged_kv(a->kv, "attn_prompt_paged", &kv);
  if (st != QPS_OK) return st;
  if (a->reserved0 != 0) return bad("reserved fields must be 0");
  if (a->tokens < 0) return bad("tokens must be >= 0");
  if (a->batch < 1 || a->batch > 65535) return bad("batch must be in [1, 65535]");
  if (a->hq < 1 || a->hq % kv.hkv) return bad("hq must be a multiple of hkv");
  // (rows and their sums over the row tiles are 32-bit in the kernel)
  if (a->hq > 65535 || a->tokens * a->hq >= (int64_t)1 << 31) return bad("tokens * hq must be below 2^31, hq below 2^16", QPS_ERR_UNSUPPORTED);
  if (a->tokens > 0 && (!a->q || !aligned_to(a->q, 16))) return bad("q is NULL or not 16-byte aligned");
  if (a->q_tok_stride % 8 || (a->tokens > 1 && a->q_tok_stride < (int64_t)a->hq * kv.d) || a->q_tok_stride > (int64_t)1 << 31)
    return bad("q_tok_stride must be >= hq*d, a multiple of 8 and at most 2^31");
  if (!a->q_starts || !aligned_to(a->q_starts, 4) || !a->page_table || !aligned_to(a->page_table, 4) || !a->kv_lens ||
      !aligned_to(a->kv_lens, 4))
    return bad("q_starts / page_table / kv_lens are NULL or misaligned");
  const int64_t held = (int64_t)a->table_width << kv.page_shift;
  if (a->table_width < 1 || held >= ((int64_t)1 << 31) - 1024) return bad("need table_width >= 1 and table_width * page_size < 2^31 - 1024");
  if (a->batch > 1 && a->table_stride < a->table_width) return bad("table_stride must be >= table_width");
  if (a->o_dtype != QPS_DT_F16 && a->o_dtype != QPS_DT_BF16 && a->o_dtype != QPS_DT_F32) return bad("unknown o_dtype");
  if (!std::isfinite(a->scale) || !std::isfinite(a->softcap)) return bad("scale and softcap must be finite");
  if (a->window < 0 || a->sinks < 0) return bad("window and sinks must be >= 0");
  const int sms = sm_count_current();
  if (sms <= 0) return bad("cannot query the current device's SM count", QPS_ERR_CUDA);

  PromptParams& p = out->p;
  p = PromptParams{};
  p.q = reinterpret_cast<const __half*>(a->q);
  p.tokens = a->tokens;
  p.q_tok = a->tokens > 1 ? a->q_tok_stride : (int64_t)a->hq * kv.d;
  p.batch = a->batch;
  p.hq = a->hq;
  p.hkv = kv.hkv;
  p.d = kv.d;
  p.group = a->hq / kv.hkv;
  p.starts = a->q_starts;
  p.table = a->page_table;
  p.table_stride = a->batch > 1 ? a->table_stride : a->table_width;
  p.table_width = a->table_width;
  p.page_shift = kv.page_shift;
  p.n_pages = kv.n_pages;
  p.lens = a->kv_lens;
  p.scale = a->scale;
  p.softcap = a->softcap > 0.f ? a->softcap : 0.f;
  // (a window that no sequence outgrows is none)
  p.window = a->window > 0 && a->window < held && a->sinks < held ? a->window : 0;
  p.sinks = p.window ? a->sinks : 0;
  p.out_dtype = a->o_dtype;
  p.kfmt = kv.kfmt;
  p.vfmt = kv.vfmt;
  p.v_parts = kv.vfmt != QPS_FMT_F16 && a->o_dtype != QPS_DT_BF16 ? 2 : 1;
  for (int i = 0; i < 3; ++i) {
    p.k[i] = kv.k[i];
    p.v[i] = kv.v[i];
  }
  if (is_tq(kv.vfmt)) {
    p.tq_block = a->kv.tq_block == 0 ? kv.d : a->kv.tq_block;
    p.tq_scale = (float)(1.0 / std::sqrt((double)kv.d * p.tq_block));
    for (int i = 0; i < kv.d / 32; ++i) {
      p.signs1[i] = a->kv.signs1[i];
      p.signs2[i] = a->kv.signs2 ? a->kv.signs2[i] : 0u;
    }
    const Codebook* cb = tq_codebook(tq_bits(kv.vfmt));
    for (int i = 0; i < cb->n; ++i) p.tq_levels[i] = cb->levels[i];
  }
  // row tiles: full ones, and at most one that is not for each sequence
  const int64_t rows = a->tokens * p.group;
  p.tiles = (int)std::min<int64_t>(rows / prompt_rows(kv.d) + std::min<int64_t>(a->batch, a->tokens), rows);
  // tiles of positions that a sequence's tokens see, at most
  int64_t most = (held + kPromptTile - 1) / kPromptTile;
  if (p.window) most = std::min(most, ((int64_t)p.window + p.sinks + a->tokens + 4 * kPromptTile) / kPromptTile);
  // Row tiles that leave SMs without work share their positions among several CTAs.
  const int64_t ctas = std::max<int64_t>(1, (int64_t)p.tiles * kv.hkv * prompt_col_ctas(kv.d));
  p.n_split = (int)std::max<int64_t>(1, std::min<int64_t>(sms / ctas, most));
  if ((int64_t)p.tiles * p.n_split * prompt_col_ctas(kv.d) * kv.hkv >= (int64_t)1 << 31)
    return bad("too many row tiles", QPS_ERR_UNSUPPORTED);
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t parts = p.n_split > 1 ? (size_t)p.n_split * a->tokens * a->hq : 0;
  out->off_lse = up(parts * kv.d * sizeof(float));
  out->off_k = out->off_lse + up(parts * sizeof(float));
  out->off_v = out->bytes = out->off_k;
  if (kv.kfmt != QPS_FMT_F16 || kv.vfmt != QPS_FMT_F16) {
    p.dense_tiles = (int)most;
    if (a->batch * most * (kPromptTile / kDecodeRows) >= (int64_t)1 << 31)
      return bad("batch * table_width * page_size is too large for compressed rows", QPS_ERR_UNSUPPORTED);
    const size_t side = (size_t)a->batch * most * kv.hkv * kPromptTile * kv.d * sizeof(__half);
    out->off_v = out->off_k + (kv.kfmt != QPS_FMT_F16 ? up(2 * side) : 0);
    out->bytes = out->off_v + (kv.vfmt != QPS_FMT_F16 ? up(p.v_parts * side) : 0);
  }
  return QPS_OK;
}

bool meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const char *pa = (const char*)a, *pb = (const char*)b;
  return na > 0 && nb > 0 && pa < pb + nb && pb < pa + na;
}

qps_status attn_prompt_paged(const qps_paged_prompt_args* a, cudaStream_t s) {
  Plan pl;
  qps_status st = plan_prompt(a, &pl);
  if (st != QPS_OK || a->tokens == 0) return st;
  PromptParams& p = pl.p;
  if (!a->o || !aligned_to(a->o, 16) || !a->lse || !aligned_to(a->lse, 4)) return bad("o / lse are NULL or misaligned (o: 16 bytes)");
  if (pl.bytes > 0 && (!a->workspace || a->workspace_bytes < pl.bytes))
    return bad("workspace missing or smaller than qps_attn_prompt_plan reports");
  if (!aligned_to(a->workspace, 256)) return bad("workspace must be 256-byte aligned");
  // what is written lies apart from the queries (read until the last CTA) and from the rest
  const int64_t rows = a->tokens * a->hq;
  const int64_t q_bytes = ((a->tokens - 1) * p.q_tok + (int64_t)a->hq * p.d) * (int64_t)sizeof(__half);
  const struct { const void* at; int64_t bytes; } out[3] = {
      {a->o, rows * p.d * dtype_bytes(a->o_dtype)}, {a->lse, rows * (int64_t)sizeof(float)}, {a->workspace, (int64_t)pl.bytes}};
  for (int i = 0; i < 3; ++i)
    if (meet(out[i].at, out[i].bytes, a->q, q_bytes) ||
        meet(out[i].at, out[i].bytes, out[(i + 1) % 3].at, out[(i + 1) % 3].bytes))
      return bad("o, lse and workspace overlap one another or q");
  p.err = device_error_word();
  if (!p.err) return bad("cannot allocate the device error word", QPS_ERR_CUDA);
  char* ws = reinterpret_cast<char*>(a->workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_lse = reinterpret_cast<float*>(ws + pl.off_lse);
  p.dense_k = p.kfmt != QPS_FMT_F16 ? reinterpret_cast<__half*>(ws + pl.off_k) : nullptr;
  p.dense_v = p.vfmt != QPS_FMT_F16 ? reinterpret_cast<__half*>(ws + pl.off_v) : nullptr;
  p.out = a->o;
  p.out_lse = a->lse;
  const uint64_t fault = take_paged_fault();
  p.drop_tile = (int)(fault & 0xffffffffu) - 1;
  p.wait_ns = fault ? (uint32_t)(fault >> 32) * 1000000u : (uint32_t)kWaitLimitNs;
  if (p.dense_tiles > 0) {
    st = p.d == 64 ? launch_decode<64>(p, s) : p.d == 128 ? launch_decode<128>(p, s) : p.d == 256 ? launch_decode<256>(p, s) : launch_decode<512>(p, s);
    if (st != QPS_OK) return st;
  }
  using Launch = qps_status (*)(const PromptParams&, cudaStream_t);
  static const Launch launches[4][2] = {{launch_prompt_d64, launch_prompt_d64_q},
                                        {launch_prompt_d128, launch_prompt_d128_q},
                                        {launch_prompt_d256, launch_prompt_d256_q},
                                        {launch_prompt_d512, launch_prompt_d512_q}};
  st = launches[p.d == 64 ? 0 : p.d == 128 ? 1 : p.d == 256 ? 2 : 3][p.dense_k ? 1 : 0](p, s);
  if (st != QPS_OK || p.n_split == 1) return st;
  switch (p.d) {
    case 64: return launch_merge<64>(p, s);
    case 128: return launch_merge<128>(p, s);
    case 256: return launch_merge<256>(p, s);
    default: return launch_merge<512>(p, s);
  }
}

}  // namespace
}  // namespace qps

using namespace qps;

extern "C" {

qps_status qps_attn_prompt_plan(const qps_paged_prompt_args* a, size_t* workspace_bytes) {
  try {
    Plan pl;
    const qps_status st = plan_prompt(a, &pl);
    if (st == QPS_OK && workspace_bytes) *workspace_bytes = pl.bytes;
    return st;
  } catch (const std::exception&) {
    return QPS_ERR_INTERNAL;
  }
}

qps_status qps_attn_prompt_paged(const qps_paged_prompt_args* a, void* stream) {
  try {
    return attn_prompt_paged(a, reinterpret_cast<cudaStream_t>(stream));
  } catch (const std::exception&) {
    return QPS_ERR_INTERNAL;
  }
}

}  // extern "C"
