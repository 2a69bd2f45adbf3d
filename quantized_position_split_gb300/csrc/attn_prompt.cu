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
// times its scale may pass it by a rounding: 127 x 516).  A tile decoded here is read by many row
// tiles; over the row tiles themselves the decoding would be repeated for each.
//
// A lane holds 16 elements of a row, a warp 512 / D rows at a time and kAhead such groups under way:
// compressed rows are small, and what bounds this is how many bytes are (13
// sequences of 1040 to 3500 positions, 8 heads of 128, q8_0 to 182 MB of bytes read and written:
// 32 us; a warp with one row, four under way, took 52).  A grid of a few CTAs an SM goes over all tiles: the lengths are on the device, and a CTA
// for each tile that there may be spent most of its time on those that are not.
constexpr int kDecodeWarps = 8, kAhead = 4;

// 16 elements as they are stored, and their scale or norm.
struct Raw {
  uint4 a, b;
  __half s;
};
// What a lane keeps from row to row: the rotation's signs of its elements.
struct LaneSigns {
  uint32_t s1, s2;
};

template <int D>
__device__ __forceinline__ Raw load_raw(int fmt, const uint8_t* const (&plane)[3], int64_t row, int c) {
  Raw r;
  r.a = r.b = make_uint4(0, 0, 0, 0);
  r.s = __float2half_rn(0.f);
  if (row < 0) return r;
  if (fmt == QPS_FMT_F16) {
    const uint4* src = reinterpret_cast<const uint4*>(plane[0] + row * (2 * D)) + 2 * c;
    r.a = src[0];
    r.b = src[1];
  } else if (fmt == QPS_FMT_Q8_0) {
    r.a = reinterpret_cast<const uint4*>(plane[0] + row * D)[c];
    r.s = reinterpret_cast<const __half*>(plane[1])[row * (D / 32) + c / 2];
  } else if (fmt == QPS_FMT_TQ4) {
    const uint2 x = reinterpret_cast<const uint2*>(plane[0] + row * (D / 2))[c];
    r.a.x = x.x;
    r.a.y = x.y;
    r.s = reinterpret_cast<const __half*>(plane[1])[row];
  } else {
    r.a.x = reinterpret_cast<const uint32_t*>(plane[0] + row * (D / 4))[c];
    if (fmt == QPS_FMT_TQ3) r.a.z = reinterpret_cast<const uint16_t*>(plane[1] + row * (D / 8))[c];
    r.s = reinterpret_cast<const __half*>(fmt == QPS_FMT_TQ3 ? plane[2] : plane[1])[row];
  }
  return r;
}

__device__ __forceinline__ float in_range(float x) { return fabsf(x) < INFINITY ? fminf(fmaxf(x, -65504.f), 65504.f) : x; }
// Two values as fp16, and what that left.
__device__ __forceinline__ void split2(float a, float b, uint32_t* hi, uint32_t* lo) {
  const __half2 h = __floats2half2_rn(in_range(a), in_range(b));
  const float2 f = __half22float2(h);
  const float c = a - f.x, d = b - f.y;
  const __half2 l = __floats2half2_rn(fabsf(c) <= 65504.f ? c : 0.f, fabsf(d) <= 65504.f ? d : 0.f);
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = *reinterpret_cast<const uint32_t*>(&l);
}

// levels: the codebook, in shared memory (the parameters' constant bank serves one address at a time).
template <int D>
__device__ __forceinline__ void decode_raw(const PromptParams& p, int fmt, const Raw& r, int lane, const LaneSigns& sg,
                                           const float* levels, uint32_t (&hi)[8], uint32_t (&lo)[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  const float f = __half2float(r.s);
  if (fmt == QPS_FMT_F16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi[i] = w[i];
      lo[i] = 0u;
    }
  } else if (fmt == QPS_FMT_Q8_0) {
    if (fabsf(f) <= 512.f) {  // the product fits fp16, and what its rounding leaves is exact
      const __half2 s2 = __half2half2(r.s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // code + 128 in the low bits of 1024 is exact
        const uint32_t c = __byte_perm(w[i / 2] ^ 0x80808080u, 0x64646464u, i & 1 ? 0x4342 : 0x4140);
        const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&c), __float2half2_rn(1152.f));
        const __half2 h = __hmul2(x, s2), l = __hfma2(x, s2, __hneg2(h));
        hi[i] = *reinterpret_cast<const uint32_t*>(&h);
        lo[i] = *reinterpret_cast<const uint32_t*>(&l);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t c = w[i / 2] >> (16 * (i & 1));
        split2((float)(int8_t)c * f, (float)(int8_t)(c >> 8) * f, &hi[i], &lo[i]);
      }
    }
  } else {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      int k;
      if (fmt == QPS_FMT_TQ4) {
        const int c = (int)(w[i / 8] >> (4 * (i % 8))) & 15;
        k = c & 8 ? c : 7 - c;
      } else {
        const int c = (int)(w[0] >> (2 * i)) & 3;
        if (fmt == QPS_FMT_TQ3) k = w[2] >> i & 1 ? 4 + c : 3 - c;
        else k = c & 2 ? c : 1 - c;
      }
      x[i] = __uint_as_float(__float_as_uint(levels[k]) ^ (sg.s2 >> i << 31));
    }
    // (a + b, a - b) over spans 1 .. G / 2: in the lane below 16, between lanes from there
#pragma unroll
    for (int h = 1; h < 16; h *= 2)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (!(i & h)) {
          const float a = x[i], b = x[i + h];
          x[i] = a + b;
          x[i + h] = a - b;
        }
#pragma unroll
    for (int o = 1; o < D / 16; o *= 2)
      if (16 * o < p.tq_block)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float other = __shfl_xor_sync(0xffffffffu, x[i], o);
          x[i] = lane & o ? other - x[i] : x[i] + other;
        }
    const float g = f * p.tq_scale;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(__float_as_uint(x[i] * g) ^ (sg.s1 >> i << 31));
#pragma unroll
    for (int i = 0; i < 8; ++i) split2(x[2 * i], x[2 * i + 1], &hi[i], &lo[i]);
  }
}

template <int D>
__global__ void __launch_bounds__(32 * kDecodeWarps) prompt_decode_kernel(const __grid_constant__ PromptParams p) {
  constexpr int LANES = D / 16, ROWS = 32 / LANES;      // lanes of a row, rows at a time
  constexpr int R = kPromptTile / kDecodeWarps, N = R / ROWS, A = N < kAhead ? N : kAhead;  // rows of a warp, its groups
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LANES;
  __shared__ float levels[16];
  if (threadIdx.x < 16) levels[threadIdx.x] = p.tq_levels[threadIdx.x];
  __syncthreads();
  const LaneSigns sg = {p.signs1[c / 2] >> (16 * (c & 1)), p.signs2[c / 2] >> (16 * (c & 1))};
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the sequences from b0 on, one a lane; the tiles before them, and up to each
  int b0 = 0, before = 0, upto = 0, cnt = 0;
  PromptSeq mine = {0, 0, 0};
  auto load = [&]() {
    mine = {0, 0, 0};
    if (b0 + lane < p.batch) mine = prompt_seq(p, b0 + lane);
    cnt = upto = mine.n > 0 ? prompt_tiles(p, mine.len - mine.n, mine.len - 1).count : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
  };
  load();
  const int head = blockIdx.y;
  for (int tile = blockIdx.x;; tile += gridDim.x) {
    unsigned hit;
    while (!(hit = __ballot_sync(0xffffffffu, before + upto > tile))) {
      before += __shfl_sync(0xffffffffu, upto, 31);
      b0 += 32;
      if (b0 >= p.batch) return;
      load();
    }
    if (tile >= p.dense_tiles) {  // (starts out of order can name more tokens than there are)
      if (lane == 0) atomicOr(p.err, kErrIndex);
      return;
    }
    const int src = __ffs(hit) - 1, b = b0 + src;
    const int n = __shfl_sync(0xffffffffu, mine.n, src), len = __shfl_sync(0xffffffffu, mine.len, src);
    const int at = tile - before - (__shfl_sync(0xffffffffu, upto, src) - __shfl_sync(0xffffffffu, cnt, src));
    const int first = prompt_tile(prompt_tiles(p, len - n, len - 1), at) * kPromptTile;
    const int low = p.window ? max(0, len - n - p.window + 1) : 0;
    // the page of position lane of the warp's rows (what no query token sees is zeros, and its page is
    // not looked up)
    int page = -1;
    const int pos = first + warp * R + lane % R;
    if (pos < len && (pos >= low || pos < p.sinks) && in_bounds(pos >> p.page_shift < p.table_width, p.err)) {
      page = p.table[b * p.table_stride + (pos >> p.page_shift)];
      if ((uint64_t)(int64_t)page >= (uint64_t)p.n_pages) {
        atomicOr(p.err, kErrIndex);
        page = -1;
      }
    }
    const int64_t to = ((int64_t)tile * p.hkv + head) * kPromptTile + warp * R;
#pragma unroll 1
    for (int g0 = blockIdx.z * A; g0 < N; g0 += gridDim.z * A) {
      int64_t row[A];
#pragma unroll
      for (int g = 0; g < A; ++g) {
        const int r = (g0 + g) * ROWS + lane / LANES, pg = __shfl_sync(0xffffffffu, page, r);
        row[g] = pg < 0 ? -1 : (((int64_t)pg * p.hkv + head) << p.page_shift) + ((first + warp * R + r) & ((1 << p.page_shift) - 1));
      }
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        __half* dst = side ? p.dense_v : p.dense_k;
        if (!dst) continue;
        const int fmt = side ? p.vfmt : p.kfmt;
        const bool two = !side || p.v_parts == 2;
        Raw raw[A];
#pragma unroll
        for (int g = 0; g < A; ++g) raw[g] = load_raw<D>(fmt, side ? p.v : p.k, row[g], c);
#pragma unroll
        for (int g = 0; g < A; ++g) {
          uint32_t hi[8], lo[8];
          decode_raw<D>(p, fmt, raw[g], lane, sg, levels, hi, lo);
          const int r = (g0 + g) * ROWS + lane / LANES;
          uint4* out = reinterpret_cast<uint4*>(dst + (to + r) * (two ? 2 * D : D) + 16 * c);
          out[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          out[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
          if (two) {
            out[D / 8] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            out[D / 8 + 1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
          }
        }
      }
    }
  }
}

template <int D>
qps_status launch_decode(const PromptParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  // (few tiles of wide rows: the rows of a warp are shared out)
  const int sms = sm_count_current(), most = std::max(1, kPromptTile / kDecodeWarps / (512 / D) / kAhead);
  const int parts = std::min<int64_t>(most, std::max<int64_t>(1, sms * 4 / ((int64_t)p.dense_tiles * p.hkv)));
  cfg.gridDim = dim3((unsigned)std::min(p.dense_tiles, (sms * 4 + p.hkv - 1) / p.hkv), p.hkv, parts);
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
  p.resident = sms;
  const int64_t rows = a->tokens * p.group;
  p.tiles = (int)std::min<int64_t>(rows / prompt_rows(kv.d) + std::min<int64_t>(a->batch, a->tokens), rows);
  // tiles of positions that a sequence's tokens see, at most
  int64_t most = (held + kPromptTile - 1) / kPromptTile;
  if (p.window) most = std::min(most, ((int64_t)p.window + p.sinks + a->tokens + 4 * kPromptTile) / kPromptTile);
  // Row tiles that leave SMs without work share their positions among several CTAs.
  const int64_t ctas = std::max<int64_t>(1, (int64_t)p.tiles * kv.hkv * prompt_col_ctas(kv.d));
  p.n_split = (int)std::max<int64_t>(1, std::min<int64_t>(sms / ctas, most));
  // A ragged batch of few tokens: cut finer, so that one long sequence is not a few CTAs' work (its
  // tiles stay 16 to a part at least, beside a part's start and end of about 6), as long as the
  // parts stay small.
  const int64_t part = a->tokens * a->hq * kv.d * (int64_t)sizeof(float);
  if (a->batch > 1) p.n_split = (int)std::max<int64_t>(p.n_split, std::min({4 * sms / ctas, most / 16, ((int64_t)32 << 20) / std::max<int64_t>(1, part)}));
  // (a part's row is counted in 32 bits; tokens that fill the SMs are not split)
  if (p.n_split * a->tokens * a->hq >= (int64_t)1 << 32) p.n_split = 1;
  if ((int64_t)p.tiles * p.n_split * prompt_col_ctas(kv.d) * kv.hkv >= (int64_t)1 << 31)
    return bad("too many row tiles", QPS_ERR_UNSUPPORTED);
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t parts = p.n_split > 1 ? (size_t)p.n_split * a->tokens * a->hq : 0;
  out->off_lse = up(parts * kv.d * sizeof(float));
  out->off_k = out->off_lse + up(parts * sizeof(float));
  out->off_v = out->bytes = out->off_k;
  if (kv.kfmt != QPS_FMT_F16 || kv.vfmt != QPS_FMT_F16) {
    // tiles of all sequences that have tokens; a window leaves each its own length, its sinks and
    // what its tokens add
    const int64_t some = std::min<int64_t>(a->batch, a->tokens);
    int64_t dense = some * ((held + kPromptTile - 1) / kPromptTile);
    if (p.window)
      dense = std::min(dense, some * ((p.sinks + kPromptTile - 1) / kPromptTile + p.window / kPromptTile + 3) + a->tokens / kPromptTile);
    if (dense >= (int64_t)1 << 30) return bad("batch * table_width * page_size is too large for compressed rows", QPS_ERR_UNSUPPORTED);
    p.dense_tiles = (int)std::max<int64_t>(1, dense);
    const size_t side = (size_t)p.dense_tiles * kv.hkv * kPromptTile * kv.d * sizeof(__half);
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
