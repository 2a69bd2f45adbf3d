// Attention of prompt chunks over a paged cache: parameters shared by the checks and plan
// (attn_prompt.cu), the kernel's instances (attn_prompt.cuh) and the decoding of compressed rows.
#pragma once

#include "paged.h"

namespace qps {

constexpr int kPromptTile = 128;  // positions per tile

struct PromptParams {
  const __half* q;
  int64_t q_tok;          // elements between query tokens
  int64_t tokens;
  int batch, hq, hkv, d, group;
  const int32_t* starts;  // [batch + 1] first query token of each sequence
  const int32_t* table;
  int64_t table_stride;
  int table_width, page_shift;
  int64_t n_pages;
  const int32_t* lens;
  float scale, softcap;
  int window, sinks;      // window 0: none
  int tiles;              // row tiles there can be
  int resident;           // CTAs that run at once
  int n_split;            // parts a row tile's positions are cut into
  float* part_o;          // f32 [n_split][tokens * hq][D], [n_split][tokens * hq]
  float* part_lse;
  void* out;
  float* out_lse;
  int out_dtype;
  unsigned int* err;
  int drop_tile;          // (see qps_paged_inject_fault)
  uint32_t wait_ns;
  // Compressed rows decoded to fp16: [dense_tiles][KV head][128 positions][columns], columns = 2 D
  // (value, what its rounding left), or D for values where v_parts is 1; NULL: fp16 pages.  The
  // tiles of the sequences follow one another.
  __half *dense_k, *dense_v;
  int v_parts;
  int dense_tiles;        // tiles there is room for
  // the cache's planes, for the decoding
  int kfmt, vfmt;
  const uint8_t *k[3], *v[3];
  uint32_t signs1[kMaxSignWords], signs2[kMaxSignWords];
  int tq_block;
  float tq_scale;         // 1 / sqrt(D G)
  float tq_levels[16];
};

// Query tokens and positions of sequence b.  A start that is out of order leaves its sequence
// without tokens.
struct PromptSeq {
  int first, n, len;
};
__device__ __forceinline__ PromptSeq prompt_seq(const PromptParams& p, int b) {
  const int s0 = p.starts[b], s1 = p.starts[b + 1], n = p.lens[b];
  const int most = p.table_width << p.page_shift;
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= p.tokens;
  const int cut = min(max(n, 0), most);
  if (!ok || cut != n) atomicOr(p.err, kErrIndex);
  return PromptSeq{ok ? s0 : 0, ok ? s1 - s0 : 0, cut};
}

// The tiles (of 128 positions) that query tokens at positions [q0, q1] of a sequence see: the
// first `few`, then those of [low, end).
struct PromptTiles {
  int few, low, end, count;
};
__device__ __forceinline__ PromptTiles prompt_tiles(const PromptParams& p, int q0, int q1) {
  PromptTiles t = {0, 0, 0, 0};
  t.end = q1 < 0 ? 0 : q1 / kPromptTile + 1;
  if (p.window) {
    const int first = max(0, q0 - p.window + 1);
    t.few = (min(p.sinks, first) + kPromptTile - 1) / kPromptTile;
    t.low = max(t.few, first / kPromptTile);
  }
  t.few = min(t.few, t.end);
  t.low = min(t.low, t.end);
  t.count = t.few + t.end - t.low;
  return t;
}
__device__ __forceinline__ int prompt_tile(const PromptTiles& t, int i) { return i < t.few ? i : i - t.few + t.low; }
// A tile's place among those of the whole sequence that are decoded (-1: it is not).
__device__ __forceinline__ int prompt_dense(const PromptTiles& seq, int tile) {
  return tile < seq.few ? tile : tile >= seq.low && tile < seq.end ? tile - seq.low + seq.few : -1;
}

// The kernel for fp16 keys, and for keys in two parts.
qps_status launch_prompt_d64(const PromptParams& p, cudaStream_t s);
qps_status launch_prompt_d64_q(const PromptParams& p, cudaStream_t s);
qps_status launch_prompt_d128(const PromptParams& p, cudaStream_t s);
qps_status launch_prompt_d128_q(const PromptParams& p, cudaStream_t s);
qps_status launch_prompt_d256(const PromptParams& p, cudaStream_t s);
qps_status launch_prompt_d256_q(const PromptParams& p, cudaStream_t s);
qps_status launch_prompt_d512(const PromptParams& p, cudaStream_t s);
qps_status launch_prompt_d512_q(const PromptParams& p, cudaStream_t s);

// Query rows (tokens x heads of a group) per CTA, and CTAs that share a row's columns.
__host__ __device__ constexpr int prompt_rows(int d) { return d <= 128 ? 256 : 128; }
__host__ __device__ constexpr int prompt_col_ctas(int d) { return d == 512 ? 2 : 1; }

}  // namespace qps
