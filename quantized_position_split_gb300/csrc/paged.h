// Shared by the calls around the paged KV cache: argument checks, the resolved cache and
// the attention's parameters.
#pragma once

#include "internal.h"

namespace qps {

// Sizes of a checked qps_paged_kv (page_size is a power of two).
struct PagedKv {
  int kfmt, vfmt, hkv, d, page_shift;
  int64_t n_pages;
  uint8_t *k[3], *v[3];  // data, aux, aux2
};

inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline int dtype_bytes(int dt) { return dt == QPS_DT_F32 ? 4 : 2; }

qps_status check_paged_kv(const qps_paged_kv& kv, const char* call, PagedKv* out);

// Parameters of the paged attention kernels: the tensor-core kernel's own (q, heads,
// scales, rotation; n_split, chunk and part_offset are the prefix's) and the page tables.
struct PagedAttnParams : AttnParams {
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  int64_t n_pages;
  int page_shift, table_width;
  int prefix_len;     // positions attended by the prefix launch (a multiple of 32)
  int target;         // chunks per (KV head, row group) the sequences are cut into, about
  int min_units;      // smallest chunk, in units
  int unit_round;     // chunks are multiples of this many units (a power of two)
  int max_chunks;     // chunks there can be, by the tables' width
  int kernel;         // PagedKernel of this launch
  int n_prefix;       // parts of the prefix
  float* pre_o;       // f32 [n_prefix][rows_total][D], [n_prefix][rows_total]
  float* pre_lse;
  float* own_o;       // f32 [chunk][n_q*hq][D], [chunk][n_q*hq]
  float* own_lse;
  int2* chunks;       // [batch] first chunk and count, for the merge; written by first chunks
  int drop_tile;      // (tcgen05 kernels) the tile of each chunk whose keys are not brought (-1:
                      // none; see qps_paged_inject_fault), and the limit of the waits
  uint32_t wait_ns;
  void* out;          // the call's o (out_dtype) and lse
  float* out_lse;
  int out_dtype;
};

// The chunking of the sequences' own positions [prefix_len, len), the same in the
// attention and in the merge: units of 32 positions, C units a chunk (a multiple of
// unit_round), sequence b's chunks numbered behind those of the sequences before it.  C is
// such that all chunks together number at most `target` + batch.  A sequence without own
// positions has one chunk, which writes an empty part.
__device__ __forceinline__ int paged_len(const PagedAttnParams& p, int b) {
  const int n = p.lens[b];
  const int most = p.table_width << p.page_shift;
  const int cut = min(max(n, 0), most);
  if (cut != n) atomicOr(p.err, kErrIndex);
  return cut;
}
// What the checked build holds the paged kernels' accesses against: entry `at` of the page
// tables, 16 bytes of the queries from element `at`, row `at` of the outputs or of a part
// (its number and its row).
__device__ __forceinline__ bool entry_in_bounds(const PagedAttnParams& p, int64_t at) {
  return in_bounds(at >= 0 && at < (p.batch - 1) * p.table_stride + p.table_width, p.err);
}
__device__ __forceinline__ bool q_in_bounds(const PagedAttnParams& p, int64_t at) {
  return in_bounds(at >= 0 && at + 8 <= p.q_elems, p.err);
}
__device__ __forceinline__ bool out_in_bounds(const PagedAttnParams& p, bool whole, int part, int64_t row) {
  return in_bounds(whole      ? row >= 0 && row < p.rows_total
                   : p.shared ? part >= 0 && part < p.n_prefix && row >= 0 && row < p.rows_total
                              : part >= 0 && part < p.max_chunks && row >= 0 && row < (int64_t)p.n_q * p.hq,
                   p.err);
}
constexpr int kPagedUnit = 32;  // a whole number of any instance's tiles
__device__ __forceinline__ int paged_units(int len, int prefix) {
  return len > prefix ? (len - prefix + kPagedUnit - 1) / kPagedUnit : 0;
}
__device__ __forceinline__ int paged_chunks(const PagedAttnParams& p, int len, int cu) {
  const int units = paged_units(len, p.prefix_len);
  return units <= cu ? 1 : (units + cu - 1) / cu;
}

// The prefix as the batch has it, the same in every lane: its positions, and the sequence
// through whose entries they are read.  The pages behind the longest sequence's end hold no
// one's rows, and a NaN there would pass a weight of zero (0 x NaN), so the prefix ends with
// it; the entries are those of the first sequence that has all of these positions (a padding
// row's may name any page).
struct PagedPrefix {
  int len, b;
};
__device__ __forceinline__ PagedPrefix paged_prefix(const PagedAttnParams& p, int lane) {
  int len = -1, first = 0;
#pragma unroll 4
  for (int b = lane; b < p.batch; b += 32) {
    const int n = min(paged_len(p, b), p.prefix_len);
    if (n > len) {
      len = n;
      first = b;
    }
  }
  PagedPrefix r;
  r.len = __reduce_max_sync(0xffffffffu, len);
  r.b = __reduce_min_sync(0xffffffffu, len == r.len ? first : 0x7fffffff);
  return r;
}

// Chunk number `index` of the batch: its sequence (-1: there are fewer chunks), positions
// [t0, t1), whether it is its sequence's first (of `count`) and its only part; the same in
// every lane.
struct PagedChunk {
  int b, t0, t1, count;
  bool first, whole;
};
__device__ __forceinline__ PagedChunk paged_find(const PagedAttnParams& p, int index, int lane) {
  // every CTA goes this way before its first load of a position: the first 128 lengths are
  // read together, once
  constexpr int R = 4;
  int len[R];
#pragma unroll
  for (int i = 0; i < R; ++i) len[i] = lane + 32 * i < p.batch ? paged_len(p, lane + 32 * i) : 0;
  int total = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) total += paged_units(len[i], p.prefix_len);
#pragma unroll 4
  for (int b = lane + 32 * R; b < p.batch; b += 32) total += paged_units(paged_len(p, b), p.prefix_len);
  total = __reduce_add_sync(0xffffffffu, total);
  int cu = p.min_units;  // chunk length in units
  if (total > cu * p.target) cu = (total + p.target - 1) / p.target;
  cu = (cu + p.unit_round - 1) & ~(p.unit_round - 1);
  PagedChunk r = {-1, 0, 0, 0, false, false};
  int before = 0;
  auto look = [&](int b0, int bl) -> bool {
    const int cnt = b0 + lane < p.batch ? paged_chunks(p, bl, cu) : 0;
    int sum = cnt;  // inclusive scan over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + sum > index);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int n = __shfl_sync(0xffffffffu, cnt, src);
      const int at = index - (before + __shfl_sync(0xffffffffu, sum, src) - n);
      r.b = b0 + src;
      r.t0 = p.prefix_len + at * cu * kPagedUnit;
      r.t1 = (int)min((int64_t)__shfl_sync(0xffffffffu, bl, src), r.t0 + (int64_t)cu * kPagedUnit);
      r.count = n;
      r.first = at == 0;
      r.whole = n == 1 && p.prefix_len == 0;
      return true;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
    return false;
  };
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (32 * i >= p.batch) return r;
    if (look(32 * i, len[i])) return r;
  }
  for (int b0 = 32 * R; b0 < p.batch; b0 += 32)
    if (look(b0, b0 + lane < p.batch ? paged_len(p, b0 + lane) : 0)) break;
  return r;
}

qps_status launch_paged_mma_d64(const PagedAttnParams& p, cudaStream_t s);
qps_status launch_paged_mma_d128(const PagedAttnParams& p, cudaStream_t s);
qps_status launch_paged_mma_d256(const PagedAttnParams& p, cudaStream_t s);
qps_status launch_paged_mma_d512(const PagedAttnParams& p, cudaStream_t s);
qps_status launch_paged_tm_d64(const PagedAttnParams& p, cudaStream_t s);
qps_status launch_paged_tm_d128(const PagedAttnParams& p, cudaStream_t s);
qps_status launch_paged_tt_d128(const PagedAttnParams& p, cudaStream_t s);
qps_status launch_paged_tt_d256(const PagedAttnParams& p, cudaStream_t s);
qps_status launch_paged_tt_d512(const PagedAttnParams& p, cudaStream_t s);

// The softmax's reference is kept below the maximum, so that the largest operand of P V is
// 2^kRefShift, 2^(kRefShift + kRefLazy) at most before the reference is raised: fp16 holds
// that, and weights down to 2^-(14 + kRefShift) of the largest keep all their bits.  With the
// reference at the maximum, a key whose logit is 16 above the others (e^-16 = 2^-23) and whose
// value is near zero, as a first position's may be, left an output off by 3e-2 of its size.
constexpr float kRefShift = 11.f, kRefLazy = 4.f;

// The kernels of a paged launch: attn_mma.cuh's, attn_tm.cuh's, attn_tt.cuh's.
enum PagedKernel { kMma, kTm, kTt };

}  // namespace qps
