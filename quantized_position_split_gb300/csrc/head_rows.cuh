// Rows of one head on their way between the projections and the cache: RMS norm and
// position rotation of query and key rows, and the append of key / value rows to a paged
// cache in its stored format.
//
// Per row x [D] (float32 throughout, one rounding at the end):
//   inv = 1 / sqrt(sum x^2 / D + eps),  y = (x * inv) * (w + offset)
//   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s) for the pairs of the first `dim` elements.
// Every step is an explicitly rounded operation in a fixed order (no contraction), so an
// appended key's codes are the same bits wherever the formula is evaluated that way: the
// encoders of kv_quant.cu are bit-exact contracts, and so is what reaches them.
//
// Layout: a lane holds two groups of 8 neighbouring elements (16-byte accesses of fp16 /
// bf16), D / 2 apart: group j of the row is group sub = j % (D / 16) of half c.  A row takes
// D / 16 lanes, a warp works on 512 / D rows of ONE token and side, so
//   * both members of a rotated pair (halves or neighbours) are in one lane's registers, and
//     the sum of squares needs log2(D / 16) shuffles (with one group a lane, each element's
//     partner came by a shuffle: 8192 tokens x 48 heads of 128 took 72.4 us, instruction
//     bound at 36 instructions an element);
//   * the token's cosines and sines, and the weights, are loaded once per warp and stay in
//     registers for all of its heads;
//   * products and sums run two to an instruction (f32x2, each half rounded to nearest).
// Measured: 8192 tokens x 48 heads of 128, fp16, normed and rotated: 40.7 us, 5.1 TB/s (55% of
// the issue slots; steps of a warp over several tokens were no faster, nor were other counts of
// rounds under way and blocks per SM; the instance spills 28 bytes of stores, 48 of loads).
// 8191 tokens x 8 heads of 128, K and V, bf16 into q8_0: 24.2 us, 2.3 TB/s, 50% of the issue
// slots: held to 80 registers, the instance spills 152 bytes of stores and 104 of loads.
// One token: 2.0 us on the GPU, launch and load latency.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>

#include "paged.h"

namespace qps {

// ---- parameters (rows are checked by head_rows.cu) --------------------------------------
struct NormP {
  const void* w;
  int w_dtype, on;
  float eps, offset;
};
struct RotP {
  const float* table;
  const int64_t* pos;
  int64_t len;
  int dim, pairs;
};

struct RowsP {
  const void* in;
  void* out;
  int64_t in_tok, in_head, out_tok, out_head;
  int heads;
  int64_t in_elems, out_elems;  // extents that the checked build holds accesses against
};

struct RopeP {
  int64_t tokens;
  float one;  // 1 (see add2)
  RowsP q, k;
  NormP qn, kn;
  RotP rot;
  int out_dtype;
  int q_iters, k_iters;  // groups of PER_WARP heads per warp
  int q_units, units;    // warps per token: of its query heads, of all
  unsigned int* err;
};

struct TqP {
  uint32_t s1[kMaxSignWords], s2[kMaxSignWords];
  float thresholds[15];
  float kappa;
  int block, bits;
};

struct SideP {
  const void* in;
  int64_t tok, head;
  int64_t elems;  // (as above)
  int fmt;
  uint8_t *data, *aux, *aux2;
};

struct AppendP {
  int64_t tokens;
  float one;  // 1 (see add2)
  SideP k, v;
  NormP kn;
  RotP rot;
  const int64_t* slots;
  int64_t n_slots;
  int hkv, page_shift;
  int iters;  // groups of PER_WARP heads per warp
  int units;  // warps per token and side
  TqP tq;
  unsigned int* err;
};

qps_status rope_f16(int d, const RopeP& p, cudaStream_t s);
qps_status rope_bf16(int d, const RopeP& p, cudaStream_t s);
qps_status rope_f32(int d, const RopeP& p, cudaStream_t s);
qps_status append_f16(int d, const AppendP& p, cudaStream_t s);
qps_status append_bf16(int d, const AppendP& p, cudaStream_t s);
qps_status append_f32(int d, const AppendP& p, cudaStream_t s);

namespace rows {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 128;
constexpr int kAhead = 2;  // groups of rows under way per warp
// Blocks per SM the registers are sized for: element-by-element angles (neighbours, a part
// of the row) take 32 registers, the halves' 16.
template <int D, typename T, int MODE>
constexpr int kBlocksPerSm = MODE == 1 || MODE == 3 ? 4 : 6;

template <int D>
struct Row {
  static constexpr int LANES = D / 16;          // lanes per row
  static constexpr int PER_WARP = 32 / LANES;   // rows per warp
};

// ---- loads and stores of 8 neighbouring elements ------------------------------------
// (Plain loads, not the read-only path: under programmatic launch the rows may have been
// written by a grid that was still running when this one started.)
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]);
template <>
__device__ __forceinline__ void unpack8<__half>(const uint4& r, float (&x)[8]) {
  const __half2* h = reinterpret_cast<const __half2*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// 8 elements as they lie in memory, so that several loads can be under way at once
template <typename T>
struct Raw8 {
  uint4 r[sizeof(T) == 4 ? 2 : 1];
  __device__ __forceinline__ void load(const T* p) {
    r[0] = *reinterpret_cast<const uint4*>(p);
    if constexpr (sizeof(T) == 4) r[1] = *(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() {
    r[0] = make_uint4(0, 0, 0, 0);
    if constexpr (sizeof(T) == 4) r[1] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (sizeof(T) == 4) {
      const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    } else {
      unpack8<T>(r[0], x);
    }
  }
};

__device__ __forceinline__ void load8_any(const void* p, int dtype, int at, float (&x)[8]) {
  if (dtype == QPS_DT_F32) {
    Raw8<float> r;
    r.load(reinterpret_cast<const float*>(p) + at);
    r.get(x);
  } else if (dtype == QPS_DT_BF16) {
    Raw8<__nv_bfloat16> r;
    r.load(reinterpret_cast<const __nv_bfloat16*>(p) + at);
    r.get(x);
  } else {
    Raw8<__half> r;
    r.load(reinterpret_cast<const __half*>(p) + at);
    r.get(x);
  }
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t bf162_bits(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- pairs of float32 in one instruction ------------------------------------------------
// (each half rounded to nearest: the same bits as two scalar operations).  A sum is
// written as a * one + b, `one` being 1 from the launch's parameters: written as
// add.rn.f32x2, a product and its sum came back contracted (a row of 128 differed in its
// last bit from the separately rounded order).
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b, f2 one) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(one), "l"(b));
  return r;
}

// A lane's part of a row: pair i of half c is elements 2i, 2i + 1 of its group there.
struct Part {
  f2 v[2][4];
};
// first element of the lane's group of half c
template <int D>
__device__ __forceinline__ int elem0(int sub, int c) {
  return c * (D / 2) + 8 * sub;
}

// (checked build) `n` elements or rows from `at` on lie within `extent`.
__device__ __forceinline__ bool row_in_bounds(int64_t at, int n, int64_t extent, unsigned int* err) {
  return in_bounds(at >= 0 && at + n <= extent, err);
}

template <typename T>
struct Raw {
  Raw8<T> g[2];
  template <int D>
  __device__ __forceinline__ void load(const T* row, int sub) {
    g[0].load(row + elem0<D>(sub, 0));
    g[1].load(row + elem0<D>(sub, 1));
  }
  __device__ __forceinline__ void zero() {
    g[0].zero();
    g[1].zero();
  }
  __device__ __forceinline__ void get(Part& x) const {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float f[8];
      g[c].get(f);
#pragma unroll
      for (int i = 0; i < 4; ++i) x.v[c][i] = pack2(f[2 * i], f[2 * i + 1]);
    }
  }
};

// ---- norm and rotation ----------------------------------------------------------------
// The side's weights, offset added, of this lane's elements.
template <int D>
__device__ __forceinline__ void load_weights(Part& w, const NormP& n, int sub, f2 one) {
  const f2 off = pack2(n.offset, n.offset);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float f[8];
    load8_any(n.w, n.w_dtype, elem0<D>(sub, c), f);
#pragma unroll
    for (int i = 0; i < 4; ++i) w.v[c][i] = add2(pack2(f[2 * i], f[2 * i + 1]), off, one);
  }
}

template <int D>
__device__ __forceinline__ void norm_row(Part& x, const NormP& n, const Part& w, f2 one) {
  float s[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    f2 t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = mul2(x.v[c][i], x.v[c][i]);
    t[0] = add2(add2(t[0], t[2], one), add2(t[1], t[3], one), one);  // the folds h = 4 (pairs i, i + 2), then h = 2
    float a, b;
    unpack2(t[0], a, b);
    s[c] = __fadd_rn(a, b);
  }
  float ss = __fadd_rn(s[0], s[1]);  // groups j and j + D/16
#pragma unroll
  for (int h = Row<D>::LANES / 2; h >= 1; h /= 2) ss = __fadd_rn(ss, __shfl_xor_sync(kFull, ss, h));
  const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.0f / D), n.eps)));
  const f2 i2 = pack2(inv, inv);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x.v[c][i] = mul2(x.v[c][i], i2);
      if (n.w) x.v[c][i] = mul2(x.v[c][i], w.v[c][i]);
    }
}

// Which elements rotate together.  kNext: neighbours (2j, 2j + 1) of the first dim
// elements; kHalves: (j, j + D/2), the whole row; kPart: (j, j + dim/2) with dim < D,
// whose partners are other lanes' (by shuffles).
enum RotMode { kNone, kNext, kHalves, kPart };

// The token's angles for this lane.  kHalves: cosines in co.v[0], sines in si.v[0] (both
// halves' elements turn by the same angles).  kNext / kPart: element by element, the sine
// with the sign of the second product (first members: -, second: +); elements behind dim
// are not touched.
struct Angles {
  Part co, si;
};
__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x;
  f[1] = v.y;
  f[2] = v.z;
  f[3] = v.w;
}
template <int D, int MODE>
__device__ __forceinline__ void load_angles(Angles& a, const RotP& r, int64_t pos, int sub) {
  const float* row = r.table + pos * r.dim;
  const int half = r.dim / 2;
#pragma unroll
  for (int c = 0; c < (MODE == kHalves ? 1 : 2); ++c) {
    const int e = elem0<D>(sub, c);
    if (e >= r.dim) continue;
    if constexpr (MODE == kNext) {  // four angles
      float co[4], si[4];
      load4(row + e / 2, co);
      load4(row + half + e / 2, si);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a.co.v[c][i] = pack2(co[i], co[i]);
        a.si.v[c][i] = pack2(-si[i], si[i]);
      }
    } else {
      const bool second = e >= half;
      const float* cp = row + (second ? e - half : e);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float co[4], si[4];
        load4(cp + 4 * q, co);
        load4(cp + half + 4 * q, si);
        if (MODE == kPart && !second) {
#pragma unroll
          for (int i = 0; i < 4; ++i) si[i] = -si[i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a.co.v[c][2 * q + i] = pack2(co[2 * i], co[2 * i + 1]);
          a.si.v[c][2 * q + i] = pack2(si[2 * i], si[2 * i + 1]);
        }
      }
    }
  }
}

// Both products rounded, then their sum (a - b = a + (-b) exactly).
template <int D, int MODE>
__device__ __forceinline__ void rotate_row(Part& x, const Angles& a, const RotP& r, int sub, int lane, f2 one) {
  if constexpr (MODE == kHalves) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f2 p = x.v[0][i], q = x.v[1][i], co = a.co.v[0][i], si = a.si.v[0][i];
      x.v[0][i] = add2(mul2(p, co), mul2(q, si ^ 0x8000000080000000ull), one);
      x.v[1][i] = add2(mul2(q, co), mul2(p, si), one);
    }
  } else if constexpr (MODE == kNext) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (elem0<D>(sub, c) >= r.dim) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float p, q;
        unpack2(x.v[c][i], p, q);
        x.v[c][i] = add2(mul2(x.v[c][i], a.co.v[c][i]), mul2(pack2(q, p), a.si.v[c][i]), one);
      }
    }
  } else if constexpr (MODE == kPart) {
    // the partner of the row's group j is group j +- dim / 16
    constexpr int L = Row<D>::LANES;
    const int step = r.dim / 16;
    Part other;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int j = sub + L * c;
      int pj = j < step ? j + step : j - step;
      if (8 * j >= r.dim) pj = j;
      const int src = (lane - sub) + pj % L;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 v0 = __shfl_sync(kFull, x.v[0][i], src), v1 = __shfl_sync(kFull, x.v[1][i], src);
        other.v[c][i] = pj >= L ? v1 : v0;
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (elem0<D>(sub, c) >= r.dim) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x.v[c][i] = add2(mul2(x.v[c][i], a.co.v[c][i]), mul2(other.v[c][i], a.si.v[c][i]), one);
    }
  }
}

__device__ __forceinline__ uint4 pack_half(const f2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack2(v[i], a, b);
    w[i] = half2_bits(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack_bf16(const f2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack2(v[i], a, b);
    w[i] = bf162_bits(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---- norm + rotation of query and key rows -------------------------------------------

// One warp: `iters` groups of PER_WARP heads of one token and side, the rows of the next
// kAhead groups under way while one's are worked on.
template <int D, typename T, int MODE>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<D, T, MODE>)
    qk_norm_rope_kernel(const __grid_constant__ RopeP p) {
  using R = Row<D>;
  const int lane = threadIdx.x & 31, sub = lane % R::LANES, seat = lane / R::LANES;
  const unsigned unit = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;  // (fits: checked by the host)
  const unsigned tok = unit / (unsigned)p.units;
  const int rest = (int)(unit % (unsigned)p.units);
  const bool key = rest >= p.q_units;
  const RowsP& r = key ? p.k : p.q;
  const NormP& n = key ? p.kn : p.qn;
  const int iters = key ? p.k_iters : p.q_iters;
  int h = (key ? rest - p.q_units : rest) * (iters * R::PER_WARP) + seat;
  const f2 one = pack2(p.one, p.one);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (tok >= p.tokens) return;  // (the whole warp)
  const int heads = r.heads;
  const int64_t in_step = R::PER_WARP * r.in_head, out_step = R::PER_WARP * r.out_head;
  const T* src = reinterpret_cast<const T*>(r.in) + tok * r.in_tok + h * r.in_head;
  auto row_in = [&](const T* at) { return row_in_bounds(at - reinterpret_cast<const T*>(r.in), D, r.in_elems, p.err); };
  uint16_t* dst = reinterpret_cast<uint16_t*>(r.out) + tok * r.out_tok + h * r.out_head;
  Raw<T> ring[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    ring[u].zero();
    if (u < iters && h + u * R::PER_WARP < heads && row_in(src)) ring[u].template load<D>(src, sub);
    src += in_step;
  }
  Angles ang;
  if constexpr (MODE != kNone) {
    const int64_t pos = p.rot.pos[tok];
    if ((uint64_t)pos >= (uint64_t)p.rot.len) {
      if (lane == 0) atomicOr(p.err, kErrIndex);
      return;
    }
    load_angles<D, MODE>(ang, p.rot, pos, sub);
  }
  Part w;
  if (n.w) load_weights<D>(w, n, sub, one);
#pragma unroll 1
  for (int it = 0; it < iters; it += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u, h += R::PER_WARP, dst += out_step, src += in_step) {
      if (it + u >= iters) break;
      Part x;
      ring[u].get(x);
      if (it + u + kAhead < iters && h + kAhead * R::PER_WARP < heads && row_in(src)) ring[u].template load<D>(src, sub);
      if (n.on) norm_row<D>(x, n, w, one);
      if constexpr (MODE != kNone) rotate_row<D, MODE>(x, ang, p.rot, sub, lane, one);
      if (h >= heads || !row_in_bounds(dst - reinterpret_cast<uint16_t*>(r.out), D, r.out_elems, p.err)) continue;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        *reinterpret_cast<uint4*>(dst + elem0<D>(sub, c)) =
            p.out_dtype == QPS_DT_BF16 ? pack_bf16(x.v[c]) : pack_half(x.v[c]);
    }
  }
}

// ---- append -----------------------------------------------------------------------------

// q8_0: blocks of 32 are 4 neighbouring lanes' groups.  A code is the quotient x / d16,
// rounded to float32 and then to the nearest whole number, halves away from zero.  As
// |x / d16| <= 128, z = x times the correctly rounded reciprocal is within 2^-16 of it and
// the rounded quotient within 2^-17: unless z is within 2^-15 of a half, both give the same
// code, which z + 1.5 * 2^23 holds in its low byte.  Only near a half, and where the scale
// is not a normal number (a code could leave +-127) or a value is NaN, is the division made.
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <int D>
__device__ __forceinline__ void store_q8(const float (&x)[2][8], uint8_t* data, uint8_t* aux, int64_t row, int sub,
                                         bool on, f2 one) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  const f2 magic = pack2(kMagic, kMagic), unmagic = pack2(-kMagic, -kMagic), minus = pack2(-1.f, -1.f);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[c][i]));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    const __half d16 = __float2half_rn(__fdiv_rn(amax, 127.0f));
    const float dd = __half2float(d16);
    const float rcp = __frcp_rn(dd);
    const f2 r2 = pack2(rcp, rcp);
    float off = 0.f;  // the largest distance of a z from its code
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f2 z = mul2(pack2(x[c][2 * i], x[c][2 * i + 1]), r2);
      const f2 m = add2(z, magic, one);
      float a, b, u, v;
      unpack2(m, a, b);
      q[2 * i] = __float_as_uint(a);
      q[2 * i + 1] = __float_as_uint(b);
      unpack2(add2(z, add2(m, unmagic, one), minus), u, v);  // code - z (the product with -1 is exact)
      off = max_nan(max_nan(off, fabsf(u)), fabsf(v));
    }
    if (!(off < 0.5f - 0x1p-15f && dd >= 0x1p-14f && dd < 65536.f)) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[i] = dd != 0.f ? (uint32_t)(int)fminf(fmaxf(roundf(__fdiv_rn(x[c][i], dd)), -127.f), 127.f) : 0u;
    }
    if (!on) continue;
    uint32_t packed[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      packed[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040), __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040), 0x5410);
    const int e = elem0<D>(sub, c);
    *reinterpret_cast<uint2*>(data + row * D + e) = make_uint2(packed[0], packed[1]);
    if ((sub & 3) == 0) reinterpret_cast<__half*>(aux)[row * (D / 32) + e / 32] = d16;
  }
}

// TurboQuant tiers, in the order of kv_quant.cu: squares folded by halves over the whole
// row, sign vector, transform of spans 1 .. G/2, second signs, codes.
template <int D>
__device__ __forceinline__ void store_tq(const float (&x)[2][8], const TqP& q, uint8_t* data, uint8_t* aux,
                                         uint8_t* aux2, int64_t row, int sub, bool on) {
  constexpr int L = Row<D>::LANES;
  float t[8], u[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = __fadd_rn(__fmul_rn(x[0][i], x[0][i]), __fmul_rn(x[1][i], x[1][i]));  // h = D/2
#pragma unroll
  for (int h = L / 2; h >= 1; h /= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = __fadd_rn(t[i], __shfl_xor_sync(kFull, t[i], h));
#pragma unroll
  for (int h = 4; h >= 1; h /= 2)
#pragma unroll
    for (int i = 0; i < h; ++i) t[i] = __fadd_rn(t[i], t[i + h]);
  const float n = __fsqrt_rn(t[0]);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int e = elem0<D>(sub, c);
    const uint32_t s = q.s1[e >> 5] >> (e & 31);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[c][i] = ((s >> i) & 1u) ? -x[c][i] : x[c][i];
#pragma unroll
    for (int h = 1; h < 8; h *= 2)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(i & h)) {
          const float a = u[c][i], b = u[c][i + h];
          u[c][i] = __fadd_rn(a, b);
          u[c][i + h] = __fsub_rn(a, b);
        }
#pragma unroll
    for (int h = 1; h < L; h *= 2) {
      if (8 * h >= q.block) break;  // the block width ends the transform
      const bool upper = (sub & h) != 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_xor_sync(kFull, u[c][i], h);
        u[c][i] = upper ? __fsub_rn(o, u[c][i]) : __fadd_rn(u[c][i], o);
      }
    }
  }
  if (q.block == D) {  // span D / 2: the lane's two groups
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = u[0][i], b = u[1][i];
      u[0][i] = __fadd_rn(a, b);
      u[1][i] = __fsub_rn(a, b);
    }
  }
  const int half = 1 << (q.bits - 1);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int e = elem0<D>(sub, c), g = e / 8;
    const uint32_t s = q.s2[e >> 5] >> (e & 31);
    uint32_t mags = 0u, signs = 0u;  // fields of 4 bits, one bit each
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int k = half - 1;
      if (n != 0.f) {
        const float z = __fdiv_rn(__fmul_rn(((s >> i) & 1u) ? -u[c][i] : u[c][i], q.kappa), n);
        k = 0;
#pragma unroll
        for (int m = 0; m < 7; ++m) k += (m < 2 * half - 1 && z >= q.thresholds[m]) ? 1 : 0;
        if (q.bits == 4)
#pragma unroll
          for (int m = 7; m < 15; ++m) k += z >= q.thresholds[m] ? 1 : 0;
      }
      const bool up = k >= half;
      mags |= (uint32_t)(up ? k - half : half - 1 - k) << (4 * i);
      signs |= (up ? 1u : 0u) << i;
    }
    if (!on) continue;
    if (q.bits == 4) {
      uint32_t f = mags;
#pragma unroll
      for (int i = 0; i < 8; ++i) f |= ((signs >> i) & 1u) << (4 * i + 3);
      *reinterpret_cast<uint32_t*>(data + row * (D / 2) + 4 * g) = f;
    } else {
      uint32_t f = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t v = (mags >> (4 * i)) & 3u;
        if (q.bits == 2) v |= ((signs >> i) & 1u) << 1;
        f |= v << (2 * i);
      }
      *reinterpret_cast<uint16_t*>(data + row * (D / 4) + 2 * g) = (uint16_t)f;
      if (q.bits == 3) aux[row * (D / 8) + g] = (uint8_t)signs;
    }
  }
  if (on && sub == 0) reinterpret_cast<__half*>(q.bits == 3 ? aux2 : aux)[row] = __float2half_rn(n);
}

// One warp: `iters` groups of PER_WARP heads of one token and side (K, then V).
template <int D, typename T, int MODE>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<D, T, MODE>)
    kv_append_kernel(const __grid_constant__ AppendP p) {
  using R = Row<D>;
  const int lane = threadIdx.x & 31, sub = lane % R::LANES, seat = lane / R::LANES;
  const unsigned unit = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;  // (fits: checked by the host)
  const unsigned tok = unit / (2u * p.units);
  const int rest = (int)(unit % (2u * p.units));
  const bool key = rest < p.units;
  const SideP& s = key ? p.k : p.v;
  int h = (key ? rest : rest - p.units) * (p.iters * R::PER_WARP) + seat;
  const f2 one = pack2(p.one, p.one);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (tok >= p.tokens) return;  // (the whole warp)
  const int64_t slot = p.slots[tok];
  int64_t pos = 0;
  if constexpr (MODE != kNone) pos = p.rot.pos[tok];
  const int64_t in_step = R::PER_WARP * s.head;
  const T* src = reinterpret_cast<const T*>(s.in) + tok * s.tok + h * s.head;
  auto row_in = [&](const T* at) { return row_in_bounds(at - reinterpret_cast<const T*>(s.in), D, s.elems, p.err); };
  Raw<T> ring[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    ring[u].zero();
    if (u < p.iters && h + u * R::PER_WARP < p.hkv && row_in(src)) ring[u].template load<D>(src, sub);
    src += in_step;
  }
  if (slot < 0) return;  // padding
  if (slot >= p.n_slots || (MODE != kNone && (uint64_t)pos >= (uint64_t)p.rot.len)) {
    if (lane == 0) atomicOr(p.err, kErrIndex);
    return;
  }
  Angles ang;
  Part w;
  if (key) {
    if constexpr (MODE != kNone) load_angles<D, MODE>(ang, p.rot, pos, sub);
    if (p.kn.w) load_weights<D>(w, p.kn, sub, one);
  }
  int64_t row = (((slot >> p.page_shift) * p.hkv + h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
#pragma unroll 1
  for (int it = 0; it < p.iters; it += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u, h += R::PER_WARP, row += (int64_t)R::PER_WARP << p.page_shift, src += in_step) {
      if (it + u >= p.iters) break;
      const bool on = h < p.hkv && row_in_bounds(row, 1, p.n_slots * p.hkv, p.err);
      Part y;
      ring[u].get(y);
      if (it + u + kAhead < p.iters && h + kAhead * R::PER_WARP < p.hkv && row_in(src)) ring[u].template load<D>(src, sub);
      if (key) {
        if (p.kn.on) norm_row<D>(y, p.kn, w, one);
        if constexpr (MODE != kNone) rotate_row<D, MODE>(y, ang, p.rot, sub, lane, one);
      }
      // the cache's input type is fp16: the one rounding before the encoder
      const uint4 h16[2] = {pack_half(y.v[0]), pack_half(y.v[1])};
      if (s.fmt == QPS_FMT_F16) {
        if (on)
#pragma unroll
          for (int c = 0; c < 2; ++c) *reinterpret_cast<uint4*>(s.data + (row * D + elem0<D>(sub, c)) * 2) = h16[c];
        continue;
      }
      float x[2][8];
#pragma unroll
      for (int c = 0; c < 2; ++c) unpack8<__half>(h16[c], x[c]);
      if (s.fmt == QPS_FMT_Q8_0) store_q8<D>(x, s.data, s.aux, row, sub, on, one);
      else store_tq<D>(x, p.tq, s.data, s.aux, s.aux2, row, sub, on);
    }
  }
}

// ---- host side ----------------------------------------------------------------------------
// Heads per warp: one group of PER_WARP while the call has fewer warps than the GPU holds
// (the shortest chain of loads), else as many as leave about kRounds rounds of warps: the
// more, the less of the time goes into angles, weights and addresses.  Few warps come in
// blocks of two, to reach more SMs.
constexpr int kRounds = 3;
template <int D>
int groups_of(int heads) {
  return (heads + Row<D>::PER_WARP - 1) / Row<D>::PER_WARP;
}
inline int iters_for(int64_t groups, int most, int blocks_per_sm) {
  const int64_t warps = (int64_t)sm_count_current() * blocks_per_sm * (kThreads / 32) * kRounds;
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, warps > 0 ? groups / warps : 1));
}

template <typename K, typename P>
qps_status launch_rows(K kernel, const P& p, int64_t warps, cudaStream_t s) {
  if (warps >= (int64_t)1 << 27) return fail(QPS_ERR_UNSUPPORTED, "rows: too many rows in one call");
  const int per_block = warps <= 2 * (int64_t)sm_count_current() ? 2 : kThreads / 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + per_block - 1) / per_block));
  cfg.blockDim = dim3(per_block * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  QPS_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, p));
  count_launch();
  QPS_CUDA_TRY(cudaGetLastError());
  return QPS_OK;
}

template <int D, typename T, int MODE>
qps_status launch_rope(RopeP p, cudaStream_t s) {
  const int gq = groups_of<D>(p.q.heads), gk = groups_of<D>(p.k.heads);
  const int iters = iters_for(p.tokens * (gq + gk), std::max(gq, gk), kBlocksPerSm<D, T, MODE>);
  p.q_units = (gq + iters - 1) / iters;
  p.units = p.q_units + (gk + iters - 1) / iters;
  p.q_iters = p.q_units ? (gq + p.q_units - 1) / p.q_units : 0;  // (evenly over the warps)
  p.k_iters = p.units > p.q_units ? (gk + p.units - p.q_units - 1) / (p.units - p.q_units) : 0;
  return launch_rows(qk_norm_rope_kernel<D, T, MODE>, p, p.tokens * p.units, s);
}

template <int D, typename T, int MODE>
qps_status launch_append(AppendP p, cudaStream_t s) {
  const int g = groups_of<D>(p.hkv);
  p.iters = iters_for(p.tokens * 2 * g, g, kBlocksPerSm<D, T, MODE>);
  p.units = (g + p.iters - 1) / p.iters;
  p.iters = (g + p.units - 1) / p.units;
  return launch_rows(kv_append_kernel<D, T, MODE>, p, p.tokens * 2 * p.units, s);
}

inline int rot_mode(const RotP& r, int d) { return r.dim == 0 ? kNone : r.pairs ? kNext : r.dim == d ? kHalves : kPart; }

template <int D, typename T>
qps_status rope_by_mode(const RopeP& p, cudaStream_t s) {
  switch (rot_mode(p.rot, D)) {
    case kNone: return launch_rope<D, T, kNone>(p, s);
    case kNext: return launch_rope<D, T, kNext>(p, s);
    case kHalves: return launch_rope<D, T, kHalves>(p, s);
    default: return launch_rope<D, T, kPart>(p, s);
  }
}
template <int D, typename T>
qps_status append_by_mode(const AppendP& p, cudaStream_t s) {
  switch (rot_mode(p.rot, D)) {
    case kNone: return launch_append<D, T, kNone>(p, s);
    case kNext: return launch_append<D, T, kNext>(p, s);
    case kHalves: return launch_append<D, T, kHalves>(p, s);
    default: return launch_append<D, T, kPart>(p, s);
  }
}

template <typename T>
qps_status rope_by_d(int d, const RopeP& p, cudaStream_t s) {
  switch (d) {
    case 32: return rope_by_mode<32, T>(p, s);
    case 64: return rope_by_mode<64, T>(p, s);
    case 128: return rope_by_mode<128, T>(p, s);
    case 256: return rope_by_mode<256, T>(p, s);
    default: return rope_by_mode<512, T>(p, s);
  }
}
template <typename T>
qps_status append_by_d(int d, const AppendP& p, cudaStream_t s) {
  switch (d) {
    case 64: return append_by_mode<64, T>(p, s);
    case 128: return append_by_mode<128, T>(p, s);
    case 256: return append_by_mode<256, T>(p, s);
    default: return append_by_mode<512, T>(p, s);
  }
}

}  // namespace rows
}  // namespace qps
