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
// Layout: a lane holds 8 neighbouring elements (one 16-byte access of fp16 / bf16), a row
// takes D / 8 lanes (two such groups per lane at D = 512), so a warp works on 256 / D rows
// of ONE token: the token's cosines and sines are loaded once per warp and stay in
// registers for all of its heads.  Both operators are bound by HBM for prompts (nothing is
// read twice) and by launch and load latency for single tokens.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <string>

#include "paged.h"

namespace qps {
namespace {

constexpr unsigned kFull = 0xffffffffu;

template <int D>
struct Row {
  static constexpr int CH = D > 256 ? D / 256 : 1;    // 8-element groups per lane
  static constexpr int LANES = D / 8 / CH;            // lanes per row
  static constexpr int PER_WARP = 32 / LANES;         // rows per warp
};

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

// ---- norm and rotation ----------------------------------------------------------------
// The row's element index of the lane's group c.
template <int D>
__device__ __forceinline__ int elem0(int sub, int c) {
  return 8 * (sub + 32 * c);
}

template <int D>
__device__ __forceinline__ void norm_row(float (&x)[Row<D>::CH][8], const NormP& n, int sub) {
  using R = Row<D>;
  float s[R::CH];
#pragma unroll
  for (int c = 0; c < R::CH; ++c) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = __fmul_rn(x[c][i], x[c][i]);
#pragma unroll
    for (int h = 4; h >= 1; h /= 2)
#pragma unroll
      for (int i = 0; i < h; ++i) t[i] = __fadd_rn(t[i], t[i + h]);
    s[c] = t[0];
  }
  float ss = s[0];
  if constexpr (R::CH == 2) ss = __fadd_rn(s[0], s[1]);
#pragma unroll
  for (int h = R::LANES / 2; h >= 1; h /= 2) ss = __fadd_rn(ss, __shfl_xor_sync(kFull, ss, h));
  const float inv = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.0f / D), n.eps)));
#pragma unroll
  for (int c = 0; c < R::CH; ++c) {
    float w[8];
    if (n.w) load8_any(n.w, n.w_dtype, elem0<D>(sub, c), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[c][i] = __fmul_rn(x[c][i], inv);
      if (n.w) x[c][i] = __fmul_rn(x[c][i], __fadd_rn(w[i], n.offset));
    }
  }
}

// The token's cosines and sines of this lane's elements: element i of group c takes
// (co, si) as its own pair member; si carries the sign of the second product (a: -, b: +).
// Elements behind `dim` get (1, 0) and are not touched.
template <int D>
struct Angles {
  float co[Row<D>::CH][8], si[Row<D>::CH][8];
};
template <int D>
__device__ __forceinline__ void load_angles(Angles<D>& a, const RotP& r, int64_t pos, int sub) {
  const float* row = r.table + pos * r.dim;
  const int half = r.dim / 2;
#pragma unroll
  for (int c = 0; c < Row<D>::CH; ++c) {
    const int e = elem0<D>(sub, c);
    if (e >= r.dim) continue;
    if (r.pairs) {  // pairs (e, e+1), ...: four angles
      const float4 co = *reinterpret_cast<const float4*>(row + e / 2);
      const float4 si = *reinterpret_cast<const float4*>(row + half + e / 2);
      const float cv[4] = {co.x, co.y, co.z, co.w}, sv[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a.co[c][i] = cv[i / 2];
        a.si[c][i] = (i & 1) ? sv[i / 2] : -sv[i / 2];
      }
    } else {
      const bool second = e >= half;
      const float* cp = row + (second ? e - half : e);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 co = reinterpret_cast<const float4*>(cp)[q];
        const float4 si = reinterpret_cast<const float4*>(cp + half)[q];
        const float cv[4] = {co.x, co.y, co.z, co.w}, sv[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a.co[c][4 * q + i] = cv[i];
          a.si[c][4 * q + i] = second ? sv[i] : -sv[i];
        }
      }
    }
  }
}

// x * c + other * (+-s): both products rounded, then their sum (a - b = a + (-b) exactly).
template <int D>
__device__ __forceinline__ void rotate_row(float (&x)[Row<D>::CH][8], const Angles<D>& a, const RotP& r, int sub,
                                           int lane) {
  using R = Row<D>;
  float other[R::CH][8];
  if (r.pairs) {
#pragma unroll
    for (int c = 0; c < R::CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) other[c][i] = x[c][i ^ 1];
  } else {
    // the partner of group g = sub + 32 c is group g +- dim / 16
    const int step = r.dim / 16;
#pragma unroll
    for (int c = 0; c < R::CH; ++c) {
      const int g = sub + 32 * c;
      int pg = g < step ? g + step : g - step;
      if (8 * g >= r.dim) pg = g;
      const int src = (lane - sub) + (pg & 31);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v0 = __shfl_sync(kFull, x[0][i], src);
        if constexpr (R::CH == 2) {
          const float v1 = __shfl_sync(kFull, x[1][i], src);
          other[c][i] = pg >= 32 ? v1 : v0;
        } else {
          other[c][i] = v0;
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < R::CH; ++c) {
    if (elem0<D>(sub, c) >= r.dim) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[c][i] = __fadd_rn(__fmul_rn(x[c][i], a.co[c][i]), __fmul_rn(other[c][i], a.si[c][i]));
  }
}

// ---- norm + rotation of query and key rows -------------------------------------------
struct RowsP {
  const void* in;
  void* out;
  int64_t in_tok, in_head, out_tok, out_head;
  int heads;
};
struct RopeP {
  int64_t tokens;
  RowsP q, k;
  NormP qn, kn;
  RotP rot;
  int out_dtype;
  int units;  // warps per token
  unsigned int* err;
};

// One warp: U x PER_WARP heads of one token (query heads, then key heads).
template <int D, typename T, int U>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const __grid_constant__ RopeP p) {
  using R = Row<D>;
  const int lane = threadIdx.x & 31, sub = lane % R::LANES, slot = lane / R::LANES;
  const int64_t unit = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t tok = unit / p.units;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (tok >= p.tokens) return;  // (the whole warp)
  const int h0 = (int)(unit % p.units) * (U * R::PER_WARP) + slot;
  const int heads = p.q.heads + p.k.heads;
  int64_t pos = 0;
  if (p.rot.dim) {
    pos = p.rot.pos[tok];
    if ((uint64_t)pos >= (uint64_t)p.rot.len) {
      if (lane == 0) atomicOr(p.err, kErrIndex);
      return;
    }
  }
  Raw8<T> raw[U][R::CH];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * R::PER_WARP;
    const bool key = h >= p.q.heads;
    const RowsP& r = key ? p.k : p.q;
    const T* src = reinterpret_cast<const T*>(r.in) + tok * r.in_tok + (int64_t)(key ? h - p.q.heads : h) * r.in_head;
#pragma unroll
    for (int c = 0; c < R::CH; ++c) {
      if (h < heads) raw[u][c].load(src + elem0<D>(sub, c));
      else raw[u][c].zero();
    }
  }
  Angles<D> ang;
  if (p.rot.dim) load_angles<D>(ang, p.rot, pos, sub);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * R::PER_WARP;
    const bool key = h >= p.q.heads;
    float x[R::CH][8];
#pragma unroll
    for (int c = 0; c < R::CH; ++c) raw[u][c].get(x[c]);
    // (a warp's rows may be of both sides: the norm's shuffles run for all of them)
    NormP n = p.qn;
    if (key) n = p.kn;
    if (p.qn.on || p.kn.on) {
      float y[R::CH][8];
#pragma unroll
      for (int c = 0; c < R::CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) y[c][i] = x[c][i];
      norm_row<D>(y, n, sub);
      if (n.on)
#pragma unroll
        for (int c = 0; c < R::CH; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) x[c][i] = y[c][i];
    }
    if (p.rot.dim) rotate_row<D>(x, ang, p.rot, sub, lane);
    if (h >= heads) continue;
    const RowsP& r = key ? p.k : p.q;
    uint16_t* dst = reinterpret_cast<uint16_t*>(r.out) + tok * r.out_tok +
                    (int64_t)(key ? h - p.q.heads : h) * r.out_head;
#pragma unroll
    for (int c = 0; c < R::CH; ++c) {
      uint4 w;
      if (p.out_dtype == QPS_DT_BF16)
        w = make_uint4(bf162_bits(x[c][0], x[c][1]), bf162_bits(x[c][2], x[c][3]), bf162_bits(x[c][4], x[c][5]),
                       bf162_bits(x[c][6], x[c][7]));
      else
        w = make_uint4(half2_bits(x[c][0], x[c][1]), half2_bits(x[c][2], x[c][3]), half2_bits(x[c][4], x[c][5]),
                       half2_bits(x[c][6], x[c][7]));
      *reinterpret_cast<uint4*>(dst + elem0<D>(sub, c)) = w;
    }
  }
}

// ---- append -----------------------------------------------------------------------------
struct TqP {
  uint32_t s1[kMaxSignWords], s2[kMaxSignWords];
  float thresholds[15];
  float kappa;
  int block, bits;
};
struct SideP {
  const void* in;
  int64_t tok, head;
  int fmt;
  uint8_t *data, *aux, *aux2;
};
struct AppendP {
  int64_t tokens;
  SideP k, v;
  NormP kn;
  RotP rot;
  const int64_t* slots;
  int64_t n_slots;
  int hkv, page_shift;
  int units;  // warps per token and side
  TqP tq;
  unsigned int* err;
};

// q8_0: blocks of 32 are 4 neighbouring lanes.
template <int D>
__device__ __forceinline__ void store_q8(const float (&x)[Row<D>::CH][8], uint8_t* data, uint8_t* aux, int64_t row,
                                         int sub, bool on) {
#pragma unroll
  for (int c = 0; c < Row<D>::CH; ++c) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[c][i]));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    const __half d16 = __float2half_rn(__fdiv_rn(amax, 127.0f));
    const float dd = __half2float(d16);
    uint32_t packed[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int q = 0;
      if (dd != 0.f) q = (int)fminf(fmaxf(roundf(__fdiv_rn(x[c][i], dd)), -127.f), 127.f);
      packed[i / 4] |= (uint32_t)(q & 0xff) << (8 * (i % 4));
    }
    if (!on) continue;
    const int g = sub + 32 * c;
    *reinterpret_cast<uint2*>(data + row * D + 8 * g) = make_uint2(packed[0], packed[1]);
    if ((g & 3) == 0) reinterpret_cast<__half*>(aux)[row * (D / 32) + g / 4] = d16;
  }
}

// TurboQuant tiers, in the order of kv_quant.cu: squares folded by halves over the whole
// row, sign vector, transform of spans 1 .. G/2, second signs, codes.
template <int D>
__device__ __forceinline__ void store_tq(const float (&x)[Row<D>::CH][8], const TqP& q, uint8_t* data, uint8_t* aux,
                                         uint8_t* aux2, int64_t row, int sub, bool on) {
  using R = Row<D>;
  constexpr int CH = R::CH;
  float t[CH][8], u[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) t[c][i] = __fmul_rn(x[c][i], x[c][i]);
  if constexpr (CH == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[0][i] = __fadd_rn(t[0][i], t[1][i]);
  }
#pragma unroll
  for (int h = R::LANES / 2; h >= 1; h /= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i) t[0][i] = __fadd_rn(t[0][i], __shfl_xor_sync(kFull, t[0][i], h));
#pragma unroll
  for (int h = 4; h >= 1; h /= 2)
#pragma unroll
    for (int i = 0; i < h; ++i) t[0][i] = __fadd_rn(t[0][i], t[0][i + h]);
  const float n = __fsqrt_rn(t[0][0]);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
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
    for (int h = 1; h < R::LANES; h *= 2) {
      if (8 * h >= q.block) break;  // the block width ends the transform
      const bool upper = (sub & h) != 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_xor_sync(kFull, u[c][i], h);
        u[c][i] = upper ? __fsub_rn(o, u[c][i]) : __fadd_rn(u[c][i], o);
      }
    }
  }
  if constexpr (CH == 2) {
    if (q.block > 256) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = u[0][i], b = u[1][i];
        u[0][i] = __fadd_rn(a, b);
        u[1][i] = __fsub_rn(a, b);
      }
    }
  }
  const int half = 1 << (q.bits - 1);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = elem0<D>(sub, c), g = sub + 32 * c;
    const uint32_t s = q.s2[e >> 5] >> (e & 31);
    uint32_t mags = 0u, signs = 0u;  // fields of 4 bits, one bit each
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int k = half - 1;
      if (n != 0.f) {
        const float z = __fdiv_rn(__fmul_rn(((s >> i) & 1u) ? -u[c][i] : u[c][i], q.kappa), n);
        k = 0;
#pragma unroll
        for (int m = 0; m < 15; ++m) k += (m < 2 * half - 1 && z >= q.thresholds[m]) ? 1 : 0;
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

// One warp: U x PER_WARP heads of one token and side (0: K, 1: V).
template <int D, typename T, int U>
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ AppendP p) {
  using R = Row<D>;
  const int lane = threadIdx.x & 31, sub = lane % R::LANES, seat = lane / R::LANES;
  const int64_t unit = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t tok = unit / (2 * p.units);
  const int rest = (int)(unit % (2 * p.units));
  const bool key = rest < p.units;
  const int h0 = (key ? rest : rest - p.units) * (U * R::PER_WARP) + seat;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (tok >= p.tokens) return;  // (the whole warp)
  const int64_t slot = p.slots[tok];
  int64_t pos = 0;
  if (p.rot.dim) pos = p.rot.pos[tok];
  if (slot < 0) return;  // padding
  if (slot >= p.n_slots || (p.rot.dim && (uint64_t)pos >= (uint64_t)p.rot.len)) {
    if (lane == 0) atomicOr(p.err, kErrIndex);
    return;
  }
  const SideP& s = key ? p.k : p.v;
  Raw8<T> raw[U][R::CH];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * R::PER_WARP;
    const T* src = reinterpret_cast<const T*>(s.in) + tok * s.tok + (int64_t)h * s.head;
#pragma unroll
    for (int c = 0; c < R::CH; ++c) {
      if (h < p.hkv) raw[u][c].load(src + elem0<D>(sub, c));
      else raw[u][c].zero();
    }
  }
  Angles<D> ang;
  if (key && p.rot.dim) load_angles<D>(ang, p.rot, pos, sub);
  const int64_t page_row = ((slot >> p.page_shift) * p.hkv << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * R::PER_WARP;
    const bool on = h < p.hkv;
    float x[R::CH][8];
#pragma unroll
    for (int c = 0; c < R::CH; ++c) raw[u][c].get(x[c]);
    if (key) {
      if (p.kn.on) norm_row<D>(x, p.kn, sub);
      if (p.rot.dim) rotate_row<D>(x, ang, p.rot, sub, lane);
    }
    const int64_t row = page_row + ((int64_t)h << p.page_shift);
    // the cache's input type is fp16: the one rounding before the encoder
    uint4 w[R::CH];
#pragma unroll
    for (int c = 0; c < R::CH; ++c) {
      w[c] = make_uint4(half2_bits(x[c][0], x[c][1]), half2_bits(x[c][2], x[c][3]), half2_bits(x[c][4], x[c][5]),
                        half2_bits(x[c][6], x[c][7]));
      unpack8<__half>(w[c], x[c]);
    }
    if (s.fmt == QPS_FMT_F16) {
      if (on)
#pragma unroll
        for (int c = 0; c < R::CH; ++c)
          *reinterpret_cast<uint4*>(s.data + (row * D + elem0<D>(sub, c)) * 2) = w[c];
    } else if (s.fmt == QPS_FMT_Q8_0) {
      store_q8<D>(x, s.data, s.aux, row, sub, on);
    } else {
      store_tq<D>(x, p.tq, s.data, s.aux, s.aux2, row, sub, on);
    }
  }
}

// ---- host side ----------------------------------------------------------------------------
// Heads per warp: one group of PER_WARP while the whole call has fewer warps than the GPU
// holds (single tokens: shortest chain of loads), else four groups, whose loads overlap
// and share the token's angles.
constexpr int kDeep = 4;
template <int D>
int groups_of(int heads, int u) {
  const int rows = u * Row<D>::PER_WARP;
  return (heads + rows - 1) / rows;
}

template <typename K, typename P>
qps_status launch_rows(K kernel, const P& p, int64_t warps, cudaStream_t s) {
  const int64_t blocks = (warps + 7) / 8;
  if (blocks > 0x7fffffffLL) return fail(QPS_ERR_UNSUPPORTED, "rows: more than 2^31 blocks");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
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

template <int D, typename T>
qps_status launch_rope(RopeP p, cudaStream_t s) {
  const int heads = p.q.heads + p.k.heads;
  const int64_t shallow = p.tokens * groups_of<D>(heads, 1);
  if (shallow <= (int64_t)sm_count_current() * 32) {
    p.units = groups_of<D>(heads, 1);
    return launch_rows(qk_norm_rope_kernel<D, T, 1>, p, shallow, s);
  }
  p.units = groups_of<D>(heads, kDeep);
  return launch_rows(qk_norm_rope_kernel<D, T, kDeep>, p, p.tokens * p.units, s);
}

template <int D, typename T>
qps_status launch_append(AppendP p, cudaStream_t s) {
  const int64_t shallow = p.tokens * 2 * groups_of<D>(p.hkv, 1);
  if (shallow <= (int64_t)sm_count_current() * 32) {
    p.units = groups_of<D>(p.hkv, 1);
    return launch_rows(kv_append_kernel<D, T, 1>, p, shallow, s);
  }
  p.units = groups_of<D>(p.hkv, kDeep);
  return launch_rows(kv_append_kernel<D, T, kDeep>, p, p.tokens * 2 * p.units, s);
}

template <typename T>
qps_status rope_by_d(int d, const RopeP& p, cudaStream_t s) {
  switch (d) {
    case 32: return launch_rope<32, T>(p, s);
    case 64: return launch_rope<64, T>(p, s);
    case 128: return launch_rope<128, T>(p, s);
    case 256: return launch_rope<256, T>(p, s);
    default: return launch_rope<512, T>(p, s);
  }
}
template <typename T>
qps_status append_by_d(int d, const AppendP& p, cudaStream_t s) {
  switch (d) {
    case 64: return launch_append<64, T>(p, s);
    case 128: return launch_append<128, T>(p, s);
    case 256: return launch_append<256, T>(p, s);
    default: return launch_append<512, T>(p, s);
  }
}

// ---- argument checks -----------------------------------------------------------------------
qps_status check_rows(const qps_rows& r, int d, const std::string& n) {
  if (r.heads < 0) return fail(QPS_ERR_INVALID_ARG, n + ": heads must be >= 0");
  if (r.heads == 0) return QPS_OK;
  if (r.dtype != QPS_DT_F16 && r.dtype != QPS_DT_BF16 && r.dtype != QPS_DT_F32)
    return fail(QPS_ERR_INVALID_ARG, n + ": unknown dtype");
  if (!r.data) return fail(QPS_ERR_INVALID_ARG, n + ": data is NULL");
  if (!aligned_to(r.data, 16) || r.tok_stride % 8 || r.head_stride % 8)
    return fail(QPS_ERR_INVALID_ARG, n + ": data must be 16-byte aligned with strides multiples of 8");
  if (r.tok_stride < 0 || r.head_stride < 0 || (r.heads > 1 && r.head_stride < d))
    return fail(QPS_ERR_INVALID_ARG, n + ": head_stride must be >= head_dim and strides >= 0");
  return QPS_OK;
}

qps_status check_norm(const qps_head_norm& n, const std::string& name) {
  if (!n.on) return QPS_OK;
  if (!std::isfinite(n.eps) || n.eps < 0.f || !std::isfinite(n.offset))
    return fail(QPS_ERR_INVALID_ARG, name + ": eps must be finite and >= 0, offset finite");
  if (n.w && n.w_dtype != QPS_DT_F16 && n.w_dtype != QPS_DT_BF16 && n.w_dtype != QPS_DT_F32)
    return fail(QPS_ERR_INVALID_ARG, name + ": unknown w_dtype");
  if (n.w && !aligned_to(n.w, 16)) return fail(QPS_ERR_INVALID_ARG, name + ": w must be 16-byte aligned");
  return QPS_OK;
}

qps_status check_rotation(const qps_rotation& r, const int64_t* positions, int d, const std::string& name) {
  if (r.dim == 0) return QPS_OK;
  if (r.dim < 0 || r.dim % 16 || r.dim > d)
    return fail(QPS_ERR_INVALID_ARG, name + ": the rotated width must be a multiple of 16 and at most head_dim");
  if (r.pairs != 0 && r.pairs != 1) return fail(QPS_ERR_INVALID_ARG, name + ": pairs must be 0 or 1");
  if (!r.table || !aligned_to(r.table, 16) || r.len < 1)
    return fail(QPS_ERR_INVALID_ARG, name + ": the rotation table must be 16-byte aligned and hold a position");
  if (!positions || !aligned_to(positions, 8))
    return fail(QPS_ERR_INVALID_ARG, name + ": positions must be given with a rotation, 8-byte aligned");
  return QPS_OK;
}

NormP norm_of(const qps_head_norm& n) { return NormP{n.on ? n.w : nullptr, n.w_dtype, n.on ? 1 : 0, n.eps, n.offset}; }

// Extent of rows in bytes from their first element.
int64_t extent(const qps_rows& r, int64_t tokens, int d) {
  return ((tokens - 1) * r.tok_stride + (int64_t)(r.heads - 1) * r.head_stride + d) * dtype_bytes(r.dtype);
}
bool overlap(const qps_rows& a, const qps_rows& b, int64_t tokens, int d) {
  const char *pa = (const char*)a.data, *pb = (const char*)b.data;
  return pa < pb + extent(b, tokens, d) && pb < pa + extent(a, tokens, d);
}
bool same_rows(const qps_rows& a, const qps_rows& b, int64_t tokens) {
  return a.data == b.data && a.dtype == b.dtype && (tokens < 2 || a.tok_stride == b.tok_stride) &&
         (a.heads < 2 || a.head_stride == b.head_stride);
}
// Whether two sets of rows interleave without touching (slices of one projection): the
// same strides, and the offset between them keeps every row apart.
bool apart_in_projection(const qps_rows& a, const qps_rows& b, int d) {
  if (dtype_bytes(a.dtype) != dtype_bytes(b.dtype) || a.tok_stride != b.tok_stride || a.tok_stride <= 0) return false;
  const int64_t sz = dtype_bytes(a.dtype), t = a.tok_stride * sz;
  const int64_t wa = ((int64_t)(a.heads - 1) * a.head_stride + d) * sz, wb = ((int64_t)(b.heads - 1) * b.head_stride + d) * sz;
  int64_t off = ((const char*)b.data - (const char*)a.data) % t;
  if (off < 0) off += t;
  return off >= wa && off + wb <= t;
}

qps_status qk_norm_rope(const qps_qk_rope_args* a, cudaStream_t s) {
  const std::string n("qk_norm_rope");
  if (!a) return fail(QPS_ERR_INVALID_ARG, n + ": args is NULL");
  if (a->tokens < 0) return fail(QPS_ERR_INVALID_ARG, n + ": tokens must be >= 0");
  if (a->reserved0 != 0) return fail(QPS_ERR_INVALID_ARG, n + ": reserved0 must be 0");
  if (a->d != 32 && a->d != 64 && a->d != 128 && a->d != 256 && a->d != 512)
    return fail(QPS_ERR_UNSUPPORTED, n + ": head_dim must be 32, 64, 128, 256 or 512");
  if (a->tokens == 0) return QPS_OK;
  const struct { const qps_rows *in, *out; const char* what; } sides[2] = {{&a->q, &a->q_out, " q"}, {&a->k, &a->k_out, " k"}};
  int in_dtype = -1, out_dtype = -1;
  for (const auto& sd : sides) {
    qps_status st = check_rows(*sd.in, a->d, n + sd.what);
    if (st == QPS_OK) st = check_rows(*sd.out, a->d, n + sd.what + "_out");
    if (st != QPS_OK) return st;
    if (sd.in->heads != sd.out->heads) return fail(QPS_ERR_INVALID_ARG, n + sd.what + ": input and output heads differ");
    if (sd.in->heads == 0) continue;
    if (sd.out->dtype == QPS_DT_F32) return fail(QPS_ERR_UNSUPPORTED, n + sd.what + "_out: the output type is F16 or BF16");
    if ((in_dtype >= 0 && in_dtype != sd.in->dtype) || (out_dtype >= 0 && out_dtype != sd.out->dtype))
      return fail(QPS_ERR_INVALID_ARG, n + ": q and k must have the same types");
    in_dtype = sd.in->dtype;
    out_dtype = sd.out->dtype;
    if (a->tokens > 1 && sd.out->tok_stride < a->d)
      return fail(QPS_ERR_INVALID_ARG, n + sd.what + "_out: tok_stride must be >= head_dim");
  }
  qps_status st = check_norm(a->q_norm, n + " q_norm");
  if (st == QPS_OK) st = check_norm(a->k_norm, n + " k_norm");
  if (st == QPS_OK) st = check_rotation(a->rot, a->positions, a->d, n);
  if (st != QPS_OK) return st;
  if (in_dtype < 0) return QPS_OK;
  if (a->q.heads > 65536 || a->k.heads > 65536) return fail(QPS_ERR_UNSUPPORTED, n + ": more than 65536 heads");
  // rows are read and written by different warps: an output overlaps an input only where
  // each row is its own
  for (int o = 0; o < 2; ++o) {
    if (sides[o].out->heads == 0) continue;
    for (int i = 0; i < 2; ++i) {
      if (sides[i].in->heads == 0 || !overlap(*sides[o].out, *sides[i].in, a->tokens, a->d)) continue;
      if (i == o && same_rows(*sides[o].out, *sides[i].in, a->tokens)) continue;
      if (!apart_in_projection(*sides[o].out, *sides[i].in, a->d))
        return fail(QPS_ERR_INVALID_ARG, n + sides[o].what + "_out: overlaps an input without being it");
    }
  }
  if (a->q.heads && a->k.heads && overlap(a->q_out, a->k_out, a->tokens, a->d) &&
      !apart_in_projection(a->q_out, a->k_out, a->d))
    return fail(QPS_ERR_INVALID_ARG, n + ": q_out and k_out overlap");
  RopeP p{};
  p.tokens = a->tokens;
  auto rows = [](const qps_rows& in, const qps_rows& out) {
    return RowsP{in.data, out.data, in.tok_stride, in.head_stride, out.tok_stride, out.head_stride, in.heads};
  };
  p.q = rows(a->q, a->q_out);
  p.k = rows(a->k, a->k_out);
  p.qn = norm_of(a->q_norm);
  p.kn = norm_of(a->k_norm);
  p.rot = RotP{a->rot.table, a->positions, a->rot.len, a->rot.dim, a->rot.pairs};
  p.out_dtype = out_dtype;
  p.err = device_error_word();
  if (!p.err) return fail(QPS_ERR_CUDA, n + ": cannot allocate the device error word");
  if (in_dtype == QPS_DT_F32) return rope_by_d<float>(a->d, p, s);
  if (in_dtype == QPS_DT_BF16) return rope_by_d<__nv_bfloat16>(a->d, p, s);
  return rope_by_d<__half>(a->d, p, s);
}

qps_status kv_append(const qps_paged_append_args* a, cudaStream_t s) {
  const std::string n("kv_append_paged");
  if (!a) return fail(QPS_ERR_INVALID_ARG, n + ": args is NULL");
  if (a->tokens < 0) return fail(QPS_ERR_INVALID_ARG, n + ": tokens must be >= 0");
  PagedKv kv;
  qps_status st = check_paged_kv(a->kv, "kv_append_paged", &kv);
  if (st == QPS_OK) st = check_norm(a->k_norm, n + " k_norm");
  if (st != QPS_OK || a->tokens == 0) return st;
  st = check_rotation(a->rot, a->positions, kv.d, n);
  if (st != QPS_OK) return st;
  if (a->k.heads != kv.hkv || a->v.heads != kv.hkv)
    return fail(QPS_ERR_INVALID_ARG, n + ": k and v must have the cache's heads");
  st = check_rows(a->k, kv.d, n + " k");
  if (st == QPS_OK) st = check_rows(a->v, kv.d, n + " v");
  if (st != QPS_OK) return st;
  if (a->k.dtype != a->v.dtype) return fail(QPS_ERR_INVALID_ARG, n + ": k and v must have the same type");
  if (!a->slots || !aligned_to(a->slots, 8)) return fail(QPS_ERR_INVALID_ARG, n + ": slots is NULL or misaligned");
  AppendP p{};
  p.tokens = a->tokens;
  p.k = SideP{a->k.data, a->k.tok_stride, a->k.head_stride, kv.kfmt, kv.k[0], kv.k[1], kv.k[2]};
  p.v = SideP{a->v.data, a->v.tok_stride, a->v.head_stride, kv.vfmt, kv.v[0], kv.v[1], kv.v[2]};
  p.kn = norm_of(a->k_norm);
  p.rot = RotP{a->rot.table, a->positions, a->rot.len, a->rot.dim, a->rot.pairs};
  p.slots = a->slots;
  p.n_slots = kv.n_pages << kv.page_shift;
  p.hkv = kv.hkv;
  p.page_shift = kv.page_shift;
  if (is_tq(kv.vfmt)) {
    const int g = a->kv.tq_block == 0 ? kv.d : a->kv.tq_block;
    for (int i = 0; i < kv.d / 32; ++i) {
      p.tq.s1[i] = a->kv.signs1[i];
      p.tq.s2[i] = a->kv.signs2 ? a->kv.signs2[i] : 0u;
    }
    p.tq.bits = tq_bits(kv.vfmt);
    const Codebook* cb = tq_codebook(p.tq.bits);
    for (int i = 0; i < cb->n - 1; ++i) p.tq.thresholds[i] = cb->thresholds[i];
    p.tq.kappa = std::sqrt((float)(kv.d / g));
    p.tq.block = g;
  }
  p.err = device_error_word();
  if (!p.err) return fail(QPS_ERR_CUDA, n + ": cannot allocate the device error word");
  if (a->k.dtype == QPS_DT_F32) return append_by_d<float>(kv.d, p, s);
  if (a->k.dtype == QPS_DT_BF16) return append_by_d<__nv_bfloat16>(kv.d, p, s);
  return append_by_d<__half>(kv.d, p, s);
}

}  // namespace

qps_status check_paged_kv(const qps_paged_kv& kv, const char* call, PagedKv* out) {
  const std::string n = std::string(call) + " kv";
  if (kv.reserved0 != 0 || kv.reserved1 != 0) return fail(QPS_ERR_INVALID_ARG, n + ": reserved fields must be 0");
  if (kv.d != 64 && kv.d != 128 && kv.d != 256 && kv.d != 512)
    return fail(QPS_ERR_UNSUPPORTED, n + ": head_dim must be 64, 128, 256 or 512");
  if (kv.hkv < 1 || kv.hkv > 65535) return fail(QPS_ERR_INVALID_ARG, n + ": hkv must be in [1, 65535]");
  const int ps = kv.page_size;
  if (ps < 16 || ps > 1024 || (ps & (ps - 1)))
    return fail(QPS_ERR_UNSUPPORTED, n + ": page_size must be a power of two in [16, 1024]");
  if (kv.n_pages < 1 || kv.n_pages >= ((int64_t)1 << 31) / ps)
    return fail(QPS_ERR_INVALID_ARG, n + ": need n_pages > 0 and n_pages * page_size < 2^31");
  const int fmts[2] = {kv.k_fmt, kv.v_fmt};
  void* const planes[2][3] = {{kv.k_data, kv.k_aux, kv.k_aux2}, {kv.v_data, kv.v_aux, kv.v_aux2}};
  for (int s = 0; s < 2; ++s) {
    if (fmts[s] != QPS_FMT_F16 && fmts[s] != QPS_FMT_Q8_0 && !is_tq(fmts[s]))
      return fail(QPS_ERR_INVALID_ARG, n + ": unknown format");
    for (int i = 0; i < plane_count(fmts[s]); ++i)
      if (!planes[s][i] || !aligned_to(planes[s][i], 16))
        return fail(QPS_ERR_INVALID_ARG, n + ": a plane is NULL or not 16-byte aligned");
  }
  if (is_tq(kv.k_fmt) && kv.v_fmt != kv.k_fmt)
    return fail(QPS_ERR_UNSUPPORTED, n + ": a TurboQuant K needs V in the same TurboQuant tier");
  if (is_tq(kv.v_fmt)) {
    if (!kv.signs1) return fail(QPS_ERR_INVALID_ARG, n + ": signs1 is required for a TurboQuant plane");
    const int g = kv.tq_block == 0 ? kv.d : kv.tq_block;
    if (g < 32 || g > kv.d || (g & (g - 1)))
      return fail(QPS_ERR_INVALID_ARG, n + ": tq_block must be 0 or a power of two in [32, head_dim]");
  }
  out->kfmt = kv.k_fmt;
  out->vfmt = kv.v_fmt;
  out->hkv = kv.hkv;
  out->d = kv.d;
  out->page_shift = 0;
  while ((1 << out->page_shift) < ps) ++out->page_shift;
  out->n_pages = kv.n_pages;
  for (int i = 0; i < 3; ++i) {
    out->k[i] = reinterpret_cast<uint8_t*>(planes[0][i]);
    out->v[i] = reinterpret_cast<uint8_t*>(planes[1][i]);
  }
  return QPS_OK;
}

}  // namespace qps

using namespace qps;

extern "C" {

qps_status qps_qk_norm_rope(const qps_qk_rope_args* a, void* stream) {
  try {
    return qk_norm_rope(a, reinterpret_cast<cudaStream_t>(stream));
  } catch (const std::exception&) {
    return QPS_ERR_INTERNAL;
  }
}

qps_status qps_kv_append_paged(const qps_paged_append_args* a, void* stream) {
  try {
    return kv_append(a, reinterpret_cast<cudaStream_t>(stream));
  } catch (const std::exception&) {
    return QPS_ERR_INTERNAL;
  }
}

}  // extern "C"
