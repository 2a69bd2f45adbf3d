// Argument checks and entry points of qk_norm_rope and kv_append_paged, and the checks of
// a paged cache; the kernels are in head_rows.cuh, their instances by input type in
// qk_rope_*.cu and kv_append_*.cu.
#include <algorithm>
#include <cmath>
#include <exception>
#include <string>

#include "head_rows.cuh"

namespace qps {
namespace {

// A refusal's message, put together only when there is one.
qps_status bad(const char* call, const char* what, const char* msg, qps_status st = QPS_ERR_INVALID_ARG) {
  return fail(st, std::string(call) + what + ": " + msg);
}

// ---- argument checks -----------------------------------------------------------------------
qps_status check_rows(const qps_rows& r, int d, const char* call, const char* what) {
  if (r.heads < 0) return bad(call, what, "heads must be >= 0");
  if (r.heads == 0) return QPS_OK;
  if (r.dtype != QPS_DT_F16 && r.dtype != QPS_DT_BF16 && r.dtype != QPS_DT_F32)
    return bad(call, what, "unknown dtype");
  if (!r.data) return bad(call, what, "data is NULL");
  if (!aligned_to(r.data, 16) || r.tok_stride % 8 || r.head_stride % 8)
    return bad(call, what, "data must be 16-byte aligned with strides multiples of 8");
  if (r.tok_stride < 0 || r.head_stride < 0 || (r.heads > 1 && r.head_stride < d))
    return bad(call, what, "head_stride must be >= head_dim and strides >= 0");
  return QPS_OK;
}

// Sizes whose products stay in 64 bits: what the checks and the kernels compute with them.
// (kMaxTokens: each token takes a warp at least, and launch_rows holds the warps to this.)
constexpr int64_t kMaxTokens = (int64_t)1 << 27;
bool reachable(const qps_rows& r, int64_t tokens, int d) {
  const __int128 last = (__int128)(tokens - 1) * r.tok_stride + (__int128)(r.heads - 1) * r.head_stride + d;
  return r.heads == 0 || last < (__int128)1 << 56;
}

qps_status check_norm(const qps_head_norm& n, const char* call, const char* what) {
  if (!n.on) return QPS_OK;
  if (!std::isfinite(n.eps) || n.eps < 0.f || !std::isfinite(n.offset))
    return bad(call, what, "eps must be finite and >= 0, offset finite");
  if (n.w && n.w_dtype != QPS_DT_F16 && n.w_dtype != QPS_DT_BF16 && n.w_dtype != QPS_DT_F32)
    return bad(call, what, "unknown w_dtype");
  if (n.w && !aligned_to(n.w, 16)) return bad(call, what, "w must be 16-byte aligned");
  return QPS_OK;
}

qps_status check_rotation(const qps_rotation& r, const int64_t* positions, int d, const char* call) {
  if (r.dim == 0) return QPS_OK;
  if (r.dim < 0 || r.dim % 16 || r.dim > d)
    return bad(call, "", "the rotated width must be a multiple of 16 and at most head_dim");
  if (r.pairs != 0 && r.pairs != 1) return bad(call, "", "pairs must be 0 or 1");
  if (!r.table || !aligned_to(r.table, 16) || r.len < 1)
    return bad(call, "", "the rotation table must be 16-byte aligned and hold a position");
  if (!positions || !aligned_to(positions, 8))
    return bad(call, "", "positions must be given with a rotation, 8-byte aligned");
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
// Whether two sets of rows whose extents meet interleave without touching (slices of one
// projection, side by side or head by head): the same distance of tokens, and no row of one
// within a row's width of a row of the other.  More pairs of heads than this looks through
// count as touching.
bool apart(const qps_rows& a, const qps_rows& b, int64_t tokens, int d) {
  const int64_t sa = dtype_bytes(a.dtype), sb = dtype_bytes(b.dtype), t = a.tok_stride * sa;
  if (tokens > 1 && (t != b.tok_stride * sb || t <= 0)) return false;
  const int64_t ha = a.head_stride * sa, hb = b.head_stride * sb, wa = d * sa, wb = d * sb;
  const int64_t base = (const char*)b.data - (const char*)a.data;
  if (tokens > 1) {  // whole tokens side by side
    const int64_t off = (base % t + t) % t;
    if (off >= (a.heads - 1) * ha + wa && off + (b.heads - 1) * hb + wb <= t) return true;
  }
  auto touch = [&](int64_t x) {  // rows x bytes apart, or any token distance n, |n| < tokens, more?
    const int64_t n = tokens > 1 ? std::max(-(tokens - 1), std::min(tokens - 1, -(x / t))) : 0;
    for (int64_t m = std::max(n - 1, -(tokens - 1)); m <= std::min(n + 1, tokens - 1); ++m)
      if (x + m * t > -wb && x + m * t < wa) return true;
    return false;
  };
  if (ha == hb) {  // only the distance of the heads counts
    for (int64_t i = -(int64_t)(a.heads - 1); i < b.heads; ++i)
      if (touch(base + i * hb)) return false;
    return true;
  }
  if ((int64_t)a.heads * b.heads > 1 << 16) return false;
  for (int64_t i = 0; i < a.heads; ++i)
    for (int64_t j = 0; j < b.heads; ++j)
      if (touch(base + j * hb - i * ha)) return false;
  return true;
}
// Whether no row of the set touches another of it.
bool apart_itself(const qps_rows& r, int64_t tokens, int d) {
  const int64_t t = r.tok_stride, h = r.head_stride;
  if (tokens < 2 || r.heads < 2 || t >= (r.heads - 1) * h + d || h >= (tokens - 1) * t + d) return true;
  for (int64_t i = 1; i < r.heads; ++i) {  // rows i heads and n tokens apart
    const int64_t x = i * h, n = std::min(tokens - 1, x / t);
    for (int64_t m = n; m <= std::min(n + 1, tokens - 1); ++m)
      if (x - m * t > -d && x - m * t < d) return false;
  }
  return true;
}

qps_status qk_norm_rope(const qps_qk_rope_args* a, cudaStream_t s) {
  const char* const n = "qk_norm_rope";
  if (!a) return bad(n, "", "args is NULL");
  if (a->tokens < 0) return bad(n, "", "tokens must be >= 0");
  if (a->reserved0 != 0) return bad(n, "", "reserved0 must be 0");
  if (a->d != 32 && a->d != 64 && a->d != 128 && a->d != 256 && a->d != 512)
    return bad(n, "", "head_dim must be 32, 64, 128, 256 or 512", QPS_ERR_UNSUPPORTED);
  if (a->tokens == 0) return QPS_OK;
  if (a->tokens >= kMaxTokens) return bad(n, "", "too many tokens in one call", QPS_ERR_UNSUPPORTED);
  const struct { const qps_rows *in, *out; const char *what, *out_what; } sides[2] = {
      {&a->q, &a->q_out, " q", " q_out"}, {&a->k, &a->k_out, " k", " k_out"}};
  int in_dtype = -1, out_dtype = -1;
  for (const auto& sd : sides) {
    qps_status st = check_rows(*sd.in, a->d, n, sd.what);
    if (st == QPS_OK) st = check_rows(*sd.out, a->d, n, sd.out_what);
    if (st != QPS_OK) return st;
    if (!reachable(*sd.in, a->tokens, a->d) || !reachable(*sd.out, a->tokens, a->d))
      return bad(n, sd.what, "strides reach behind any memory");
    if (sd.in->heads != sd.out->heads) return bad(n, sd.what, "input and output heads differ");
    if (sd.in->heads == 0) continue;
    if (sd.out->dtype == QPS_DT_F32) return bad(n, sd.out_what, "the output type is F16 or BF16", QPS_ERR_UNSUPPORTED);
    if ((in_dtype >= 0 && in_dtype != sd.in->dtype) || (out_dtype >= 0 && out_dtype != sd.out->dtype))
      return bad(n, "", "q and k must have the same types");
    in_dtype = sd.in->dtype;
    out_dtype = sd.out->dtype;
    if (a->tokens > 1 && sd.out->tok_stride < a->d)
      return bad(n, sd.out_what, "tok_stride must be >= head_dim");
    if (!apart_itself(*sd.out, a->tokens, a->d)) return bad(n, sd.out_what, "rows overlap one another");
  }
  qps_status st = check_norm(a->q_norm, n, " q_norm");
  if (st == QPS_OK) st = check_norm(a->k_norm, n, " k_norm");
  if (st == QPS_OK) st = check_rotation(a->rot, a->positions, a->d, n);
  if (st != QPS_OK) return st;
  if (in_dtype < 0) return QPS_OK;
  if (a->q.heads > 65536 || a->k.heads > 65536) return bad(n, "", "more than 65536 heads", QPS_ERR_UNSUPPORTED);
  // rows are read and written by different warps: an output overlaps an input only where
  // each row is its own
  for (int o = 0; o < 2; ++o) {
    if (sides[o].out->heads == 0) continue;
    for (int i = 0; i < 2; ++i) {
      if (sides[i].in->heads == 0 || !overlap(*sides[o].out, *sides[i].in, a->tokens, a->d)) continue;
      if (i == o && same_rows(*sides[o].out, *sides[i].in, a->tokens)) continue;
      if (!apart(*sides[o].out, *sides[i].in, a->tokens, a->d))
        return bad(n, sides[o].out_what, "overlaps an input without being it");
    }
  }
  if (a->q.heads && a->k.heads && overlap(a->q_out, a->k_out, a->tokens, a->d) &&
      !apart(a->q_out, a->k_out, a->tokens, a->d))
    return bad(n, "", "q_out and k_out overlap");
  RopeP p{};
  p.tokens = a->tokens;
  p.one = 1.0f;
  auto elems = [a](const qps_rows& r) { return r.heads ? extent(r, a->tokens, a->d) / dtype_bytes(r.dtype) : 0; };
  auto rows = [&](const qps_rows& in, const qps_rows& out) {
    return RowsP{in.data, out.data, in.tok_stride, in.head_stride, out.tok_stride, out.head_stride, in.heads, elems(in), elems(out)};
  };
  p.q = rows(a->q, a->q_out);
  p.k = rows(a->k, a->k_out);
  p.qn = norm_of(a->q_norm);
  p.kn = norm_of(a->k_norm);
  p.rot = RotP{a->rot.table, a->positions, a->rot.len, a->rot.dim, a->rot.pairs};
  p.out_dtype = out_dtype;
  p.err = device_error_word();
  if (!p.err) return bad(n, "", "cannot allocate the device error word", QPS_ERR_CUDA);
  if (in_dtype == QPS_DT_F32) return rope_f32(a->d, p, s);
  if (in_dtype == QPS_DT_BF16) return rope_bf16(a->d, p, s);
  return rope_f16(a->d, p, s);
}

qps_status kv_append(const qps_paged_append_args* a, cudaStream_t s) {
  const char* const n = "kv_append_paged";
  if (!a) return bad(n, "", "args is NULL");
  if (a->tokens < 0) return bad(n, "", "tokens must be >= 0");
  PagedKv kv;
  qps_status st = check_paged_kv(a->kv, "kv_append_paged", &kv);
  if (st == QPS_OK) st = check_norm(a->k_norm, n, " k_norm");
  if (st != QPS_OK || a->tokens == 0) return st;
  if (a->tokens >= kMaxTokens) return bad(n, "", "too many tokens in one call", QPS_ERR_UNSUPPORTED);
  st = check_rotation(a->rot, a->positions, kv.d, n);
  if (st != QPS_OK) return st;
  if (a->k.heads != kv.hkv || a->v.heads != kv.hkv)
    return bad(n, "", "k and v must have the cache's heads");
  st = check_rows(a->k, kv.d, n, " k");
  if (st == QPS_OK) st = check_rows(a->v, kv.d, n, " v");
  if (st != QPS_OK) return st;
  if (!reachable(a->k, a->tokens, kv.d) || !reachable(a->v, a->tokens, kv.d))
    return bad(n, "", "strides reach behind any memory");
  if (a->k.dtype != a->v.dtype) return bad(n, "", "k and v must have the same type");
  if (!a->slots || !aligned_to(a->slots, 8)) return bad(n, "", "slots is NULL or misaligned");
  AppendP p{};
  p.tokens = a->tokens;
  p.one = 1.0f;
  auto elems = [&](const qps_rows& r) { return extent(r, a->tokens, kv.d) / dtype_bytes(r.dtype); };
  p.k = SideP{a->k.data, a->k.tok_stride, a->k.head_stride, elems(a->k), kv.kfmt, kv.k[0], kv.k[1], kv.k[2]};
  p.v = SideP{a->v.data, a->v.tok_stride, a->v.head_stride, elems(a->v), kv.vfmt, kv.v[0], kv.v[1], kv.v[2]};
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
  if (!p.err) return bad(n, "", "cannot allocate the device error word", QPS_ERR_CUDA);
  if (a->k.dtype == QPS_DT_F32) return append_f32(kv.d, p, s);
  if (a->k.dtype == QPS_DT_BF16) return append_bf16(kv.d, p, s);
  return append_f16(kv.d, p, s);
}

}  // namespace

qps_status check_paged_kv(const qps_paged_kv& kv, const char* call, PagedKv* out) {
  const char* const n = " kv";
  if (kv.reserved0 != 0 || kv.reserved1 != 0) return bad(call, n, "reserved fields must be 0");
  if (kv.d != 64 && kv.d != 128 && kv.d != 256 && kv.d != 512)
    return bad(call, n, "head_dim must be 64, 128, 256 or 512", QPS_ERR_UNSUPPORTED);
  if (kv.hkv < 1 || kv.hkv > 65535) return bad(call, n, "hkv must be in [1, 65535]");
  const int ps = kv.page_size;
  if (ps < 16 || ps > 1024 || (ps & (ps - 1)))
    return bad(call, n, "page_size must be a power of two in [16, 1024]", QPS_ERR_UNSUPPORTED);
  if (kv.n_pages < 1 || kv.n_pages >= ((int64_t)1 << 31) / ps)
    return bad(call, n, "need n_pages > 0 and n_pages * page_size < 2^31");
  const int fmts[2] = {kv.k_fmt, kv.v_fmt};
  void* const planes[2][3] = {{kv.k_data, kv.k_aux, kv.k_aux2}, {kv.v_data, kv.v_aux, kv.v_aux2}};
  for (int s = 0; s < 2; ++s) {
    if (fmts[s] != QPS_FMT_F16 && fmts[s] != QPS_FMT_Q8_0 && !is_tq(fmts[s]))
      return bad(call, n, "unknown format");
    for (int i = 0; i < plane_count(fmts[s]); ++i)
      if (!planes[s][i] || !aligned_to(planes[s][i], 16))
        return bad(call, n, "a plane is NULL or not 16-byte aligned");
  }
  if (is_tq(kv.k_fmt) && kv.v_fmt != kv.k_fmt)
    return bad(call, n, "a TurboQuant K needs V in the same TurboQuant tier", QPS_ERR_UNSUPPORTED);
  if (is_tq(kv.v_fmt)) {
    if (!kv.signs1) return bad(call, n, "signs1 is required for a TurboQuant plane");
    const int g = kv.tq_block == 0 ? kv.d : kv.tq_block;
    if (g < 32 || g > kv.d || (g & (g - 1)))
      return bad(call, n, "tq_block must be 0 or a power of two in [32, head_dim]");
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
