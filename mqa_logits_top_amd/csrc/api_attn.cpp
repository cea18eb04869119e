// C ABI of the operators around the indexer: rotary positions, cache writes and reads, attention
// over the selection and over paged caches, the RMS norm.  Argument checks and launch descriptions, as in api.cpp.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/idx.h"
#include "api_internal.h"
#include "attn.h"
#include "norm.h"
#include "paged.h"
#include "rows.h"

namespace {

constexpr int32_t MAX_D = 512;
constexpr int32_t MAX_ROT = 512;
constexpr int32_t MAX_NORM = 32768;
constexpr int32_t MAX_GROUP = 512;             // values with a scale of their own, where a row has several
constexpr int32_t MAX_REQUESTS = 1 << 16;
constexpr int32_t MAX_POOL = 64;
constexpr int64_t MAX_LD = (int64_t)1 << 31;   // strides: their products with 32-bit counts stay inside 64 bits
constexpr int64_t MAX_ROW = (int64_t)1 << 30;  // elements of an attention cache's slot: 32 bits of bytes

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
idx_status launched(hipError_t e) { return e == hipSuccess ? IDX_OK : IDX_E_LAUNCH; }

// Bits of an element.
int bits(int32_t fmt) {
  switch (fmt) {
    case IDX_K_FP8_E4M3: return 8;
    case IDX_K_MXFP4: return 4;
    case IDX_K_BF16:
    case IDX_K_F16: return 16;
    case IDX_K_F32: return 32;
  }
  return 0;
}
bool value_type(int32_t f) { return f == IDX_K_BF16 || f == IDX_K_F16 || f == IDX_K_F32; }

// Rows of values; written: rows may not share memory.
idx_status check_rows(const idx_rows &x, bool written, int32_t max_d = MAX_D) {
  if (x.T < 0 || x.H < 0 || x.D <= 0) return IDX_E_SHAPE;
  if (!value_type(x.dtype)) return IDX_E_FORMAT;
  if (x.D % 8 || x.D > max_d) return IDX_E_UNSUPPORTED;
  if (x.ld_t < 0 || x.ld_h < 0 || x.ld_t > MAX_LD || x.ld_h > MAX_LD) return IDX_E_SHAPE;
  if (x.T == 0 || x.H == 0) return IDX_OK;
  if (!x.data) return IDX_E_NULL;
  if (written) {
    if ((x.H > 1 && x.ld_h < x.D) || (x.T > 1 && x.ld_t < x.D)) return IDX_E_SHAPE;
    if (x.T > 1 && x.H > 1 && x.ld_t < (x.H - 1) * x.ld_h + x.D && x.ld_h < (x.T - 1) * x.ld_t + x.D)
      return IDX_E_SHAPE;
  }
  const int64_t per = 128 / bits(x.dtype);
  if (!aligned(x.data, 16) || (x.T > 1 && x.ld_t % per) || (x.H > 1 && x.ld_h % per)) return IDX_E_ALIGN;
  return IDX_OK;
}

idx_status check_cache(const idx_cache &c, int32_t max_d = MAX_D) {
  if (c.rows < 0 || c.rows > INT32_MAX || c.H <= 0 || c.D <= 0) return IDX_E_SHAPE;
  const int b = bits(c.fmt);
  if (!b) return IDX_E_FORMAT;
  if (c.D % (c.fmt == IDX_K_MXFP4 ? 32 : 8) || c.D > max_d) return IDX_E_UNSUPPORTED;
  const int64_t width = (int64_t)c.H * c.D;
  const bool scaled = c.fmt == IDX_K_FP8_E4M3 || c.fmt == IDX_K_MXFP4;
  const int64_t swidth = c.fmt == IDX_K_MXFP4 ? width / 32 : c.H;
  if (c.ld > MAX_LD || c.ld < 0 || (c.rows > 1 && c.ld < width)) return IDX_E_SHAPE;
  if (scaled && (c.ld_scale > MAX_LD || c.ld_scale < 0 || (c.rows > 1 && c.ld_scale < swidth))) return IDX_E_SHAPE;
  if (c.rows == 0) return IDX_OK;
  if (!c.data || (scaled && !c.scale)) return IDX_E_NULL;
  if (!aligned(c.data, 16) || (c.rows > 1 && c.ld % 8)) return IDX_E_ALIGN;   // every access takes 8 elements
  if (c.fmt == IDX_K_FP8_E4M3 && !aligned(c.scale, 4)) return IDX_E_ALIGN;
  return IDX_OK;
}

idx_status check_rotary(const idx_rotary &r, int32_t D, int32_t T) {
  if (r.layout != IDX_ROPE_HALF && r.layout != IDX_ROPE_INTERLEAVED) return IDX_E_FORMAT;
  if (r.rot < 8 || r.rot % 8 || r.rot0 < 0 || r.rot0 % 8 || r.rot > D || r.rot0 > D - r.rot) return IDX_E_SHAPE;
  if (!std::isfinite(r.mscale)) return IDX_E_PARAM;
  if (T == 0) return IDX_OK;
  if (!r.freq || !r.pos) return IDX_E_NULL;
  if (!aligned(r.freq, 8) || !aligned(r.pos, 4)) return IDX_E_ALIGN;
  return IDX_OK;
}

int64_t bytes_of(int64_t elements, int32_t fmt) { return elements * bits(fmt) / 8; }

idx::RowJob row_job(const idx_rows &x, const idx_rotary *r, const int32_t *slot, const idx_cache &to) {
  idx::RowJob j{};
  j.x = (const uint8_t *)x.data;
  j.x_t = bytes_of(x.ld_t, x.dtype);
  j.x_h = bytes_of(x.ld_h, x.dtype);
  j.out = (uint8_t *)to.data;
  j.out_t = bytes_of(to.ld, to.fmt);
  j.out_h = bytes_of(to.D, to.fmt);
  j.scale = (uint8_t *)to.scale;
  const int64_t entry = to.fmt == IDX_K_FP8_E4M3 ? 4 : 1;
  j.scale_t = to.ld_scale * entry;
  j.scale_h = to.fmt == IDX_K_FP8_E4M3 ? 4 : to.D / 32;
  j.slot = slot;
  j.rows = to.rows;
  j.T = x.T;
  j.H = x.H;
  j.D = x.D;
  j.dtype = x.dtype;
  j.fmt = to.fmt;
  if (r) {
    j.freq = r->freq;
    j.pos = r->pos;
    j.mscale = r->mscale;
    j.rot = r->rot;
    j.rot0 = r->rot0;
    j.half = r->layout == IDX_ROPE_HALF;
    j.inverse = r->inverse != 0;
  }
  return j;
}

// A launch has a lane to 8 values, and fewer than 2^32 lanes.
constexpr int64_t MAX_LANES = (int64_t)1 << 31;
int64_t lanes_of(const idx_rows &x) {
  const int64_t rows = (int64_t)x.T * x.H;
  if (rows >= MAX_LANES) return MAX_LANES;
  int64_t lanes = 1;
  while (8 * lanes < x.D) lanes *= 2;
  return rows * lanes;
}

// The scale for powers of two.
float scale2_of(float scale) { return (float)((double)scale * 1.4426950408889634); }

// Whether two row arrays that start together lie alike; true where they do not.
bool alike(const idx_rows &a, const idx_rows &b) {
  return a.data != b.data || (bits(a.dtype) == bits(b.dtype) && (a.T <= 1 || a.ld_t == b.ld_t) &&
                              (a.H <= 1 || a.ld_h == b.ld_h));
}

// Queries, outputs and caches of an attention.
template <class Attn>
idx_status check_attn_arrays(const Attn *a) {
  idx_status st;
  if ((st = check_rows(a->q, false)) || (st = check_rows(a->out, true))) return st;
  if ((st = check_cache(a->k)) || (st = check_cache(a->v))) return st;
  if (a->q.T != a->out.T || a->q.H != a->out.H || a->q.D != a->out.D) return IDX_E_SHAPE;
  if (a->k.H != a->v.H || a->k.D != a->q.D || a->v.D != a->q.D || a->k.rows != a->v.rows) return IDX_E_SHAPE;
  if (a->q.H <= 0 || a->q.H % a->k.H) return IDX_E_SHAPE;
  if (a->q.dtype == IDX_K_F32 || a->out.dtype != a->q.dtype) return IDX_E_FORMAT;
  if (a->k.fmt != a->v.fmt) return IDX_E_FORMAT;
  if (a->k.fmt != a->q.dtype && a->k.fmt != IDX_K_FP8_E4M3) return IDX_E_UNSUPPORTED;
  if (a->q.D != 64 && a->q.D != 128) return IDX_E_UNSUPPORTED;
  if (a->k.ld != a->v.ld || a->k.ld_scale != a->v.ld_scale) return IDX_E_SHAPE;
  if (a->k.ld > MAX_ROW) return IDX_E_UNSUPPORTED;
  if ((int64_t)a->q.T * a->q.H >= (int64_t)1 << 26) return IDX_E_UNSUPPORTED;   // at most a wave each: 2^32 lanes
  if (!std::isfinite(scale2_of(a->scale))) return IDX_E_PARAM;
  // the attention kernels read 16 bytes of a cache row at a time
  const int64_t per = 128 / bits(a->k.fmt);
  if (a->k.rows > 1 && (a->k.ld % per || a->v.ld % per)) return IDX_E_ALIGN;
  return aligned(a->lse, 4) ? IDX_OK : IDX_E_ALIGN;
}

idx_status check_attn(const idx_attn *a) {
  if (!a) return IDX_E_NULL;
  const idx_status st = check_attn_arrays(a);
  if (st) return st;
  if (a->L < 0 || a->n_sel < 0 || a->ld_sel < 0 || (a->q.T > 1 && a->ld_sel < a->n_sel)) return IDX_E_SHAPE;
  if (!a->slot_of_key && a->L > a->k.rows) return IDX_E_SHAPE;
  if (a->pool < 1 || a->pool > MAX_POOL || (a->pool & (a->pool - 1))) return IDX_E_UNSUPPORTED;
  if ((a->ks == nullptr) != (a->ke == nullptr) || (a->pool > 1 && !a->ks && a->q.T > 0)) return IDX_E_NULL;
  if (a->q.T > 0 && a->n_sel > 0 && !a->sel) return IDX_E_NULL;
  if (!aligned(a->sel, 4) || !aligned(a->ks, 4) || !aligned(a->ke, 4) || !aligned(a->slot_of_key, 4))
    return IDX_E_ALIGN;
  return IDX_OK;
}

idx::PagedPlan plan_of(const idx_paged *a) {
  return idx::plan_paged(a->q.T, a->B, a->k.H, a->q.H / a->k.H, a->q.D, a->n_pages * a->page,
                         a->k.fmt == IDX_K_FP8_E4M3);
}

idx_status check_paged(const idx_paged *a) {
  if (!a) return IDX_E_NULL;
  const idx_status st = check_attn_arrays(a);
  if (st) return st;
  if (a->B < 0 || a->n_pages < 0 || a->ld_pages < 0 || a->ld_pages > MAX_LD || (a->B > 1 && a->ld_pages < a->n_pages))
    return IDX_E_SHAPE;
  if (!alike(a->out, a->q)) return IDX_E_SHAPE;
  if (a->B > MAX_REQUESTS) return IDX_E_UNSUPPORTED;
  if (a->page < 1 || (a->page & (a->page - 1))) return IDX_E_UNSUPPORTED;
  if ((int64_t)a->n_pages * a->page > INT32_MAX) return IDX_E_UNSUPPORTED;
  if (a->window < 0 || a->first < 0) return IDX_E_PARAM;
  if (a->q.T > 0 && a->B > 0 && (!a->cu_q || !a->len_k || (a->n_pages > 0 && !a->pages))) return IDX_E_NULL;
  if (!aligned(a->pages, 4) || !aligned(a->cu_q, 4) || !aligned(a->len_k, 4)) return IDX_E_ALIGN;
  // workgroups of 256 lanes, fewer than 2^32 lanes
  const idx::PagedPlan plan = plan_of(a);
  return plan.max_items < (int64_t)1 << 23 && plan.grid < (int64_t)1 << 24 ? IDX_OK : IDX_E_UNSUPPORTED;
}

bool same_sizes(const idx_rows &a, const idx_rows &b) { return a.T == b.T && a.H == b.H && a.D == b.D; }

idx_status check_norm(const idx_norm *n) {
  if (!n) return IDX_E_NULL;
  idx_status st;
  const idx_rows &x = n->x;
  if ((st = check_rows(x, false, MAX_NORM))) return st;
  if (!(n->eps >= 0.f) || !std::isfinite(n->eps)) return IDX_E_PARAM;
  if (n->weight && (!value_type(n->weight_dtype))) return IDX_E_FORMAT;
  if (!aligned(n->weight, 16)) return IDX_E_ALIGN;
  if (x.T == 0 || x.H == 0) return IDX_OK;
  if (lanes_of(x) >= MAX_LANES) return IDX_E_UNSUPPORTED;
  if (!n->out.data && !n->to) return IDX_E_NULL;
  if (n->residual.data) {
    if ((st = check_rows(n->residual, false, MAX_NORM)) || (st = check_rows(n->total, true, MAX_NORM))) return st;
    if (!same_sizes(x, n->residual) || !same_sizes(x, n->total)) return IDX_E_SHAPE;
    if (n->residual.dtype != n->total.dtype) return IDX_E_FORMAT;
    if (!alike(n->total, x) || !alike(n->total, n->residual)) return IDX_E_SHAPE;
  }
  if (n->out.data) {
    if ((st = check_rows(n->out, true, MAX_NORM))) return st;
    if (!same_sizes(x, n->out) || !alike(n->out, x)) return IDX_E_SHAPE;
    if (n->residual.data && (n->out.data == n->total.data || !alike(n->out, n->residual))) return IDX_E_SHAPE;
  }
  if (n->to) {
    const idx_cache &c = *n->to;
    if ((st = check_cache(c, MAX_NORM))) return st;
    if (c.fmt != IDX_K_FP8_E4M3) return IDX_E_UNSUPPORTED;
    if (x.H == 1 ? (int64_t)c.H * c.D != x.D : c.H != x.H || c.D != x.D) return IDX_E_SHAPE;
    if (c.rows < x.T) return IDX_E_SHAPE;
    if (c.D != x.D && (c.D > MAX_GROUP || (c.D & (c.D - 1)))) return IDX_E_UNSUPPORTED;
  }
  return IDX_OK;
}

idx::NormRows norm_rows(const idx_rows &x) {
  return {(uint8_t *)x.data, bytes_of(x.ld_t, x.dtype), bytes_of(x.ld_h, x.dtype), x.dtype};
}

idx::AttnPlan plan_of(const idx_attn *a) {
  const bool fp8 = a->k.fmt == IDX_K_FP8_E4M3;
  const int64_t entries = (int64_t)a->n_sel * a->pool;
  // T * entries stays inside 64 bits: 2^26 rows of 2^37
  const int64_t slots = entries * a->q.T < a->k.rows ? entries * a->q.T : a->k.rows;
  const int64_t touched = 2 * slots * (int64_t)a->k.H * a->k.D * (fp8 ? 1 : 2);
  return idx::plan_attn(a->q.T, a->k.H, a->q.H / a->k.H, a->q.D, fp8, entries, touched);
}

}  // namespace

extern "C" {

idx_status idx_rope_freqs(int32_t rot, double base, int32_t scaling, double factor, double original, double beta_fast,
                          double beta_slow, double *freq, double *mscale) {
  if (!freq) return IDX_E_NULL;
  if (rot < 2 || rot % 2 || rot > MAX_ROT) return IDX_E_SHAPE;
  if (!(base > 1.0) || !std::isfinite(base)) return IDX_E_PARAM;
  if (scaling < IDX_ROPE_PLAIN || scaling > IDX_ROPE_PARTS) return IDX_E_FORMAT;
  if (scaling != IDX_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return IDX_E_PARAM;
  if (scaling == IDX_ROPE_BASE && rot < 4) return IDX_E_SHAPE;
  if (scaling == IDX_ROPE_PARTS && (!(original > 0.0) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) ||
                                    !std::isfinite(original) || !std::isfinite(beta_fast)))
    return IDX_E_PARAM;
  if (scaling == IDX_ROPE_BASE) base *= std::pow(factor, (double)rot / (rot - 2));
  double lo = 0.0, hi = 0.0;
  if (scaling == IDX_ROPE_PARTS) {
    // the pair that makes `turns` turns over the original context: base^(-2 i / rot) * original = 2 pi turns
    const double per = rot / (2.0 * std::log(base)), two_pi = 6.283185307179586476925;
    lo = std::floor(per * std::log(original / (beta_fast * two_pi)));
    hi = std::ceil(per * std::log(original / (beta_slow * two_pi)));
    lo = lo > 0.0 ? lo : 0.0;
    hi = hi < rot - 1 ? hi : rot - 1;
  }
  for (int32_t i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == IDX_ROPE_LINEAR) f /= factor;
    if (scaling == IDX_ROPE_PARTS) {
      const double span = hi - lo > 0.001 ? hi - lo : 0.001;
      double r = (i - lo) / span;
      r = r < 0.0 ? 0.0 : r > 1.0 ? 1.0 : r;
      f = f * (1.0 - r) + f / factor * r;
    }
    freq[i] = f;
  }
  if (mscale) *mscale = scaling == IDX_ROPE_PARTS ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return IDX_OK;
}

idx_status idx_rope(const idx_rows *x, const idx_rotary *r, const idx_rows *out, void *stream) {
  if (!x || !r || !out) return IDX_E_NULL;
  idx_status st;
  if ((st = check_rows(*x, false)) || (st = check_rows(*out, true)) || (st = check_rotary(*r, x->D, x->T))) return st;
  if (x->T != out->T || x->H != out->H || x->D != out->D) return IDX_E_SHAPE;
  if (x->dtype != out->dtype) return IDX_E_FORMAT;
  if (x->data == out->data && ((x->T > 1 && x->ld_t != out->ld_t) || (x->H > 1 && x->ld_h != out->ld_h)))
    return IDX_E_SHAPE;
  if (lanes_of(*x) >= MAX_LANES) return IDX_E_UNSUPPORTED;
  const idx_cache to{out->data, nullptr, out->T, out->ld_t, 0, out->dtype, out->H, out->D};
  idx::RowJobs jobs{};
  jobs.job[0] = row_job(*x, r, nullptr, to);
  jobs.job[0].out_h = bytes_of(out->ld_h, out->dtype);
  jobs.n = 1;
  return launched(idx::launch_rows(jobs, (hipStream_t)stream));
}

idx_status idx_cache_write(const idx_write *w, int32_t n, void *stream) {
  if (n < 0 || n > IDX_MAX_WRITES) return IDX_E_PARAM;
  if (n > 0 && !w) return IDX_E_NULL;
  idx::RowJobs jobs{};
  int64_t lanes = 0;
  for (int32_t i = 0; i < n; ++i) {
    idx_status st;
    if ((st = check_rows(w[i].x, false)) || (st = check_cache(w[i].to))) return st;
    if (w[i].rotary && (st = check_rotary(*w[i].rotary, w[i].x.D, w[i].x.T))) return st;
    if (w[i].x.H != w[i].to.H || w[i].x.D != w[i].to.D) return IDX_E_SHAPE;
    if (!w[i].slot && w[i].x.T > w[i].to.rows) return IDX_E_SHAPE;
    if (!aligned(w[i].slot, 4)) return IDX_E_ALIGN;
    lanes += lanes_of(w[i].x);
    if (lanes >= MAX_LANES) return IDX_E_UNSUPPORTED;
    jobs.job[i] = row_job(w[i].x, w[i].rotary, w[i].slot, w[i].to);
  }
  jobs.n = n;
  for (int32_t i = 0; i < n; ++i) {
    const idx_status st = idx::debug_check_slots(w[i].slot, w[i].x.T, w[i].to.rows, stream);
    if (st) return st;
  }
  return launched(idx::launch_rows(jobs, (hipStream_t)stream));
}

idx_status idx_cache_read(const idx_cache *c, const int32_t *rows, const idx_rows *out, void *stream) {
  if (!c || !out) return IDX_E_NULL;
  idx_status st;
  if ((st = check_cache(*c)) || (st = check_rows(*out, true))) return st;
  if (c->H != out->H || c->D != out->D) return IDX_E_SHAPE;
  if (!aligned(rows, 4)) return IDX_E_ALIGN;
  if (lanes_of(*out) >= MAX_LANES) return IDX_E_UNSUPPORTED;
  idx::ReadJob j{};
  j.data = (const uint8_t *)c->data;
  j.data_t = bytes_of(c->ld, c->fmt);
  j.data_h = bytes_of(c->D, c->fmt);
  j.scale = (const uint8_t *)c->scale;
  j.scale_t = c->ld_scale * (c->fmt == IDX_K_FP8_E4M3 ? 4 : 1);
  j.scale_h = c->fmt == IDX_K_FP8_E4M3 ? 4 : c->D / 32;
  j.rows = c->rows;
  j.list = rows;
  j.out = (uint8_t *)out->data;
  j.out_t = bytes_of(out->ld_t, out->dtype);
  j.out_h = bytes_of(out->ld_h, out->dtype);
  j.T = out->T;
  j.H = out->H;
  j.D = out->D;
  j.fmt = c->fmt;
  j.dtype = out->dtype;
  return launched(idx::launch_read(j, (hipStream_t)stream));
}

idx_status idx_sparse_attn_workspace(const idx_attn *a, size_t *bytes) {
  if (!bytes) return IDX_E_NULL;
  const idx_status st = check_attn(a);
  if (st) return st;
  *bytes = plan_of(a).bytes;
  return IDX_OK;
}

idx_status idx_sparse_attn(const idx_attn *a, void *ws, size_t ws_bytes, void *stream) {
  idx_status st = check_attn(a);
  if (st) return st;
  if (a->q.T == 0) return IDX_OK;
  const idx::AttnPlan plan = plan_of(a);
  if (plan.bytes) {
    if (!ws) return IDX_E_NULL;
    if (ws_bytes < plan.bytes) return IDX_E_WORKSPACE;
    if (!aligned(ws, 256)) return IDX_E_ALIGN;
  }
  if (a->ks && (st = idx::debug_check(a->ks, a->ke, a->q.T, a->L, -1, nullptr, stream))) return st;
  idx::AttnArgs g{};
  g.q = (const uint8_t *)a->q.data;
  g.q_t = 2 * a->q.ld_t;
  g.q_h = 2 * a->q.ld_h;
  g.out = (uint8_t *)a->out.data;
  g.out_t = 2 * a->out.ld_t;
  g.out_h = 2 * a->out.ld_h;
  g.k = (const uint8_t *)a->k.data;
  g.v = (const uint8_t *)a->v.data;
  g.row_bytes = (uint32_t)bytes_of(a->k.ld, a->k.fmt);
  g.k_scale = (const float *)a->k.scale;
  g.v_scale = (const float *)a->v.scale;
  g.scale_row = a->k.ld_scale;
  g.rows = a->k.rows;
  g.sel = a->sel;
  g.ld_sel = a->ld_sel;
  g.n_sel = a->n_sel;
  while ((1 << g.pool_sh) < a->pool) ++g.pool_sh;
  g.ks = a->ks;
  g.ke = a->ke;
  g.table = a->slot_of_key;
  g.L = a->L;
  g.T = a->q.T;
  g.Hq = a->q.H;
  g.Hkv = a->k.H;
  g.G = a->q.H / a->k.H;
  g.scale2 = scale2_of(a->scale);
  g.lse = a->lse;
  return launched(idx::launch_attn(g, a->q.dtype, a->k.fmt, a->q.D, plan, ws, (hipStream_t)stream));
}

idx_status idx_paged_attn_workspace(const idx_paged *a, size_t *bytes) {
  if (!bytes) return IDX_E_NULL;
  const idx_status st = check_paged(a);
  if (st) return st;
  *bytes = plan_of(a).bytes;
  return IDX_OK;
}

idx_status idx_paged_attn(const idx_paged *a, void *ws, size_t ws_bytes, void *stream) {
  idx_status st = check_paged(a);
  if (st) return st;
  if (a->q.T == 0 || a->B == 0) return IDX_OK;
  const idx::PagedPlan plan = plan_of(a);
  if (plan.bytes) {
    if (!ws) return IDX_E_NULL;
    if (ws_bytes < plan.bytes) return IDX_E_WORKSPACE;
    if (!aligned(ws, 256)) return IDX_E_ALIGN;
  }
  idx::PagedArgs g{};
  g.q = (const uint8_t *)a->q.data;
  g.q_t = 2 * a->q.ld_t;
  g.q_h = 2 * a->q.ld_h;
  g.out = (uint8_t *)a->out.data;
  g.out_t = 2 * a->out.ld_t;
  g.out_h = 2 * a->out.ld_h;
  g.k = (const uint8_t *)a->k.data;
  g.v = (const uint8_t *)a->v.data;
  g.row_bytes = (uint32_t)bytes_of(a->k.ld, a->k.fmt);
  g.k_scale = (const float *)a->k.scale;
  g.v_scale = (const float *)a->v.scale;
  g.scale_row = a->k.ld_scale;
  g.rows = a->k.rows;
  g.pages = a->pages;
  g.ld_pages = a->ld_pages;
  while ((1 << g.page_sh) < a->page) ++g.page_sh;
  g.max_len = a->n_pages * a->page;
  g.cu_q = a->cu_q;
  g.len_k = a->len_k;
  g.B = a->B;
  g.T = a->q.T;
  g.Hq = a->q.H;
  g.Hkv = a->k.H;
  g.G = a->q.H / a->k.H;
  g.window = a->window;
  g.first = a->first;
  g.scale2 = scale2_of(a->scale);
  g.lse = a->lse;
  if ((st = idx::debug_check_paged(g, stream))) return st;
  return launched(idx::launch_paged(g, a->q.dtype, a->k.fmt, a->q.D, plan, ws, (hipStream_t)stream));
}

idx_status idx_rms_norm(const idx_norm *n, void *stream) {
  const idx_status st = check_norm(n);
  if (st) return st;
  if (n->x.T == 0 || n->x.H == 0) return IDX_OK;
  idx::NormJob j{};
  j.x = norm_rows(n->x);
  if (n->residual.data) {
    j.residual = norm_rows(n->residual);
    j.total = norm_rows(n->total);
  }
  if (n->out.data) j.out = norm_rows(n->out);
  j.group = n->x.D;
  if (n->to) {
    j.codes = (uint8_t *)n->to->data;
    j.codes_t = n->to->ld;
    j.codes_h = n->to->D;
    j.scale = (float *)n->to->scale;
    j.scale_t = n->to->ld_scale;
    j.group = n->to->D;
  }
  j.weight = (const uint8_t *)n->weight;
  j.weight_dtype = n->weight_dtype;
  j.T = n->x.T;
  j.H = n->x.H;
  j.D = n->x.D;
  j.eps = n->eps;
  return launched(idx::launch_norm(j, (hipStream_t)stream));
}

}  // extern "C"
