// Rows on their way into and out of caches.
//  - write: rotary positions, then E4M3 / MXFP4 / 16- or 32-bit storage at a slot.  idx_rope is
//    this kernel with a 16- or 32-bit output and no slots.
//  - read: cache rows as values, by slot.
// Both move each byte once.  Measured (a large copy moves 4.9 TB/s here, reads and writes counted):
//   16384 rows x 64 heads of 128 rotated, bf16: 93 us, 5.8 TB/s (the copy's rate: 110 us);
//   30720 rows x 8 heads, keys rotated and values, to E4M3 slots in any order: 48 us, 4.0 TB/s (39 us);
//   2048 rows x 64 heads rotated to E4M3: 17 us (10.5 us): the lanes' loads are all under way at once, and the
//     800 instructions of a wave follow them;
//   102400 MXFP4 rows read: 8.1 us, 4.1 TB/s (6.9 us); one row of 32 heads rotated: 2.9 us, the launch.
#include "common.h"
#include "rows.h"

namespace idx {
namespace {

constexpr int HEADS = 4;       // heads a lane takes of one token at most: they share the sines and cosines
constexpr int THREADS = 256;

template <bool F32>
struct Raw {   // 8 elements
  uint4 w[F32 ? 2 : 1];
};

__device__ __forceinline__ float bf16_val(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float f16_val(uint32_t u) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)u);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  const v2 p = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  typedef _Float16 v2 __attribute__((ext_vector_type(2)));
  const v2 p = {(_Float16)lo, (_Float16)hi};
  return __builtin_bit_cast(uint32_t, p);
}

// Four 16-bit or fp32 values of a word group.
__device__ __forceinline__ void unpack4(uint32_t w0, uint32_t w1, int dtype, float *v) {
  if (dtype == IDX_K_BF16) {
    v[0] = bf16_val(w0 & 0xFFFFu);
    v[1] = __uint_as_float(w0 & 0xFFFF0000u);
    v[2] = bf16_val(w1 & 0xFFFFu);
    v[3] = __uint_as_float(w1 & 0xFFFF0000u);
  } else {
    v[0] = f16_val(w0 & 0xFFFFu);
    v[1] = f16_val(w0 >> 16);
    v[2] = f16_val(w1 & 0xFFFFu);
    v[3] = f16_val(w1 >> 16);
  }
}

// The lane's 8 elements: two groups of four at element offsets e0 and e1 (e1 = e0 + 4 unless the
// lane holds both halves of four rotated pairs).
template <bool F32>
__device__ __forceinline__ Raw<F32> load8(const uint8_t *p, int dtype, int e0, int e1, bool split) {
  Raw<F32> r;
  if constexpr (F32) {
    if (dtype == IDX_K_F32) {
      r.w[0] = *(const uint4 *)(p + 4 * e0);
      r.w[1] = *(const uint4 *)(p + 4 * e1);
      return r;
    }
  }
  if (split) {
    const uint2 lo = *(const uint2 *)(p + 2 * e0), hi = *(const uint2 *)(p + 2 * e1);
    r.w[0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
  } else {
    r.w[0] = *(const uint4 *)(p + 2 * e0);
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ void values8(const Raw<F32> &r, int dtype, float *v) {
  if constexpr (F32) {
    if (dtype == IDX_K_F32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[4 * i] = __uint_as_float(r.w[i].x);
        v[4 * i + 1] = __uint_as_float(r.w[i].y);
        v[4 * i + 2] = __uint_as_float(r.w[i].z);
        v[4 * i + 3] = __uint_as_float(r.w[i].w);
      }
      return;
    }
  }
  unpack4(r.w[0].x, r.w[0].y, dtype, v);
  unpack4(r.w[0].z, r.w[0].w, dtype, v + 4);
}

// Largest of x over aligned groups of 2^sh lanes.
__device__ __forceinline__ uint32_t group_max(uint32_t x, int sh) {
  if (sh > 0) x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, false));
  if (sh > 1) x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, false));
  if (sh > 2) x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xF, 0xF, false));
  if (sh > 3) x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x140, 0xF, 0xF, false));
  if (sh > 4) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = max(r[0], r[1]);
  }
  if (sh > 5) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = max(r[0], r[1]);
  }
  return x;
}

__device__ __forceinline__ uint32_t e4m3x4(const float *v) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
  return (uint32_t)w;
}

template <int LANE>   // x of that lane of the quad
__device__ __forceinline__ float of_quad(float x) {
  return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), LANE * 0x55, 0xF, 0xF, false));
}
// 448 / amax less its rounded value inv: with it x * 448 / amax is rounded once, so that values half way between
// two codes (16-bit values often are) go to the even one.  One more fma a value (no time); 0.1% of a bf16
// array's codes would go to the other one without it.
__device__ __forceinline__ float inverse_rest(float amax, float inv) {
  return __builtin_fmaf(-inv, amax, 448.0f) * (inv * (1.0f / 448.0f));
}

// Sine and cosine of an angle below 2^32, within 2^-45 (fp32 keeps 2^-24): the angle less its nearest multiple of
// pi/2 (pi/2 in three parts of 53 bits; each fma is exact but for its one rounding, and the angle's multiple k of
// pi/2 is below 2^32), then the Taylor series on [-pi/4, pi/4], the sine's to x^13 (the next term is below 2^-45.4),
// the cosine's to x^14 (2^-49.7), and the quadrant's exchange of the two.  No branch, a quarter of the library
// function's instructions, which took more time than the rotation.
__device__ __forceinline__ void sin_cos(double x, double *sn, double *cs) {
  const double k = __builtin_rint(x * 0.63661977236758134308);   // 2 / pi
  double r = __builtin_fma(-k, 1.57079632679489655800, x);
  r = __builtin_fma(-k, 6.12323399573676603587e-17, r);
  r = __builtin_fma(-k, -1.49738490485916983280e-33, r);
  const double z = r * r;
  double s = 1.0 / 6227020800.0;
  s = __builtin_fma(s, z, -1.0 / 39916800.0);
  s = __builtin_fma(s, z, 1.0 / 362880.0);
  s = __builtin_fma(s, z, -1.0 / 5040.0);
  s = __builtin_fma(s, z, 1.0 / 120.0);
  s = __builtin_fma(s, z, -1.0 / 6.0);
  s = __builtin_fma(s * z, r, r);
  double c = -1.0 / 87178291200.0;
  c = __builtin_fma(c, z, 1.0 / 479001600.0);
  c = __builtin_fma(c, z, -1.0 / 3628800.0);
  c = __builtin_fma(c, z, 1.0 / 40320.0);
  c = __builtin_fma(c, z, -1.0 / 720.0);
  c = __builtin_fma(c, z, 1.0 / 24.0);
  c = __builtin_fma(c, z, -0.5);
  c = __builtin_fma(c, z, 1.0);
  const uint32_t q = (uint32_t)(int32_t)__builtin_fma(-4.0, __builtin_floor(k * 0.25), k);   // k modulo 4
  const double a = q & 1u ? c : s, b = q & 1u ? s : c;
  *sn = q & 2u ? -a : a;
  *cs = (q + 1u) & 2u ? -b : b;
}

// The lane's four pairs: (v[e], v[4 + e]) for split halves, else neighbours.  In fp64, each result rounded once.
template <bool SPLIT>
__device__ __forceinline__ void rotate4(float *v, const double *cs, const double *sn) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float &x = v[SPLIT ? e : 2 * e], &y = v[SPLIT ? 4 + e : 2 * e + 1];
    const double a = x, b = y;
    x = (float)(a * cs[e] - b * sn[e]);
    y = (float)(b * cs[e] + a * sn[e]);
  }
}

constexpr uint32_t TINY = 0x0D800000u;   // bits of 2^-100
constexpr uint32_t INF = 0x7F800000u;

// The first N of a launch's jobs, as the kernel's argument.  A single one has a kernel of its own: no search, and
// 0.2 KB for the host to write a launch instead of 1.3 (one row of 32 heads 2.9 us, 3.2 among eight; 16384 rows of
// 64 heads 93.4, 95.3; the call 0.3 us less on the host).
template <int N>
struct Jobs {
  RowJob job[N];
  int32_t first[N];
  int32_t n;
};

// A lane takes 8 dims of up to four heads of one token: its loads are under way before the angles are computed, and
// the heads share them (two heads a lane: 10% slower; eight: no gain).  A lane of a rotated part of halves holds four dims
// of either half, so that every pair is one lane's.  A row's largest magnitude is reduced over its lanes.
// F32: some array of the call holds or receives fp32 values (the others then keep fewer registers).
template <bool F32, int N>
__global__ __launch_bounds__(THREADS) void write_kernel(Jobs<N> jobs) {
  int ji = 0;
  if constexpr (N > 1)
    while (ji + 1 < jobs.n && (int)blockIdx.x >= jobs.first[ji + 1]) ++ji;
  const RowJob &j = jobs.job[ji];
  const int sh = j.lanes_sh;
  const uint32_t unit = ((blockIdx.x - (uint32_t)jobs.first[ji]) << (8 - sh)) + (threadIdx.x >> sh);
  const int c = threadIdx.x & ((1 << sh) - 1);
  const uint32_t tu = unit / (uint32_t)j.groups;
  const int hs = (int)(unit - tu * (uint32_t)j.groups);
  if (tu >= (uint32_t)j.T) return;        // whole lane groups leave together
  const int t = (int)tu;
  const bool live = c * 8 < j.D;
  const int64_t slot = j.slot ? (int64_t)j.slot[t] : (int64_t)t;
  if (slot < 0 || slot >= j.rows) return;

  // this lane's elements, and its pairs
  int e0 = c * 8, e1 = e0 + 4;
  const int part = e0 - j.rot0;
  const bool turned = j.freq && part >= 0 && part < j.rot && live;
  const bool split = turned && j.half;
  if (split) {
    e0 = j.rot0 + part / 2;
    e1 = e0 + j.rot / 2;
  }
  Raw<F32> raw[HEADS];
  const uint8_t *xt = j.x + (int64_t)t * j.x_t;
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = hs + i * j.groups;
    if (live && h < j.H) raw[i] = load8<F32>(xt + (int64_t)h * j.x_h, j.dtype, e0, e1, split);
  }
  double cs[4], sn[4];
  if (turned) {
    const double p = (double)j.pos[t], gain_s = j.inverse ? -j.mscale : j.mscale;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      double s, k;
      sin_cos(p * j.freq[part / 2 + i], &s, &k);
      cs[i] = k * j.mscale;
      sn[i] = s * gain_s;
    }
  }
  float v[HEADS][8];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    if (hs + i * j.groups >= j.H) break;         // the same for the whole lane group
    if (live) {
      values8<F32>(raw[i], j.dtype, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
    if (j.half) {
      if (turned) rotate4<true>(v[i], cs, sn);
    } else {
      if (turned) rotate4<false>(v[i], cs, sn);
    }
  }
  uint8_t *const out = j.out + slot * j.out_t;

  if (j.fmt == IDX_K_FP8_E4M3) {
    // Lane 4 n + i of a group divides for head i (lanes_sh >= 2; else every lane for each): two divisions for
    // all heads instead of two a head
    uint32_t m[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      m[i] = 0;
      if (hs + i * j.groups >= j.H) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) m[i] = max(m[i], __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
      m[i] = group_max(m[i], sh);
    }
    static_assert(HEADS == 4, "one lane of a quad to a head");
    const int mine = c & 3;
    const uint32_t ml = mine & 2 ? (mine & 1 ? m[3] : m[2]) : (mine & 1 ? m[1] : m[0]);
    const float amax = __uint_as_float(ml);
    const float inv = ml >= TINY ? 448.0f / amax : 0.f, more = inverse_rest(amax, inv);
    if (sh >= 2) {
      // a NaN or an infinity in the row makes the scale NaN, and with it the whole row
      const int h = hs + mine * j.groups;
      if (c < 4 && h < j.H)
        *(float *)(j.scale + slot * j.scale_t + (int64_t)h * j.scale_h) =
            ml >= INF ? __uint_as_float(0x7FC00000u) : ml >= TINY ? amax / 448.0f : 1.0f;
    }
    const float quad[HEADS] = {of_quad<0>(inv), of_quad<1>(inv), of_quad<2>(inv), of_quad<3>(inv)};
    const float rest[HEADS] = {of_quad<0>(more), of_quad<1>(more), of_quad<2>(more), of_quad<3>(more)};
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      const int h = hs + i * j.groups;
      if (h >= j.H) break;
      float f = quad[i], f1 = rest[i];
      if (sh < 2) {   // rows of one or two lanes: no quad of their own
        const float am = __uint_as_float(m[i]);
        f = m[i] >= TINY ? 448.0f / am : 0.f;
        f1 = inverse_rest(am, f);
        if (c == 0)
          *(float *)(j.scale + slot * j.scale_t + (int64_t)h * j.scale_h) =
              m[i] >= INF ? __uint_as_float(0x7FC00000u) : m[i] >= TINY ? am / 448.0f : 1.0f;
      }
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(v[i][e], f, v[i][e] * f1);
      if (live) {
        uint8_t *o = out + (int64_t)h * j.out_h;
        const uint32_t w0 = e4m3x4(y), w1 = e4m3x4(y + 4);
        if (split) {
          *(uint32_t *)(o + e0) = w0;
          *(uint32_t *)(o + e1) = w1;
        } else {
          *(uint2 *)(o + e0) = make_uint2(w0, w1);
        }
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = hs + i * j.groups;
    if (h >= j.H) break;
    uint8_t *o = out + (int64_t)h * j.out_h;
    float *x = v[i];
    if (j.fmt == IDX_K_MXFP4) {
      // The lane's two groups of four lie in blocks of 32 of their own when it holds the halves of
      // pairs: bring the values back into order, lane c holding elements 8c .. 8c + 7.
      if (j.freq && j.half) {
        const int lo = (j.rot0 >> 3), n = j.rot >> 3;        // rotated lanes [lo, lo + n)
        const int base = (threadIdx.x & 63) - c;
        const bool in = c >= lo && c < lo + n;
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int q = 2 * (c - lo) + (e >> 2);             // group of four inside the part
          const int src = in ? lo + (q < n ? q : q - n) : c;
          const float va = __shfl(x[e & 3], base + src), vb = __shfl(x[4 + (e & 3)], base + src);
          w[e] = in ? (q < n ? va : vb) : x[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = w[e];
      }
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7FFFFFFFu);
      m = group_max(m, 2);       // 4 lanes hold a block of 32
      const int ex = (int)(m >> 23) - 127 - 2;
      const int e8 = m >= TINY ? min(max(ex + 127, 0), 254) : 0;
      // 2^(e8 - 127) divides the values; 2^127 leaves none of a block of zeros
      const float unit = m >= TINY ? __uint_as_float((uint32_t)e8 << 23) : 0x1p127f;
      if (live) {
        uint32_t w = 0;   // to nearest even, saturating
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], unit, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], unit, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], unit, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], unit, 3);
        *(uint32_t *)(o + c * 4) = w;
        if ((c & 3) == 0)
          j.scale[slot * j.scale_t + (int64_t)h * j.scale_h + (c >> 2)] = m >= INF ? 0xFFu : (uint8_t)e8;
      }
    } else if (live) {
      if (F32 && j.fmt == IDX_K_F32) {
        *(float4 *)(o + 4 * e0) = make_float4(x[0], x[1], x[2], x[3]);
        *(float4 *)(o + 4 * e1) = make_float4(x[4], x[5], x[6], x[7]);
      } else {
        uint4 w;
        if (j.fmt == IDX_K_BF16)
          w = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
        else
          w = make_uint4(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]), pack_f16(x[4], x[5]), pack_f16(x[6], x[7]));
        if (split) {
          *(uint2 *)(o + 2 * e0) = make_uint2(w.x, w.y);
          *(uint2 *)(o + 2 * e1) = make_uint2(w.z, w.w);
        } else {
          *(uint4 *)(o + 2 * e0) = w;
        }
      }
    }
  }
}

// One lane to 8 elements of a row, READS rows: their loads are under way together (102400 MXFP4 rows: 8.1 us, 13.2
// one at a time).
constexpr int READS = 4;
template <int FMT>   // the cache's; IDX_K_BF16 stands for both 16-bit ones
__global__ __launch_bounds__(THREADS) void read_kernel(ReadJob j) {
  constexpr bool F32 = FMT == IDX_K_F32;
  const int c = threadIdx.x & ((1 << j.lanes_sh) - 1);
  const bool live = c * 8 < j.D;
  const uint32_t units = (uint32_t)j.T * (uint32_t)j.H, per = THREADS >> j.lanes_sh;
  const uint32_t first = blockIdx.x * per * READS + (threadIdx.x >> j.lanes_sh);
  uint32_t t[READS], h[READS];
  int32_t row[READS];
#pragma unroll
  for (int i = 0; i < READS; ++i) {
    const uint32_t u = first + i * per;
    t[i] = j.H == 1 ? u : u / (uint32_t)j.H;
    h[i] = u - t[i] * (uint32_t)j.H;
    row[i] = u < units && live ? j.list ? j.list[t[i]] : (int32_t)t[i] : -1;
    if (row[i] >= j.rows) row[i] = -1;
  }
  Raw<F32> raw[READS];
  uint32_t scale[READS];
#pragma unroll
  for (int i = 0; i < READS; ++i) {
    if (row[i] < 0) continue;
    const uint8_t *p = j.data + row[i] * j.data_t + (int64_t)h[i] * j.data_h;
    if constexpr (FMT == IDX_K_FP8_E4M3) {
      const uint2 w = *(const uint2 *)(p + 8 * c);
      raw[i].w[0] = make_uint4(w.x, w.y, 0u, 0u);
      scale[i] = *(const uint32_t *)(j.scale + row[i] * j.scale_t + (int64_t)h[i] * j.scale_h);
    } else if constexpr (FMT == IDX_K_MXFP4) {
      raw[i].w[0] = make_uint4(*(const uint32_t *)(p + 4 * c), 0u, 0u, 0u);
      scale[i] = (j.scale + row[i] * j.scale_t + (int64_t)h[i] * j.scale_h)[c >> 2];
    } else {
      raw[i] = load8<F32>(p, F32 ? IDX_K_F32 : IDX_K_BF16, 8 * c, 8 * c + 4, false);
    }
  }
#pragma unroll
  for (int i = 0; i < READS; ++i) {
    if (first + i * per >= units || !live) continue;
    float v[8];
    if (row[i] < 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    } else if constexpr (FMT == IDX_K_FP8_E4M3) {
      const float sc = __uint_as_float(scale[i]);
      const int w0 = (int)raw[i].w[0].x, w1 = (int)raw[i].w[0].y;
      const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(w0, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w0, true);
      const auto d = __builtin_amdgcn_cvt_pk_f32_fp8(w1, false), f = __builtin_amdgcn_cvt_pk_f32_fp8(w1, true);
      v[0] = a[0] * sc;
      v[1] = a[1] * sc;
      v[2] = b[0] * sc;
      v[3] = b[1] * sc;
      v[4] = d[0] * sc;
      v[5] = d[1] * sc;
      v[6] = f[0] * sc;
      v[7] = f[1] * sc;
    } else if constexpr (FMT == IDX_K_MXFP4) {
      const uint32_t w = raw[i].w[0].x, e8 = scale[i];
      // E8M0 code 0 stands for 2^-127, a subnormal; 0xFF is NaN
      const float sc = e8 == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float(e8 ? e8 << 23 : 0x00400000u);
      const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
      const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
      const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
      const auto f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
      v[0] = a[0] * sc;
      v[1] = a[1] * sc;
      v[2] = b[0] * sc;
      v[3] = b[1] * sc;
      v[4] = d[0] * sc;
      v[5] = d[1] * sc;
      v[6] = f[0] * sc;
      v[7] = f[1] * sc;
    } else {
      values8<F32>(raw[i], j.fmt, v);
    }
    uint8_t *o = j.out + (int64_t)t[i] * j.out_t + (int64_t)h[i] * j.out_h;
    if (j.dtype == IDX_K_F32) {
      *(float4 *)(o + 32 * c) = make_float4(v[0], v[1], v[2], v[3]);
      *(float4 *)(o + 32 * c + 16) = make_float4(v[4], v[5], v[6], v[7]);
    } else if (j.dtype == IDX_K_BF16) {
      *(uint4 *)(o + 16 * c) =
          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else {
      *(uint4 *)(o + 16 * c) =
          make_uint4(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]), pack_f16(v[6], v[7]));
    }
  }
}

// Every pair of rows: quadratic, for debugging only.
__global__ __launch_bounds__(THREADS) void slot_check_kernel(const int32_t *slot, int32_t T, int64_t rows,
                                                             uint32_t *word) {
  const int64_t t = (int64_t)blockIdx.x * THREADS + threadIdx.x;
  if (t >= T) return;
  const int32_t s = slot[t];
  if (s < 0 || s >= rows) return;
  for (int64_t u = 0; u < t; ++u)
    if (slot[u] == s) {
      atomicOr(word, 32u);
      return;
    }
}

}  // namespace

template <bool F32, int N>
static void launch_jobs(const RowJobs &jobs, hipStream_t s) {
  Jobs<N> few;
  for (int i = 0; i < N; ++i) {
    few.job[i] = jobs.job[i];
    few.first[i] = jobs.first[i];
  }
  few.n = jobs.n;
  hipLaunchKernelGGL((write_kernel<F32, N>), dim3((unsigned)jobs.first[jobs.n]), dim3(THREADS), 0, s, few);
}
template <bool F32>
static void launch_some(const RowJobs &jobs, hipStream_t s) {
  if (jobs.n == 1)
    launch_jobs<F32, 1>(jobs, s);
  else
    launch_jobs<F32, IDX_MAX_WRITES>(jobs, s);
}

// log2 of the lanes of a row: the power of two at or above D / 8
static int lanes_of(int32_t D) {
  int sh = 0;
  while ((8 << sh) < D) ++sh;
  return sh;
}

hipError_t launch_rows(RowJobs &jobs, hipStream_t s) {
  int64_t blocks = 0;
  int m = 0;
  bool f32 = false;
  for (int i = 0; i < jobs.n; ++i) {
    RowJob j = jobs.job[i];
    if (j.T <= 0 || j.H <= 0 || j.rows <= 0) continue;
    j.lanes_sh = lanes_of(j.D);
    f32 = f32 || j.dtype == IDX_K_F32 || j.fmt == IDX_K_F32;
    // as many heads to a lane as still leave every SIMD eight waves: few rows spread over the machine, and
    // run one head's code only (one row of 32 heads: 3.6 us, 4.7 us with four heads to a lane)
    int heads = HEADS;
    while (heads > 1 && (((int64_t)j.T * ((j.H + heads - 1) / heads)) << j.lanes_sh) < 8192 * 64) heads /= 2;
    j.groups = (j.H + heads - 1) / heads;
    jobs.job[m] = j;
    jobs.first[m++] = (int32_t)blocks;
    static_assert(THREADS == 256, "the kernel's units of a workgroup: 256 >> lanes_sh");
    const int per = THREADS >> j.lanes_sh;
    blocks += ((int64_t)j.T * j.groups + per - 1) / per;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
  }
  jobs.n = m;
  jobs.first[m] = (int32_t)blocks;
  if (!m) return hipSuccess;
  if (f32)
    launch_some<true>(jobs, s);
  else
    launch_some<false>(jobs, s);
  return hipGetLastError();
}

hipError_t launch_read(ReadJob &j, hipStream_t s) {
  if (j.T <= 0 || j.H <= 0) return hipSuccess;
  j.lanes_sh = lanes_of(j.D);
  const int64_t per = (THREADS >> j.lanes_sh) * READS;
  const int64_t blocks = ((int64_t)j.T * j.H + per - 1) / per;
  const dim3 grid((unsigned)blocks), threads(THREADS);
  if (j.fmt == IDX_K_FP8_E4M3)
    hipLaunchKernelGGL(read_kernel<IDX_K_FP8_E4M3>, grid, threads, 0, s, j);
  else if (j.fmt == IDX_K_MXFP4)
    hipLaunchKernelGGL(read_kernel<IDX_K_MXFP4>, grid, threads, 0, s, j);
  else if (j.fmt == IDX_K_F32)
    hipLaunchKernelGGL(read_kernel<IDX_K_F32>, grid, threads, 0, s, j);
  else
    hipLaunchKernelGGL(read_kernel<IDX_K_BF16>, grid, threads, 0, s, j);
  return hipGetLastError();
}

hipError_t launch_slot_check(const int32_t *slot, int32_t T, int64_t rows, uint32_t *word, hipStream_t s) {
  if (T <= 0) return hipSuccess;
  hipLaunchKernelGGL(slot_check_kernel, dim3((unsigned)((T + THREADS - 1) / THREADS)), dim3(THREADS), 0, s, slot, T,
                     rows, word);
  return hipGetLastError();
}

}  // namespace idx
