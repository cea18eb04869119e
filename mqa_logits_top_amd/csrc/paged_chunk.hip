// Attention over a paged cache for requests of many rows: 64 rows (tokens x heads of one cache head) to a wave, four waves
// to a workgroup, which share tiles of 64 keys in LDS.
#include <cmath>
#include <type_traits>

#include "attn_dev.h"
#include "paged_dev.h"

namespace idx {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int KT = 64;        // keys of a tile
constexpr int WAVES = 4;
constexpr int M = 64 * WAVES; // rows of a workgroup
constexpr int KSTAGES = 4, VSTAGES = 3, IDS = 8;

template <bool BF16>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Over the two lanes that hold one row (l, l ^ 32).
__device__ __forceinline__ float pair_max(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

template <bool FP8, int D>
constexpr int chunk_lds() {
  return (KSTAGES + VSTAGES) * KT * (FP8 ? D : 2 * D) + WAVES * IDS * KT * 4 + (FP8 ? KSTAGES * WAVES * 256 : 0);
}

template <bool BF16, bool FP8, int D>
__global__ __launch_bounds__(64 * WAVES, D == 64 ? 2 : 1) void chunk_kernel(PagedArgs a) {
  constexpr bool PV_BF16 = BF16 || FP8;   // weights times E4M3 scales need bf16's range
  constexpr bool TWO = FP8 && !BF16;      // ... and, for fp16 results, two parts
  constexpr float LIFT = !PV_BF16 ? 7.f : 0.f;
  constexpr int RB = FP8 ? D : 2 * D;     // bytes of a cache row
  constexpr int CH = RB / 16;             // its 16-byte chunks
  constexpr int PER = 256 / RB;           // rows of 256 bytes of LDS
  constexpr int RPC = 64 / CH;            // rows of a copy
  constexpr int NI = 16 / RPC;            // copies of a wave's 16 rows of a tile
  constexpr int KS = D / 16;              // steps of the first product
  constexpr int DN = D / 32;              // tiles of the second product
  constexpr int NKL = FP8 ? KS / 2 : KS;  // loads of a K operand
  constexpr int NSTEP = 2 * NI + 1 + (FP8 ? 1 : 0);   // copies of a step
  constexpr int KV = KT * RB;
  constexpr int V_AT = KSTAGES * KV, IDS_AT = V_AT + VSTAGES * KV, SCALES_AT = IDS_AT + WAVES * IDS * KT * 4;
  extern __shared__ __attribute__((aligned(256))) uint8_t lds[];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int c = lane & 31, hl = lane >> 5;
  const uint32_t mu = (uint32_t)(a.Hkv * a.blocks);
  const uint32_t member = blockIdx.x % mu;
  const int kvh = (int)(member % (uint32_t)a.Hkv), hb = (int)(member / (uint32_t)a.Hkv);
  Item w;
  if (!find_item<KT, true, false>(a, blockIdx.x / mu, w)) return;
  const int head0 = kvh * a.G + hb * a.Gt, heads = min(a.Gt, a.G - hb * a.Gt);
  const KeyTiles kt = key_tiles<KT>(a, w.r, w.row0, a.R);
  const int v0 = (int)((int64_t)kt.count * w.split / w.splits), v1 = (int)((int64_t)kt.count * (w.split + 1) / w.splits);
  const int nv = v1 - v0;

  // this lane's rows
  int32_t pos[2], lb[2];      // last key a row sees; keys above lb, or below a.first, are in its window
  int64_t q_at[2];
  int32_t t[2], h[2];
  bool real[2];
  int32_t min_pos = INT32_MAX, max_lb = -1;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int row = wave * 64 + m * 32 + c, tok = row / a.Gt;
    h[m] = row - tok * a.Gt;
    real[m] = tok < a.R && h[m] < heads && w.row0 + tok < w.r.n;
    t[m] = w.r.from + w.row0 + tok;
    h[m] += head0;
    pos[m] = real[m] ? w.r.len - w.r.n + w.row0 + tok : -1;
    lb[m] = a.window && real[m] ? (int32_t)max((int64_t)pos[m] - a.window, (int64_t)-1) : -1;
    q_at[m] = (int64_t)t[m] * a.q_t + (int64_t)h[m] * a.q_h;
    if (real[m]) {
      min_pos = min(min_pos, pos[m]);
      max_lb = max(max_lb, lb[m]);
    }
  }
  min_pos = (int32_t)wave_min((uint32_t)min_pos ^ 0x80000000u) ^ 0x80000000u;
  max_lb = (int32_t)(wave_max((uint32_t)(max_lb + 1)) - 1u);
  const bool any_row = __any(real[0] || real[1]);

  // ---- copies
  const int32_t *table = a.pages + (int64_t)w.b * a.ld_pages;
  uint32_t *const ids = (uint32_t *)(lds + IDS_AT) + wave * IDS * KT;
  const uint32_t page_mask = (1u << a.page_sh) - 1u, rows = (uint32_t)a.rows, max_page = (rows - 1u) >> a.page_sh;
  const int32_t last_key = kt.hi - 1;
  auto key0 = [&](int v) {    // of the split's v-th tile; behind its last one, that one
    const int x = v0 + min(v, nv - 1);
    return x < kt.firsts ? x * KT : kt.base + (x - kt.firsts) * KT;
  };
  auto request_ids = [&](int v) {
    const int32_t key = min(key0(v) + lane, last_key);
    copy4((const float *)(table + (key >> a.page_sh)), lds_addr(ids + (v & (IDS - 1)) * KT));
  };
  // slot of a key, from its page's id; a page outside the cache gives slot 0 and does not count
  auto slot_of = [&](uint32_t id, int32_t key, bool &ok) -> uint32_t {
    const uint32_t s = (id << a.page_sh) + ((uint32_t)key & page_mask);
    ok = id <= max_page && s < rows;
    return ok ? s : 0u;
  };
  const int my_row = lane / CH;   // of a copy
  auto swizzle_k = [](int r) { return (r / PER) & (CH - 1); };
  auto swizzle_v = [](int r) {
    if constexpr (FP8) return D == 128 ? (((r >> 1) & 1) << 1) | (((r >> 3) & 1) << 2) : ((r >> 3) & 1) << 1;
    return D == 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2;
  };
  const uint8_t *kbase = a.k + (int64_t)RB * kvh, *vbase = a.v + (int64_t)RB * kvh;
  auto row_slot = [&](int v, int u) {
    const int r = 16 * wave + u * RPC + my_row;
    bool ok;
    return slot_of(ids[(v & (IDS - 1)) * KT + r], min(key0(v) + r, last_key), ok);
  };
  auto request_k = [&](int v, int stage, int u) {
    const int r = 16 * wave + u * RPC + my_row;
    copy16(kbase, (uint64_t)row_slot(v, u) * a.row_bytes + ((((lane & (CH - 1)) ^ swizzle_k(r))) << 4),
           lds_addr(lds + stage * KV + (16 * wave + u * RPC) * RB));
  };
  auto request_v = [&](int v, int stage, int u) {
    const int r = 16 * wave + u * RPC + my_row;
    copy16(vbase, (uint64_t)row_slot(v, u) * a.row_bytes + ((((lane & (CH - 1)) ^ swizzle_v(r))) << 4),
           lds_addr(lds + V_AT + stage * KV + (16 * wave + u * RPC) * RB));
  };
  // lanes 0 .. 15 bring the wave's keys' scales, 16 .. 31 their values', the others the same again
  auto request_scales = [&](int v) {
    if constexpr (FP8) {
      const int r = 16 * wave + (lane & 15);
      bool ok;
      const uint32_t s = slot_of(ids[(v & (IDS - 1)) * KT + r], min(key0(v) + r, last_key), ok);
      copy4((lane & 16 ? a.v_scale : a.k_scale) + (int64_t)s * a.scale_row + kvh,
            lds_addr(lds + SCALES_AT + ((v & (KSTAGES - 1)) * WAVES + wave) * 256));
    }
  };

  f32x16 o[2][DN];
  float ref[2] = {NEG_INF, NEG_INF}, sum[2] = {0.f, 0.f};
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int d = 0; d < DN; ++d) o[m][d] = f32x16{};

  if (nv > 0) {
#pragma unroll
    for (int i = 0; i < 5; ++i) request_ids(i);
    copies_left<0>();
    request_scales(0);
#pragma unroll
    for (int u = 0; u < NI; ++u) request_k(0, 0, u);
    request_scales(1);
#pragma unroll
    for (int u = 0; u < NI; ++u) request_k(1, 1, u);
#pragma unroll
    for (int u = 0; u < NI; ++u) request_v(0, 0, u);
    // as many as a step has
    request_scales(2);
#pragma unroll
    for (int u = 0; u < NI; ++u) request_k(2, 2, u);
#pragma unroll
    for (int u = 0; u < NI; ++u) request_v(1, 1, u);
    request_ids(4);
  }
  auto meet = [&] {   // all but the last step's copies are there, the other waves' too
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(NSTEP) : "memory");
  };
  int vs = 0;         // stage of V(j)
  if (!any_row) {
    // no row of its own: the wave's share of the copies only
    for (int j = 0; j < nv; ++j) {
      meet();
      const int vn = vs == 0 ? 2 : vs - 1;
      request_scales(j + 3);
      for (int u = 0; u < NI; ++u) request_k(j + 3, (j + 3) & (KSTAGES - 1), u);
      for (int u = 0; u < NI; ++u) request_v(j + 2, vn, u);
      request_ids(j + 5);
      vs = vs == 2 ? 0 : vs + 1;
    }
  } else if (nv > 0) {
    // Q^T as B operands: lane l holds row l % 32 and 8 dims of each 16
    u32x4 q[2][KS];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int e = FP8 ? 32 * (s >> 1) + 16 * hl + 8 * (s & 1) : 16 * s + 8 * hl;
        u32x4 x = {0u, 0u, 0u, 0u};
        if (real[m]) x = *(const u32x4 *)(a.q + q_at[m] + 2 * e);
        q[m][s] = (x & a.q_keep) ^ a.q_sign;
      }
    const uint32_t k_row = (uint32_t)(c * RB), k_sw = (uint32_t)swizzle_k(c);
    // V^T: lane 4 r + x of a group points to key r, dims 4 x (E4M3: lane 2 r + x, dims 8 x)
    const int g16 = lane & 15;
    const int vr = FP8 ? (g16 >> 1) : (g16 >> 2);
    const int vkey = FP8 ? (vr < 4 ? 4 * hl + vr : 4 + 4 * hl + vr) : 4 * hl + vr;   // of the 16 (FP8) or of each 8
    const uint32_t v_row = (uint32_t)(vkey * RB + 8 * (g16 & 1));
    const uint32_t v_ch = FP8 ? (uint32_t)((lane >> 4) & 1) : (uint32_t)(2 * ((lane >> 4) & 1) + ((g16 & 3) >> 1));
    const uint32_t v_sw = (uint32_t)swizzle_v(vkey);

    float sc[2] = {a.scale2, a.scale2}, nb[2] = {0.f, 0.f};
    bool big = false, masked = false;

    auto load_k = [&](const uint8_t *kp, int g) {
      return *(const u32x4 *)(kp + k_row + (((uint32_t)(2 * g + hl) ^ k_sw) << 4));
    };
    // scores of 32 keys: S^T = K Q^T
    f32x16 sa[2], sb[2];
    auto k_scales = [&](int v, int half, f32x16 *s) {
      if constexpr (FP8) {
        const float *p = (const float *)(lds + SCALES_AT + (v & (KSTAGES - 1)) * WAVES * 256);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = 32 * half + 8 * x + 4 * hl;
          const f32x4 f = *(const f32x4 *)(p + (key >> 4) * 64 + (key & 15));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[0][4 * x + j] *= f[j];
            s[1][4 * x + j] *= f[j];
          }
        }
      }
    };
    // which of the 32 keys from k0 on, half a tile, have a slot
    auto good_keys = [&](int v, int half) -> uint32_t {
      bool ok;
      const int r = 32 * half + c;
      slot_of(ids[(v & (IDS - 1)) * KT + r], min(key0(v) + r, last_key), ok);
      return (uint32_t)__ballot(ok);
    };
    auto mask = [&](int v, int half, f32x16 *s) -> bool {
      const int32_t k0 = key0(v) + 32 * half;
      const uint32_t good = good_keys(v, half);
      const bool whole = k0 + 31 <= min_pos && (k0 > max_lb || k0 + 31 < a.first) && good == ~0u;
      if (whole) return false;
      asm volatile("");   // stays a branch
      const uint32_t mine = good >> (4 * hl);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int off = 8 * (i / 4) + i % 4;
        const int32_t key = k0 + off + 4 * hl;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const bool sees = key <= pos[m] && (key > lb[m] || key < a.first) && ((mine >> off) & 1u);
          s[m][i] = sees ? s[m][i] : NEG_INF;
        }
      }
      return true;
    };
    auto settle = [&](f32x16 *s, const float *top) {
      // The reference moves only when a score is 2^8 above it (LIFT lower than the largest): see attn.hip
      if (__any(top[0] * a.scale2 > ref[0] + (8.f + LIFT) || top[1] * a.scale2 > ref[1] + (8.f + LIFT))) {
        bool far = false;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          // each row by its own scores, so that its bits do not depend on its neighbours'
          const float high = pair_max(top[m] * a.scale2);
          const float to = high > ref[m] + (8.f + LIFT) ? high - LIFT : ref[m];
          const float f = to == ref[m] ? 1.f : __builtin_amdgcn_exp2f(ref[m] - to);
          sum[m] *= f;
#pragma unroll
          for (int d = 0; d < DN; ++d) o[m][d] *= f;
          ref[m] = to;
          nb[m] = to == NEG_INF ? 0.f : -to;
          far |= __builtin_fabsf(to) >= BIG && to != NEG_INF;
        }
        big = __any(far);
      }
      if (big) {
        // The reference's own rounding passes the exponential's range: products are rounded like it, then it is taken off
        asm volatile("");
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const bool far = __builtin_fabsf(ref[m]) >= BIG && ref[m] != NEG_INF;
#pragma unroll
          for (int i = 0; i < 16; ++i) s[m][i] = far ? product(s[m][i], a.scale2) - ref[m] : s[m][i];
          sc[m] = far ? 1.f : a.scale2;
          nb[m] = far || ref[m] == NEG_INF ? 0.f : -ref[m];
        }
      }
    };
    auto first_max = [&](const f32x16 *s, float *top) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        top[m] = s[m][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top[m] = __builtin_fmaxf(top[m], s[m][i]);
      }
    };
    auto qk = [&](const uint8_t *kp, f32x16 *s) {
      s[0] = f32x16{};
      s[1] = f32x16{};
      static_for<NKL>([&](auto gc) {
        constexpr int g = decltype(gc)::value;
        const u32x4 x = load_k(kp, g);
        if constexpr (FP8) {
          const u32x4 lo = {codes2<BF16, false>(x.x), codes2<BF16, true>(x.x), codes2<BF16, false>(x.y),
                            codes2<BF16, true>(x.y)};
          const u32x4 hi = {codes2<BF16, false>(x.z), codes2<BF16, true>(x.z), codes2<BF16, false>(x.w),
                            codes2<BF16, true>(x.w)};
#pragma unroll
          for (int m = 0; m < 2; ++m) s[m] = mfma32<BF16>(lo, q[m][2 * g], s[m]);
#pragma unroll
          for (int m = 0; m < 2; ++m) s[m] = mfma32<BF16>(hi, q[m][2 * g + 1], s[m]);
        } else {
#pragma unroll
          for (int m = 0; m < 2; ++m) s[m] = mfma32<BF16>(x, q[m][g], s[m]);
        }
      });
    };
    // V^T of dims 32 d .. and the 16 keys from 16 u on
    auto load_v = [&](const uint8_t *vp, int u, int d) -> u32x4 {
      if constexpr (FP8) {
        const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2 *)(vp + 16 * u * RB + v_row + (((uint32_t)(2 * d) + v_ch) ^ v_sw) * 16));
        return u32x4{(uint32_t)x[0], (uint32_t)x[1], 0u, 0u};
      } else {
        u32x4 r;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const i32x2 x = __builtin_bit_cast(
              i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4 *)(
                         vp + (16 * u + 8 * e) * RB + v_row + (((uint32_t)(4 * d) + v_ch) ^ v_sw) * 16)));
          r[2 * e] = (uint32_t)x[0];
          r[2 * e + 1] = (uint32_t)x[1];
        }
        return r;
      }
    };
    auto weights = [&](int v, int half, f32x16 *s, u32x4 (*p)[2], u32x4 (*rest)[2]) {
      f32x4 vsc[4];
      if constexpr (FP8) {
        const float *f = (const float *)(lds + SCALES_AT + (v & (KSTAGES - 1)) * WAVES * 256) + 16;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = 32 * half + 8 * x + 4 * hl;
          vsc[x] = *(const f32x4 *)(f + (key >> 4) * 64 + (key & 15));
        }
        if (masked) {   // scales that are not finite reach the rows that see their keys through add_odd
          asm volatile("");
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) vsc[x][j] = vsc[x][j] - vsc[x][j] == 0.f ? vsc[x][j] : 0.f;
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[m][i], sc[m], nb[m]));
          float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[m][i + 1], sc[m], nb[m]));
          sum[m] += x + y;
          if constexpr (FP8) {
            x *= vsc[i / 4][i % 4];
            y *= vsc[i / 4][i % 4 + 1];
          }
          const uint32_t b = pack2<PV_BF16>(x, y);
          p[m][i / 8][i % 8 / 2] = b;
          if constexpr (TWO)
            rest[m][i / 8][i % 8 / 2] =
                pack2<true>(x - __uint_as_float(b << 16), y - __uint_as_float(b & 0xFFFF0000u));
        }
    };
    // Bits of a value that is not finite (E4M3: of a NaN, in the lowest byte).
    auto odd_value = [](uint32_t x) {
      constexpr uint32_t E = FP8 ? 0x7Fu : BF16 ? 0x7F80u : 0x7C00u;
      return (x & E) == E;
    };
    // Keys that not every row sees may hold values that are not finite, and weight 0 times those is NaN.  Returns the
    // keys of the 32 that hold one (a bit each, of the lane's own rows of the tile in LDS).
    auto odd_values = [&](int v, int half, const uint8_t *vp) -> uint32_t {
      bool odd = false;
#pragma unroll
      for (int x = 0; x < CH / 2; ++x) {   // lane: key lane % 32, half of its chunks
        const u32x4 z = *(const u32x4 *)(vp + c * RB + (hl * (CH / 2) + x) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int y = 0; y < 32; y += FP8 ? 8 : 16) odd |= odd_value(z[i] >> y);
      }
      if constexpr (FP8) {
        const int key = 32 * half + c;
        const uint32_t e = ((const uint32_t *)(lds + SCALES_AT + (v & (KSTAGES - 1)) * WAVES * 256))[(key >> 4) * 64 + 16 +
                                                                                                     (key & 15)];
        odd |= (e & 0x7F800000u) == 0x7F800000u;
      }
      const uint64_t m = __ballot(odd);
      return (uint32_t)m | (uint32_t)(m >> 32);
    };
    auto pv = [&](auto with_odd, const uint8_t *vp, u32x4 (*p)[2], u32x4 (*rest)[2]) {
      static_for<2 * DN>([&](auto gc) {
        constexpr int u = decltype(gc)::value / DN, d = decltype(gc)::value % DN;
        u32x4 x = load_v(vp, u, d);
        if constexpr (decltype(with_odd)::value) {   // without the values that are not finite
#pragma unroll
          for (int i = 0; i < (FP8 ? 2 : 4); ++i)
#pragma unroll
            for (int y = 0; y < 32; y += FP8 ? 8 : 16)
              if (odd_value((x[i] >> y) & 0xFFFFu)) x[i] &= ~((FP8 ? 0xFFu : 0xFFFFu) << y);
        }
        if constexpr (FP8)
          x = u32x4{codes2<true, false>(x.x), codes2<true, true>(x.x), codes2<true, false>(x.y), codes2<true, true>(x.y)};
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          o[m][d] = mfma32<PV_BF16>(x, p[m][u], o[m][d]);
          if constexpr (TWO) o[m][d] = mfma32<true>(x, rest[m][u], o[m][d]);
        }
      });
    };
    // The values left out, key by key, for the rows that see them: weights x values by the vector unit
    auto add_odd = [&](int v, int half, const uint8_t *vp, u32x4 (*p)[2], u32x4 (*rest)[2], uint32_t odd) {
      const int32_t k0 = key0(v) + 32 * half;
      const uint32_t good = good_keys(v, half);
      while (odd) {
        const int key = __builtin_ctz(odd);
        odd &= odd - 1;
        // the weight is the i-th of lane half own
        const int i = 4 * (key >> 3) + (key & 3), own = (key >> 2) & 1;
        const float vs1 = FP8 ? ((const float *)(lds + SCALES_AT + (v & (KSTAGES - 1)) * WAVES * 256))[((32 * half + key) >> 4) * 64 + 16 + (key & 15)] : 1.f;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t word = 0, less = 0;
#pragma unroll
          for (int z = 0; z < 8; ++z)
            if (z == (i >> 1)) {
              word = p[m][z / 4][z % 4];
              if constexpr (TWO) less = rest[m][z / 4][z % 4];
            }
          const uint32_t bits = (i & 1) ? word >> 16 : word & 0xFFFFu;
          float wgt = PV_BF16 ? __uint_as_float(bits << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
          if constexpr (TWO) wgt += __uint_as_float((i & 1) ? less & 0xFFFF0000u : less << 16);
          const uint32_t wu = __float_as_uint(wgt);
          const auto sw = __builtin_amdgcn_permlane32_swap(wu, wu, false, false);
          wgt = __uint_as_float(own ? sw[1] : sw[0]);
          const int32_t s = k0 + key;
          const bool sees = s <= pos[m] && (s > lb[m] || s < a.first) && ((good >> key) & 1u);
          if (FP8 && !(vs1 - vs1 == 0.f)) wgt = vs1;   // a scale that is not finite makes the whole row so
#pragma unroll
          for (int d = 0; d < DN; ++d)
#pragma unroll
            for (int z = 0; z < 16; ++z) {
              const int dim = 32 * d + 8 * (z / 4) + 4 * hl + z % 4;
              const int chunk = (dim * (FP8 ? 1 : 2) / 16) ^ swizzle_v(key);
              const uint8_t *at = vp + key * RB + chunk * 16 + (dim * (FP8 ? 1 : 2)) % 16;
              float val;
              bool left;
              if constexpr (FP8) {
                val = __builtin_amdgcn_cvt_f32_fp8((int)*at, 0);
                left = odd_value(*at) || !(vs1 - vs1 == 0.f);
              } else {
                const uint32_t x = *(const uint16_t *)at;
                val = BF16 ? __uint_as_float(x << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)x);
                left = odd_value(x);
              }
              if (sees && left) o[m][d][z] = __builtin_fmaf(wgt, val, o[m][d][z]);
            }
        }
      }
    };

    meet();
    qk(lds, sa);
    k_scales(0, 0, sa);
    masked = mask(0, 0, sa);
    {
      float top[2];
      first_max(sa, top);
      settle(sa, top);
    }
    for (int j = 0; j < nv; ++j) {
      if (j > 0) meet();
      const int vn = vs == 0 ? 2 : vs - 1;
      request_scales(j + 3);
#pragma unroll
      for (int u = 0; u < NI; ++u) request_k(j + 3, (j + 3) & (KSTAGES - 1), u);
#pragma unroll
      for (int u = 0; u < NI; ++u) request_v(j + 2, vn, u);
      request_ids(j + 5);
      const uint8_t *kp = lds + (j & (KSTAGES - 1)) * KV, *kn = lds + ((j + 1) & (KSTAGES - 1)) * KV, *vp = lds + V_AT + vs * KV;
      auto half = [&](auto hc, f32x16 *cur, f32x16 *nxt) {
        constexpr int hh = decltype(hc)::value;
        u32x4 p[2][2], rest[2][2];
        qk(hh == 0 ? kp + 32 * RB : kn, nxt);
        weights(j, hh, cur, p, rest);
        k_scales(j + hh, 1 - hh, nxt);
        uint32_t odd = 0;
        if (masked) odd = odd_values(j, hh, vp + hh * 32 * RB);
        const bool m2 = mask(j + hh, 1 - hh, nxt);
        if (odd) {
          asm volatile("");
          pv(std::true_type{}, vp + hh * 32 * RB, p, rest);
          add_odd(j, hh, vp + hh * 32 * RB, p, rest, odd);
        } else {
          pv(std::false_type{}, vp + hh * 32 * RB, p, rest);
        }
        masked = m2;
        float top[2];
        first_max(nxt, top);
        sc[0] = sc[1] = a.scale2;
        nb[0] = ref[0] == NEG_INF ? 0.f : -ref[0];
        nb[1] = ref[1] == NEG_INF ? 0.f : -ref[1];
        settle(nxt, top);
      };
      half(std::integral_constant<int, 0>{}, sa, sb);
      half(std::integral_constant<int, 1>{}, sb, sa);
      vs = vs == 2 ? 0 : vs + 1;
    }
  }
  copies_left<0>();   // none may write LDS that is another workgroup's by then

  // lane l holds row l % 32 and dims 32 d + 8 (z / 4) + 4 (l / 32) + z % 4
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float l = pair_sum(sum[m]);
    if (!real[m]) continue;
    if (w.splits > 1) {
      const int64_t item = (int64_t)(w.first_item + w.split * w.next) * mu + member;
      const int64_t at = item * M + wave * 64 + m * 32 + c;
      if (hl == 0) *(float2 *)(a.part_ml + 2 * at) = make_float2(ref[m], l);
#pragma unroll
      for (int d = 0; d < DN; ++d)
#pragma unroll
        for (int z = 0; z < 16; z += 4)
          *(f32x4 *)(a.part + at * D + 32 * d + 2 * z + 4 * hl) =
              f32x4{o[m][d][z], o[m][d][z + 1], o[m][d][z + 2], o[m][d][z + 3]};
    } else {
      const float f = finish(l);
      uint8_t *dst = a.out + (int64_t)t[m] * a.out_t + (int64_t)h[m] * a.out_h;
#pragma unroll
      for (int d = 0; d < DN; ++d)
#pragma unroll
        for (int z = 0; z < 16; z += 4)
          *(uint2 *)(dst + 2 * (32 * d + 2 * z + 4 * hl)) =
              make_uint2(pack2<BF16>(o[m][d][z] * f, o[m][d][z + 1] * f), pack2<BF16>(o[m][d][z + 2] * f, o[m][d][z + 3] * f));
      if (hl == 0 && a.lse) a.lse[(int64_t)t[m] * a.Hq + h[m]] = lse_of(ref[m], l);
    }
  }
}

template <bool BF16, bool FP8, int D>
hipError_t launch_one(const PagedArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((chunk_kernel<BF16, FP8, D>), dim3((unsigned)a.max_items), dim3(64 * WAVES), (chunk_lds<FP8, D>()), s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_paged_chunk(const PagedArgs &a, int32_t dtype, int32_t fmt, int32_t D, hipStream_t s) {
  const bool bf16 = dtype == IDX_K_BF16, fp8 = fmt == IDX_K_FP8_E4M3;
  if (D == 64)
    return bf16 ? (fp8 ? launch_one<true, true, 64>(a, s) : launch_one<true, false, 64>(a, s))
                : (fp8 ? launch_one<false, true, 64>(a, s) : launch_one<false, false, 64>(a, s));
  return bf16 ? (fp8 ? launch_one<true, true, 128>(a, s) : launch_one<true, false, 128>(a, s))
              : (fp8 ? launch_one<false, true, 128>(a, s) : launch_one<false, false, 128>(a, s));
}

}  // namespace idx
