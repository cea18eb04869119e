// Attention over a paged cache for requests of one or a few rows: 16 or 32 rows (tokens x heads of one cache head) to a
// workgroup, whose four waves divide the keys, 32 at a time, without a barrier until their parts are done.
//
// The same pass as paged_chunk.hip's, on 16-row tiles: few rows read every key for little work, so that memory bounds it and
// waves that never wait for each other keep the most requests under way.  Medians of traced launches: 64 rows of 32 heads on
// 8 of 4100 keys each, bf16: 189 us, 5.7 TB/s (a large copy: 4.8 read and written); 32 of 1700 to 16384, E4M3, pages of 16:
// 130 us, 4.8 TB/s, and the join, 6.  One row on 4000 keys: 7.2 us of latencies (lengths, pages, keys, the waves' join), and
// 4.6 for the join.
#include <array>
#include <cmath>
#include <type_traits>

#include "attn_dev.h"
#include "paged_dev.h"

namespace idx {
namespace {

constexpr int KT = 32;        // keys of a tile
constexpr int WAVES = 4;
constexpr int IDS = 4;

#define INLINE __attribute__((always_inline))

template <bool BF16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// x plus a pair's two values, rounded once.
template <bool BF16>
__device__ __forceinline__ float add_pair(float x, uint32_t pair) {
  if constexpr (BF16) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2, pair), v2{(__bf16)1.f, (__bf16)1.f}, x, false);
  } else {
    typedef _Float16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(v2, pair), v2{(_Float16)1.f, (_Float16)1.f}, x, false);
  }
}

// Over the four lanes that hold one row (l, l ^ 16, l ^ 32, l ^ 48).
template <class Op>
__device__ __forceinline__ float over_row(float x, Op op) {
  const uint32_t u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t w = __float_as_uint(op(__uint_as_float(a[0]), __uint_as_float(a[1])));
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return op(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// Bytes of LDS of a wave: K and V of a tile (the join's output afterwards), page ids, scales.
template <bool FP8, int D, int MT>
constexpr int step_wave_lds() {
  constexpr int kv = 2 * KT * (FP8 ? D : 2 * D), join = MT * 16 * D * 4;
  return (kv > join ? kv : join) + IDS * 256 + (FP8 ? 2 * 256 : 0);
}
template <bool FP8, int D, int MT>
constexpr int step_lds() {
  return WAVES * step_wave_lds<FP8, D, MT>() + WAVES * MT * 16 * 16;
}

// RUNS: has_runs.
template <bool BF16, bool FP8, int D, int MT, bool RUNS>
__global__ __launch_bounds__(64 * WAVES, FP8 && MT == 1 ? 3 : 2) void step_kernel(PagedArgs a) {
  // E4M3: a key's scale enters its weight, which then needs bf16's range, and two parts of it, so that a value is not rounded
  // by its scale and again as a result.  (32 rows on 1700 to 16384 keys: 142 us with one part or two.)
  constexpr bool PV_BF16 = BF16 || FP8;
  constexpr float LIFT = !PV_BF16 ? 7.f : 0.f;
  constexpr int M = 16 * MT;
  constexpr int RB = FP8 ? D : 2 * D, CH = RB / 16, PER = 256 / RB, RPC = 64 / CH;
  constexpr int NI = KT / RPC;            // copies of a tile's K or V
  constexpr int KS = D / 32;              // steps of the first product
  constexpr int DN = D / 16;              // tiles of the second product
  constexpr int NK = NI + (RUNS ? 0 : 1) + (FP8 ? 1 : 0);   // copies of a tile's K, scales and page ids
  constexpr int WAVE_LDS = step_wave_lds<FP8, D, MT>();
  constexpr int SCALES_AT = WAVE_LDS - (FP8 ? 2 * 256 : 0), IDS_AT = SCALES_AT - IDS * 256;
  extern __shared__ __attribute__((aligned(256))) uint8_t lds[];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int c = lane & 15, g = lane >> 4;
  uint8_t *const kbuf = lds + wave * WAVE_LDS, *const vbuf = kbuf + KT * RB;
  uint32_t *const ids = (uint32_t *)(kbuf + IDS_AT);
  const uint32_t mu = (uint32_t)(a.Hkv * a.blocks);
  // Workgroup b runs on XCD b % 8.  E4M3 rows of several cache heads share lines, their scales if nothing else: there all
  // heads of an item run on one XCD.
  uint32_t id = blockIdx.x / mu, member = blockIdx.x % mu;
  if (FP8 || a.blocks > 1) {   // PagedPlan::by_xcd
    const uint32_t local = blockIdx.x >> 3;
    id = local / mu * 8 + (blockIdx.x & 7u);
    member = local % mu;
  }
  Item found;
  if (!find_item<KT, false, ITEM>(a, id, found)) return;
  const Item w = uniform(found);
  const int kvh = (int)(member % (uint32_t)a.Hkv), hb = (int)(member / (uint32_t)a.Hkv);
  const int head0 = kvh * a.G + hb * a.Gt, heads = min(a.Gt, a.G - hb * a.Gt);
  const KeyTiles kt = key_tiles<KT>(a, w.r, w.row0, a.R);
  const int v0 = (int)((int64_t)kt.count * w.split / w.splits), v1 = (int)((int64_t)kt.count * (w.split + 1) / w.splits);
  const int nv = (v1 - v0 - wave + WAVES - 1) / WAVES;   // this wave's tiles: v0 + wave, and every fourth on

  int32_t pos[MT], lb[MT];    // last key a row sees; keys above lb, or below a.first, are in its window
  bool real[MT];
  int64_t q_at[MT];
  int32_t min_pos = INT32_MAX, max_lb = -1;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = m * 16 + c, tok = row / a.Gt, h = row - tok * a.Gt;
    real[m] = tok < a.R && h < heads && w.row0 + tok < w.r.n;
    pos[m] = real[m] ? w.r.len - w.r.n + w.row0 + tok : -1;
    lb[m] = a.window && real[m] ? (int32_t)max((int64_t)pos[m] - a.window, (int64_t)-1) : -1;
    q_at[m] = (int64_t)(w.r.from + w.row0 + tok) * a.q_t + (int64_t)(head0 + h) * a.q_h;
    if (real[m]) {
      min_pos = min(min_pos, pos[m]);
      max_lb = max(max_lb, lb[m]);
    }
  }
  const int32_t p0 = w.r.len - w.r.n + w.row0;   // keys above lb0, or below a.first, are in the first row's window
  const int32_t lb0 = a.window ? (int32_t)max((int64_t)p0 - a.window, (int64_t)-1) : -1;
  min_pos = uniform((int32_t)(wave_min((uint32_t)min_pos ^ 0x80000000u) ^ 0x80000000u));
  max_lb = uniform((int32_t)(wave_max((uint32_t)(max_lb + 1)) - 1u));
  const uint32_t whole0 = min_pos - 31 > max_lb ? (uint32_t)max_lb + 1u : ~0u;
  const uint32_t whole_span = min_pos - 31 > max_lb ? (uint32_t)(min_pos - 31 - max_lb - 1) : 0u;

  // ---- copies
  const int32_t *table = a.pages + (int64_t)w.b * a.ld_pages;
  const uint32_t page_mask = (1u << a.page_sh) - 1u, rows = (uint32_t)a.rows, max_page = (rows - 1u) >> a.page_sh;
  const int32_t last_key = kt.hi - 1;
  auto key0 = [&](int j) INLINE {    // of the wave's j-th tile; behind its last one, that one
    const int x = v0 + wave + WAVES * min(j, nv - 1);
    return x < kt.firsts ? x * KT : kt.base + (x - kt.firsts) * KT;
  };
  auto slot_of = [&](uint32_t page, int32_t key, bool &ok) INLINE -> uint32_t {
    const uint32_t s = (page << a.page_sh) + ((uint32_t)key & page_mask);
    ok = page <= max_page && s < rows;
    return ok ? s : 0u;
  };
  auto request_ids = [&](int j) INLINE {
    if constexpr (!RUNS) {
      const int32_t key = min(key0(j) + (lane & 31), last_key);
      copy4((const float *)(table + (key >> a.page_sh)), lds_addr(ids + (j & (IDS - 1)) * 64));
    }
  };
  // page of the run of 16 keys from k on, by a scalar load (the table is not written while the kernel runs)
  typedef __attribute__((address_space(4))) const uint32_t scalar_u32;
  auto page_of = [&](int32_t k) INLINE -> uint32_t {
    return *(scalar_u32 *)(uintptr_t)(table + uniform(min(k, last_key) >> a.page_sh));
  };
  const int my_row = lane / CH;   // of a copy
  auto swizzle_k = [](int r) INLINE { return (r / PER) & (CH - 1); };
  auto swizzle_v = [](int r) INLINE {
    if constexpr (FP8)
      return D == 128 ? ((r >> 1) & 3) | (((r >> 4) & 1) << 2) : ((r >> 2) & 1) | (((r >> 4) & 1) << 1);
    return D == 128 ? (r & 7) << 1 : ((r >> 1) & 3) << 1;
  };
  const uint8_t *kbase = a.k + (int64_t)RB * kvh, *vbase = a.v + (int64_t)RB * kvh;
  // slots of a tile's rows: with RUNS those of its two runs of 16, else of the lane's rows
  struct Slots {
    uint32_t s[RUNS ? 2 : NI];
  };
  uint32_t good = ~0u;            // keys of the tile whose K was requested last that have a slot
  auto slots_of = [&](int j) INLINE -> Slots {
    Slots x;
    const int32_t k0 = key0(j);
    bool ok;
    if constexpr (RUNS) {
      good = 0u;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        x.s[u] = slot_of(page_of(k0 + 16 * u), min(k0 + 16 * u, last_key) & ~15, ok);
        good |= ok ? 0xFFFFu << (16 * u) : 0u;
      }
    } else {
      const uint32_t *p = ids + (j & (IDS - 1)) * 64;
      slot_of(p[lane & 31], min(k0 + (lane & 31), last_key), ok);
      good = (uint32_t)__ballot(ok);
#pragma unroll
      for (int u = 0; u < NI; ++u) {
        const int r = u * RPC + my_row;
        x.s[u] = slot_of(p[r], min(k0 + r, last_key), ok);
      }
    }
    return x;
  };
  // offsets of the lane's chunks: with RUNS also of its row in the run, else one, from which the others are an exclusive or
  // away (a swizzle's bits are bits of the row's number)
  constexpr int NO = RUNS ? NI : 1;
  uint32_t k_off[NO], v_off[NO];
#pragma unroll
  for (int u = 0; u < NO; ++u) {
    const int r = u * RPC + my_row;
    k_off[u] = (uint32_t)(((lane & (CH - 1)) ^ swizzle_k(r)) << 4) + (RUNS ? (uint32_t)(r & 15) * a.row_bytes : 0u);
    v_off[u] = (uint32_t)(((lane & (CH - 1)) ^ swizzle_v(r)) << 4) + (RUNS ? (uint32_t)(r & 15) * a.row_bytes : 0u);
  }
  auto request = [&](const uint8_t *base, const Slots &x, const uint32_t *off, auto swizzle, uint8_t *to) INLINE {
#pragma unroll
    for (int u = 0; u < NI; ++u) {
      if constexpr (RUNS) {
        copy16(uniform(base + (uint64_t)x.s[u * RPC / 16] * a.row_bytes), off[u], lds_addr(to) + u * 1024);
      } else {
        uint64_t at = (uint64_t)x.s[u] * a.row_bytes + (off[0] ^ (uint32_t)(swizzle(u * RPC) << 4));
        asm volatile("" : "+v"(at));   // the base is added here; added to every offset before the loop it fills registers
        copy16(base, at, lds_addr(to) + u * 1024);
      }
    }
  };
  // lanes 0 .. 31 bring their key's scale, the others their value's
  auto request_scales = [&](int j, const Slots &x) INLINE {
    if constexpr (FP8) {
      uint32_t s;
      if constexpr (RUNS) {
        const uint32_t other = -(uint32_t)((lane >> 4) & 1);   // (a choice of the two would go through memory)
        s = (x.s[0] ^ ((x.s[0] ^ x.s[1]) & other)) + (uint32_t)(lane & 15);
      } else {
        bool ok;
        s = slot_of(ids[(j & (IDS - 1)) * 64 + (lane & 31)], min(key0(j) + (lane & 31), last_key), ok);
      }
      copy4((lane < 32 ? a.k_scale : a.v_scale) + (int64_t)s * a.scale_row + kvh,
            lds_addr(kbuf + SCALES_AT + (j & 1) * 256));
    }
  };

  f32x4 o[MT][DN];
  float ref[MT], sum[MT], high[MT];
  float rounded[MT];   // 16-bit caches: the sum of the weights as rounded, by which the output is divided (attn.hip); no time
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    ref[m] = high[m] = NEG_INF;
    sum[m] = rounded[m] = 0.f;
#pragma unroll
    for (int d = 0; d < DN; ++d) o[m][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  if (nv > 0) {
    request_ids(0);
    request_ids(1);
    if constexpr (!RUNS) copies_left<0>();
    Slots slots = slots_of(0);
    uint32_t good_now = good;
    request_scales(0, slots);
    request(kbase, slots, k_off, swizzle_k, kbuf);
    request(vbase, slots, v_off, swizzle_v, vbuf);
    // Q^T as B operands: lane l holds row l % 16 and the dims its K piece holds in that step
    u32x4 q[MT][KS];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int e = FP8 ? 16 * ((s >> 1) * 4 + g) + 8 * (s & 1) : 32 * s + 8 * g;
        u32x4 x = {0u, 0u, 0u, 0u};
        if (real[m]) x = *(const u32x4 *)(a.q + q_at[m] + 2 * e);
        q[m][s] = (x & a.q_keep) ^ a.q_sign;
      }
    const int vr = FP8 ? c >> 1 : c >> 2;
    const int vkey = FP8 ? (vr < 4 ? 4 * g + vr : 12 + 4 * g + vr) : 4 * g + vr;
    const uint32_t v_row = (uint32_t)(vkey * RB + 8 * (c & 1)), v_ch = FP8 ? 0u : (uint32_t)((c & 3) >> 1);
    const uint32_t v_sw = (uint32_t)swizzle_v(vkey);
    const uint32_t k_sw = (uint32_t)swizzle_k(c);
    auto odd_value = [](uint32_t x) INLINE {
      constexpr uint32_t E = FP8 ? 0x7Fu : BF16 ? 0x7F80u : 0x7C00u;
      return (x & E) == E;
    };

    for (int j = 0; j < nv; ++j) {
      copies_left<NI>();   // this tile's K, scales and the next one's page ids are there (its V followed)
      u32x4 kf[2][KS];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int s = 0; s < KS; s += FP8 ? 2 : 1) {
          kf[h][s] = *(const u32x4 *)(kbuf + (16 * h + c) * RB + (((uint32_t)((FP8 ? 2 : 4) * s + g) ^ k_sw) << 4));
        }
      f32x4 ksc[2], vsc[2];
      if constexpr (FP8) {
        const float *p = (const float *)(kbuf + SCALES_AT + (j & 1) * 256);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ksc[h] = *(const f32x4 *)(p + 16 * h + 4 * g);
          vsc[h] = *(const f32x4 *)(p + 32 + 16 * h + 4 * g);
        }
      }
      const int32_t k0 = key0(j);
      const Slots next = slots_of(j + 1);
      lds_done();
      // behind the last tile it is requested once more and not used: the waits count on it
      request_ids(j + 2);
      request_scales(j + 1, next);
      request(kbase, next, k_off, swizzle_k, kbuf);
      if constexpr (FP8) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int s = 0; s < KS; s += 2) {
            const u32x4 x = kf[h][s];
            kf[h][s] = u32x4{codes2<BF16, false>(x.x), codes2<BF16, true>(x.x), codes2<BF16, false>(x.y),
                             codes2<BF16, true>(x.y)};
            kf[h][s + 1] = u32x4{codes2<BF16, false>(x.z), codes2<BF16, true>(x.z), codes2<BF16, false>(x.w),
                                 codes2<BF16, true>(x.w)};
          }
      }
      f32x4 sc[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < KS; ++s) acc = mfma16<BF16>(kf[h][s], q[m][s], acc);
          sc[m][h] = FP8 ? acc * ksc[h] : acc;
        }
      // lane l: row l % 16, keys 16 h + 4 g + i
      const bool masked = (uint32_t)k0 - whole0 > whole_span || good_now != ~0u;
      if (masked) {
        asm volatile("");   // stays a branch
        const uint32_t mine = good_now >> (4 * g);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int32_t key = k0 + 16 * h + 4 * g + i;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const bool sees = (key <= pos[m]) & ((key > lb[m]) | (key < a.first)) & ((mine >> (16 * h + i)) & 1u);
              sc[m][h][i] = sees ? sc[m][h][i] : NEG_INF;
            }
            if constexpr (FP8) vsc[h][i] = finite(vsc[h][i]) ? vsc[h][i] : 0.f;   // back through add_odd
          }
      }
      u32x4 p[MT], rest[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float top = sc[m][0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, sc[m][i / 4][i % 4]);
        // The reference moves only when a score is 2^8 above it (LIFT lower than the largest), each row's by its own
        // scores; one that is far is looked at in every tile, and its products are rounded like it (attn.hip)
        bool far = false;
        if (__any(top > high[m])) {
          const float all = over_row(top, [](float x, float y) { return __builtin_fmaxf(x, y); });
          const float to = all > high[m] ? __builtin_fmaxf(ref[m], product(all, a.scale2) - LIFT) : ref[m];
          const float f = to == ref[m] ? 1.f : __builtin_amdgcn_exp2f(ref[m] - to);
          sum[m] *= f;
          rounded[m] *= f;
#pragma unroll
          for (int d = 0; d < DN; ++d) o[m][d] *= f;
          ref[m] = to;
          far = __builtin_fabsf(to) >= BIG && to != NEG_INF;
          high[m] = far ? NEG_INF : (to + (8.f + LIFT)) / a.scale2;
        }
        const float nb = ref[m] == NEG_INF ? 0.f : -ref[m];
        if (__any(far)) {
          asm volatile("");
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = sc[m][i / 4][i % 4];
            sc[m][i / 4][i % 4] = far ? product(x, a.scale2) + nb : __builtin_fmaf(x, a.scale2, nb);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) sc[m][i / 4][i % 4] = __builtin_fmaf(sc[m][i / 4][i % 4], a.scale2, nb);
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          float x = __builtin_amdgcn_exp2f(sc[m][i / 4][i % 4]), y = __builtin_amdgcn_exp2f(sc[m][i / 4][i % 4 + 1]);
          sum[m] += x + y;
          if constexpr (FP8) {
            x *= vsc[i / 4][i % 4];
            y *= vsc[i / 4][i % 4 + 1];
          }
          p[m][i / 2] = pack2<PV_BF16>(x, y);
          if constexpr (!FP8) rounded[m] = add_pair<BF16>(rounded[m], p[m][i / 2]);
          if constexpr (FP8)
            rest[m][i / 2] =
                pack2<true>(x - __uint_as_float(p[m][i / 2] << 16), y - __uint_as_float(p[m][i / 2] & 0xFFFF0000u));
        }
      }

      // V^T operands: keys 4 g .. 4 g + 3 of either 16, of dim 16 d + c
      copies_left<NK>();   // this tile's V is there (the next one's K followed)
      u32x4 vt[DN];
#pragma unroll
      for (int d = 0; d < DN; ++d) {
        if constexpr (FP8) {
          const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2 *)(
              vbuf + v_row + (((uint32_t)d ^ v_sw) << 4)));
          vt[d][0] = (uint32_t)x[0];
          vt[d][1] = (uint32_t)x[1];
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const i32x2 x = __builtin_bit_cast(
                i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4 *)(
                           vbuf + 16 * h * RB + v_row + ((((uint32_t)(2 * d) + v_ch) ^ v_sw) << 4))));
            vt[d][2 * h] = (uint32_t)x[0];
            vt[d][2 * h + 1] = (uint32_t)x[1];
          }
        }
      }
      lds_done();
      if (masked) {
        // Keys that not every row sees may hold values that are not finite, and weight 0 times those is NaN.  Those of keys
        // that no row sees (behind the last key, before the window, without a slot: any memory's) become zeros; others are
        // left out of the product, and added for the rows that see their keys.
        auto below = [&](int32_t key) INLINE -> uint32_t {   // of the 32 keys from k0 on
          return key <= k0 ? 0u : key - k0 >= 32 ? ~0u : (1u << (key - k0)) - 1u;
        };
        const uint32_t seen = below(last_key + 1) & (~below(lb0 + 1) | below(a.first)) & good_now;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < (FP8 ? 2 : 4); ++i) {
          const uint32_t bits = seen >> (4 * g) >> (FP8 ? 16 * i : 16 * (i >> 1) + 2 * (i & 1));
          uint32_t keep = 0;
#pragma unroll
          for (int y = 0; y < (FP8 ? 4 : 2); ++y) keep |= -((bits >> y) & 1u) & (FP8 ? 0xFFu << (8 * y) : 0xFFFFu << (16 * y));
#pragma unroll
          for (int d = 0; d < DN; ++d) vt[d][i] &= keep;
        }
#pragma unroll
        for (int d = 0; d < DN; ++d)
#pragma unroll
          for (int i = 0; i < (FP8 ? 2 : 4); ++i)
#pragma unroll
            for (int y = 0; y < 32; y += FP8 ? 8 : 16) odd |= odd_value(vt[d][i] >> y);
        const float *vs1 = (const float *)(kbuf + SCALES_AT + (j & 1) * 256) + 32;
        if constexpr (FP8) odd |= !finite(vs1[lane & 31]) && ((seen >> (lane & 31)) & 1u);
        if (__any(odd)) {
          asm volatile("");
#pragma unroll
          for (int d = 0; d < DN; ++d)
#pragma unroll
            for (int i = 0; i < (FP8 ? 2 : 4); ++i)
#pragma unroll
              for (int y = 0; y < 32; y += FP8 ? 8 : 16)
                if (odd_value(vt[d][i] >> y)) vt[d][i] &= ~((FP8 ? 0xFFu : 0xFFFFu) << y);
          for (int key = 0; key < KT; ++key) {
            if (!((seen >> key) & 1u)) continue;
            float scale = 1.f;
            if constexpr (FP8) scale = vs1[key];
            const bool bad_scale = !finite(scale);
            const int from = ((key >> 2) & 3) * 16 + c, i = 4 * (key >> 4) + (key & 3);   // lane and weight of the row
            const int32_t s = k0 + key;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              uint32_t word = 0, less = 0;
#pragma unroll
              for (int z = 0; z < 4; ++z)
                if (z == i >> 1) {
                  word = p[m][z];
                  if constexpr (FP8) less = rest[m][z];
                }
              word = (uint32_t)__shfl((int)word, from);
              const uint32_t bits = i & 1 ? word >> 16 : word & 0xFFFFu;
              float weight = PV_BF16 ? __uint_as_float(bits << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
              if constexpr (FP8) {
                less = (uint32_t)__shfl((int)less, from);
                weight += __uint_as_float(i & 1 ? less & 0xFFFF0000u : less << 16);
              }
              if (bad_scale) weight = scale;
              const bool sees = s <= pos[m] && (s > lb[m] || s < a.first) && ((good_now >> key) & 1u);
#pragma unroll
              for (int d = 0; d < DN; ++d)
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  const int at = (16 * d + 4 * g + z) * (FP8 ? 1 : 2);
                  const uint8_t *x = vbuf + key * RB + (((at >> 4) ^ swizzle_v(key)) << 4) + (at & 15);
                  float val;
                  bool left;
                  if constexpr (FP8) {
                    val = __builtin_amdgcn_cvt_f32_fp8((int)*x, 0);
                    left = odd_value(*x) || bad_scale;
                  } else {
                    const uint32_t u = *(const uint16_t *)x;
                    val = BF16 ? __uint_as_float(u << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)u);
                    left = odd_value(u);
                  }
                  if (sees && left) o[m][d][z] = __builtin_fmaf(weight, val, o[m][d][z]);
                }
            }
          }
          lds_done();
        }
      }
      request(vbase, next, v_off, swizzle_v, vbuf);
      good_now = good;
      if constexpr (FP8) {
#pragma unroll
        for (int d = 0; d < DN; ++d)
          vt[d] = u32x4{codes2<true, false>(vt[d][0]), codes2<true, true>(vt[d][0]), codes2<true, false>(vt[d][1]),
                        codes2<true, true>(vt[d][1])};
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int d = 0; d < DN; ++d) {
          o[m][d] = mfma16<PV_BF16>(vt[d], p[m], o[m][d]);
          if constexpr (FP8) o[m][d] = mfma16<true>(vt[d], rest[m], o[m][d]);
        }
    }
  }
  copies_left<0>();   // none may write LDS that holds something else by then

  // The waves' outputs, references and sums through LDS; quads of dims exchanged against bank conflicts
  constexpr int QUADS = D / 4;
  float *const ml = (float *)(lds + WAVES * WAVE_LDS);   // [waves][M][4]
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    auto plus = [](float x, float y) { return x + y; };
    const float l = over_row(sum[m], plus), div = FP8 ? l : over_row(rounded[m], plus);
    const int row = m * 16 + c;
#pragma unroll
    for (int d = 0; d < DN; ++d) *(f32x4 *)(kbuf + row * D * 4 + ((4 * d + g) ^ (c & 7)) * 16) = o[m][d];
    if (g == 0) *(f32x4 *)(ml + (wave * M + row) * 4) = f32x4{ref[m], l, div, 0.f};
  }
  __syncthreads();
  for (int x = threadIdx.x; x < M * QUADS; x += 64 * WAVES) {
    const int row = x / QUADS, y = x % QUADS, tok = row / a.Gt, h = row - tok * a.Gt;
    if (tok >= a.R || h >= heads || w.row0 + tok >= w.r.n) continue;
    float top = NEG_INF;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) top = __builtin_fmaxf(top, ml[(i * M + row) * 4]);
    const float base = top == NEG_INF ? 0.f : top;
    float total = 0.f, div = 0.f;
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      const f32x4 x = *(const f32x4 *)(ml + (i * M + row) * 4);
      const float f = __builtin_amdgcn_exp2f(x[0] - base);
      total += f * x[1];
      div += f * x[2];
      r += f * *(const f32x4 *)(lds + i * WAVE_LDS + row * D * 4 + (y ^ (row & 7)) * 16);
    }
    const int64_t t = w.r.from + w.row0 + tok, hq = head0 + h;
    if (w.splits > 1) {
      const int64_t at = ((int64_t)id * mu + member) * M + row;
      *(f32x4 *)(a.part + at * D + 4 * y) = r;
      if (y == 0) *(f32x4 *)(a.part_ml + 4 * at) = f32x4{top, total, div, 0.f};
    } else {
      r *= finish(div);
      *(uint2 *)(a.out + t * a.out_t + hq * a.out_h + 8 * y) =
          make_uint2(pack2<BF16>(r[0], r[1]), pack2<BF16>(r[2], r[3]));
      if (y == 0 && a.lse) a.lse[t * a.Hq + hq] = lse_of(top, total);
    }
  }
}

template <bool BF16, bool FP8, int D, int MT>
hipError_t launch_tiles(const PagedArgs &a, hipStream_t s) {
  constexpr int lds = step_lds<FP8, D, MT>();
  if (has_runs(a))
    hipLaunchKernelGGL((step_kernel<BF16, FP8, D, MT, true>), dim3((unsigned)a.grid), dim3(64 * WAVES), lds, s, a);
  else
    hipLaunchKernelGGL((step_kernel<BF16, FP8, D, MT, false>), dim3((unsigned)a.grid), dim3(64 * WAVES), lds, s, a);
  return hipGetLastError();
}
template <bool BF16, bool FP8>
hipError_t launch_dims(const PagedArgs &a, int D, int M, hipStream_t s) {
  if (D == 64) return M == 16 ? launch_tiles<BF16, FP8, 64, 1>(a, s) : launch_tiles<BF16, FP8, 64, 2>(a, s);
  return M == 16 ? launch_tiles<BF16, FP8, 128, 1>(a, s) : launch_tiles<BF16, FP8, 128, 2>(a, s);
}

}  // namespace

hipError_t launch_paged_step(const PagedArgs &a, int32_t dtype, int32_t fmt, int32_t D, int32_t M, hipStream_t s) {
  const bool bf16 = dtype == IDX_K_BF16, fp8 = fmt == IDX_K_FP8_E4M3;
  if (bf16) return fp8 ? launch_dims<true, true>(a, D, M, s) : launch_dims<true, false>(a, D, M, s);
  return fp8 ? launch_dims<false, true>(a, D, M, s) : launch_dims<false, false>(a, D, M, s);
}

}  // namespace idx
