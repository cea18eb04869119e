// Attention over a paged cache for requests of many rows: 64 rows (tokens x heads of one cache head) to a wave, four waves
// to a workgroup, which share tiles of 64 keys in LDS.
//
// One pass: S^T = K Q^T, weights exp2(scale2 S - ref) with a running reference, O^T += V^T P^T; transposed, so that a lane
// holds one row's scores and the weights are the second product's operands as they come out.  64 rows a wave, because every
// operand read from LDS then feeds two matrix instructions; four waves share a tile, so that a key comes from memory once
// for 256 rows; what the registers then hold (queries, two tiles' scores, outputs) leaves room for one wave a SIMD, two with
// 64 dims.  Among captured calls, joins included: 2048 rows of 32 heads on 8, 65536 keys, 128 dims, bf16: 2096 us, 1033
// TFLOP/s (a large library product: 1200); 1000 of 64 heads on to 30001 keys, E4M3, whose codes every wave converts for
// itself: 1723 us, 486.  What bounds it is one wave's issue, an instruction in 4 cycles, an exponential in 16: of the 4400
// cycles of a tile 60% are issue, 23% waits for results, 17% waits for LDS and the other waves; the matrix pipes are busy for
// 49%.  Moving the second product of 32 keys behind the first product of the next 64, so that weights lie beside both, gave 1%
// and cost E4M3 16%: not kept.
// An item takes about 12 us besides its tiles of 2 us each (latencies of lengths, pages and keys, 7; code that runs once).
#include <array>
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

#define INLINE __attribute__((always_inline))

template <bool BF16>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// c plus the sum of the lane's own four values, in every element: 16 products of 4 x 4 x 4, by ones.  (16-bit caches, whose
// outputs are divided by the sum of the weights as rounded (attn.hip).  2048 rows on 65536 keys: 2054 us, without that sum
// 2010, with it by pairs, v_dot2, 2171; with 64 dims 133, 127 and 142.)
template <bool BF16>
__device__ __forceinline__ f32x4 add_own(uint32_t lo, uint32_t hi, f32x4 c) {
  constexpr uint32_t ONES = BF16 ? 0x3F803F80u : 0x3C003C00u;
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  const u32x2 one = {ONES, ONES}, x = {lo, hi};
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(i16x4, one), __builtin_bit_cast(i16x4, x), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(f16x4, one), __builtin_bit_cast(f16x4, x), c, 0, 0, 0);
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

// RUNS (has_runs): the 16 keys of a tile that a wave brings follow each other in a cache, and their copies have one scalar
// address.
template <bool BF16, bool FP8, int D, bool RUNS>
__global__ __launch_bounds__(64 * WAVES, D == 64 ? 2 : 1) void chunk_kernel(PagedArgs a) {
  // E4M3: a key's scale enters its weight, which then needs bf16's range, and two parts of it, so that a value is not rounded
  // by its scale and again as a result.  (1000 rows of 64 heads on to 30001 keys: 1723 us, 1325 with one part.)
  constexpr bool PV_BF16 = BF16 || FP8;
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
  Item found;
  if (!find_item<KT, true, ITEM>(a, blockIdx.x / mu, found)) return;
  const Item w = uniform(found);
  const int head0 = kvh * a.G + hb * a.Gt, heads = min(a.Gt, a.G - hb * a.Gt);
  const KeyTiles kt = key_tiles<KT>(a, w.r, w.row0, a.R);
  const int v0 = (int)((int64_t)kt.count * w.split / w.splits), v1 = (int)((int64_t)kt.count * (w.split + 1) / w.splits);
  const int nv = v1 - v0;

  // this lane's rows: the m-th of them is row 64 wave + 32 m + l % 32 of the tile
  struct Row {
    int32_t t, h;             // token and query head
    bool real;
  };
  auto row_of = [&](int m) INLINE -> Row {
    const int row = wave * 64 + m * 32 + c, tok = row / a.Gt, h = row - tok * a.Gt;
    return {w.r.from + w.row0 + tok, head0 + h, tok < a.R && h < heads && w.row0 + tok < w.r.n};
  };
  int32_t pos[2], lb[2];      // last key a row sees; keys above lb, or below a.first, are in its window
  int32_t min_pos = INT32_MAX, max_lb = -1;
  bool some = false;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const Row r = row_of(m);
    pos[m] = r.real ? w.r.len - w.r.n + (r.t - w.r.from) : -1;
    lb[m] = a.window && r.real ? (int32_t)max((int64_t)pos[m] - a.window, (int64_t)-1) : -1;
    if (r.real) {
      min_pos = min(min_pos, pos[m]);
      max_lb = max(max_lb, lb[m]);
      some = true;
    }
  }
  min_pos = uniform((int32_t)(wave_min((uint32_t)min_pos ^ 0x80000000u) ^ 0x80000000u));
  max_lb = uniform((int32_t)(wave_max((uint32_t)(max_lb + 1)) - 1u));
  const bool any_row = __any(some);

  // ---- copies
  const int32_t *table = a.pages + (int64_t)w.b * a.ld_pages;
  uint32_t *const ids = (uint32_t *)(lds + IDS_AT) + wave * IDS * KT;
  const uint32_t page_mask = (1u << a.page_sh) - 1u, rows = (uint32_t)a.rows, max_page = (rows - 1u) >> a.page_sh;
  const int32_t last_key = kt.hi - 1;
  auto key0 = [&](int v) INLINE {    // of the split's v-th tile; behind its last one, that one
    const int x = v0 + min(v, nv - 1);
    return x < kt.firsts ? x * KT : kt.base + (x - kt.firsts) * KT;
  };
  auto request_ids = [&](int v) INLINE {
    const int32_t key = min(key0(v) + lane, last_key);
    copy4((const float *)(table + (key >> a.page_sh)), lds_addr(ids + (v & (IDS - 1)) * KT));
  };
  // slot of a key, from its page's id; a page outside the cache gives slot 0 and does not count
  auto slot_of = [&](uint32_t id, int32_t key, bool &ok) INLINE -> uint32_t {
    const uint32_t s = (id << a.page_sh) + ((uint32_t)key & page_mask);
    ok = id <= max_page && s < rows;
    return ok ? s : 0u;
  };
  const int my_row = lane / CH;   // of a copy
  auto swizzle_k = [](int r) INLINE { return (r / PER) & (CH - 1); };
  auto swizzle_v = [](int r) INLINE {
    if constexpr (FP8) return D == 128 ? (((r >> 1) & 1) << 1) | (((r >> 3) & 1) << 2) : ((r >> 3) & 1) << 1;
    return D == 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2;
  };
  const uint8_t *kbase = a.k + (int64_t)RB * kvh, *vbase = a.v + (int64_t)RB * kvh;
  // The wave's 16 rows of a tile: their slots, or with RUNS the byte offset of the first, the lanes' being a constant on.
  using Slots = std::conditional_t<RUNS, uint64_t, std::array<uint32_t, NI>>;
  auto slots_of = [&](int v) INLINE -> Slots {
    const uint32_t *p = ids + (v & (IDS - 1)) * KT + 16 * wave;
    const int32_t k0 = key0(v) + 16 * wave;
    bool ok;
    if constexpr (RUNS) {
      const uint32_t id = (uint32_t)__builtin_amdgcn_readfirstlane((int)p[0]);
      return (uint64_t)slot_of(id, min(k0, last_key) & ~15, ok) * a.row_bytes;
    } else {
      Slots s;
#pragma unroll
      for (int u = 0; u < NI; ++u) {
        const int r = u * RPC + my_row;
        s[u] = slot_of(p[r], min(k0 + r, last_key), ok);
      }
      return s;
    }
  };
  uint32_t k_off[NI], v_off[NI];   // of the lane's chunk: with RUNS also of its row
#pragma unroll
  for (int u = 0; u < NI; ++u) {
    const int r = u * RPC + my_row;
    k_off[u] = (uint32_t)(((lane & (CH - 1)) ^ swizzle_k(r)) << 4) + (RUNS ? (uint32_t)r * a.row_bytes : 0u);
    v_off[u] = (uint32_t)(((lane & (CH - 1)) ^ swizzle_v(r)) << 4) + (RUNS ? (uint32_t)r * a.row_bytes : 0u);
  }
  auto request = [&](const uint8_t *base, const Slots &s, uint32_t off, int u, uint32_t at) INLINE {
    if constexpr (RUNS) {
      copy16(uniform(base + s), off, at);
    } else {
      uint64_t x = (uint64_t)s[u] * a.row_bytes + off;
      asm volatile("" : "+v"(x));   // the base is added here; added to every offset before the loop it fills registers
      copy16(base, x, at);
    }
  };
  auto request_k = [&](int stage, const Slots &s, int u) INLINE {
    request(kbase, s, k_off[u], u, lds_addr(lds + stage * KV + (16 * wave + u * RPC) * RB));
  };
  auto request_v = [&](int stage, const Slots &s, int u) INLINE {
    request(vbase, s, v_off[u], u, lds_addr(lds + V_AT + stage * KV + (16 * wave + u * RPC) * RB));
  };
  // lanes 0 .. 15 bring the wave's keys' scales, 16 .. 31 their values', the others the same again
  auto request_scales = [&](int v) INLINE {
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
  f32x4 rounded[2] = {};   // 16-bit caches: the sum of the weights as rounded
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int d = 0; d < DN; ++d) o[m][d] = f32x16{};

  // Q^T as B operands: lane l holds row l % 32 and 8 dims of each 16
  u32x4 q[2][KS];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const Row r = row_of(m);
    const uint8_t *at = a.q + (r.real ? (int64_t)r.t * a.q_t + (int64_t)r.h * a.q_h : 0);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int e = FP8 ? 32 * (s >> 1) + 16 * hl + 8 * (s & 1) : 16 * s + 8 * hl;
      q[m][s] = *(const u32x4 *)(at + 2 * e);   // rows that are not there: any row's, masked and not stored
    }
  }

  Slots ks, vs;       // of K(j + 3) and V(j + 2) in step j
  if (nv > 0) {
#pragma unroll
    for (int i = 0; i < 6; ++i) request_ids(i);
    copies_left<0>();
    const Slots s0 = slots_of(0), s1 = slots_of(1);
    vs = slots_of(2);
    ks = slots_of(3);
    request_scales(0);
#pragma unroll
    for (int u = 0; u < NI; ++u) request_k(0, s0, u);
    request_scales(1);
#pragma unroll
    for (int u = 0; u < NI; ++u) request_k(1, s1, u);
#pragma unroll
    for (int u = 0; u < NI; ++u) request_v(0, s0, u);
    // as many as a step has
    request_scales(2);
#pragma unroll
    for (int u = 0; u < NI; ++u) request_k(2, vs, u);
#pragma unroll
    for (int u = 0; u < NI; ++u) request_v(1, s1, u);
    request_ids(5);
  }
  auto meet = [&]() INLINE {   // all but the last step's copies are there, the other waves' too
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(NSTEP) : "memory");
  };
  int vst = 0;        // stage of V(j)
  // Keys that not every row sees may hold values that are not finite, and weight 0 times those is NaN.  Before such a tile
  // (an edge) is used each wave takes them out of its rows of it in LDS; at the end the rows that see them get them.  Those
  // that no row sees (behind the last key, before the window, without a slot) may be any memory's, and cost no more.
  int32_t odd_lo = INT32_MAX, odd_hi = -1;   // tiles, from the first to the last, with some that a row sees
  const int32_t p0 = w.r.len - w.r.n + w.row0, p1 = last_key;   // the workgroup's first and last row
  const int32_t lb0 = a.window ? (int32_t)max((int64_t)p0 - a.window, (int64_t)-1) : -1;
  const int32_t lb1 = a.window ? (int32_t)max((int64_t)p1 - a.window, (int64_t)-1) : -1;
  auto edge = [&](int32_t k0, uint64_t good) INLINE {
    return !(k0 + KT - 1 <= p0 && (k0 > lb1 || k0 + KT - 1 < a.first) && good == ~0ull);
  };
  auto some_row_sees = [&](int32_t key, bool ok) INLINE { return ok && key <= p1 && (key > lb0 || key < a.first); };
  auto good_keys = [&](int v) INLINE -> uint64_t {   // keys of a tile that have a slot
    const uint32_t id = ids[(v & (IDS - 1)) * KT + lane];
    if constexpr (RUNS) return __ballot(id <= max_page);
    bool ok;
    slot_of(id, min(key0(v) + lane, last_key), ok);
    return __ballot(ok);
  };
  auto clean = [&](int v, int32_t k0, uint64_t good) INLINE {
    if (!edge(k0, good)) return;
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NSTEP) : "memory");   // its own rows are there
    bool odd = false;
#pragma unroll
    for (int i = 0; i < CH / 4; ++i) {
      u32x4 *const at = (u32x4 *)(lds + V_AT + vst * KV + 16 * wave * RB) + i * 64 + lane;
      u32x4 z = *at;
      bool here = false;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t bits;   // of the values that are not finite (E4M3: of NaNs)
        if constexpr (FP8) {
          bits = ((((z[x] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu;
        } else {
          constexpr uint32_t E = BF16 ? 0x7F80u : 0x7C00u;
          bits = ((z[x] & E) == E ? 0xFFFFu : 0u) | ((z[x] >> 16 & E) == E ? 0xFFFF0000u : 0u);
        }
        z[x] &= ~bits;
        here |= bits != 0u;
      }
      if (here) {
        *at = z;
        const int r = 16 * wave + i * RPC + my_row;
        odd |= some_row_sees(k0 + r, (good >> r) & 1u);
      }
    }
    if constexpr (FP8) {
      float *const at = (float *)(lds + SCALES_AT + ((v & (KSTAGES - 1)) * WAVES + wave) * 256) + 16 + (lane & 15);
      if (!finite(*at)) {
        *at = 0.f;
        const int r = 16 * wave + (lane & 15);
        odd |= some_row_sees(k0 + r, (good >> r) & 1u);
      }
    }
    if (__any(odd)) {
      odd_lo = min(odd_lo, v);
      odd_hi = v;
    }
    lds_done();
  };
  uint64_t good = 0;
  int32_t k0 = 0;
  if (nv > 0) {
    good = good_keys(0);
    k0 = key0(0);
    clean(0, k0, good);
  }
  if (!any_row) {
    // no row of its own: the wave's share of the copies only
    for (int j = 0; j < nv; ++j) {
      if (j > 0) {
        good = good_keys(j);
        clean(j, key0(j), good);
      }
      meet();
      request_scales(j + 3);
#pragma unroll
      for (int u = 0; u < NI; ++u) request_k((j + 3) & (KSTAGES - 1), ks, u);
#pragma unroll
      for (int u = 0; u < NI; ++u) request_v(vst == 0 ? 2 : vst - 1, vs, u);
      request_ids(j + 6);
      vs = ks;
      ks = slots_of(j + 4);
      vst = vst == 2 ? 0 : vst + 1;
    }
  } else if (nv > 0) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        q[m][s] = (q[m][s] & a.q_keep) ^ a.q_sign;
        // with 128 dims the queries' place is the accumulation registers, which the products read as well
        if constexpr (D == 128) asm volatile("" : "+a"(q[m][s]));
      }
    // LDS addresses of the lane's operands in the first tile.  A chunk's number enters by exclusive or, and so do the
    // swizzles: the next operand's address is one exclusive or with a constant away.
    const uint32_t k_lane = lds_addr(lds) + (uint32_t)(c * RB + ((hl ^ swizzle_k(c)) << 4));
    // V^T: lane 4 r + x of a group points to key r, dims 4 x (E4M3: lane 2 r + x, dims 8 x)
    const int g16 = lane & 15;
    const int vr = FP8 ? (g16 >> 1) : (g16 >> 2);
    const int vkey = FP8 ? (vr < 4 ? 4 * hl + vr : 4 + 4 * hl + vr) : 4 * hl + vr;   // of the 16 (FP8) or of each 8
    const int v_ch = FP8 ? (lane >> 4) & 1 : 2 * ((lane >> 4) & 1) + ((g16 & 3) >> 1);
    const uint32_t v_lane =
        lds_addr(lds) + (uint32_t)(V_AT + vkey * RB + 8 * (g16 & 1) + ((v_ch ^ swizzle_v(vkey)) << 4));

    float nb[2] = {0.f, 0.f};   // -ref, or 0 while there is none
    bool big = false;

    typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
    // K of 16 dims (E4M3: 32) from 16 g (32 g) on; at: k_lane in the tile and half
    auto load_k = [&](uint32_t at, int g) INLINE { return *(lds_u32x4 *)(uintptr_t)(at ^ (uint32_t)(32 * g)); };
    // scores of 32 keys: S^T = K Q^T
    f32x16 sa[2], sb[2];
    auto scales_at = [&](int v, int half, int x, int value) INLINE {   // of keys 32 half + 8 x + 4 (l / 32) .. + 3
      const float *p = (const float *)(lds + SCALES_AT + (v & (KSTAGES - 1)) * WAVES * 256) + 16 * value;
      const int key = 32 * half + 8 * x + 4 * hl;
      return *(const f32x4 *)(p + (key >> 4) * 64 + (key & 15));
    };
    // 32 keys from k0 on: every row sees them all if k0 is one of these, and the slots are good
    const uint32_t whole0 = min_pos - 31 > max_lb ? (uint32_t)max_lb + 1u : ~0u;
    const uint32_t whole_span = min_pos - 31 > max_lb ? (uint32_t)(min_pos - 31 - max_lb - 1) : 0u;
    auto mask = [&](int32_t k0, uint32_t good, f32x16 *s) INLINE -> bool {
      if ((uint32_t)k0 - whole0 <= whole_span && good == ~0u) return false;
      asm volatile("");   // stays a branch
      // a bit for each key that the row sees
      auto below = [&](int32_t key) INLINE -> uint32_t {   // of the 32 keys from k0 on
        return key <= k0 ? 0u : key - k0 >= 32 ? ~0u : (1u << (key - k0)) - 1u;
      };
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t sees = (below(pos[m] + 1) & (~below(lb[m] + 1) | below(a.first)) & good) >> (4 * hl);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t keep = (uint32_t)((int32_t)(sees << (31 - (8 * (i / 4) + i % 4))) >> 31);
          s[m][i] = __uint_as_float((__float_as_uint(s[m][i]) & keep) | (0xFF800000u & ~keep));
        }
      }
      return true;
    };
    // The reference moves only when a score is 2^8 above it (LIFT lower than the largest): the accumulators are rescaled
    // a few times a row instead of at most tiles.  Each row by its own scores, so that its bits do not depend on its
    // neighbours'.
    float high[2] = {NEG_INF, NEG_INF};   // scores, before their scale, from which on it moves
    auto settle = [&](f32x16 *s, const float *top) INLINE {
      if (__any(top[0] > high[0] || top[1] > high[1])) {
        bool far = false;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float both = pair_max(top[m]);
          const float to = both > high[m] ? __builtin_fmaxf(ref[m], product(both, a.scale2) - LIFT) : ref[m];
          const float f = to == ref[m] ? 1.f : __builtin_amdgcn_exp2f(ref[m] - to);
          sum[m] *= f;
          rounded[m] *= f;
#pragma unroll
          for (int d = 0; d < DN; ++d) o[m][d] *= f;
          ref[m] = to;
          const bool rounds = __builtin_fabsf(to) >= BIG && to != NEG_INF;   // then every tile is looked at
          high[m] = rounds ? NEG_INF : (to + (8.f + LIFT)) / a.scale2;
          nb[m] = to == NEG_INF ? 0.f : -to;
          far |= rounds;
        }
        big = __any(far);
      }
      if (big) {
        // The reference's own rounding passes the exponential's range: products are rounded like it, then it is taken off.
        // (What is left is small where it matters, and comes back through the scale within 2^-22 of itself.)
        asm volatile("");
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const bool far = __builtin_fabsf(ref[m]) >= BIG && ref[m] != NEG_INF;
#pragma unroll
          for (int i = 0; i < 16; ++i) s[m][i] = far ? (product(s[m][i], a.scale2) - ref[m]) / a.scale2 : s[m][i];
          nb[m] = far || ref[m] == NEG_INF ? 0.f : -ref[m];
        }
      }
    };
    auto first_max = [&](const f32x16 *s, float *top) INLINE {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        top[m] = s[m][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top[m] = __builtin_fmaxf(top[m], s[m][i]);
      }
    };
    // One load's share of S^T += K Q^T
    auto qk = [&](auto gc, u32x4 x, f32x16 *s) INLINE {
      constexpr int g = decltype(gc)::value;
      if constexpr (g == 0) s[0] = s[1] = f32x16{};
      if constexpr (FP8) {
        const u32x4 lo = {codes2<BF16, false>(x.x), codes2<BF16, true>(x.x), codes2<BF16, false>(x.y), codes2<BF16, true>(x.y)};
        const u32x4 hi = {codes2<BF16, false>(x.z), codes2<BF16, true>(x.z), codes2<BF16, false>(x.w), codes2<BF16, true>(x.w)};
#pragma unroll
        for (int m = 0; m < 2; ++m) s[m] = mfma32<BF16>(lo, q[m][2 * g], s[m]);
#pragma unroll
        for (int m = 0; m < 2; ++m) s[m] = mfma32<BF16>(hi, q[m][2 * g + 1], s[m]);
      } else {
#pragma unroll
        for (int m = 0; m < 2; ++m) s[m] = mfma32<BF16>(x, q[m][g], s[m]);
      }
    };
    // V^T of dims 32 d .. and the 16 keys from 16 u on; at: v_lane in the tile and half
    auto load_v = [&](uint32_t at, int u, int d) INLINE -> u32x4 {
      if constexpr (FP8) {
        const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2 *)(uintptr_t)((at ^ (uint32_t)(32 * d)) + 16 * u * RB));
        return u32x4{(uint32_t)x[0], (uint32_t)x[1], 0u, 0u};
      } else {
        u32x4 r;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const i32x2 x = __builtin_bit_cast(
              i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4 *)(uintptr_t)(
                         (at ^ (uint32_t)(64 * d)) + (16 * u + 8 * e) * RB)));
          r[2 * e] = (uint32_t)x[0];
          r[2 * e + 1] = (uint32_t)x[1];
        }
        return r;
      }
    };
    u32x4 p[2][2], rest[2][2];   // weights of 16 keys each, and their second parts
    f32x4 vsc;   // E4M3: scales of the values of four keys
    // Weights of two keys, the n-th pair of the 16: keys in the order of the second product's steps
    auto weigh = [&](int n, const f32x16 *s, int v, int half) INLINE {
      const int m = n & 1, i = n >> 1 << 1;
      if constexpr (FP8) {
        if (n % 4 == 0) vsc = scales_at(v, half, i / 4, 1);
      }
      float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[m][i], a.scale2, nb[m]));
      float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[m][i + 1], a.scale2, nb[m]));
      sum[m] += x;
      sum[m] += y;
      if constexpr (FP8) {
        x *= vsc[i % 4];
        y *= vsc[i % 4 + 1];
      }
      uint32_t b = pack2<PV_BF16>(x, y);
      if constexpr (FP8) {
        uint32_t r = pack2<true>(x - __uint_as_float(b << 16), y - __uint_as_float(b & 0xFFFF0000u));
        asm volatile("" : "+v"(r));
        rest[m][i / 8][i % 8 / 2] = r;
      }
      asm volatile("" : "+v"(b));   // here, not where it is used
      p[m][i / 8][i % 8 / 2] = b;
      if constexpr (!FP8) {
        if (i % 4 == 2) rounded[m] = add_own<BF16>(p[m][i / 8][i % 8 / 2 - 1], b, rounded[m]);
      }
    };
    // One load's share of O^T += V^T P^T
    auto pv = [&](auto gc, u32x4 x) INLINE {
      constexpr int u = decltype(gc)::value / DN, d = decltype(gc)::value % DN;
      if constexpr (FP8)
        x = u32x4{codes2<true, false>(x.x), codes2<true, true>(x.x), codes2<true, false>(x.y), codes2<true, true>(x.y)};
#pragma unroll
      for (int m = 0; m < 2; ++m) o[m][d] = mfma32<PV_BF16>(x, p[m][u], o[m][d]);
      if constexpr (FP8) {
#pragma unroll
        for (int m = 0; m < 2; ++m) o[m][d] = mfma32<true>(x, rest[m][u], o[m][d]);
      }
    };
    meet();
    static_for<NKL>([&](auto g) INLINE { qk(g, load_k(k_lane, decltype(g)::value), sa); });
    float top[2];
    if constexpr (FP8)
      for (int x = 0; x < 4; ++x) {
        const f32x4 f = scales_at(0, 0, x, 0);
        for (int i = 0; i < 4; ++i) {
          sa[0][4 * x + i] *= f[i];
          sa[1][4 * x + i] *= f[i];
        }
      }
    first_max(sa, top);
    // Operands are read two products ahead
    u32x4 kf[2] = {load_k(k_lane + 32 * RB, 0), load_k(k_lane + 32 * RB, 1)}, vf[2];
    for (int j = 0; j < nv; ++j) {
      if (j > 0) {
        clean(j, k0, good);
        meet();
      }
      const uint32_t kp = k_lane + (uint32_t)((j & (KSTAGES - 1)) * KV), kn = k_lane + (uint32_t)(((j + 1) & (KSTAGES - 1)) * KV);
      const uint32_t vp = v_lane + (uint32_t)(vst * KV);
      // 32 keys: their weights and second product, beside the first product of the next 32
      auto half = [&](auto hc, f32x16 *cur, f32x16 *nxt) INLINE {
        constexpr int hh = decltype(hc)::value;
        constexpr int NB = 2 * DN;
        const uint32_t kc = hh == 0 ? kp + 32 * RB : kn, kd = hh == 0 ? kn : kn + 32 * RB, vc = vp + hh * 32 * RB;
        auto copies = [&](auto gc) INLINE {   // one load's share of the step's
          constexpr int g = decltype(gc)::value;
          if constexpr (hh == 0) {
            if constexpr (g == 0) request_scales(j + 3);
            if constexpr (g % (NKL / NI) == 0) request_k((j + 3) & (KSTAGES - 1), ks, g / (NKL / NI));
          } else {
            if constexpr (g == 0) request_ids(j + 6);
            if constexpr (g % (NKL / NI) == 0) request_v(vst == 0 ? 2 : vst - 1, vs, g / (NKL / NI));
          }
        };
        auto scale_next = [&](int i) INLINE {
          if constexpr (FP8) {
            const float f = scales_at(j + hh, 1 - hh, i / 4, 0)[i % 4];
            nxt[0][i] *= f;
            nxt[1][i] *= f;
          }
        };
        auto first_product = [&](auto gc) INLINE {   // one load's share, and the next but one's operands
          constexpr int g = decltype(gc)::value;
          qk(gc, kf[g & 1], nxt);
          if constexpr (g + 2 < NKL)
            kf[g & 1] = load_k(kc, g + 2);
          else
            vf[g & 1] = load_v(vc, (g + 2 - NKL) / DN, (g + 2 - NKL) % DN);
          copies(gc);
        };
        // A few products ahead of what the weights wait for: the mask, the maximum against the reference
        constexpr int AHEAD = FP8 ? 0 : NKL >= 8 ? 2 : 1;
        static_for<AHEAD>([&](auto gc) INLINE { first_product(gc); });
        if (mask(k0 + 32 * hh, (uint32_t)(good >> (32 * hh)), cur)) first_max(cur, top);
        settle(cur, top);
        static_for<NKL - AHEAD>([&](auto xc) INLINE {
          constexpr int x = decltype(xc)::value, g = x + AHEAD, ON = NKL - AHEAD;
          first_product(std::integral_constant<int, g>{});
          static_for<(x + 1) * 16 / ON - x * 16 / ON>([&](auto n) INLINE { weigh(x * 16 / ON + decltype(n)::value, cur, j, hh); });
          if constexpr (!FP8 && hh == 1 && x == ON - 1) {
            vs = ks;
            ks = slots_of(j + 4);
            good = good_keys(j + 1);
            k0 = key0(j + 1);
          }
        });
        static_for<NB>([&](auto gc) INLINE {
          constexpr int g = decltype(gc)::value;
          pv(gc, vf[g & 1]);
          if constexpr (g + 2 < NB)
            vf[g & 1] = load_v(vc, (g + 2) / DN, (g + 2) % DN);
          else
            kf[g & 1] = load_k(kd, g + 2 - NB);
          static_for<16 / NB>([&](auto ic) INLINE {
            constexpr int i = g * (16 / NB) + decltype(ic)::value;
            scale_next(i);
#pragma unroll
            for (int m = 0; m < 2; ++m) top[m] = i == 0 ? nxt[m][0] : __builtin_fmaxf(top[m], nxt[m][i]);
          });
        });
        if constexpr (FP8 && hh == 1) {
            vs = ks;
            ks = slots_of(j + 4);
            good = good_keys(j + 1);
            k0 = key0(j + 1);
        }
      };
      half(std::integral_constant<int, 0>{}, sa, sb);
      half(std::integral_constant<int, 1>{}, sb, sa);
      vst = vst == 2 ? 0 : vst + 1;
    }
  }
  copies_left<0>();   // none may write LDS that is another workgroup's by then

  // whether any wave left some values out; and the others have read their last tile
  constexpr int OUT_CH = D / 8;   // 16-byte chunks of a row of out
  uint8_t *const mine = lds + wave * 64 * 2 * D;
  int32_t *const word = (int32_t *)(lds + M * 2 * D);
  static_assert(M * 2 * D + 8 * WAVES <= chunk_lds<FP8, D>(), "the output fits");
  if (nv > 0) {
    __syncthreads();
    if (lane == 0) {
      word[2 * wave] = odd_lo;
      word[2 * wave + 1] = odd_hi;
    }
    __syncthreads();
    for (int x = 0; x < WAVES; ++x) {
      odd_lo = min(odd_lo, uniform(word[2 * x]));
      odd_hi = max(odd_hi, uniform(word[2 * x + 1]));
    }
  }
  // lane l holds row l % 32 and dims 32 d + 8 (z / 4) + 4 (l / 32) + z % 4
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float l = pair_sum(sum[m]), div = FP8 ? l : pair_sum(rounded[m][0]);
    const Row r = row_of(m);
    if (!r.real) continue;
    if (w.splits > 1) {
      const int64_t at = (int64_t)blockIdx.x * M + wave * 64 + m * 32 + c;
      if (hl == 0) *(f32x4 *)(a.part_ml + 4 * at) = f32x4{ref[m], l, div, 0.f};
#pragma unroll
      for (int d = 0; d < DN; ++d)
#pragma unroll
        for (int z = 0; z < 16; z += 4)
          *(f32x4 *)(a.part + at * D + 32 * d + 2 * z + 4 * hl) =
              f32x4{o[m][d][z], o[m][d][z + 1], o[m][d][z + 2], o[m][d][z + 3]};
    } else {
      const float f = finish(div);
#pragma unroll
      for (int d = 0; d < DN; ++d)
#pragma unroll
        for (int z = 0; z < 16; z += 4)
          *(uint2 *)(mine + (m * 32 + c) * 2 * D + (((4 * d + z / 4) ^ (c & (OUT_CH - 1))) << 4) + 8 * hl) =
              make_uint2(pack2<BF16>(o[m][d][z] * f, o[m][d][z + 1] * f), pack2<BF16>(o[m][d][z + 2] * f, o[m][d][z + 3] * f));
      if (hl == 0 && a.lse) a.lse[(int64_t)r.t * a.Hq + r.h] = lse_of(ref[m], l);
    }
  }
  if (w.splits == 1) {   // through LDS, so that whole rows are stored at a time
    wave_sync();
    for (int i = 0; i < OUT_CH; ++i) {
      const int x = i * (64 / OUT_CH) + lane / OUT_CH, ch = lane & (OUT_CH - 1);
      const int row = wave * 64 + x, tok = row / a.Gt, h = row - tok * a.Gt;
      if (tok < a.R && h < heads && w.row0 + tok < w.r.n)
        *(u32x4 *)(a.out + (int64_t)(w.r.from + w.row0 + tok) * a.out_t + (int64_t)(head0 + h) * a.out_h + 16 * ch) =
            *(const u32x4 *)(mine + x * 2 * D + ((ch ^ (x & (OUT_CH - 1))) << 4));
    }
  }
  if (odd_hi >= 0) {
    asm volatile("");   // stays a branch
    __threadfence();    // the outputs are other lanes'
    constexpr int E = D / 64;
    for (int j = odd_lo; j <= odd_hi; ++j) {
      const int32_t k0 = key0(j), mine = min(k0 + lane, last_key);
      bool ok;
      const uint32_t slot0 = slot_of((uint32_t)table[mine >> a.page_sh], mine, ok);
      const uint64_t have = __ballot(ok);
      if (!edge(k0, have)) continue;   // none was taken out
      for (int i = 0; i < KT; ++i) {
        const int32_t key = k0 + i;
        if (!some_row_sees(key, (have >> i) & 1u)) continue;
        const uint32_t slot = (uint32_t)__builtin_amdgcn_readlane((int)slot0, i);
        // by the code and the scale, as they were taken out: a product past fp32's range has been counted with its weight
        float scale = 1.f, val[E];
        bool odd[E], some_odd = false;
        if constexpr (FP8) scale = a.v_scale[(int64_t)slot * a.scale_row + kvh];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint8_t *at = vbase + (uint64_t)slot * a.row_bytes + (lane * E + e) * (FP8 ? 1 : 2);
          if constexpr (FP8) {
            val[e] = __builtin_amdgcn_cvt_f32_fp8((int)*at, 0) * scale;
            odd[e] = (*at & 0x7Fu) == 0x7Fu || !finite(scale);
          } else {
            val[e] = BF16 ? __uint_as_float((uint32_t) * (const uint16_t *)at << 16) : (float)*(const _Float16 *)at;
            odd[e] = !finite(val[e]);
          }
          some_odd |= odd[e];
        }
        if (!__any(some_odd)) continue;
        for (int row = wave * 64; row < wave * 64 + 64; ++row) {
          const int tok = row / a.Gt, h = row - tok * a.Gt;
          if (tok >= a.R || h >= heads || w.row0 + tok >= w.r.n) continue;
          const int32_t p = w.r.len - w.r.n + w.row0 + tok;
          if (key > p || (a.window && (int64_t)key <= (int64_t)p - a.window && key >= a.first)) continue;
          const int64_t tq = w.r.from + w.row0 + tok;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (!odd[e]) continue;
            if (w.splits > 1) {
              float *to = a.part + ((int64_t)blockIdx.x * M + row) * D + lane * E + e;
              *to += val[e];
            } else {
              uint16_t *to = (uint16_t *)(a.out + tq * a.out_t + (int64_t)(head0 + h) * a.out_h) + lane * E + e;
              if constexpr (BF16)
                *to = __builtin_bit_cast(uint16_t, (__bf16)(__uint_as_float((uint32_t)*to << 16) + val[e]));
              else
                *to = __builtin_bit_cast(uint16_t, (_Float16)((float)__builtin_bit_cast(_Float16, *to) + val[e]));
            }
          }
        }
      }
    }
  }
}

template <bool BF16, bool FP8, int D>
hipError_t launch_one(const PagedArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)a.max_items), block(64 * WAVES);
  constexpr int lds = chunk_lds<FP8, D>();
  if (has_runs(a))
    hipLaunchKernelGGL((chunk_kernel<BF16, FP8, D, true>), grid, block, lds, s, a);
  else
    hipLaunchKernelGGL((chunk_kernel<BF16, FP8, D, false>), grid, block, lds, s, a);
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
