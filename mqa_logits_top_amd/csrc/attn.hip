// Attention of each query row over the keys its list selects.
//
// A wave serves one row t, one cache head and 16 or 32 of its query heads, without a barrier until its part of the
// list is done.  The list's entries that count go, without gaps, to a queue in LDS; a step takes 32 of them:
//   S^T = K Q^T  (v_mfma 16x16x32, twice 16 keys): A = keys x 32 dims, lane l holds key l % 16 and 8 dims of
//     group g = l / 16; the result gives lane l head l % 16 and keys 4 g .. 4 g + 3 of the 16.
//   O^T += V^T P^T: B = P^T, lane l holds head l % 16 and 8 of the 32 keys.  The product sums over keys, so
//     their order is free: with positions 8 g + 4 h + j for the keys 4 g + j of the h-th 16, the two S^T
//     results, exponentiated, are the operand as they stand.  A = V^T comes transposed out of LDS.
// The softmax is the running one: a reference near the maximum, the sum, the unnormalised output.  The weights
// of the second product are rounded to 16 bits; the output is divided by the sum of the rounded ones (a product
// with ones), so that a row whose weight lies on few keys gains little error from it.  E4M3 caches put a key's
// scale into its weight, whose rounding has no such sum (one key's value would come out rounded twice): there weights
// are two parts of 8 bits, in every variant, so that a row's precision is the same whatever rows are beside it.  The
// second part takes 18% of the time of 32 heads a wave (2048 rows x 512 keys, 64 heads: 61 us without it), none of 16
// heads a wave (40 rows x 8 cache heads: 49.8 us, 49.6).
// Cache rows reach LDS by memory-to-LDS copies that each bring whole rows, K for the next step while this one
// multiplies, V while the next one's scores are computed.  Waves of the 2000 rows that are resident at once
// walk their ascending lists at the same pace, so each XCD's L2 meets a row's neighbours' keys soon after.
//
// What bounds it: every row gathers its own keys, so cache rows pass the L2 once for each query row and cache head,
// however few they are in memory.  D = 128, 2 waves a SIMD by registers.
//   2048 rows x 2048 of 65536 keys, 32 heads on one bf16 cache head: 100 us, 690 TFLOP/s (58 us at the rate of a
//     large product); 2.1 GB through the L2s at 21 TB/s, which reach 27 with nothing but such loads (80 us).
//   2048 rows x 512 of 102400, 64 heads, E4M3: 73 us, 470 TFLOP/s (29 us): vector instructions, nearly half of
//     them conversions of codes and of weights, and matrix instructions, a third of them for the weights' second part.
//   40 rows x 2048 of 4000 each, 32 heads on 8, E4M3, paged: 48 us, 3.6 TB/s (36 us): scattered 1 KB slots.
//   1023 rows x 96 blocks of 8 keys, 16 heads of 64 on 2, fp16: 22 us: 0.4 GB gathered at 18 TB/s.
//   1 row x 512 keys, 64 heads, bf16: 8.4 us, of which 3.6 are a launch and the rest three loads' latencies in turn
//     (list, rows, output) and the waves' join.
#include "attn.h"

#include <cmath>
#include <type_traits>

#include "attn_dev.h"
#include "common.h"

namespace idx {
namespace {

constexpr int TILE = 32;      // keys of a step
constexpr int CHUNK = 256;    // list entries resolved at a time
constexpr int QUEUE = 512;    // rows waiting: under two tiles when a chunk is added
constexpr int MAX_WAVES = 8;  // of a workgroup
constexpr int MAX_SPLITS = 256;
constexpr int64_t FROM_MEMORY = (int64_t)128 << 20;   // bytes: half of the last cache

template <bool BF16>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// The largest / the sum over the four lanes that hold one head (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float head_max(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float y = __builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t w = __float_as_uint(y);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __builtin_fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float head_sum(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float y = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const uint32_t w = __float_as_uint(y);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ float max8(const float *x) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __builtin_fmaxf(m, x[i]);
  return m;
}

// Bytes of LDS of a wave.
constexpr int wave_lds(bool fp8, int D, bool wide) {
  return 2 * TILE * (fp8 ? D : 2 * D) + 4 * QUEUE * (fp8 && !wide ? 2 : 1) + (fp8 ? 8 * TILE : 0);
}

// Waves a SIMD, asked for so that a register more does not cost one (E4M3, 128 dims, 600 rows x 4 cache heads: 63 us
// with three, 70 with two).  The registers do not quite allow them in some variants, which keep one to three in scratch
// memory while the tiles run: stored before their loop, loaded behind it.
constexpr int waves_a_simd(bool fp8, int D, int mt) {
  return (D == 64 ? 3 : 2) + (mt == 1 && (fp8 || D == 64) ? 1 : 0);
}

// BF16: q's type; FP8: E4M3 caches (else of q's type); MT: 16-head tiles.
// WIDE: caches past 2^32 bytes (64-bit offsets of rows instead of 32-bit ones beside a uniform base).
// MT = 1 may run several waves a workgroup, which divide the entries and join through LDS.
template <bool BF16, bool FP8, int D, int MT, bool WIDE>
__global__ __launch_bounds__(MT == 1 ? 64 * MAX_WAVES : 64, waves_a_simd(FP8, D, MT)) void attn_kernel(AttnArgs a) {
  constexpr bool PV_BF16 = BF16 || FP8;   // weights times E4M3 scales need bf16's range, and two parts for precision
  // Weights are exp2(score - reference), below 2^8 with the reference where it was when last moved.  In fp16 they lie
  // 2^7 higher, below 2^15 (of 2^16): those under its smallest normal number, which lose up to 2^-25 whatever their
  // size, are then 2^-21 of the largest and less instead of 2^-14, and long lists of small weights keep their sum.
  // No time: 1023 rows of 8-key blocks 23.6 us, 23.3 without it.
  constexpr float LIFT = !PV_BF16 ? 7.f : 0.f;
  constexpr uint32_t ONES = BF16 ? 0x3F803F80u : 0x3C003C00u;
  constexpr int KS = D / 32;              // steps of the first product
  constexpr int DN = D / 16;              // tiles of the second product
  constexpr int HEADS = MT * 16;
  constexpr int RB = FP8 ? D : 2 * D;     // bytes of a cache row
  constexpr int CH = RB / 16;             // its 16-byte chunks
  constexpr int NI = CH / 2;              // copies of a tile's K or V: 64 / CH rows each
  constexpr int PER = 16 / CH;            // rows a 16-lane group brings in one copy
  constexpr int NK = NI + (FP8 ? 1 : 0);  // copies of a tile's K and scales
  constexpr int OUT_CH = D / 8;           // 16-byte chunks of a row of out
  // a wave's LDS: K, V (the join's output afterwards), the queue, scales
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int V_AT = TILE * RB, QUEUE_AT = 2 * TILE * RB;
  constexpr int OFFSETS_AT = QUEUE_AT + (WIDE || FP8 ? 4 * QUEUE : 0), SCALES_AT = OFFSETS_AT + (WIDE ? 0 : 4 * QUEUE);
  constexpr int WAVE_LDS = SCALES_AT + (FP8 ? 8 * TILE : 0);
  static_assert(WAVE_LDS == wave_lds(FP8, D, WIDE), "the launch's LDS");
  static_assert(HEADS * D * (MT > 1 ? 2 : 4) <= 2 * TILE * RB, "the output fits K and V");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t *const kbuf = lds + wave * WAVE_LDS, *const vbuf = kbuf + V_AT;
  uint32_t *const queue = (uint32_t *)(kbuf + QUEUE_AT), *const offsets = (uint32_t *)(kbuf + OFFSETS_AT);
  const float *const scales = (const float *)(kbuf + SCALES_AT);
  using Off = std::conditional_t<WIDE, uint64_t, uint32_t>;

  const int lane = threadIdx.x & 63;
  const int c = lane & 15, g = lane >> 4;
  // Workgroup b runs on XCD b % 8.  Those that read the same lines share one: the head blocks of a row's part, and
  // for E4M3, whose rows of 64 bytes and scales share lines, its cache heads too (40 rows x 8 cache heads of 64
  // dims, 2048 keys: 28 us, 42 without).  Other cache heads keep XCDs of their own, whose L2 holds more rows then
  // (1023 rows x 2 cache heads of 64 dims: 22.8 us, 24.3 together).
  const uint32_t kvs = FP8 ? 1u : (uint32_t)a.Hkv, same = (uint32_t)(a.Hkv * a.blocks) / kvs;
  const uint32_t parts = (uint32_t)a.T * kvs * (uint32_t)a.splits, even = parts & ~7u;
  const bool last = blockIdx.x >= even * same;                 // one of the parts behind the last multiple of 8
  const uint32_t i = last ? blockIdx.x - even * same : blockIdx.x >> 3;
  uint32_t part_of = last ? even + i / same : i / same * 8 + (blockIdx.x & 7u);
  const uint32_t member = i % same;
  const int split = (int)(part_of % (uint32_t)a.splits);
  part_of /= (uint32_t)a.splits;
  const int t = (int)(part_of / kvs), hb = (int)(member % (uint32_t)a.blocks);
  const int kvh = FP8 ? (int)(member / (uint32_t)a.blocks) : (int)(part_of % kvs);
  const int64_t item = (((int64_t)t * a.Hkv + kvh) * a.blocks + hb) * a.splits + split;
  const int head0 = kvh * a.G + hb * HEADS;                    // first query head
  const int heads = min(HEADS, a.G - hb * HEADS);

  // ---- the list: this wave's entries, 256 at a time, through registers into the queue of cache rows
  const int32_t win0 = a.ks ? max(a.ks[t], 0) : 0, win1 = a.ke ? min(a.ke[t], a.L) : a.L;
  const int64_t entries = (int64_t)a.n_sel << a.pool_sh;
  const int part = split * a.waves + wave;
  const int64_t e_end = min(entries, (part + 1) * a.per);
  int64_t e_next = part * a.per;          // first entry whose id is not loaded
  const int32_t *list = a.sel + (int64_t)t * a.ld_sel;
  // Three chunks are under way: the one that fill() appends (row), whose slots are loading (row, once it
  // is appended), and the one behind it, whose ids are loading (id).  Nothing waits for a load just issued.
  int32_t id[4], row[4];
  auto load_ids = [&] {
#pragma unroll
    for (int r = 0; r < 4; ++r) id[r] = list[min(e_next + 64 * r + lane, e_end - 1) >> a.pool_sh];
    e_next += CHUNK;
  };
  auto load_rows = [&] {   // of the ids loaded last
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t e = e_next - CHUNK + 64 * r + lane;
      int64_t key = id[r];
      if (a.pool_sh) key = (key * (1 << a.pool_sh)) + win0 + (e & ((1 << a.pool_sh) - 1));
      const bool ok = e < e_end && id[r] >= 0 && key >= win0 && key < win1;
      row[r] = ok ? (int32_t)key : -1;
      if (a.table && ok) row[r] = a.table[key];
    }
  };
  int64_t e_left = e_end - e_next;        // entries not in the queue yet
  // the queue holds positions [head, tail): entries that count, in order, no gaps; head is the current
  // tile's first, a multiple of TILE
  uint32_t head = 0, tail = 0;
  // Makes the tile after the current one whole, if the list has that much left; behind the list's last
  // entry the last tile repeats it.
  auto fill = [&] {
    if (tail - head >= 2 * TILE || e_left <= 0) return;
    do {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool ok = row[r] >= 0 && row[r] < a.rows;
        const uint64_t m = __ballot(ok);
        if (ok) {
          const uint32_t at = (tail + (uint32_t)__popcll(m & lanemask_lt(lane))) & (QUEUE - 1);
          if constexpr (WIDE || FP8) queue[at] = (uint32_t)row[r];
          if constexpr (!WIDE) offsets[at] = (uint32_t)row[r] * a.row_bytes;
        }
        tail += (uint32_t)__popcll(m);
      }
      e_left -= CHUNK;
      if (e_left > 0) {
        load_rows();
        if (e_left > CHUNK) load_ids();
      }
    } while (tail - head < 2 * TILE && e_left > 0);
    wave_sync();
    if (e_left <= 0 && (tail & (TILE - 1))) {
      const uint32_t last = (tail - 1) & (QUEUE - 1), at = tail + (uint32_t)lane;
      if ((uint32_t)lane < (-tail & (TILE - 1))) {
        if constexpr (WIDE || FP8) queue[at & (QUEUE - 1)] = queue[last];
        if constexpr (!WIDE) offsets[at & (QUEUE - 1)] = offsets[last];
      }
      wave_sync();
    }
  };
  if (e_left > 0) {
    load_ids();
    load_rows();
    if (e_left > CHUNK) load_ids();
  }

  // Q^T as B operands: lane l holds head l % 16 and the dims its K piece holds in that step
  u32x4 q[MT][KS];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int e = FP8 ? 16 * ((s >> 1) * 4 + g) + 8 * (s & 1) : 8 * (4 * s + g);
      u32x4 w = {0u, 0u, 0u, 0u};
      if (m * 16 + c < heads)
        w = *(const u32x4 *)(a.q + (int64_t)t * a.q_t + (int64_t)(head0 + m * 16 + c) * a.q_h + 2 * e);
      q[m][s] = (w & a.q_keep) ^ a.q_sign;
    }

  f32x4 o[MT][DN], rounded[MT];           // rounded: sum of the weights as the second product has them
  float ref[MT], neg[MT], sum[MT];        // neg: -ref, or 0 while there is none
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    ref[m] = NEG_INF;
    neg[m] = 0.f;
    sum[m] = 0.f;
    rounded[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < DN; ++n) o[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const uint8_t *kbase = a.k + (int64_t)RB * kvh, *vbase = a.v + (int64_t)RB * kvh;
  const float *sbase = (lane < TILE ? a.k_scale : a.v_scale) + kvh;
  // Copy u brings position 8 g + e, e = PER u + c / CH, of the tile to LDS row u 4 PER + lane / CH, its chunks
  // exchanged (xor) so that lanes that read together meet different banks.  K: 16 lanes read one chunk of 16
  // rows, in passes that mix lanes 0-3, 12-15 of one group with 4-11 of the next.  V: a pass of 32 lanes reads
  // 32 bytes of 8 rows, or 16 bytes (E4M3) of 16.
  auto ldsrow = [](int g, int e) { return e / PER * 4 * PER + g * PER + e % PER; };
  auto swizzle_k = [](int g, int e) {
    return CH == 16 ? (g << 2) | (e & 3) : CH == 8 ? (g << 1) | ((e >> 1) & 1) : (g & 1) * 3;
  };
  auto swizzle_v = [](int g, int e) {
    if constexpr (FP8) return (e / PER << 1) | (g & 1);
    return ((CH == 16 ? e & 3 : (e >> 1) & 1) << 2) | ((g & 1) << 1) | (g >> 1);
  };
  Off off[8];                             // of the lane's 8 positions 8 g .. 8 g + 7
  uint32_t scale_row = 0;                 // E4M3: of position lane % 32

  auto copy_row = [&](int u) -> Off {
    Off b = off[PER * u];
    if constexpr (PER > 1) {
      const Off b1 = off[PER * u + 1];
      b = c / CH == 1 ? b1 : b;
    }
    if constexpr (PER > 2) {
      const Off b2 = off[PER * u + 2], b3 = off[PER * u + 3];
      b = c / CH == 2 ? b2 : c / CH == 3 ? b3 : b;
    }
    return b;
  };
  auto request_k = [&] {
#pragma unroll
    for (int u = 0; u < NI; ++u)
      copy16(kbase, (Off)(copy_row(u) + (((lane & (CH - 1)) ^ swizzle_k(g, PER * u + c / CH)) << 4)),
             lds_addr(kbuf) + u * 1024);
    // lanes 0 .. 31 bring their key's scale, the others their value's
    if constexpr (FP8) copy4(sbase + (int64_t)scale_row * a.scale_row, lds_addr(scales));
  };
  auto request_v = [&] {
#pragma unroll
    for (int u = 0; u < NI; ++u)
      copy16(vbase, (Off)(copy_row(u) + (((lane & (CH - 1)) ^ swizzle_v(g, PER * u + c / CH)) << 4)),
             lds_addr(vbuf) + u * 1024);
  };
  // addresses of the tile at queue position `at`; spread 0: of its first rows only, over and over
  auto next_tile = [&](uint32_t at, int spread) {
    at &= QUEUE - 1;
    const u32x4 lo = *(const u32x4 *)&(WIDE ? queue : offsets)[at + (8 * g & spread)];
    const u32x4 hi = *(const u32x4 *)&(WIDE ? queue : offsets)[at + (8 * g & spread) + 4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      off[i] = i < 4 ? lo[i & 3] : hi[i & 3];
      if constexpr (WIDE) off[i] *= a.row_bytes;
    }
    if constexpr (FP8) scale_row = queue[at + (lane & (TILE - 1) & spread)];
  };

  fill();
  bool more = tail != 0;
  if (more) {
    next_tile(0, -1);
    request_k();
    request_v();
  }
  for (; more; head += TILE) {
    copies_left<NI>();   // this tile's K is there (its V followed)
    fill();
    // the list's last tile may be partial; the others are whole
    const int n = (int)(tail - head);
    more = n > TILE;
    // K from LDS into operands, then the copy of the next tile's may start
    u32x4 kt[2][KS];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kg = c >> 2, ke = 4 * h + (c & 3);   // the position of key c of the h-th 16
      const uint8_t *p = kbuf + ldsrow(kg, ke) * RB;
#pragma unroll
      for (int s = 0; s < KS; s += FP8 ? 2 : 1)
        kt[h][s] = *(const u32x4 *)(p + ((((FP8 ? 2 : 4) * s + g) ^ swizzle_k(kg, ke)) << 4));
    }
    float ksc[8], vsc[8];
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ksc[i] = scales[8 * g + i];
        vsc[i] = scales[TILE + 8 * g + i];
      }
    }
    // behind the last tile its first rows are requested once more and not used: the waits count on it
    next_tile(more ? head + TILE : head, more ? -1 : 0);
    lds_done();
    request_k();
    if constexpr (FP8) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int s = 0; s < KS; s += 2) {
          const u32x4 w = kt[h][s];
          kt[h][s] = u32x4{codes2<BF16, false>(w.x), codes2<BF16, true>(w.x), codes2<BF16, false>(w.y),
                           codes2<BF16, true>(w.y)};
          kt[h][s + 1] = u32x4{codes2<BF16, false>(w.z), codes2<BF16, true>(w.z), codes2<BF16, false>(w.w),
                               codes2<BF16, true>(w.w)};
        }
    }

    float sc[MT][8];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) acc = mfma<BF16>(kt[h][s], q[m][s], acc);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * h + j;
          sc[m][i] = FP8 ? acc[j] * ksc[i] : acc[j];
        }
      }
    if (!more) {
      asm volatile("");   // stays a branch; the compiler would select in every tile
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * g + i >= n) sc[m][i] = NEG_INF;
    }
    u32x4 p[MT], rest[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float top = max8(sc[m]) * a.scale2;   // scale2 > 0: the largest product is the largest dot's
      // The reference (LIFT below the largest score) moves only when a score is 2^8 above that: the
      // accumulators are rescaled a few times a row instead of at most tiles.  The four lanes of a head
      // share their reference, so a lane's own scores decide whether there is anything to do.
      // A large reference itself is off by more than the exponential's range (by 2^7 from 2^31 on), so that one fma a
      // weight, exact in the product, would leave infinities or zeros: from BIG on, which is looked at in every
      // tile then, the products are rounded like the reference.
      bool big = false;
      if (__any(top > (__builtin_fabsf(ref[m]) < BIG ? ref[m] + (8.f + LIFT) : NEG_INF))) {
        const float to = __builtin_fmaxf(ref[m], head_max(top) - LIFT);
        big = __any(__builtin_fabsf(to) >= BIG);
        const float f = to == ref[m] ? 1.f : __builtin_amdgcn_exp2f(ref[m] - to);
        sum[m] *= f;
        rounded[m] *= f;
#pragma unroll
        for (int d = 0; d < DN; ++d) o[m][d] *= f;
        ref[m] = to;
        neg[m] = to == NEG_INF ? 0.f : -to;
      }
      if (big) {
        asm volatile("");   // stays a branch
#pragma unroll
        for (int i = 0; i < 8; ++i) sc[m][i] = product(sc[m][i], a.scale2) + neg[m];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) sc[m][i] = __builtin_fmaf(sc[m][i], a.scale2, neg[m]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x = __builtin_amdgcn_exp2f(sc[m][2 * i]);
        float y = __builtin_amdgcn_exp2f(sc[m][2 * i + 1]);
        sum[m] += x + y;
        if constexpr (FP8) {
          x *= vsc[2 * i];
          y *= vsc[2 * i + 1];
        }
        p[m][i] = pack2<PV_BF16>(x, y);
        if constexpr (FP8)
          rest[m][i] = pack2<PV_BF16>(x - __uint_as_float(p[m][i] << 16), y - __uint_as_float(p[m][i] & 0xFFFF0000u));
      }
    }

    // V^T operands: the 8 keys 8 g .. 8 g + 7 of dim 16 d + c
    copies_left<NK>();   // this tile's V is there (the next one's K followed)
    u32x4 vt[DN];
    if constexpr (FP8) {
      // transposed 8 keys x 16 dims of a group: lane 2 r + x points to key r, dims 8 x .. 8 x + 7
      const uint8_t *p = vbuf + ldsrow(g, c >> 1) * RB + 8 * (c & 1);
#pragma unroll
      for (int d = 0; d < DN; ++d) {
        const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2 *)(p + ((d ^ swizzle_v(g, c >> 1)) << 4)));
        vt[d][0] = (uint32_t)w[0];
        vt[d][1] = (uint32_t)w[1];
      }
    } else {
      // transposed 4 keys x 16 dims: lane 4 r + x points to key r, dims 4 x .. 4 x + 3
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int ve = 4 * h + (c >> 2);
        const uint8_t *p = vbuf + ldsrow(g, ve) * RB + 8 * (c & 1);
#pragma unroll
        for (int d = 0; d < DN; ++d) {
          const i32x2 w = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) i16x4 *)(p + (((2 * d + ((c & 3) >> 1)) ^ swizzle_v(g, ve)) << 4))));
          vt[d][2 * h] = (uint32_t)w[0];
          vt[d][2 * h + 1] = (uint32_t)w[1];
        }
      }
    }
    lds_done();
    request_v();
    if (!more) {   // keys behind the list's end are zeros
      const int left = n - 8 * g;
#pragma unroll
      for (int y = 0; y < (FP8 ? 2 : 4); ++y) {
        constexpr int PACK = FP8 ? 4 : 2, BITS = FP8 ? 8 : 16;   // keys of a word
        const int keys = min(max(left - PACK * y, 0), PACK);
        const uint32_t keep = keys == PACK ? ~0u : (1u << (keys * BITS)) - 1u;
#pragma unroll
        for (int d = 0; d < DN; ++d) vt[d][y] &= keep;
      }
    }
    if constexpr (FP8) {
#pragma unroll
      for (int d = 0; d < DN; ++d)
        vt[d] = u32x4{codes2<true, false>(vt[d][0]), codes2<true, true>(vt[d][0]), codes2<true, false>(vt[d][1]),
                      codes2<true, true>(vt[d][1])};
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if constexpr (!FP8) rounded[m] = mfma<BF16>(u32x4{ONES, ONES, ONES, ONES}, p[m], rounded[m]);
#pragma unroll
      for (int d = 0; d < DN; ++d) {
        o[m][d] = mfma<PV_BF16>(vt[d], p[m], o[m][d]);
        if constexpr (FP8) o[m][d] = mfma<PV_BF16>(vt[d], rest[m], o[m][d]);
      }
    }
  }

  copies_left<0>();   // none may write LDS that is another wave's by then

  if constexpr (MT == 1) {
    if (a.waves > 1) {
      // each wave's output, sum and reference through LDS; quads of dims exchanged against bank conflicts
      constexpr int QUADS = D / 4;
      float *const ml = (float *)(lds + a.waves * WAVE_LDS);    // [waves][3][16]
      const float l = head_sum(sum[0]);
#pragma unroll
      for (int d = 0; d < DN; ++d)
        *(f32x4 *)(kbuf + c * D * 4 + ((4 * d + g) ^ (c & 7)) * 16) = o[0][d];
      if (g == 0) {
        ml[wave * 48 + c] = ref[0];
        ml[wave * 48 + 16 + c] = l;
        ml[wave * 48 + 32 + c] = FP8 ? l : rounded[0][0];
      }
      __syncthreads();
      for (int x = threadIdx.x; x < heads * QUADS; x += 64 * a.waves) {
        const int h = x / QUADS, y = x % QUADS;
        float top = NEG_INF;
        for (int w = 0; w < a.waves; ++w) top = __builtin_fmaxf(top, ml[w * 48 + h]);
        const float base = top == NEG_INF ? 0.f : top;
        float total = 0.f, div = 0.f;
        f32x4 r = {0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < a.waves; ++w) {
          const float f = __builtin_amdgcn_exp2f(ml[w * 48 + h] - base);
          total += f * ml[w * 48 + 16 + h];
          div += f * ml[w * 48 + 32 + h];
          r += f * *(const f32x4 *)(lds + w * WAVE_LDS + h * D * 4 + (y ^ (h & 7)) * 16);
        }
        if (a.splits > 1) {
          const int64_t at = item * HEADS + h;
          *(f32x4 *)(a.part + at * D + 4 * y) = r;
          if (y == 0) *(f32x4 *)(a.part_ml + 4 * at) = f32x4{top, total, div, 0.f};
        } else {
          r *= finish(div);
          *(uint2 *)(a.out + (int64_t)t * a.out_t + (int64_t)(head0 + h) * a.out_h + 8 * y) =
              make_uint2(pack2<BF16>(r[0], r[1]), pack2<BF16>(r[2], r[3]));
          if (y == 0 && a.lse) a.lse[(int64_t)t * a.Hq + head0 + h] = lse_of(top, total);
        }
      }
      return;
    }
  }
  // lane l holds head l % 16 and dims 16 d + 4 g + j
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const float l = head_sum(sum[m]), div = FP8 ? l : rounded[m][0];
    const int h = m * 16 + c;
    if (a.splits > 1) {
      if (h >= heads) continue;
      const int64_t at = item * HEADS + h;
      if (g == 0) *(f32x4 *)(a.part_ml + 4 * at) = f32x4{ref[m], l, div, 0.f};
#pragma unroll
      for (int d = 0; d < DN; ++d) *(f32x4 *)(a.part + at * D + 16 * d + 4 * g) = o[m][d];
    } else {
      const float f = finish(div);
#pragma unroll
      for (int d = 0; d < DN; ++d)
        *(uint2 *)(kbuf + h * 2 * D + (((2 * d + (g >> 1)) ^ (h & (OUT_CH - 1))) << 4) + 8 * (g & 1)) =
            make_uint2(pack2<BF16>(o[m][d][0] * f, o[m][d][1] * f), pack2<BF16>(o[m][d][2] * f, o[m][d][3] * f));
      if (g == 0 && h < heads && a.lse) a.lse[(int64_t)t * a.Hq + head0 + h] = lse_of(ref[m], l);
    }
  }
  if (a.splits > 1) return;
  // through LDS, so that whole rows are stored at a time
  wave_sync();
  uint8_t *const dst = a.out + (int64_t)t * a.out_t;
#pragma unroll
  for (int i = 0; i < HEADS * OUT_CH / 64; ++i) {
    const int h = i * (64 / OUT_CH) + lane / OUT_CH, ch = lane & (OUT_CH - 1);
    if (h < heads)
      *(u32x4 *)(dst + (int64_t)(head0 + h) * a.out_h + 16 * ch) =
          *(const u32x4 *)(kbuf + h * 2 * D + ((ch ^ (h & (OUT_CH - 1))) << 4));
  }
}

// Joins the splits of a row's head: D / 4 threads to four dims each, MERGE / (D / 4) groups of splits.
constexpr int MERGE = 256;
template <bool BF16, int D>
__global__ __launch_bounds__(MERGE) void merge_splits_kernel(AttnArgs a, int HEADS) {
  constexpr int QUADS = D / 4, GROUPS = MERGE / QUADS;
  __shared__ __attribute__((aligned(16))) float acc[GROUPS][D];
  __shared__ float factor[MAX_SPLITS];
  __shared__ float shared[3];
  const uint32_t th = blockIdx.x;
  const int t = (int)(th / (uint32_t)a.Hq), hq = (int)(th % (uint32_t)a.Hq);
  const int kvh = hq / a.G, in = hq % a.G;
  const int d = 4 * (threadIdx.x % QUADS), gr = threadIdx.x / QUADS;
  const int64_t at0 = ((((int64_t)t * a.Hkv + kvh) * a.blocks + in / HEADS) * a.splits) * HEADS + in % HEADS;
  if (threadIdx.x < 64) {   // one wave: every split's reference and sum at once
    float m[MAX_SPLITS / 64], l[MAX_SPLITS / 64], div[MAX_SPLITS / 64];
#pragma unroll
    for (int i = 0; i < MAX_SPLITS / 64; ++i) {
      const int s = threadIdx.x + 64 * i;
      m[i] = NEG_INF;
      l[i] = div[i] = 0.f;
      if (s < a.splits) {
        const f32x4 ml = *(const f32x4 *)(a.part_ml + 4 * (at0 + (int64_t)s * HEADS));
        m[i] = ml[0];
        l[i] = ml[1];
        div[i] = ml[2];
      }
    }
    float top = m[0];
#pragma unroll
    for (int i = 1; i < MAX_SPLITS / 64; ++i) top = __builtin_fmaxf(top, m[i]);
    top = wave_reduce_f32(top, [](float x, float y) { return __builtin_fmaxf(x, y); });
    const float ref = top == NEG_INF ? 0.f : top;
    float total = 0.f, divide = 0.f;
#pragma unroll
    for (int i = 0; i < MAX_SPLITS / 64; ++i) {
      const int s = threadIdx.x + 64 * i;
      const float f = __builtin_amdgcn_exp2f(m[i] - ref);
      if (s < a.splits) {
        factor[s] = f;
        total += f * l[i];
        divide += f * div[i];
      }
    }
    total = wave_reduce_f32(total, [](float x, float y) { return x + y; });
    divide = wave_reduce_f32(divide, [](float x, float y) { return x + y; });
    if (threadIdx.x == 0) {
      shared[0] = top;
      shared[1] = total;
      shared[2] = divide;
    }
  }
  __syncthreads();
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = gr; s < a.splits; s += GROUPS) r += factor[s] * *(const f32x4 *)(a.part + (at0 + (int64_t)s * HEADS) * D + d);
  *(f32x4 *)&acc[gr][d] = r;
  __syncthreads();
  if (gr) return;
#pragma unroll
  for (int x = 1; x < GROUPS; ++x) r += *(const f32x4 *)&acc[x][d];
  r *= finish(shared[2]);
  *(uint2 *)(a.out + (int64_t)t * a.out_t + (int64_t)hq * a.out_h + 2 * d) =
      make_uint2(pack2<BF16>(r[0], r[1]), pack2<BF16>(r[2], r[3]));
  if (d == 0 && a.lse) a.lse[th] = lse_of(shared[0], shared[1]);
}

template <bool BF16, bool FP8, int D, int MT, bool WIDE>
hipError_t launch_width(const AttnArgs &a, unsigned blocks, hipStream_t s) {
  const size_t lds = (size_t)a.waves * wave_lds(FP8, D, WIDE) + (a.waves > 1 ? 192 * a.waves : 0);
  hipLaunchKernelGGL((attn_kernel<BF16, FP8, D, MT, WIDE>), dim3(blocks), dim3(64 * a.waves), lds, s, a);
  return hipGetLastError();
}
template <bool BF16, bool FP8, int D, int MT>
hipError_t launch_one(const AttnArgs &a, unsigned blocks, hipStream_t s) {
  return (uint64_t)a.rows * a.row_bytes > 0xFFFFFFFFull ? launch_width<BF16, FP8, D, MT, true>(a, blocks, s)
                                                        : launch_width<BF16, FP8, D, MT, false>(a, blocks, s);
}
template <bool BF16, bool FP8, int D>
hipError_t launch_tiles(const AttnArgs &a, int tiles, unsigned blocks, hipStream_t s) {
  return tiles == 1 ? launch_one<BF16, FP8, D, 1>(a, blocks, s) : launch_one<BF16, FP8, D, 2>(a, blocks, s);
}
template <bool BF16, bool FP8>
hipError_t launch_dim(const AttnArgs &a, int D, int tiles, unsigned blocks, hipStream_t s) {
  return D == 64 ? launch_tiles<BF16, FP8, 64>(a, tiles, blocks, s) : launch_tiles<BF16, FP8, 128>(a, tiles, blocks, s);
}

}  // namespace

AttnPlan plan_attn(int32_t T, int32_t Hkv, int32_t G, int32_t D, bool fp8, int64_t entries, int64_t touched) {
  AttnPlan p{};
  const int64_t tiles = entries > 0 ? (entries + TILE - 1) / TILE : 1;
  // 32 heads to a wave where rows alone nearly fill the machine (2 waves a SIMD): each key is fetched once for them.
  // From 768 waves on 32 heads are as fast or faster with 24, 32 and 64 query heads, 64 and 128 dims, 512 and 2048
  // keys, either type of cache.  us with 16 heads a wave and with 32, 2048 keys, 32 heads of 128 and of 64: E4M3,
  // 512 rows 53, 82 and 41, 63; 768 rows 81, 83 and 64, 63; 1024 rows 90, 83 and 67, 63; 2048 rows 160, 123 and 127,
  // 90; bf16, 512 rows 53, 58 and 31, 47; 768 rows 75, 57 and 46, 47; 1024 rows 90, 60 and 52, 49; 2048 rows 171, 99
  // and 97, 65
  p.tiles = G > 16 && (int64_t)T * Hkv * ((G + 31) / 32) >= 768 ? 2 : 1;
  const int32_t heads = 16 * p.tiles;
  p.blocks = (G + heads - 1) / heads;
  const int64_t items = (int64_t)T * Hkv * p.blocks;
  // Fewer rows than that: a row's entries are divided over the waves of a workgroup, which join through LDS, or
  // over workgroups, which a second kernel joins (4 us).  A 32-key step takes a lone wave about 1 us.
  p.waves = p.splits = 1;
  if (p.tiles == 1 && items <= 256) {
    if (tiles > 32 && items <= 128) {
      // few rows, long lists: about one step to a wave.  1 row, 64 heads, 2048 keys: 9.9 us, 15.8 with eight
      // waves alone; 8 rows: 11.8 and 17.8.  Up to half the CUs: 128 items, us with four waves and two workgroups and
      // with eight waves alone, E4M3 and bf16: 16 rows x 8 cache heads 24, 29 and 33, 38; 128 rows of 16 heads, cache
      // rows of their own 24, 23 and 34, 33, shared 18, 17 and 17, 18; 32 rows of 64 heads 18, 16 and 18, 18
      p.waves = 4;
      while (items * p.waves * p.splits < 1024 && p.waves * p.splits < tiles && p.splits < MAX_SPLITS) p.splits *= 2;
    } else {
      // One workgroup for 129 to 256 items: of 20 divisions up to 8 waves and 16 workgroups the best one, or within 5%
      // of it, for 16 and 64 heads on one cache head and from 24 rows x 8 on (200 rows of 16 heads, E4M3: 33 us, 43
      // with eight workgroups of a wave; 24 rows x 8: 35.5, 34.5); 17 to 20 rows x 8 in E4M3 lose 14% (31.6, 27.1).
      // 256 rows, 16 heads, 512 keys: 15.9 us, 17.3 with one wave
      while (p.waves < MAX_WAVES && p.waves < tiles && items * p.waves < 1024) p.waves *= 2;
    }
  } else if (p.tiles == 1 && items <= 384 && tiles > 32 && Hkv > 1 && touched > FROM_MEMORY) {
    // More items than CUs, and up to one and a half: a workgroup each leaves some CUs twice the others' share of what
    // memory brings.  2048 keys of 128 dims through a slot table, us, four workgroups of a wave and one of four, E4M3
    // and bf16: 33 rows x 8 cache heads 47, 53 and 68, 76; 40 rows 51, 63 and 75, 80; 48 rows 59, 65 and 87, 85; 96
    // rows x 4 58, 60 and 89, 86; 180 rows x 2 56, 57 and 81, 80 (slots in order: 51, 47 and 81, 78).  Past it a
    // workgroup each is as fast or faster (52 rows x 8 66, 67 and 95, 88), and so it is for one cache head (400 rows of
    // 16 heads 78, 66 and 95, 84), rows that a cache on the chip holds (300 of 16 heads 35, 26) and shorter lists
    // (33 rows x 8, 512 keys: 17.5, 15.5)
    p.splits = 4;
  } else if (p.tiles == 1) {
    // Two or four waves to a workgroup while all fit the machine about at once (LDS and registers: 2048 waves of
    // 16-bit rows of 128 dims, which also meet the memory's rate first; up to 4000 of the others).  512 rows of 16
    // heads, 2048 keys, us, one wave and this: bf16 of 64 dims 38, 18, of 128 48, 35; E4M3 49, 23 and 60, 29;
    // past the limits, 2046 rows of 768 keys: 25 and two waves 29; 38, 44
    const int64_t most = fp8 ? 2560 : D == 64 ? 2048 : 1536;
    while (p.waves < 4 && 4 * p.waves < tiles && 2 * items * p.waves <= most) p.waves *= 2;
  }
  const int64_t parts = (int64_t)p.waves * p.splits;
  p.per = ((tiles + parts - 1) / parts) * TILE;
  p.bytes = p.splits > 1 ? (size_t)items * p.splits * heads * (D + 4) * 4 : 0;
  return p;
}

template <bool BF16>
hipError_t launch_merge_splits(const AttnArgs &a, int D, int heads, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.T * a.Hq));
  if (D == 64)
    hipLaunchKernelGGL((merge_splits_kernel<BF16, 64>), grid, dim3(MERGE), 0, s, a, heads);
  else
    hipLaunchKernelGGL((merge_splits_kernel<BF16, 128>), grid, dim3(MERGE), 0, s, a, heads);
  return hipGetLastError();
}

hipError_t launch_attn(AttnArgs &a, int32_t dtype, int32_t fmt, int32_t D, const AttnPlan &plan, void *ws,
                       hipStream_t s) {
  const int64_t blocks = (int64_t)a.T * a.Hkv * plan.blocks * plan.splits;
  if (blocks <= 0) return hipSuccess;
  if (blocks > INT32_MAX || (int64_t)a.T * a.Hq > INT32_MAX) return hipErrorInvalidValue;
  const int heads = 16 * plan.tiles;
  a.blocks = plan.blocks;
  a.splits = plan.splits;
  a.waves = plan.waves;
  a.per = plan.per;
  a.part = (float *)ws;
  a.part_ml = a.part + (size_t)blocks * heads * D;
  // a negative factor turns q over instead, so that the largest product comes from the largest dot
  a.q_sign = a.scale2 < 0.f ? 0x80008000u : 0u;
  // and a factor of zero zeroes q, so that the product of the mask's -inf with it stays -inf
  a.q_keep = a.scale2 == 0.f ? 0u : ~0u;
  a.scale2 = a.scale2 == 0.f ? 1.f : std::fabs(a.scale2);
  const bool bf16 = dtype == IDX_K_BF16, fp8 = fmt == IDX_K_FP8_E4M3;
  hipError_t e;
  if (bf16)
    e = fp8 ? launch_dim<true, true>(a, D, plan.tiles, (unsigned)blocks, s)
            : launch_dim<true, false>(a, D, plan.tiles, (unsigned)blocks, s);
  else
    e = fp8 ? launch_dim<false, true>(a, D, plan.tiles, (unsigned)blocks, s)
            : launch_dim<false, false>(a, D, plan.tiles, (unsigned)blocks, s);
  if (e != hipSuccess || plan.splits == 1) return e;
  return bf16 ? launch_merge_splits<true>(a, D, heads, s) : launch_merge_splits<false>(a, D, heads, s);
}

}  // namespace idx
