// Attention of each query row over the keys its list selects.
//
// A workgroup serves one row t, one cache head and up to 64 of its query heads.  Its four waves
// take 32-key tiles of the list in turn, each with a softmax of its own (running maximum m, sum l
// and unnormalised output O), joined through LDS at the end.  Keys and values go straight from
// memory to the matrix cores' operand registers:
//   S^T = K Q^T  (v_mfma 16x16x32): A = 16 keys x 32 dims, lane l holds key l % 16, 8 dims of group
//     g = l / 16; the result gives lane l head l % 16 and keys 4 g .. 4 g + 3 of the tile.
//   O^T += V^T P^T: B = P^T, lane l holds head l % 16 and 8 of the 32 keys.  The product sums over
//     keys, so their order is free: taking keys 4g + j and 16 + 4g + j for group g makes the two S^T
//     results, exponentiated, the operand as they stand.  A = V^T: lane l reads dims
//     [c D/16, (c + 1) D/16), c = l % 16, of the same 8 keys (16 lanes read a whole row) and
//     transposes 8 keys x D/16 dims in registers; tile n's row c is then dim c D/16 + n.
// So no tile passes through LDS and no barrier stands in the loop.
#include "attn.h"

#include <cmath>
#include <type_traits>

#include "common.h"

namespace idx {
namespace {

constexpr int TILE = 32;      // keys of a step
constexpr int CHUNK = 256;    // list entries resolved at a time
constexpr int QUEUE = 512;    // rows waiting: under two tiles when a chunk is added
constexpr float NEG_INF = -__builtin_inff();

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <bool BF16>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    const v2 p = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, p);
  } else {
    typedef _Float16 v2 __attribute__((ext_vector_type(2)));
    const v2 p = {(_Float16)lo, (_Float16)hi};
    return __builtin_bit_cast(uint32_t, p);
  }
}

// Two E4M3 codes (low or high half of w) as two 16-bit values, exactly.
template <bool BF16, bool HI>
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
  if constexpr (BF16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
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

// Lanes of the wave exchange data through LDS: its accesses complete in order, the compiler must not move them.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
// Every LDS read so far has its data: the memory they read may be written by a copy.
__device__ __forceinline__ void lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Factor of the unnormalised output, and ln of the sum of exponentials.
__device__ __forceinline__ float finish(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float lse_of(float ref, float l) {
  return l == 0.f ? NEG_INF : 0.69314718055994531f * (ref + __builtin_amdgcn_logf(l));
}

// BF16: q's type; FP8: E4M3 caches (else of q's type); MT: 16-head tiles.
// WIDE: caches past 2^32 bytes (64-bit offsets of rows instead of 32-bit ones beside a uniform base).
template <bool BF16, bool FP8, int D, int MT, bool WIDE>
__global__ __launch_bounds__(64, MT == 4 ? 1 : 2) void attn_kernel(AttnArgs a) {
  constexpr bool PV_BF16 = BF16 || FP8;   // weights times E4M3 scales need bf16's range
  constexpr int KS = D / 32;              // steps of the first product
  constexpr int DN = D / 16;              // dims of a lane's V piece, and tiles of the second product
  constexpr int HEADS = MT * 16;
  constexpr int RB = FP8 ? D : 2 * D;     // bytes of a cache row
  constexpr int CH = RB / 16;             // its 16-byte chunks
  constexpr int NI = CH / 2;              // copies of a tile's K: 64 / CH rows each
  constexpr int PER = 16 / CH;            // rows a 16-lane group brings in one copy
  __shared__ __attribute__((aligned(16))) uint8_t kbuf[TILE * RB];
  __shared__ __attribute__((aligned(16))) uint32_t queue[QUEUE];
  __shared__ __attribute__((aligned(16))) uint32_t offsets[WIDE ? 1 : QUEUE];   // the queue's rows in bytes
  __shared__ __attribute__((aligned(16))) float scales[FP8 ? 2 * TILE : 1];
  using Off = std::conditional_t<WIDE, uint64_t, uint32_t>;

  const int lane = threadIdx.x;
  const int c = lane & 15, g = lane >> 4;
  int64_t item = blockIdx.x;
  const int split = (int)(item % a.splits);
  item /= a.splits;
  const int hb = (int)(item % a.blocks);
  item /= a.blocks;
  const int kvh = (int)(item % a.Hkv);
  const int t = (int)(item / a.Hkv);
  const int head0 = kvh * a.G + hb * HEADS;                    // first query head
  const int heads = min(HEADS, a.G - hb * HEADS);

  // ---- the list: this split's entries, 256 at a time, through registers into the queue of cache rows
  const int32_t win0 = a.ks ? max(a.ks[t], 0) : 0, win1 = a.ke ? min(a.ke[t], a.L) : a.L;
  const int64_t entries = (int64_t)a.n_sel << a.pool_sh;
  const int64_t per = ((entries + a.splits - 1) / a.splits + TILE - 1) / TILE * TILE;
  const int64_t e_end = min(entries, (split + 1) * per);
  int64_t e_next = split * per;           // first entry whose id is not loaded
  const int32_t *list = a.sel + (int64_t)t * a.ld_sel;
  int32_t key[4], row[4];                 // the chunk after next: keys; the next chunk: rows
  auto load_keys = [&] {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t e = e_next + 64 * r + lane;
      int64_t k = -1;
      if (e < e_end) {
        const int32_t id = list[e >> a.pool_sh];
        k = id;
        if (a.pool_sh && id >= 0) k = (int64_t)win0 + ((int64_t)id << a.pool_sh) + (e & ((1 << a.pool_sh) - 1));
      }
      key[r] = k >= win0 && k < win1 ? (int32_t)k : -1;
    }
    e_next += CHUNK;
  };
  auto load_rows = [&] {
#pragma unroll
    for (int r = 0; r < 4; ++r) row[r] = a.table && key[r] >= 0 ? a.table[key[r]] : key[r];
  };
  int64_t e_left = e_end - e_next;        // entries not in the queue yet
  uint32_t head = 0, tail = 0;            // queue positions (modulo QUEUE); entries in order, no gaps
  auto fill = [&] {
    while (tail - head < 2 * TILE && e_left > 0) {
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
        if (e_left > CHUNK) load_keys();
      }
    }
    wave_sync();
  };
  if (e_left > 0) {
    load_keys();
    load_rows();
    if (e_left > CHUNK) load_keys();
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
      q[m][s] = w ^ a.q_sign;
    }

  f32x4 o[MT][DN];
  float ref[MT], sum[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    ref[m] = NEG_INF;
    sum[m] = 0.f;
#pragma unroll
    for (int n = 0; n < DN; ++n) o[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const uint8_t *kbase = a.k + (int64_t)RB * kvh, *vbase = a.v + (int64_t)RB * kvh;
  const float *sbase = (lane < TILE ? a.k_scale : a.v_scale) + kvh;
  // K copy u brings position 8 g + PER u + c / CH of the tile to LDS row u 4 PER + lane / CH, chunks swizzled
  // so that 16 lanes reading one chunk of 16 rows meet every bank once
  auto ldsrow = [](int p) { return (p & 7) / PER * 4 * PER + (p >> 3) * PER + (p & 7) % PER; };
  auto swizzle = [](int r) { return (r / PER) & (CH - 1); };
  Off off[8];                             // of the lane's 8 positions 8 g .. 8 g + 7
  float scale_in = 0.f;
  uint32_t vr[8][DN / 2];                 // V: DN dims of them (E4M3: their codes in the first words)

  auto request_k = [&] {
#pragma unroll
    for (int u = 0; u < NI; ++u) {
      Off b = off[PER * u];
      if constexpr (PER > 1) {
        const Off b1 = off[PER * u + 1];
        b = c / CH == 1 ? b1 : b;
      }
      if constexpr (PER > 2) {
        const Off b2 = off[PER * u + 2], b3 = off[PER * u + 3];
        b = c / CH == 2 ? b2 : c / CH == 3 ? b3 : b;
      }
      const int r = u * 4 * PER + lane / CH;
      const uint8_t *p = kbase + (Off)(b + (((lane & (CH - 1)) ^ swizzle(r)) << 4));
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)p,
                                       (__attribute__((address_space(3))) void *)(kbuf + u * 1024), 16, 0, 0);
    }
  };
  auto request_v = [&] {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint8_t *p = vbase + (Off)(off[i] + (RB / 16) * c);
      if constexpr (RB == 256)
        *(u32x4 *)vr[i] = *(const u32x4 *)p;
      else if constexpr (RB == 128)
        *(uint2 *)vr[i] = *(const uint2 *)p;
      else
        vr[i][0] = *(const uint32_t *)p;
    }
  };
  // the next tile's addresses, from the queue; returns how many of its positions count
  auto next_tile = [&]() -> int {
    fill();
    const int n = min((int)(tail - head), TILE);
    if (n > 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t at = (head + (uint32_t)min(8 * g + i, n - 1)) & (QUEUE - 1);
        off[i] = WIDE ? (Off)queue[at] * a.row_bytes : (Off)offsets[at];
      }
      if constexpr (FP8) {
        const uint32_t r = queue[(head + (uint32_t)min(lane & (TILE - 1), n - 1)) & (QUEUE - 1)];
        scale_in = sbase[(int64_t)r * a.scale_row];
      }
    }
    head += (uint32_t)n;
    return n;
  };

  int n = next_tile();
  if (n > 0) {
    request_k();
    request_v();
  }
  while (n > 0) {
    // this tile's K from LDS into operands, then the copy of the next tile's may start
    u32x4 kt[2][KS];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = ldsrow(8 * (c >> 2) + 4 * h + (c & 3));
      const uint8_t *p = kbuf + r * RB;
      if constexpr (FP8) {
#pragma unroll
        for (int s = 0; s < KS; s += 2) kt[h][s] = *(const u32x4 *)(p + (((2 * s + g) ^ swizzle(r)) << 4));
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s) kt[h][s] = *(const u32x4 *)(p + (((4 * s + g) ^ swizzle(r)) << 4));
      }
    }
    float ksc[8], vsc[8];
    if constexpr (FP8) {
      scales[lane] = scale_in;
      wave_sync();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ksc[i] = scales[8 * g + i] * a.scale2;
        vsc[i] = 8 * g + i < n ? scales[TILE + 8 * g + i] : 0.f;
      }
    }
    const int now_n = n;
    n = next_tile();
    lds_done();
    if (n > 0) request_k();
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

    u32x4 p[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float sc[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) acc = mfma<BF16>(kt[h][s], q[m][s], acc);
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[4 * h + j] = FP8 ? acc[j] * ksc[4 * h + j] : acc[j];
      }
      if (now_n < TILE) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * g + i >= now_n) sc[i] = NEG_INF;
      }
      float top = sc[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, sc[i]);
      if constexpr (!FP8) top *= a.scale2;     // scale2 >= 0: the largest product is the largest dot's
      const float now = head_max(top);
      // the reference moves only when a score is 2^8 above it: weights then stay below 2^8, and the
      // accumulators are rescaled a few times a row instead of at most tiles
      if (__any(now > ref[m] + 8.f)) {
        const float to = __builtin_fmaxf(ref[m], now);
        const float f = to == ref[m] ? 1.f : __builtin_amdgcn_exp2f(ref[m] - to);
        sum[m] *= f;
#pragma unroll
        for (int n2 = 0; n2 < DN; ++n2) o[m][n2] *= f;
        ref[m] = to;
      }
      const float base = ref[m] == NEG_INF ? 0.f : ref[m];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x, y;
        if constexpr (FP8) {
          x = __builtin_amdgcn_exp2f(sc[2 * i] - base);
          y = __builtin_amdgcn_exp2f(sc[2 * i + 1] - base);
        } else {
          x = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[2 * i], a.scale2, -base));
          y = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[2 * i + 1], a.scale2, -base));
        }
        sum[m] += x + y;
        if constexpr (FP8) {
          x *= vsc[2 * i];
          y *= vsc[2 * i + 1];
        }
        p[m][i] = pack2<PV_BF16>(x, y);
      }
    }

    // V^T operands: vt[d] packs the 8 keys of dim c DN + d
    if (now_n < TILE) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * g + i >= now_n) {
#pragma unroll
          for (int x = 0; x < DN / 2; ++x) vr[i][x] = 0u;
        }
    }
    u32x4 vt[DN];
    if constexpr (FP8) {
#pragma unroll
      for (int x = 0; x < DN / 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t e = vr[2 * y][x], f = vr[2 * y + 1][x];
          const uint32_t lo0 = codes2<true, false>(e), lo1 = codes2<true, false>(f);
          const uint32_t hi0 = codes2<true, true>(e), hi1 = codes2<true, true>(f);
          vt[4 * x][y] = __builtin_amdgcn_perm(lo1, lo0, 0x05040100u);
          vt[4 * x + 1][y] = __builtin_amdgcn_perm(lo1, lo0, 0x07060302u);
          vt[4 * x + 2][y] = __builtin_amdgcn_perm(hi1, hi0, 0x05040100u);
          vt[4 * x + 3][y] = __builtin_amdgcn_perm(hi1, hi0, 0x07060302u);
        }
    } else {
#pragma unroll
      for (int x = 0; x < DN / 2; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          vt[2 * x][y] = __builtin_amdgcn_perm(vr[2 * y + 1][x], vr[2 * y][x], 0x05040100u);
          vt[2 * x + 1][y] = __builtin_amdgcn_perm(vr[2 * y + 1][x], vr[2 * y][x], 0x07060302u);
        }
    }
    if (n > 0) request_v();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int d = 0; d < DN; ++d) o[m][d] = mfma<PV_BF16>(vt[d], p[m], o[m][d]);
  }

  // lane l holds head l % 16 and dims (4 g + j) DN + d
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const float l = head_sum(sum[m]);
    const int h = m * 16 + c;
    if (h >= heads) continue;
    if (a.splits > 1) {
      const int64_t at = (int64_t)blockIdx.x * HEADS + h;
      if (g == 0) {
        a.part_ml[2 * at] = ref[m];
        a.part_ml[2 * at + 1] = l;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int d = 0; d < DN; d += 4)
          *(f32x4 *)(a.part + at * D + (4 * g + j) * DN + d) =
              f32x4{o[m][d][j], o[m][d + 1][j], o[m][d + 2][j], o[m][d + 3][j]};
    } else {
      const float f = finish(l);
      uint8_t *dst = a.out + (int64_t)t * a.out_t + (int64_t)(head0 + h) * a.out_h;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int d = 0; d < DN; d += 4)
          *(uint2 *)(dst + 2 * ((4 * g + j) * DN + d)) =
              make_uint2(pack2<BF16>(o[m][d][j] * f, o[m][d + 1][j] * f),
                         pack2<BF16>(o[m][d + 2][j] * f, o[m][d + 3][j] * f));
      if (g == 0 && a.lse) a.lse[(int64_t)t * a.Hq + head0 + h] = lse_of(ref[m], l);
    }
  }
}

// Joins the splits of a row's head: D / 4 threads to four dims each, MERGE / (D / 4) groups of splits.
constexpr int MERGE = 256;
template <bool BF16, int D>
__global__ __launch_bounds__(MERGE) void merge_splits_kernel(AttnArgs a, int HEADS) {
  constexpr int QUADS = D / 4, GROUPS = MERGE / QUADS;
  __shared__ __attribute__((aligned(16))) float acc[GROUPS][D];
  __shared__ float sums[GROUPS];
  const int64_t th = blockIdx.x;
  const int t = (int)(th / a.Hq), hq = (int)(th % a.Hq);
  const int kvh = hq / a.G, in = hq % a.G;
  const int d = 4 * (threadIdx.x % QUADS), gr = threadIdx.x / QUADS;
  const int64_t at0 = ((((int64_t)t * a.Hkv + kvh) * a.blocks + in / HEADS) * a.splits) * HEADS + in % HEADS;
  float top = NEG_INF;
  for (int s = 0; s < a.splits; ++s) top = __builtin_fmaxf(top, a.part_ml[2 * (at0 + (int64_t)s * HEADS)]);
  const float ref = top == NEG_INF ? 0.f : top;
  float l = 0.f;
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = gr; s < a.splits; s += GROUPS) {
    const int64_t at = at0 + (int64_t)s * HEADS;
    const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * at] - ref);
    l += f * a.part_ml[2 * at + 1];
    r += f * *(const f32x4 *)(a.part + at * D + d);
  }
  *(f32x4 *)&acc[gr][d] = r;
  if (d == 0) sums[gr] = l;
  __syncthreads();
  if (gr) return;
#pragma unroll
  for (int x = 1; x < GROUPS; ++x) {
    r += *(const f32x4 *)&acc[x][d];
    l += sums[x];
  }
  if (d) {
    l = 0.f;
#pragma unroll
    for (int x = 0; x < GROUPS; ++x) l += sums[x];
  }
  r *= finish(l);
  *(uint2 *)(a.out + (int64_t)t * a.out_t + (int64_t)hq * a.out_h + 2 * d) =
      make_uint2(pack2<BF16>(r[0], r[1]), pack2<BF16>(r[2], r[3]));
  if (d == 0 && a.lse) a.lse[th] = lse_of(top, l);
}

template <bool BF16, bool FP8, int D, int MT>
hipError_t launch_one(const AttnArgs &a, unsigned blocks, hipStream_t s) {
  if ((uint64_t)a.rows * a.row_bytes > 0xFFFFFFFFull) {
    hipLaunchKernelGGL((attn_kernel<BF16, FP8, D, MT, true>), dim3(blocks), dim3(64), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((attn_kernel<BF16, FP8, D, MT, false>), dim3(blocks), dim3(64), 0, s, a);
  return hipGetLastError();
}
template <bool BF16, bool FP8, int D>
hipError_t launch_tiles(const AttnArgs &a, int tiles, unsigned blocks, hipStream_t s) {
  if (tiles == 1) return launch_one<BF16, FP8, D, 1>(a, blocks, s);
  if (tiles == 2) return launch_one<BF16, FP8, D, 2>(a, blocks, s);
  return launch_one<BF16, FP8, D, 4>(a, blocks, s);
}
template <bool BF16, bool FP8>
hipError_t launch_dim(const AttnArgs &a, int D, int tiles, unsigned blocks, hipStream_t s) {
  return D == 64 ? launch_tiles<BF16, FP8, 64>(a, tiles, blocks, s) : launch_tiles<BF16, FP8, 128>(a, tiles, blocks, s);
}

}  // namespace

AttnPlan plan_attn(int32_t T, int32_t Hkv, int32_t G, int32_t D, int64_t entries) {
  AttnPlan p{};
  p.tiles = G <= 16 ? 1 : G <= 32 ? 2 : 4;
  int64_t items = 0;
  for (;; p.tiles /= 2) {
    const int32_t heads = 16 * p.tiles;
    p.blocks = (G + heads - 1) / heads;
    items = (int64_t)T * Hkv * p.blocks;
    if (p.tiles == 1 || items >= 64) break;
  }
  const int64_t most = (entries + TILE - 1) / TILE;
  int64_t splits = items > 0 ? 2048 / items : 1;
  splits = splits < most ? splits : most;
  p.splits = (int32_t)(splits < 1 ? 1 : splits);
  p.bytes = p.splits > 1 ? (size_t)items * p.splits * 16 * p.tiles * (D + 2) * 4 : 0;
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
  a.part = (float *)ws;
  a.part_ml = a.part + (size_t)blocks * heads * D;
  // a negative factor turns q over instead, so that the largest product comes from the largest dot
  a.q_sign = a.scale2 < 0.f ? 0x80008000u : 0u;
  a.scale2 = std::fabs(a.scale2);
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
