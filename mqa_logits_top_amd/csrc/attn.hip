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
#include "common.h"

namespace idx {
namespace {

constexpr int WAVES = 4;
constexpr int TILE = 32;
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

// BF16: q's type; FP8: E4M3 caches (else of q's type); MT: 16-head tiles.
template <bool BF16, bool FP8, int D, int MT>
__global__ __launch_bounds__(WAVES * 64) void attn_kernel(AttnArgs a) {
  constexpr bool PV_BF16 = BF16 || FP8;   // weights times E4M3 scales need bf16's range
  constexpr int KS = D / 32;              // steps of the first product
  constexpr int DN = D / 16;              // dims of a lane's V piece, and tiles of the second product
  constexpr int HEADS = MT * 16;
  __shared__ __attribute__((aligned(16))) float lds[WAVES * HEADS * (D + 2)];   // [WAVES][HEADS][D] out, then (m, l)

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
      q[m][s] = w;
    }

  f32x4 o[MT][DN];
  float mx[MT], sum[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    mx[m] = NEG_INF;
    sum[m] = 0.f;
#pragma unroll
    for (int n = 0; n < DN; ++n) o[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int32_t win0 = a.ks ? max(a.ks[t], 0) : 0, win1 = a.ke ? min(a.ke[t], a.L) : a.L;
  const int64_t entries = (int64_t)a.n_sel << a.pool_sh;
  const int64_t tiles = (entries + TILE - 1) / TILE;
  const int32_t *list = a.sel + (int64_t)t * a.ld_sel;
  const uint8_t *kbase = a.k + (FP8 ? D : 2 * D) * (int64_t)kvh, *vbase = a.v + (FP8 ? D : 2 * D) * (int64_t)kvh;

  for (int64_t tile = (int64_t)split * WAVES + wave; tile < tiles; tile += (int64_t)a.splits * WAVES) {
    // the cache row of entry lane % 32, or -1
    const int64_t e = tile * TILE + (lane & 31);
    int64_t key = -1;
    if (e < entries) {
      const int32_t id = list[e >> a.pool_sh];
      if (id >= 0)
        key = a.pool_sh ? (int64_t)win0 + ((int64_t)id << a.pool_sh) + (e & ((1 << a.pool_sh) - 1)) : (int64_t)id;
    }
    int32_t row = -1;
    if (key >= win0 && key < win1) {
      const int64_t r = a.table ? (int64_t)a.table[key] : key;
      if (r >= 0 && r < a.rows) row = (int32_t)r;
    }
    const uint64_t some = __ballot(row >= 0);
    if (!some) continue;
    const bool all = some == ~0ull;
    // rows that do not count read a row that does; their scores and values are replaced below
    const int32_t first = __builtin_amdgcn_readlane(row, __builtin_ctzll(some));
    const int32_t safe = row >= 0 ? row : first;

    u32x4 kt[2][KS];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = __shfl(safe, 16 * h + c);
      const uint8_t *p = kbase + r * a.k_t;
      if constexpr (FP8) {
#pragma unroll
        for (int s = 0; s < KS; s += 2) {
          const u32x4 w = *(const u32x4 *)(p + 16 * ((s >> 1) * 4 + g));
          kt[h][s] = u32x4{codes2<BF16, false>(w.x), codes2<BF16, true>(w.x), codes2<BF16, false>(w.y),
                           codes2<BF16, true>(w.y)};
          kt[h][s + 1] = u32x4{codes2<BF16, false>(w.z), codes2<BF16, true>(w.z), codes2<BF16, false>(w.w),
                               codes2<BF16, true>(w.w)};
        }
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s) kt[h][s] = *(const u32x4 *)(p + 16 * (4 * s + g));
      }
    }
    // V: DN dims of 8 keys; vt[n] packs the 8 keys of dim c DN + n
    uint32_t vr[8][DN / 2];
    int32_t vrow[8];
    float ksc[8], vsc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int src = (i >> 2) * 16 + 4 * g + (i & 3);
      vrow[i] = __shfl(row, src);
      const int64_t r = __shfl(safe, src);
      const uint8_t *p = vbase + r * a.v_t;
      if constexpr (FP8) {
        ksc[i] = a.k_scale[r * a.ks_t + kvh];
        vsc[i] = a.v_scale[r * a.vs_t + kvh];
        if (vrow[i] < 0) vsc[i] = 0.f;
        uint32_t w[DN / 4];
        if constexpr (D == 128)
          *(uint2 *)w = *(const uint2 *)(p + DN * c);
        else
          w[0] = *(const uint32_t *)(p + DN * c);
#pragma unroll
        for (int x = 0; x < DN / 4; ++x) {
          if (!all && vrow[i] < 0) w[x] = 0u;
          vr[i][2 * x] = codes2<true, false>(w[x]);
          vr[i][2 * x + 1] = codes2<true, true>(w[x]);
        }
      } else {
        if constexpr (D == 128)
          *(u32x4 *)vr[i] = *(const u32x4 *)(p + 2 * DN * c);
        else
          *(uint2 *)vr[i] = *(const uint2 *)(p + 2 * DN * c);
        if (!all && vrow[i] < 0) {
#pragma unroll
          for (int x = 0; x < DN / 2; ++x) vr[i][x] = 0u;
        }
      }
    }
    u32x4 vt[DN];
#pragma unroll
    for (int x = 0; x < DN / 2; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        vt[2 * x][y] = __builtin_amdgcn_perm(vr[2 * y + 1][x], vr[2 * y][x], 0x05040100u);
        vt[2 * x + 1][y] = __builtin_amdgcn_perm(vr[2 * y + 1][x], vr[2 * y][x], 0x07060302u);
      }

#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float sc[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) acc = mfma<BF16>(kt[h][s], q[m][s], acc);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x = acc[j] * a.scale2;
          if constexpr (FP8) x *= ksc[4 * h + j];
          sc[4 * h + j] = vrow[4 * h + j] >= 0 ? x : NEG_INF;
        }
      }
      float top = sc[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, sc[i]);
      const float was = mx[m], now = __builtin_fmaxf(was, head_max(top));
      const float ref = now == NEG_INF ? 0.f : now;
      if (__any(now != was)) {
        const float f = __builtin_amdgcn_exp2f(was - ref);
        sum[m] *= f;
#pragma unroll
        for (int n = 0; n < DN; ++n) o[m][n] *= f;
        mx[m] = now;
      }
      u32x4 p;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x = __builtin_amdgcn_exp2f(sc[2 * i] - ref), y = __builtin_amdgcn_exp2f(sc[2 * i + 1] - ref);
        sum[m] += x + y;
        if constexpr (FP8) {
          x *= vsc[2 * i];
          y *= vsc[2 * i + 1];
        }
        p[i] = pack2<PV_BF16>(x, y);
      }
#pragma unroll
      for (int n = 0; n < DN; ++n) o[m][n] = mfma<PV_BF16>(vt[n], p, o[m][n]);
    }
  }

  // join the waves: lane l holds head l % 16 and dims (4 g + j) DN + n
  float *ml = lds + WAVES * HEADS * D;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const float l = head_sum(sum[m]);
    const int h = m * 16 + c;
    if (g == 0) {
      ml[2 * (wave * HEADS + h)] = mx[m];
      ml[2 * (wave * HEADS + h) + 1] = l;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int n = 0; n < DN; ++n) lds[(wave * HEADS + h) * D + (4 * g + j) * DN + n] = o[m][n][j];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < heads * (D / 4); x += WAVES * 64) {
    const int h = x / (D / 4), d = 4 * (x % (D / 4));
    float top = NEG_INF;
    for (int w = 0; w < WAVES; ++w) top = __builtin_fmaxf(top, ml[2 * (w * HEADS + h)]);
    const float ref = top == NEG_INF ? 0.f : top;
    float l = 0.f;
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
    for (int w = 0; w < WAVES; ++w) {
      const float f = __builtin_amdgcn_exp2f(ml[2 * (w * HEADS + h)] - ref);
      l += f * ml[2 * (w * HEADS + h) + 1];
      r += f * *(const f32x4 *)&lds[(w * HEADS + h) * D + d];
    }
    if (a.splits > 1) {
      const int64_t at = (int64_t)blockIdx.x * HEADS + h;
      *(f32x4 *)(a.part + at * D + d) = r;
      if (d == 0) {
        a.part_ml[2 * at] = top;
        a.part_ml[2 * at + 1] = l;
      }
    } else {
      const float f = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      r *= f;
      *(uint2 *)(a.out + (int64_t)t * a.out_t + (int64_t)(head0 + h) * a.out_h + 2 * d) =
          make_uint2(pack2<BF16>(r[0], r[1]), pack2<BF16>(r[2], r[3]));
      if (d == 0 && a.lse)
        a.lse[(int64_t)t * a.Hq + head0 + h] =
            l == 0.f ? NEG_INF : 0.69314718055994531f * (top + __builtin_amdgcn_logf(l));
    }
  }
}

// Joins the splits of a row: one thread to four dims of a head.
template <bool BF16>
__global__ __launch_bounds__(256) void merge_splits_kernel(AttnArgs a, int D, int HEADS) {
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int quads = D / 4;
  if (x >= (int64_t)a.T * a.Hq * quads) return;
  const int d = 4 * (int)(x % quads);
  const int64_t th = x / quads;
  const int t = (int)(th / a.Hq), hq = (int)(th % a.Hq);
  const int kvh = hq / a.G, in = hq % a.G;
  const int64_t at0 = ((((int64_t)t * a.Hkv + kvh) * a.blocks + in / HEADS) * a.splits) * HEADS + in % HEADS;
  float top = NEG_INF;
  for (int s = 0; s < a.splits; ++s) top = __builtin_fmaxf(top, a.part_ml[2 * (at0 + (int64_t)s * HEADS)]);
  const float ref = top == NEG_INF ? 0.f : top;
  float l = 0.f;
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.splits; ++s) {
    const int64_t at = at0 + (int64_t)s * HEADS;
    const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * at] - ref);
    l += f * a.part_ml[2 * at + 1];
    r += f * *(const f32x4 *)(a.part + at * D + d);
  }
  const float f = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  r *= f;
  *(uint2 *)(a.out + (int64_t)t * a.out_t + (int64_t)hq * a.out_h + 2 * d) =
      make_uint2(pack2<BF16>(r[0], r[1]), pack2<BF16>(r[2], r[3]));
  if (d == 0 && a.lse) a.lse[th] = l == 0.f ? NEG_INF : 0.69314718055994531f * (top + __builtin_amdgcn_logf(l));
}

template <bool BF16, bool FP8, int D, int MT>
hipError_t launch_one(const AttnArgs &a, unsigned blocks, hipStream_t s) {
  hipLaunchKernelGGL((attn_kernel<BF16, FP8, D, MT>), dim3(blocks), dim3(WAVES * 64), 0, s, a);
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
  const int32_t heads = 16 * p.tiles;
  p.blocks = (G + heads - 1) / heads;
  const int64_t items = (int64_t)T * Hkv * p.blocks;
  const int64_t most = (entries + WAVES * TILE - 1) / (WAVES * TILE);
  int64_t splits = items > 0 ? 512 / items : 1;
  splits = splits < most ? splits : most;
  p.splits = (int32_t)(splits < 1 ? 1 : splits);
  p.bytes = p.splits > 1 ? (size_t)items * p.splits * heads * (D + 2) * 4 : 0;
  return p;
}

hipError_t launch_attn(AttnArgs &a, int32_t dtype, int32_t fmt, int32_t D, const AttnPlan &plan, void *ws,
                       hipStream_t s) {
  const int64_t blocks = (int64_t)a.T * a.Hkv * plan.blocks * plan.splits;
  if (blocks <= 0) return hipSuccess;
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  const int heads = 16 * plan.tiles;
  a.blocks = plan.blocks;
  a.splits = plan.splits;
  a.part = (float *)ws;
  a.part_ml = a.part + (size_t)blocks * heads * D;
  const bool bf16 = dtype == IDX_K_BF16, fp8 = fmt == IDX_K_FP8_E4M3;
  hipError_t e;
  if (bf16)
    e = fp8 ? launch_dim<true, true>(a, D, plan.tiles, (unsigned)blocks, s)
            : launch_dim<true, false>(a, D, plan.tiles, (unsigned)blocks, s);
  else
    e = fp8 ? launch_dim<false, true>(a, D, plan.tiles, (unsigned)blocks, s)
            : launch_dim<false, false>(a, D, plan.tiles, (unsigned)blocks, s);
  if (e != hipSuccess || plan.splits == 1) return e;
  const int64_t threads = (int64_t)a.T * a.Hq * (D / 4);
  const unsigned mb = (unsigned)((threads + 255) / 256);
  if (bf16)
    hipLaunchKernelGGL((merge_splits_kernel<true>), dim3(mb), dim3(256), 0, s, a, (int)D, heads);
  else
    hipLaunchKernelGGL((merge_splits_kernel<false>), dim3(mb), dim3(256), 0, s, a, (int)D, heads);
  return hipGetLastError();
}

}  // namespace idx
