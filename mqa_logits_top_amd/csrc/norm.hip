// Root-mean-square norm of rows, with the residual's addition before it and E4M3 codes behind it.
//
// A row's values stay in registers from their load to the stores of its sum, its result and its codes: each byte moves
// once.  A lane holds 8 neighbouring values (V times, a workgroup's stride apart), all of whose loads are issued before the
// first is used.  Narrow rows share a wave, wide ones take 1 to 16 waves.  The squares' sum goes over the lanes by DPP and,
// with several waves, through LDS in a fixed order: results are repeatable.
//
// Memory bounds it.  Medians of traced launches: 16384 rows of 8192, bf16, with residual and E4M3 codes, 165 us, 5.7 TB/s;
// 2048 rows of 64 heads of 128, 14.8 us, 4.5; one row 3.9 us, of which the launch is 3.
#include "norm.h"

#include "common.h"
#include "rows_dev.h"

namespace idx {
namespace {

constexpr float SMALL_EPS = 0x1p-100f;   // squares lose up to 2^-150 each

// x summed over aligned groups of 2^sh lanes.
__device__ __forceinline__ float group_sum(float x, int sh) {
  auto add = [&](int on, int moved) { return on ? x + __uint_as_float((uint32_t)moved) : x; };
  x = add(sh > 0, __builtin_amdgcn_mov_dpp((int)__float_as_uint(x), 0xB1, 0xF, 0xF, false));
  x = add(sh > 1, __builtin_amdgcn_mov_dpp((int)__float_as_uint(x), 0x4E, 0xF, 0xF, false));
  x = add(sh > 2, __builtin_amdgcn_mov_dpp((int)__float_as_uint(x), 0x141, 0xF, 0xF, false));
  x = add(sh > 3, __builtin_amdgcn_mov_dpp((int)__float_as_uint(x), 0x140, 0xF, 0xF, false));
  if (sh > 4) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (sh > 5) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return x;
}

template <bool F32>
__device__ __forceinline__ void store8(uint8_t *p, int dtype, const float *v) {
  if constexpr (F32) {
    if (dtype == IDX_K_F32) {
      *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]);
      *(float4 *)(p + 16) = make_float4(v[4], v[5], v[6], v[7]);
      return;
    }
  }
  *(uint4 *)p = dtype == IDX_K_BF16
                    ? make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]))
                    : make_uint4(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]), pack_f16(v[6], v[7]));
}

// F32: some array of the call is fp32.  V: pieces of 8 values of a lane.  WAVES: of a row; 0: a row is 2^lanes_sh lanes.
template <bool F32, int V, int WAVES>
__global__ __launch_bounds__(WAVES > 4 ? 64 * WAVES : 256) void norm_kernel(NormJob j) {
  constexpr int ROWS = WAVES == 0 || WAVES >= 4 ? 1 : 4 / WAVES;   // of a workgroup of 256 threads and more, in waves
  constexpr int LANES = WAVES ? 64 * WAVES : 64;
  __shared__ float parts[WAVES > 1 ? ROWS * WAVES : 1];
  __shared__ uint32_t tops[WAVES > 1 ? ROWS * WAVES : 1];
  const int sh = WAVES ? 6 : j.lanes_sh;
  uint32_t row;
  int c;                                  // the lane's place in its row
  if constexpr (WAVES == 0) {
    row = (blockIdx.x << (8 - sh)) + (threadIdx.x >> sh);
    c = threadIdx.x & ((1 << sh) - 1);
  } else {
    row = blockIdx.x * ROWS + threadIdx.x / LANES;
    c = threadIdx.x % LANES;
  }
  const int stride = WAVES ? LANES : 1 << sh;
  const bool live_row = row < (uint32_t)j.T * (uint32_t)j.H;
  if constexpr (WAVES <= 1) {
    if (!live_row) return;                // whole lane groups leave together
  }
  const uint32_t at = live_row ? row : 0u;
  const int64_t t = j.H == 1 ? at : at / (uint32_t)j.H, h = j.H == 1 ? 0 : at % (uint32_t)j.H;
  const uint8_t *const x = j.x.p + t * j.x.t + h * j.x.h;
  const uint8_t *const res = j.residual.p + t * j.residual.t + h * j.residual.h;
  const int xs = F32 && j.x.dtype == IDX_K_F32 ? 4 : 2, rs = F32 && j.residual.dtype == IDX_K_F32 ? 4 : 2;
  const int ws = F32 && j.weight_dtype == IDX_K_F32 ? 4 : 2;
  Raw<F32> xr[V], rr[V], wr[V];
  bool live[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = (c + i * stride) * 8;
    live[i] = e < j.D && live_row;
    if (live[i]) xr[i] = load8<F32>(x + (int64_t)e * xs, j.x.dtype, 0, 4, false);
  }
  if (j.residual.p) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = (c + i * stride) * 8;
      if (live[i]) rr[i] = load8<F32>(res + (int64_t)e * rs, j.residual.dtype, 0, 4, false);
    }
  }
  if (j.weight) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = (c + i * stride) * 8;
      if (live[i]) wr[i] = load8<F32>(j.weight + (int64_t)e * ws, j.weight_dtype, 0, 4, false);
    }
  }
  float v[V][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (!live[i]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      continue;
    }
    values8<F32>(xr[i], j.x.dtype, v[i]);
    if (j.residual.p) {
      float r[8];
      values8<F32>(rr[i], j.residual.dtype, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] += r[e];
      store8<F32>(j.total.p + t * j.total.t + h * j.total.h + (int64_t)(c + i * stride) * 8 * rs, j.total.dtype, v[i]);
    }
  }
  const int wave = threadIdx.x >> 6, wave0 = WAVES > 1 ? wave / WAVES * WAVES : 0;
  // An eps too small to cover what squares lose below fp32's normal numbers (the whole launch's): rows are multiplied by a
  // power of two, which no other rounding notices, so that their largest value, or eps's root, comes to 1.
  float eps = j.eps;
  if (eps < SMALL_EPS) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
    top = group_max(top, sh);
    if constexpr (WAVES > 1) {
      if ((threadIdx.x & 63) == 0) tops[wave] = top;
      __syncthreads();
      top = tops[wave0];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) top = max(top, tops[wave0 + w]);
    }
    int up = top >= INF ? 0 : max(-__builtin_amdgcn_frexp_expf(__uint_as_float(top)), 0);
    if (eps > 0.f) up = min(up, -__builtin_amdgcn_frexp_expf(eps) / 2);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = __builtin_amdgcn_ldexpf(v[i][e], up);
    eps = __builtin_amdgcn_ldexpf(eps, 2 * up);
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(v[i][e], v[i][e], sum);
  sum = group_sum(sum, sh);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) parts[wave] = sum;
    __syncthreads();
    sum = parts[wave0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += parts[wave0 + w];
  }
  const float rstd = 1.f / __builtin_sqrtf(sum / (float)j.D + eps);
  uint32_t top = 0;
  uint8_t *const out = j.out.p + t * j.out.t + h * j.out.h;
  const int os = F32 && j.out.dtype == IDX_K_F32 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (!live[i]) continue;
    float w[8];
    if (j.weight) values8<F32>(wr[i], j.weight_dtype, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[i][e] *= rstd;
      if (j.weight) v[i][e] *= w[e];
      top = max(top, __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
    }
    if (j.out.p) store8<F32>(out + (int64_t)(c + i * stride) * 8 * os, j.out.dtype, v[i]);
  }
  if (!j.codes) return;                   // the same for the whole launch
  const bool groups = j.group != j.D;     // several scales a row, each of 2^group_sh lanes
  if (!groups) {
    top = group_max(top, sh);
    if constexpr (WAVES > 1) {
      if ((threadIdx.x & 63) == 0) tops[wave] = top;
      __syncthreads();
      top = tops[wave0];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) top = max(top, tops[wave0 + w]);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e0 = (c + i * stride) * 8;
    uint32_t m = top;
    if (groups) {
      m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
      m = group_max(m, j.group_sh);
    }
    if (!live[i]) continue;
    const float amax = __uint_as_float(m), f = m >= TINY ? 448.0f / amax : 0.f, f1 = inverse_rest(amax, f);
    const int64_t head = groups ? e0 >> (j.group_sh + 3) : h;
    if (groups ? (c & ((1 << j.group_sh) - 1)) == 0 : e0 == 0)
      j.scale[t * j.scale_t + head] = m >= INF ? __uint_as_float(0x7FC00000u) : m >= TINY ? amax / 448.0f : 1.0f;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(v[i][e], f, v[i][e] * f1);
    *(uint2 *)(j.codes + t * j.codes_t + h * j.codes_h + e0) = make_uint2(e4m3x4(y), e4m3x4(y + 4));
  }
}

template <bool F32, int V, int WAVES>
hipError_t launch_as(const NormJob &j, hipStream_t s) {
  constexpr int threads = WAVES > 4 ? 64 * WAVES : 256;
  const int64_t rows = (int64_t)j.T * j.H;
  const int64_t per = WAVES ? threads / (64 * WAVES) : 256 >> j.lanes_sh;
  hipLaunchKernelGGL((norm_kernel<F32, V, WAVES>), dim3((unsigned)((rows + per - 1) / per)), dim3(threads), 0, s, j);
  return hipGetLastError();
}

template <bool F32>
hipError_t launch_width(const NormJob &j, hipStream_t s) {
  const int pieces = (j.D + 7) / 8;
  if (pieces <= 64) return launch_as<F32, 1, 0>(j, s);
  if (pieces <= 128) return launch_as<F32, 2, 1>(j, s);
  if (pieces <= 256) return launch_as<F32, 2, 2>(j, s);
  if (pieces <= 512) return launch_as<F32, 2, 4>(j, s);
  if (pieces <= 1024) return launch_as<F32, 2, 8>(j, s);
  if (pieces <= 2048) return launch_as<F32, 2, 16>(j, s);
  return launch_as<F32, 4, 16>(j, s);
}

}  // namespace

hipError_t launch_norm(NormJob &j, hipStream_t s) {
  j.lanes_sh = 0;
  while (j.lanes_sh < 6 && 8 << j.lanes_sh < j.D) ++j.lanes_sh;
  j.group_sh = 0;
  while (8 << j.group_sh < j.group && j.group_sh < 6) ++j.group_sh;
  const bool f32 = j.x.dtype == IDX_K_F32 || (j.residual.p && j.residual.dtype == IDX_K_F32) ||
                   (j.out.p && j.out.dtype == IDX_K_F32) || (j.weight && j.weight_dtype == IDX_K_F32);
  return f32 ? launch_width<true>(j, s) : launch_width<false>(j, s);
}

}  // namespace idx
