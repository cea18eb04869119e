// Root-mean-square norm of rows, with the residual's addition before it and E4M3 codes behind it.
#include "norm.h"

#include "common.h"

namespace idx {
namespace {

constexpr int THREADS = 1024;
constexpr uint32_t TINY = 0x0D800000u;   // bits of 2^-100
constexpr uint32_t INF = 0x7F800000u;

__device__ __forceinline__ float load1(const uint8_t *p, int dtype, int e) {
  if (dtype == IDX_K_F32) return ((const float *)p)[e];
  const uint16_t u = ((const uint16_t *)p)[e];
  return dtype == IDX_K_BF16 ? __uint_as_float((uint32_t)u << 16) : (float)__builtin_bit_cast(_Float16, u);
}
__device__ __forceinline__ void store1(uint8_t *p, int dtype, int e, float x) {
  if (dtype == IDX_K_F32)
    ((float *)p)[e] = x;
  else
    ((uint16_t *)p)[e] = dtype == IDX_K_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)x) : __builtin_bit_cast(uint16_t, (_Float16)x);
}

// A workgroup takes a row, which it keeps in LDS.
__global__ __launch_bounds__(THREADS) void norm_kernel(NormJob j) {
  extern __shared__ float row[];
  __shared__ float part[THREADS / 64];
  const int t = blockIdx.x / (unsigned)j.H, h = blockIdx.x % (unsigned)j.H;
  const uint8_t *x = j.x.p + t * j.x.t + h * j.x.h;
  float sum = 0.f;
  for (int e = threadIdx.x; e < j.D; e += THREADS) {
    float v = load1(x, j.x.dtype, e);
    if (j.residual.p) {
      v += load1(j.residual.p + t * j.residual.t + h * j.residual.h, j.residual.dtype, e);
      store1(j.total.p + t * j.total.t + h * j.total.h, j.total.dtype, e, v);
    }
    row[e] = v;
    sum += v * v;
  }
  sum = wave_reduce_f32(sum, [](float a, float b) { return a + b; });
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < THREADS / 64; ++w) sum += part[w];
  const float rstd = 1.f / __builtin_sqrtf(sum / (float)j.D + j.eps);
  for (int e = threadIdx.x; e < j.D; e += THREADS) {
    float y = row[e] * rstd;
    if (j.weight) y *= load1(j.weight, j.weight_dtype, e);
    row[e] = y;
    if (j.out.p) store1(j.out.p + t * j.out.t + h * j.out.h, j.out.dtype, e, y);
  }
  if (!j.codes) return;
  __syncthreads();
  const int groups = j.D / j.group;
  for (int g = threadIdx.x >> 6; g < groups; g += THREADS / 64) {
    const float *y = row + g * j.group;
    uint32_t m = 0;
    for (int e = threadIdx.x & 63; e < j.group; e += 64) m = max(m, __float_as_uint(y[e]) & 0x7FFFFFFFu);
    m = wave_max(m);
    const float amax = __uint_as_float(m), f = m >= TINY ? 448.f / amax : 0.f;
    const float rest = m >= TINY ? __builtin_fmaf(-f, amax, 448.f) * (f * (1.f / 448.f)) : 0.f;
    const int head = j.H > 1 ? h : g;
    if ((threadIdx.x & 63) == 0)
      j.scale[t * j.scale_t + head] = m >= INF ? __uint_as_float(0x7FC00000u) : m >= TINY ? amax / 448.f : 1.f;
    for (int e = threadIdx.x & 63; e < j.group; e += 64) {
      const float q = __builtin_fmaf(y[e], f, y[e] * rest);
      j.codes[t * j.codes_t + head * j.codes_h + e] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false);
    }
  }
}

}  // namespace

hipError_t launch_norm(const NormJob &j, hipStream_t s) {
  hipLaunchKernelGGL(norm_kernel, dim3((unsigned)((int64_t)j.T * j.H)), dim3(THREADS), (size_t)j.D * 4, s, j);
  return hipGetLastError();
}

}  // namespace idx
