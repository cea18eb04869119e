// Device code that the row kernels share: 8 values of a lane, their types, E4M3 codes.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/idx.h"

namespace idx {

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

// 448 / amax less its rounded value inv: with it x * 448 / amax is rounded once, so that values half way between
// two codes (16-bit values often are) go to the even one.  One more fma a value (no time); 0.1% of a bf16
// array's codes would go to the other one without it.
__device__ __forceinline__ float inverse_rest(float amax, float inv) {
  return __builtin_fmaf(-inv, amax, 448.0f) * (inv * (1.0f / 448.0f));
}

constexpr uint32_t TINY = 0x0D800000u;   // bits of 2^-100
constexpr uint32_t INF = 0x7F800000u;

}  // namespace idx
