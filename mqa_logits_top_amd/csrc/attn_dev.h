// Device code that the attention kernels share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace idx {

constexpr float NEG_INF = -__builtin_inff();
constexpr float BIG = 0x1p20f;   // references from which on a score is rounded before the reference is taken off

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
typedef int16_t i16x4 __attribute__((ext_vector_type(4)));

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

// By its bits: x - x of a product may become an fma, and that the product's rounding error.
__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// A product rounded by itself, never part of an fma.
__device__ __forceinline__ float product(float x, float y) {
#pragma clang fp contract(off)
  return x * y;
}

// Lanes of the wave exchange data through LDS: its accesses complete in order, the compiler must not move them.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
// Memory-to-LDS copies: lane l's 16 (4) bytes land at LDS byte lds + 16 l (4 l); lds is wave-uniform and goes
// through m0, which the compiler reserves (it warns of a clobber) and no other instruction here reads.  The
// compiler does not count the copies, so the kernel waits itself: copies and loads of a wave complete in the order of
// their issue, so with at most N operations under way every copy is there that N others certainly followed; more of
// them only make the wait stricter.
typedef __attribute__((address_space(3))) uint8_t lds_u8;
__device__ __forceinline__ uint32_t lds_addr(const void *p) { return (uint32_t)(uintptr_t)(const lds_u8 *)p; }
__device__ __forceinline__ void copy16(const uint8_t *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
               : "memory");
}
__device__ __forceinline__ void copy16(const uint8_t *base, uint64_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(base + off), "s"(lds)
               : "memory");
}
__device__ __forceinline__ void copy4(const float *p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(p), "s"(lds) : "memory");
}
template <int N>
__device__ __forceinline__ void copies_left() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Every LDS read so far has its data: the memory they read may be written by a copy.
__device__ __forceinline__ void lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Factor of the unnormalised output, and ln of the sum of exponentials.
__device__ __forceinline__ float finish(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float lse_of(float ref, float l) {
  return l == 0.f ? NEG_INF : 0.69314718055994531f * (ref + __builtin_amdgcn_logf(l));
}

}  // namespace idx
