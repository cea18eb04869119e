// Attention of new rows over every key, or a window of keys, of a paged cache.
#include "paged.h"

#include <cmath>

#include "common.h"

namespace idx {
namespace {

constexpr float NEG_INF = -__builtin_inff();

__device__ __forceinline__ float value16(uint16_t u, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t)u << 16) : (float)__builtin_bit_cast(_Float16, u);
}

// The last request that starts at or before row t.
__device__ __forceinline__ int request_of(const int32_t *cu, int B, int t) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A product rounded by itself, never part of an fma: a score past 2^24 less its rounded maximum would be off otherwise.
__device__ __forceinline__ float product(float x, float y) {
#pragma clang fp contract(off)
  return x * y;
}

// A wave serves one row and query head, a key at a time; a lane holds D / 64 dims.
template <int D>
__global__ __launch_bounds__(256) void paged_kernel(PagedArgs a, bool bf16, bool fp8) {
  constexpr int N = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= (int64_t)a.T * a.Hq) return;
  const int t = (int)(item / a.Hq), h = (int)(item % a.Hq), kvh = h / a.G;
  const int b = request_of(a.cu_q, a.B, t);
  const int first_row = a.cu_q[b], n = a.cu_q[b + 1] - first_row;
  if (t < first_row || t - first_row >= n) return;
  const int64_t pos = (int64_t)min(max(a.len_k[b], 0), a.max_len) - n + (t - first_row);
  const int64_t low = a.window && pos >= a.window ? pos - a.window + 1 : 0;
  float q[N], o[N], ref = NEG_INF, sum = 0.f;
  for (int i = 0; i < N; ++i) {
    uint16_t u = *(const uint16_t *)(a.q + t * a.q_t + h * a.q_h + 2 * (lane * N + i));
    u = (u & (uint16_t)a.q_keep) ^ (uint16_t)a.q_sign;
    q[i] = value16(u, bf16);
    o[i] = 0.f;
  }
  for (int64_t s = low > 0 && a.first > 0 ? 0 : low; s <= pos; ++s) {
    if (s < low && s >= a.first) s = low;
    const int64_t slot = ((int64_t)a.pages[b * a.ld_pages + (s >> a.page_sh)] << a.page_sh) + (s & ((1ll << a.page_sh) - 1));
    if (slot < 0 || slot >= a.rows) continue;
    float k[N], v[N];
    for (int i = 0; i < N; ++i) {
      const int e = kvh * D + lane * N + i;
      if (fp8) {
        k[i] = __builtin_amdgcn_cvt_f32_fp8((int)a.k[slot * a.row_bytes + e], 0) * a.k_scale[slot * a.scale_row + kvh];
        v[i] = __builtin_amdgcn_cvt_f32_fp8((int)a.v[slot * a.row_bytes + e], 0) * a.v_scale[slot * a.scale_row + kvh];
      } else {
        k[i] = value16(*(const uint16_t *)(a.k + slot * a.row_bytes + 2 * e), bf16);
        v[i] = value16(*(const uint16_t *)(a.v + slot * a.row_bytes + 2 * e), bf16);
      }
    }
    float dot = 0.f;
    for (int i = 0; i < N; ++i) dot = __builtin_fmaf(q[i], k[i], dot);
    dot = product(wave_reduce_f32(dot, [](float x, float y) { return x + y; }), a.scale2);
    const float to = __builtin_fmaxf(ref, dot);
    const float f = to == ref ? 1.f : __builtin_amdgcn_exp2f(ref - to), p = dot == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(dot - to);
    sum = sum * f + p;
    for (int i = 0; i < N; ++i) o[i] = o[i] * f + p * v[i];
    ref = to;
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  for (int i = 0; i < N; ++i) {
    const float x = o[i] * f;
    *(uint16_t *)(a.out + t * a.out_t + h * a.out_h + 2 * (lane * N + i)) =
        bf16 ? __builtin_bit_cast(uint16_t, (__bf16)x) : __builtin_bit_cast(uint16_t, (_Float16)x);
  }
  if (lane == 0 && a.lse) a.lse[item] = sum == 0.f ? NEG_INF : 0.69314718055994531f * (ref + __builtin_amdgcn_logf(sum));
}

__global__ void check_paged_kernel(PagedArgs a, uint32_t *word) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int32_t from = a.cu_q[b], to = a.cu_q[b + 1], len = a.len_k[b];
    bool bad = from < 0 || to < from || to > a.T || len < 0 || len > a.max_len;
    if (!bad && to > from) {
      const int64_t pages = (((int64_t)len - 1) >> a.page_sh) + 1;
      const int64_t low = a.window ? (int64_t)len - (to - from) - a.window + 1 : 0;   // the first row's window
      for (int64_t i = threadIdx.x; i < pages && len > 0; i += blockDim.x) {
        if ((i + 1) << a.page_sh <= low && i << a.page_sh >= a.first) continue;        // no row sees the page
        // the last slot of the page that the length reaches
        const int64_t last = min((int64_t)len - (i << a.page_sh), (int64_t)1 << a.page_sh) - 1;
        const int64_t slot = (int64_t)a.pages[b * a.ld_pages + i] << a.page_sh;
        bad |= slot < 0 || slot + last >= a.rows;
      }
    }
    if (bad) atomicOr(word, 1u);
  }
}

}  // namespace

PagedPlan plan_paged(int32_t T, int32_t B, int32_t Hkv, int32_t G, int32_t D, bool fp8, int32_t max_len) { return {}; }

hipError_t launch_paged(PagedArgs &a, int32_t dtype, int32_t fmt, int32_t D, const PagedPlan &plan, void *ws,
                        hipStream_t s) {
  const int64_t items = (int64_t)a.T * a.Hq;
  if (items <= 0) return hipSuccess;
  // a negative factor turns q over instead, so that the largest product comes from the largest dot
  a.q_sign = a.scale2 < 0.f ? 0x80008000u : 0u;
  // and a factor of zero zeroes q, so that the product of the mask's -inf with it stays -inf
  a.q_keep = a.scale2 == 0.f ? 0u : ~0u;
  a.scale2 = a.scale2 == 0.f ? 1.f : std::fabs(a.scale2);
  const dim3 grid((unsigned)((items + 3) / 4));
  const bool bf16 = dtype == IDX_K_BF16, fp8 = fmt == IDX_K_FP8_E4M3;
  if (D == 64)
    hipLaunchKernelGGL(paged_kernel<64>, grid, dim3(256), 0, s, a, bf16, fp8);
  else
    hipLaunchKernelGGL(paged_kernel<128>, grid, dim3(256), 0, s, a, bf16, fp8);
  return hipGetLastError();
}

hipError_t launch_paged_check(const PagedArgs &a, uint32_t *word, hipStream_t s) {
  if (a.B <= 0) return hipSuccess;
  hipLaunchKernelGGL(check_paged_kernel, dim3((unsigned)(a.B < 1024 ? a.B : 1024)), dim3(64), 0, s, a, word);
  return hipGetLastError();
}

}  // namespace idx
