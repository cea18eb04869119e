// Attention of new rows over every key, or a window of keys, of a paged cache: the division of the work, and the join of
// keys that were divided.
#include <cmath>

#include "attn_dev.h"
#include "paged_dev.h"

namespace idx {
namespace {

constexpr int JOIN = 256;     // threads of a join

// Joins the parts of a row tile's rows, JOIN / (D / 4) rows at a time, D / 4 threads to one: tiles of many rows, whose keys
// are in few parts.
template <bool BF16, int D>
__global__ __launch_bounds__(JOIN) void join_tile_kernel(PagedArgs a, int M, int slices) {
  constexpr int QUADS = D / 4;
  const uint32_t mu = (uint32_t)(a.Hkv * a.blocks);
  const uint32_t member = blockIdx.x % mu, rest = blockIdx.x / mu;
  const int slice = (int)(rest % (uint32_t)slices);
  if (!*a.chunk) return;
  Item found;
  if (!find_item<64, true, TILE>(a, rest / (uint32_t)slices, found) || found.splits == 1) return;
  const Item w = uniform(found);
  const int kvh = (int)(member % (uint32_t)a.Hkv), hb = (int)(member / (uint32_t)a.Hkv);
  const int heads = min(a.Gt, a.G - hb * a.Gt), d = 4 * (threadIdx.x % QUADS);
  for (int row = slice * (M / slices) + threadIdx.x / QUADS; row < (slice + 1) * (M / slices); row += JOIN / QUADS) {
    const int tok = row / a.Gt, h = row - tok * a.Gt;
    if (tok >= a.R || h >= heads || w.row0 + tok >= w.r.n) continue;
    const int64_t at0 = ((int64_t)w.first_item * mu + member) * M + row, step = (int64_t)w.next * mu * M;
    float top = NEG_INF;
    for (int s = 0; s < w.splits; ++s) top = __builtin_fmaxf(top, a.part_ml[4 * (at0 + s * step)]);
    const float ref = top == NEG_INF ? 0.f : top;
    float total = 0.f, div = 0.f;
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < w.splits; ++s) {
      const int64_t at = at0 + s * step;
      const f32x4 m = *(const f32x4 *)(a.part_ml + 4 * at);
      const float f = __builtin_amdgcn_exp2f(m[0] - ref);
      total += f * m[1];
      div += f * m[2];
      r += f * *(const f32x4 *)(a.part + at * D + d);
    }
    r *= finish(div);
    const int64_t t = w.r.from + w.row0 + tok, hq = kvh * a.G + hb * a.Gt + h;
    *(uint2 *)(a.out + t * a.out_t + hq * a.out_h + 2 * d) =
        make_uint2(pack2<BF16>(r[0], r[1]), pack2<BF16>(r[2], r[3]));
    if (d == 0 && a.lse) a.lse[t * a.Hq + hq] = lse_of(top, total);
  }
}

// Joins the parts of one row and head, JOIN / (D / 4) of them at a time: few rows, whose keys may be in many parts.  Each
// group of threads keeps a reference of its own, so that a part's reference, sum and values are requested together: the
// kernel is three latencies long (the batch, the parts, the store).
template <bool BF16, int D>
__global__ __launch_bounds__(JOIN) void join_row_kernel(PagedArgs a, int M) {
  constexpr int QUADS = D / 4, GROUPS = JOIN / QUADS, AT_ONCE = 4;
  __shared__ __attribute__((aligned(16))) float acc[GROUPS][D];
  __shared__ f32x4 ml[GROUPS];
  const uint32_t mu = (uint32_t)(a.Hkv * a.blocks);
  const int t = (int)(blockIdx.x / (uint32_t)a.Hq), hq = (int)(blockIdx.x % (uint32_t)a.Hq);
  Item found;
  if (!find_item<32, false, ROW>(a, (uint32_t)t, found) || found.splits == 1) return;
  const Item w = uniform(found);
  const int kvh = hq / a.G, hb = (hq - kvh * a.G) / a.Gt, h = hq - kvh * a.G - hb * a.Gt;
  const int row = (t - w.r.from - w.row0) * a.Gt + h;
  const int64_t at0 = ((int64_t)w.first_item * mu + hb * a.Hkv + kvh) * M + row, step = (int64_t)w.next * mu * M;
  const int d = 4 * (threadIdx.x % QUADS), gr = threadIdx.x / QUADS;
  float top = NEG_INF, total = 0.f, div = 0.f;
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = gr; s0 < w.splits; s0 += AT_ONCE * GROUPS) {
    f32x4 m[AT_ONCE], x[AT_ONCE];
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const int s = s0 + u * GROUPS;
      m[u] = f32x4{NEG_INF, 0.f, 0.f, 0.f};
      x[u] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (s < w.splits) {
        m[u] = *(const f32x4 *)(a.part_ml + 4 * (at0 + s * step));
        x[u] = *(const f32x4 *)(a.part + (at0 + s * step) * D + d);
      }
    }
    float to = top;
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) to = __builtin_fmaxf(to, m[u][0]);
    const float ref = to == NEG_INF ? 0.f : to, by = __builtin_amdgcn_exp2f(top - ref);
    total *= by;
    div *= by;
    r *= by;
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const float f = __builtin_amdgcn_exp2f(m[u][0] - ref);
      total += f * m[u][1];
      div += f * m[u][2];
      r += f * x[u];
    }
    top = to;
  }
  *(f32x4 *)&acc[gr][d] = r;
  if (d == 0) ml[gr] = f32x4{top, total, div, 0.f};
  __syncthreads();
  if (gr) return;
#pragma unroll
  for (int x = 1; x < GROUPS; ++x) top = __builtin_fmaxf(top, ml[x][0]);
  const float ref = top == NEG_INF ? 0.f : top;
  total = div = 0.f;
  r = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int x = 0; x < GROUPS; ++x) {
    const float f = __builtin_amdgcn_exp2f(ml[x][0] - ref);
    r += f * *(const f32x4 *)&acc[x][d];
    total += f * ml[x][1];
    div += f * ml[x][2];
  }
  r *= finish(div);
  *(uint2 *)(a.out + (int64_t)t * a.out_t + (int64_t)hq * a.out_h + 2 * d) =
      make_uint2(pack2<BF16>(r[0], r[1]), pack2<BF16>(r[2], r[3]));
  if (d == 0 && a.lse) a.lse[(int64_t)t * a.Hq + hq] = lse_of(top, total);
}

template <bool BF16, int D>
hipError_t launch_join(const PagedArgs &a, const PagedPlan &plan, hipStream_t s) {
  if (plan.chunk) {
    const int slices = plan.M * (D / 4) / JOIN;
    hipLaunchKernelGGL((join_tile_kernel<BF16, D>), dim3((unsigned)(plan.tiles * slices)), dim3(JOIN), 0, s, a, plan.M, slices);
  } else {
    hipLaunchKernelGGL((join_row_kernel<BF16, D>), dim3((unsigned)((int64_t)a.T * a.Hq)), dim3(JOIN), 0, s, a, plan.M);
  }
  return hipGetLastError();
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

PagedPlan plan_paged(int32_t T, int32_t B, int32_t Hkv, int32_t G, int32_t D, int32_t max_len, bool fp8) {
  PagedPlan p{};
  const int32_t live = B < T ? (B > 0 ? B : 1) : (T > 0 ? T : 1);   // requests that can have rows
  // Rows of a request and cache head, about: tokens times query heads.  Up to 64 of them, and single tokens of up to 128
  // heads, take 16 or 32 rows to a workgroup and read the keys twice or four times, the later times out of a cache; the chunk
  // kernel, which reads them once, keeps one wave of four busy then.  us, 16 or 32 rows and chunks, 128 dims, bf16 and E4M3:
  // a token of 64 heads on 6603 keys 16, 42 and 16, 48; 64 such on 16384 133, 153 and 101, 180; 16 of 128 heads on 4096 35,
  // 40 and 35, 43; 16 times 8 tokens of 8 heads on 8192 138, 143 and 110, 172.
  // The mean decides for all requests of a call: 512 tokens of one, 32 heads on 8, beside 63 single ones on 8000 to 32000 keys
  // take 1244 us, in two calls 172 and 939; 2048 of them 2140, in two calls 588 and 939.
  const int64_t need = (int64_t)((T + live - 1) / live) * G;
  p.chunk = need > 64 && !(T == live && G <= 128);
  p.M = p.chunk ? 256 : need > 16 ? 32 : 16;
  p.Gt = G < p.M ? G : p.M;
  p.blocks = (G + p.Gt - 1) / p.Gt;
  p.R = p.M / p.Gt;
  const int64_t mu = (int64_t)Hkv * p.blocks;
  p.slots = p.chunk ? (D == 64 ? 512 : 256) : 512;
  p.min_tiles = 4;
  const int64_t divided = (T / p.R + live) * mu;      // row tiles at most
  // Requests are divided for the sake of unequal lengths; many of equal ones pay for the looking through them all.  us, divided
  // and not, 8 heads on 1, 128 dims: 128 single rows on 2000 keys each 36 and 26, on 100 to 8000 55 and 60; 512 such 120 and
  // 105, 224 and 220; 64 requests of 16 rows on 2000 56 and 69, on 100 to 8000 71 and 226; 256 such 119 and 141, 281 and 234,
  // and with one on 30000 beside shorter ones 156 and 836.  (4096 single rows on 2000: 744; 4097, not divided, 755.)
  p.divide = divided < (p.chunk ? 3 : 6) * p.slots && max_len > (p.chunk ? 512 : 256) && B <= 4096;
  if (p.divide) {
    p.tiles = divided;
    p.max_items = divided + 2 * p.slots + p.slots / 8 + mu;
    p.bytes = ((size_t)p.max_items * p.M * (D + 4) * 4 + 4 + 255) / 256 * 256;
  } else {
    p.tiles = (T / p.R + (int64_t)B) * mu;            // the numbers that tiles are looked up by
    p.max_items = p.tiles;
  }
  p.by_xcd = !p.chunk && (fp8 || p.blocks > 1);
  p.grid = p.by_xcd ? (p.max_items / mu + 8) / 8 * 8 * mu : p.max_items;
  return p;
}

hipError_t launch_paged(PagedArgs &a, int32_t dtype, int32_t fmt, int32_t D, const PagedPlan &plan, void *ws,
                        hipStream_t s) {
  if (plan.max_items <= 0) return hipSuccess;
  if (a.rows == 0) a.max_len = 0;   // no slot that could be read
  // a negative factor turns q over instead, so that the largest product comes from the largest dot
  a.q_sign = a.scale2 < 0.f ? 0x80008000u : 0u;
  // and a factor of zero zeroes q, so that the product of the mask's -inf with it stays -inf
  a.q_keep = a.scale2 == 0.f ? 0u : ~0u;
  a.scale2 = a.scale2 == 0.f ? 1.f : std::fabs(a.scale2);
  a.R = plan.R;
  a.Gt = plan.Gt;
  a.blocks = plan.blocks;
  a.divide = plan.divide;
  a.slots = plan.slots;
  a.min_tiles = plan.min_tiles;
  a.max_items = (int32_t)plan.max_items;
  a.grid = (int32_t)plan.grid;
  a.part = (float *)ws;
  a.part_ml = a.part + (size_t)plan.max_items * plan.M * D;
  a.chunk = (uint32_t *)(a.part_ml + (size_t)plan.max_items * plan.M * 4);
  const hipError_t e = plan.chunk ? launch_paged_chunk(a, dtype, fmt, D, s) : launch_paged_step(a, dtype, fmt, D, plan.M, s);
  if (e != hipSuccess || !plan.divide) return e;
  if (D == 64) return dtype == IDX_K_BF16 ? launch_join<true, 64>(a, plan, s) : launch_join<false, 64>(a, plan, s);
  return dtype == IDX_K_BF16 ? launch_join<true, 128>(a, plan, s) : launch_join<false, 128>(a, plan, s);
}

hipError_t launch_paged_check(const PagedArgs &a, uint32_t *word, hipStream_t s) {
  if (a.B <= 0) return hipSuccess;
  hipLaunchKernelGGL(check_paged_kernel, dim3((unsigned)(a.B < 1024 ? a.B : 1024)), dim3(64), 0, s, a, word);
  return hipGetLastError();
}

}  // namespace idx
