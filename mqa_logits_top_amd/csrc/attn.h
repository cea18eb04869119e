// Internal interface of the attention over selected keys (attn.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/idx.h"

namespace idx {

struct AttnArgs {
  const uint8_t *q;
  int64_t q_t, q_h;          // bytes
  uint8_t *out;
  int64_t out_t, out_h;
  const uint8_t *k, *v;
  uint32_t row_bytes;        // of a slot, in both caches; a head is D values on
  const float *k_scale, *v_scale;
  int64_t scale_row;         // floats of a slot
  int64_t rows;              // slots in both caches
  const int32_t *sel;
  int64_t ld_sel;
  int32_t n_sel, pool_sh;
  const int32_t *ks, *ke;
  const int32_t *table;
  int32_t L;
  int32_t T, Hq, Hkv, G;
  float scale2;              // scale * log2(e); launch_attn makes it > 0 ...
  uint32_t q_sign, q_keep;   // ... and flips q's signs, or zeroes q, instead (filled there)
  float *lse;
  int32_t blocks;            // head blocks of a cache head's G query heads
  int32_t splits;            // workgroups a row's entries are divided over
  int32_t waves;             // waves of a workgroup, over which its share is divided
  int64_t per;               // entries of a wave
  // splits > 1: per (row, cache head, head block, split) the unnormalised out of the split's
  // heads [heads][D], then all their (reference, sum, divisor, 0)
  float *part;
  float *part_ml;
};

struct AttnPlan {
  int32_t tiles;             // 16-head tiles a wave holds: 1 or 2
  int32_t blocks;
  int32_t splits, waves;
  int64_t per;
  size_t bytes;              // workspace
};
// entries: of a list; touched: bytes of the caches that the lists can name at most
AttnPlan plan_attn(int32_t T, int32_t Hkv, int32_t G, int32_t D, bool fp8, int64_t entries, int64_t touched);
hipError_t launch_attn(AttnArgs &a, int32_t dtype, int32_t fmt, int32_t D, const AttnPlan &plan, void *ws,
                       hipStream_t s);

}  // namespace idx
