// Internal interface of the attention over a paged cache (paged.hip, paged_chunk.hip, paged_step.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/idx.h"

namespace idx {

struct PagedArgs {
  const uint8_t *q;
  int64_t q_t, q_h;          // bytes
  uint8_t *out;
  int64_t out_t, out_h;
  const uint8_t *k, *v;
  uint32_t row_bytes;        // of a slot, in both caches; a head is D values on
  const float *k_scale, *v_scale;
  int64_t scale_row;         // floats of a slot
  int64_t rows;              // slots in both caches
  const int32_t *pages;
  int64_t ld_pages;
  int32_t page_sh;           // log2 of the slots of a page
  int32_t max_len;           // keys that a row of pages has room for
  const int32_t *cu_q, *len_k;
  int32_t B, T, Hq, Hkv, G;
  int32_t window, first;
  float scale2;              // scale * log2(e); launch_paged makes it > 0 ...
  uint32_t q_sign, q_keep;   // ... and flips q's signs, or zeroes q, instead (filled there)
  float *lse;
  // Filled by launch_paged from the plan
  int32_t R;                 // tokens of a row tile
  int32_t Gt, blocks;        // query heads of a row tile, and head blocks of a cache head
  int32_t divide;            // whether keys may be divided over workgroups
  int32_t slots, min_tiles;  // ... by aiming at this many workgroups, and at least this many key tiles for each
  int32_t max_items;         // workgroups that may have work
  int32_t grid;              // ... of the launch
  float *part;               // divided items: [max_items][M][D] unnormalised out, then
  float *part_ml;            // [max_items][M][4] reference, sum, sum of the weights as rounded, nothing
  uint32_t *chunk;           // the division, for the join (0: nothing is divided)
};

// Whether the 16 keys from a multiple of 16 on follow each other in the caches, within a 32-bit offset.
inline bool has_runs(const PagedArgs &a) {
  return a.page_sh >= 4 && a.rows >> a.page_sh << a.page_sh == a.rows && (uint64_t)a.row_bytes * 16 < (1ull << 32);
}

struct PagedPlan {
  bool chunk;                // paged_chunk.hip, else paged_step.hip
  int32_t M;                 // rows (tokens x heads) of a workgroup
  int32_t R, Gt, blocks;
  int32_t divide, slots, min_tiles;
  int64_t tiles;             // row tiles of the batch at most, times cache heads and head blocks
  int64_t max_items;
  bool by_xcd;               // all cache heads of an item on one XCD
  int64_t grid;              // workgroups: max_items, with by_xcd for a multiple of 8 items
  size_t bytes;              // workspace
};
PagedPlan plan_paged(int32_t T, int32_t B, int32_t Hkv, int32_t G, int32_t D, int32_t max_len, bool fp8);
hipError_t launch_paged(PagedArgs &a, int32_t dtype, int32_t fmt, int32_t D, const PagedPlan &plan, void *ws,
                        hipStream_t s);
hipError_t launch_paged_chunk(const PagedArgs &a, int32_t dtype, int32_t fmt, int32_t D, hipStream_t s);
hipError_t launch_paged_step(const PagedArgs &a, int32_t dtype, int32_t fmt, int32_t D, int32_t M, hipStream_t s);

// Debug check: cu_q ascending within [0, T], lengths within [0, max_len], the pages that some row sees a key of inside the
// caches; else raises *word.
hipError_t launch_paged_check(const PagedArgs &a, uint32_t *word, hipStream_t s);

}  // namespace idx
