// Internal interface of the row kernels (rows.hip): rotary positions, cache writes and reads.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/idx.h"

namespace idx {

// One array of rows through the write kernel.  Strides are bytes.
struct RowJob {
  const uint8_t *x;
  int64_t x_t, x_h;
  uint8_t *out;
  int64_t out_t, out_h;    // of a slot and of a head
  uint8_t *scale;
  int64_t scale_t, scale_h;
  const int32_t *slot;     // nullable: row t goes to slot t
  int64_t rows;            // slots (rows outside are dropped)
  const double *freq;      // nullable: no rotation
  const int32_t *pos;
  double mscale;
  int32_t T, H, D;
  int32_t rot, rot0;
  int32_t dtype, fmt;
  int32_t half, inverse;
  int32_t lanes_sh;        // log2 of the lanes of a row: the power of two at or above D / 8
  int32_t groups;          // lane groups of a token, each taking every groups-th head
};

struct RowJobs {
  RowJob job[IDX_MAX_WRITES];
  int32_t first[IDX_MAX_WRITES + 1];   // first workgroup of each job
  int32_t n;
};

// Fills the launch layout (lanes_sh, groups, first) and launches every job.
hipError_t launch_rows(RowJobs &jobs, hipStream_t s);

struct ReadJob {
  const uint8_t *data;
  int64_t data_t, data_h;  // bytes of a slot and of a head
  const uint8_t *scale;
  int64_t scale_t, scale_h;
  int64_t rows;
  const int32_t *list;     // nullable: out row t reads slot t
  uint8_t *out;
  int64_t out_t, out_h;
  int32_t T, H, D;
  int32_t fmt, dtype;
  int32_t lanes_sh;        // filled by launch_read
};
hipError_t launch_read(ReadJob &j, hipStream_t s);

// Debug check of slot lists: a slot inside [0, rows) named twice raises *word.
hipError_t launch_slot_check(const int32_t *slot, int32_t T, int64_t rows, uint32_t *word, hipStream_t s);

}  // namespace idx
