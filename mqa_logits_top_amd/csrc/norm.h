// Internal interface of the RMS norm (norm.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/idx.h"

namespace idx {

// A row array; strides are bytes.  p null: absent.
struct NormRows {
  uint8_t *p;
  int64_t t, h;
  int32_t dtype;
};

struct NormJob {
  NormRows x, residual, total, out;
  uint8_t *codes;          // null: none
  int64_t codes_t, codes_h;
  float *scale;
  int64_t scale_t;         // floats
  const uint8_t *weight;   // null: ones
  int32_t weight_dtype;
  int32_t group;           // values that share a scale
  int32_t T, H, D;
  float eps;
  int32_t lanes_sh;        // log2 of the lanes of a row of up to 512 values; filled by launch_norm
  int32_t group_sh;        // ... of the lanes of a group
};
hipError_t launch_norm(NormJob &j, hipStream_t s);

}  // namespace idx
