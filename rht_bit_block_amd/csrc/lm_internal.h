// Internal interface between the C ABI of the language-model operators
// (api_lm.cpp: validation, planning) and their HIP kernels (glu.hip).
// Host-visible structs only; every pointer is a device pointer.
#pragma once

#include "ufp4_internal.h"

namespace ufp4 {

struct GluLaunch {
  const void* gate;        // forward inputs, dtype, row pitch ld
  const void* up;
  int64_t ld;
  const float* row_scale;  // null: 1
  uint16_t* h;             // bf16 output (backward: recomputed), null in a backward without it
  int64_t ldh;
  uint8_t* gate_codes;     // checkpoint (forward: written or null; backward: read)
  uint8_t* gate_scales;
  uint8_t* up_codes;
  uint8_t* up_scales;
  const void* dh;          // backward input, dtype, row pitch lddh
  int64_t lddh;
  uint16_t* dgate;         // backward outputs, bf16, row pitch ldd
  uint16_t* dup;
  int64_t ldd;
  float* drow;             // backward output, null to skip
  int64_t rows, cols;
  int32_t dtype, act;
};

hipError_t launch_glu_fwd(const GluLaunch& g, hipStream_t s);
hipError_t launch_glu_bwd(const GluLaunch& g, hipStream_t s);

}  // namespace ufp4
