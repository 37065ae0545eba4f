// Internal interface between the C ABI of the language-model operators
// (api_lm.cpp: validation, planning) and their HIP kernels (glu.hip, xent.hip).
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

struct XentLaunch {
  const uint16_t* h;       // bf16 [T][ldh]
  const uint16_t* w;       // bf16 [V][ldw]
  const int64_t* targets;  // [T]; outside 0 .. V-1: no class
  int64_t T, V, D, ldh, ldw;
  float* loss;             // forward outputs [T]
  float* lse_out;
  const float* lse;        // backward inputs [T]
  const float* dloss;
  const float* dlse;       // or null
  uint16_t* dh;            // backward outputs, bf16 [T][lddh], [V][lddw]
  uint16_t* dw;
  int64_t lddh, lddw;
  uint8_t* ws;
};

// Workspace of both directions and how the backward pass cuts the vocabulary.
struct XentPlan {
  int64_t parts;                 // statistics per token in the forward pass
  int64_t fwd_bytes, bwd_bytes;
  int64_t piece, pieces;         // classes per piece (a multiple of 256), pieces
  int64_t Tp;                    // tokens rounded up to 64
  int32_t splits;                // of the dh product's K
  int64_t g, gt, wt, ht, slab;   // offsets of the backward workspace's parts
};
XentPlan xent_plan(int64_t T, int64_t V, int64_t D);
hipError_t launch_xent_fwd(const XentLaunch& x, hipStream_t s);
hipError_t launch_xent_bwd(const XentLaunch& x, hipStream_t s);

}  // namespace ufp4
