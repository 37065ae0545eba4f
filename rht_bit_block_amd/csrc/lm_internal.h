// Internal interface between the C ABI of the language-model operators
// (api_lm.cpp: validation, planning) and their HIP kernels (glu.hip, xent.hip,
// moe_tokens.hip).
// Host-visible structs only; every pointer is a device pointer.
#pragma once

#include "ufp4_internal.h"

namespace ufp4 {

// Checks of a quantized operand shared by every entry point that takes one
// (sizes, configuration, storage, alignment); UFP4_OK or a status (api.cpp).
int check_operand(const ufp4_qtensor* t);
// The sign bits of 128 consecutive elements that start a chunk (the n-bit
// pattern of the configuration's seed, repeated), bit i of word i / 32 (api.cpp).
void sign_bits128(const ufp4_quant_cfg* c, uint32_t out[4]);

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
  int64_t Tp;                    // tokens rounded up to 8
  int32_t splits;                // of the dh product's K
  int64_t g, gt, wt, ht, slab, scale;   // offsets of the backward workspace's parts
};
XentPlan xent_plan(int64_t T, int64_t V, int64_t D);
hipError_t launch_xent_fwd(const XentLaunch& x, hipStream_t s);
hipError_t launch_xent_bwd(const XentLaunch& x, hipStream_t s);

constexpr int kMoeMaxTokens = 64, kMoeMaxExperts = 256, kMoeMaxChoices = 16;
constexpr int64_t kMoeMaxWidth = 1 << 20;   // 32-bit offsets inside a 16-row tile and x
// Up to here the up product's workgroups route and rotate x themselves.
constexpr int kMoeFusedTokens = 8;

// One expert matrix, stacked over the experts: codes of row r at r K / 2,
// scales of row r at (r >> row_shift) * scale_pitch bytes.
struct MoeWeight {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t scale_pitch;
  int32_t row_shift;
  int32_t grid;
  int32_t kind;      // 0 fp32 / 32, 1 fp32 / 16, 2 E8M0 / 32, 3 E8M0 / 16
  float factor;      // per-tensor factor of two-level scaling, else 1
};

struct MoeLaunch {
  const uint16_t* x;       // bf16 [T][ldx]
  const float* logits;     // [T][ldl]
  uint16_t* y;             // bf16 [T][ldy]
  int64_t ldx, ldl, ldy;
  int64_t T, H, F;
  int32_t E, k, renorm, act;
  MoeWeight wg, wu, wd;
  int32_t nx, nh;          // rotation of x and of the intermediate
  float cnx, cnh;
  uint32_t sign_x[4], sign_h[4];   // sign bits of 128 consecutive elements
  // set by moe_plan
  int32_t by_pair, fused, slots;   // slots: the T k choices, or all experts if fewer
  int32_t run_up, run_down;        // pairs of tiles per workgroup of the two products
  int* ids;                // [T][k] chosen experts, -1: none
  float* share;            // [T][k]
  int* expert;             // [slots] a slot's expert
  int* count;              // [slots] its tokens
  int* row0;               // [slots] first row of its tokens in h and partial
  int* place;              // [T][k] row of a choice, -1: none
  uint8_t* xr;             // rotated x: [T][H], 4 bytes an element
  float* h;                // weighted intermediate: [T k][F], by experts
  float* partial;          // down products: [T k][H]
};

// Fills the plan and returns the workspace's size in bytes (ws may be null).
int64_t moe_plan(MoeLaunch& p, uint8_t* ws);
hipError_t launch_moe_tokens(const MoeLaunch& p, hipStream_t s);

}  // namespace ufp4
