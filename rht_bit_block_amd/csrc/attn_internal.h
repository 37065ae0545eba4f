// Internal interface between the C ABI of the attention operators
// (api_attn.cpp: validation, planning) and their HIP kernels (attn.hip,
// attn_grad.hip, kv_attn.hip, kv_rows.h).  Host-visible structs only; every
// pointer is a device pointer.
#pragma once

#include "lm_internal.h"

namespace ufp4 {

constexpr int kAttnTile = 128;                       // queries (or keys) of a workgroup
// Workgroups of four waves that the chip holds at once: launches of no more take eight waves
// each (see in_parts).
constexpr int64_t kInParts = 512;
constexpr int64_t kAttnMaxRows = (int64_t)1 << 30, kAttnMaxSeqs = (int64_t)1 << 20;
constexpr int64_t kAttnMaxPitch = (int64_t)1 << 22;  // 32-bit offsets inside a tile of 128 rows
constexpr int kAttnMaxHeads = 1024, kAttnMaxWidth = 128;

struct AttnLaunch {
  const uint16_t* q;       // bf16 [T][ldq], head h at h D
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* starts;   // [B + 1]
  int64_t ldq, ldk, ldv, ldo;
  uint16_t* o;             // written forward, read backward
  float* lse;              // [T][heads]; null: not wanted
  const uint16_t* dout;    // backward
  int64_t lddo, lddq, lddk, lddv;
  uint16_t* dq;
  uint16_t* dk;
  uint16_t* dv;
  float* lw;               // workspace: lse log2(e), [heads][T]
  float* delta;            // workspace: do . o, [heads][T]
  int64_t T;
  int32_t B, heads, kv_heads, group, D;
  FastDiv by_heads, by_kv_heads;
  float scale;
};
int64_t attn_workspace(int64_t T, int32_t heads);
hipError_t launch_attn_fwd(const AttnLaunch& p, hipStream_t s);
hipError_t launch_attn_bwd(const AttnLaunch& p, hipStream_t s);

// Where a cache's tokens lie.
struct KvPlace {
  const int32_t* starts;   // [B + 1]
  const int32_t* lens;     // [B]
  const int32_t* table;    // [B][ldt]
  int64_t ldt, width, T, pages;
  int32_t B, page_shift, kv_heads, D;
};

struct KvRows {            // write and read
  KvPlace at;
  uint16_t* k;             // bf16 [T][ldk] (read by a write)
  uint16_t* v;
  int64_t ldk, ldv, t0;    // t0: first row of a launch
  uint8_t* codes[2];       // of k, v
  void* scales[2];
  uint32_t sign_pat[4];    // as QuantLaunch
  float cn;
  int32_t n, grid, scale_mode, bc;
  int32_t items;           // heads of k and v that a lane takes one after another (set by the launcher)
  // what the quantizer's lane function asks of its launch
  float* rotated;          // null
  float tmul;              // 1
  uint64_t sr_seed;
  uint32_t sr_stream;
};
hipError_t launch_kv_write(const KvRows& p, hipStream_t s);
hipError_t launch_kv_read(const KvRows& p, hipStream_t s);

constexpr int kKvGroups = 512;   // workgroups of the attention over a cache: two per compute unit
struct KvAttn {
  KvPlace at;
  const uint16_t* q;
  uint16_t* o;
  int64_t ldq, ldo;
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  uint32_t sign[4];        // of 128 consecutive elements
  float cn, scale;
  int32_t n, grid, kind;   // kind: 0 fp32 / 32, 1 fp32 / 16, 2 E8M0 / 32
  int32_t heads, group, rows16;   // rows16: 16-row tiles that a workgroup takes at once
  float* partial;          // [2 kKvGroups][16 rows16][D + 2]
};
int32_t kv_attn_rows16(int64_t T, int32_t B, int32_t group);
int64_t kv_attn_workspace(int64_t T, int32_t B, int32_t heads, int32_t kv_heads, int32_t D);
hipError_t launch_kv_attn(const KvAttn& p, hipStream_t s);

}  // namespace ufp4
