// C ABI of the language-model operators around the 4-bit GEMMs: argument
// validation and launch planning.  As in api.cpp every check runs before any
// HIP call, so a rejected call has no side effect and needs no GPU.
#include <cstring>

#include "../../include/ufp4.h"
#include "lm_internal.h"

using namespace ufp4;

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? UFP4_OK : UFP4_ERR_HIP; }

// rows x pitch elements of `elem` bytes must be addressable (and the sizes
// multiply without overflow).
bool sizes_ok(int64_t rows, int64_t pitch) {
  return rows >= 0 && pitch >= 0 && (pitch == 0 || rows <= ((int64_t)1 << 50) / pitch);
}

bool dtype_ok(int32_t d) { return d == UFP4_BF16 || d == UFP4_FP32; }
bool act_ok(int32_t a) { return a == UFP4_ACT_SILU || a == UFP4_ACT_GELU; }
uintptr_t elem_bytes(int32_t d) { return d == UFP4_BF16 ? 2 : 4; }

constexpr int64_t kMaxGluCols = (int64_t)1 << 30;   // a row's 8-element chunks in one launch

}  // namespace

extern "C" {

int ufp4_glu_fwd(const void* gate, const void* up, int32_t dtype, int64_t rows, int64_t cols,
                 int64_t ld, int32_t act, const float* row_scale, void* h, int64_t ldh,
                 uint8_t* gate_codes, uint8_t* gate_scales, uint8_t* up_codes,
                 uint8_t* up_scales, void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || rows < 0 || cols < 0) return UFP4_ERR_INVALID_ARG;
  if (rows > 0 && (ld < cols || ldh < cols)) return UFP4_ERR_INVALID_ARG;
  const int kept = !!gate_codes + !!gate_scales + !!up_codes + !!up_scales;
  if (rows == 0 || cols == 0) return UFP4_OK;
  if (kept != 0 && kept != 4) return UFP4_ERR_INVALID_ARG;
  if (!gate || !up || !h) return UFP4_ERR_INVALID_ARG;
  if (!sizes_ok(rows, ld) || !sizes_ok(rows, ldh)) return UFP4_ERR_INVALID_ARG;
  const uintptr_t es = elem_bytes(dtype);
  if (!aligned(gate, es) || !aligned(up, es) || !aligned(h, 2) || !aligned(row_scale, 4))
    return UFP4_ERR_INVALID_ARG;
  if (cols > kMaxGluCols) return UFP4_ERR_UNSUPPORTED;
  GluLaunch g;
  std::memset(&g, 0, sizeof(g));
  g.gate = gate;
  g.up = up;
  g.ld = ld;
  g.row_scale = row_scale;
  g.h = static_cast<uint16_t*>(h);
  g.ldh = ldh;
  g.gate_codes = gate_codes;
  g.gate_scales = gate_scales;
  g.up_codes = up_codes;
  g.up_scales = up_scales;
  g.rows = rows;
  g.cols = cols;
  g.dtype = dtype;
  g.act = act;
  return hip_status(launch_glu_fwd(g, (hipStream_t)stream));
}

int ufp4_glu_bwd(const uint8_t* gate_codes, const uint8_t* gate_scales, const uint8_t* up_codes,
                 const uint8_t* up_scales, int64_t rows, int64_t cols, int32_t act,
                 const float* row_scale, const void* dh, int32_t dtype, int64_t lddh, void* dgate,
                 void* dup, int64_t ldd, float* drow_scale, void* h, int64_t ldh, void* stream) {
  if (!dtype_ok(dtype) || !act_ok(act) || rows < 0 || cols < 0) return UFP4_ERR_INVALID_ARG;
  if (rows > 0 && (lddh < cols || ldd < cols || (h && ldh < cols))) return UFP4_ERR_INVALID_ARG;
  if (drow_scale && !row_scale) return UFP4_ERR_INVALID_ARG;
  if (rows == 0 || (cols == 0 && !drow_scale)) return UFP4_OK;
  if (!aligned(row_scale, 4) || !aligned(drow_scale, 4)) return UFP4_ERR_INVALID_ARG;
  if (cols > 0) {   // an empty row still has a gradient of its factor: zero
    if (!gate_codes || !gate_scales || !up_codes || !up_scales || !dh || !dgate || !dup)
      return UFP4_ERR_INVALID_ARG;
    if (!sizes_ok(rows, lddh) || !sizes_ok(rows, ldd) || (h && !sizes_ok(rows, ldh)))
      return UFP4_ERR_INVALID_ARG;
    if (!aligned(dh, elem_bytes(dtype)) || !aligned(dgate, 2) || !aligned(dup, 2) || !aligned(h, 2))
      return UFP4_ERR_INVALID_ARG;
    if (cols > kMaxGluCols) return UFP4_ERR_UNSUPPORTED;
  } else if (rows > ((int64_t)1 << 50)) {
    return UFP4_ERR_INVALID_ARG;
  }
  GluLaunch g;
  std::memset(&g, 0, sizeof(g));
  g.row_scale = row_scale;
  g.h = static_cast<uint16_t*>(h);
  g.ldh = ldh;
  g.gate_codes = const_cast<uint8_t*>(gate_codes);
  g.gate_scales = const_cast<uint8_t*>(gate_scales);
  g.up_codes = const_cast<uint8_t*>(up_codes);
  g.up_scales = const_cast<uint8_t*>(up_scales);
  g.dh = dh;
  g.lddh = lddh;
  g.dgate = static_cast<uint16_t*>(dgate);
  g.dup = static_cast<uint16_t*>(dup);
  g.ldd = ldd;
  g.drow = drow_scale;
  g.rows = rows;
  g.cols = cols;
  g.dtype = dtype;
  g.act = act;
  return hip_status(launch_glu_bwd(g, (hipStream_t)stream));
}

}  // extern "C"
