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

// Sizes of a linear cross entropy: 32-bit offsets inside a 256-row tile and
// grids of a launch bound them.
int xent_sizes(int64_t T, int64_t V, int64_t D) {
  if (T < 0 || V < 1 || D < 1) return UFP4_ERR_INVALID_ARG;
  if (D % 8) return UFP4_ERR_SHAPE;
  if (T > ((int64_t)1 << 21) || V > ((int64_t)1 << 30) || D > ((int64_t)1 << 20))
    return UFP4_ERR_UNSUPPORTED;
  return UFP4_OK;
}

int xent_matrix(const void* p, int64_t ld, int64_t cols) {
  if (!p || ld < cols || ld % 8 || !aligned(p, 16)) return UFP4_ERR_INVALID_ARG;
  return ld > ((int64_t)1 << 20) ? UFP4_ERR_UNSUPPORTED : UFP4_OK;
}

}  // namespace

extern "C" {

size_t ufp4_linear_xent_workspace_bytes(int64_t T, int64_t V, int64_t D, int32_t backward) {
  if (xent_sizes(T, V, D) || T == 0) return 0;
  const XentPlan p = xent_plan(T, V, D);
  return (size_t)(backward ? p.bwd_bytes : p.fwd_bytes);
}

int ufp4_linear_xent_fwd(const void* h, int64_t ldh, const void* w, int64_t ldw,
                         const int64_t* targets, int64_t T, int64_t V, int64_t D, float* loss,
                         float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  int st = xent_sizes(T, V, D);
  if (st) return st;
  if (T == 0) return UFP4_OK;
  if ((st = xent_matrix(h, ldh, D)) || (st = xent_matrix(w, ldw, D))) return st;
  if (!targets || !loss || !lse || !workspace) return UFP4_ERR_INVALID_ARG;
  if (!aligned(targets, 8) || !aligned(loss, 4) || !aligned(lse, 4) || !aligned(workspace, 256))
    return UFP4_ERR_INVALID_ARG;
  if (workspace_bytes < ufp4_linear_xent_workspace_bytes(T, V, D, 0)) return UFP4_ERR_INVALID_ARG;
  XentLaunch x;
  std::memset(&x, 0, sizeof(x));
  x.h = static_cast<const uint16_t*>(h);
  x.w = static_cast<const uint16_t*>(w);
  x.targets = targets;
  x.T = T;
  x.V = V;
  x.D = D;
  x.ldh = ldh;
  x.ldw = ldw;
  x.loss = loss;
  x.lse_out = lse;
  x.ws = static_cast<uint8_t*>(workspace);
  return hip_status(launch_xent_fwd(x, (hipStream_t)stream));
}

int ufp4_linear_xent_bwd(const void* h, int64_t ldh, const void* w, int64_t ldw,
                         const int64_t* targets, int64_t T, int64_t V, int64_t D, const float* lse,
                         const float* dloss, const float* dlse, void* dh, int64_t lddh, void* dw,
                         int64_t lddw, void* workspace, size_t workspace_bytes, void* stream) {
  int st = xent_sizes(T, V, D);
  if (st) return st;
  if ((st = xent_matrix(dw, lddw, D))) return st;
  if (T > 0) {
    if ((st = xent_matrix(h, ldh, D)) || (st = xent_matrix(w, ldw, D)) ||
        (st = xent_matrix(dh, lddh, D)))
      return st;
    if (!targets || !lse || !dloss || !workspace) return UFP4_ERR_INVALID_ARG;
    if (!aligned(targets, 8) || !aligned(lse, 4) || !aligned(dloss, 4) || !aligned(dlse, 4) ||
        !aligned(workspace, 256))
      return UFP4_ERR_INVALID_ARG;
    if (workspace_bytes < ufp4_linear_xent_workspace_bytes(T, V, D, 1))
      return UFP4_ERR_INVALID_ARG;
  }
  XentLaunch x;
  std::memset(&x, 0, sizeof(x));
  x.h = static_cast<const uint16_t*>(h);
  x.w = static_cast<const uint16_t*>(w);
  x.targets = targets;
  x.T = T;
  x.V = V;
  x.D = D;
  x.ldh = ldh;
  x.ldw = ldw;
  x.lse = lse;
  x.dloss = dloss;
  x.dlse = dlse;
  x.dh = static_cast<uint16_t*>(dh);
  x.dw = static_cast<uint16_t*>(dw);
  x.lddh = lddh;
  x.lddw = lddw;
  x.ws = static_cast<uint8_t*>(workspace);
  return hip_status(launch_xent_bwd(x, (hipStream_t)stream));
}

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
