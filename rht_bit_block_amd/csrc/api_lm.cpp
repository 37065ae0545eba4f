// C ABI of the language-model operators around the 4-bit GEMMs: argument
// validation and launch planning.  As in api.cpp every check runs before any
// HIP call, so a rejected call has no side effect and needs no GPU.
#include <cmath>
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

// Sizes of a linear cross entropy: 32-bit offsets inside a 256-row tile bound T
// (a pitch of the turned operands) and D, 2^22 tiles of classes V, and as many
// tiles of dh T D (512 GiB of h).
int xent_sizes(int64_t T, int64_t V, int64_t D) {
  if (T < 0 || V < 1 || D < 1) return UFP4_ERR_INVALID_ARG;
  if (D % 8) return UFP4_ERR_SHAPE;
  if (T > ((int64_t)1 << 21) || V > ((int64_t)1 << 30) || D > ((int64_t)1 << 20) ||
      T * D > ((int64_t)1 << 38))
    return UFP4_ERR_UNSUPPORTED;
  return UFP4_OK;
}

int xent_matrix(const void* p, int64_t ld, int64_t cols) {
  if (!p || ld < cols || ld % 8 || !aligned(p, 16)) return UFP4_ERR_INVALID_ARG;
  return ld > ((int64_t)1 << 20) ? UFP4_ERR_UNSUPPORTED : UFP4_OK;
}

int moe_sizes(int64_t T, int64_t E, int64_t k, int64_t H, int64_t F) {
  if (T < 0 || E < 1 || k < 1 || k > E || H < 1 || F < 1) return UFP4_ERR_INVALID_ARG;
  if (H % 32 || F % 32) return UFP4_ERR_SHAPE;
  if (T > kMoeMaxTokens || E > kMoeMaxExperts || k > kMoeMaxChoices || H > kMoeMaxWidth ||
      F > kMoeMaxWidth)
    return UFP4_ERR_UNSUPPORTED;
  return UFP4_OK;
}

MoeWeight moe_weight(const ufp4_qtensor* t) {
  MoeWeight w;
  w.codes = t->codes;
  w.scales = static_cast<const uint8_t*>(t->scales);
  const bool e8 = t->cfg.scale_mode == UFP4_SCALE_POW2;
  w.scale_pitch = t->K / t->cfg.block_cols * (e8 ? 1 : 4);
  w.row_shift = t->cfg.block_rows == 32 ? 5 : t->cfg.block_rows == 16 ? 4 : 0;
  w.grid = t->cfg.grid;
  w.kind = (e8 ? 2 : 0) + (t->cfg.block_cols == 16 ? 1 : 0);
  w.factor = t->cfg.tensor_scale != 0.0f ? t->cfg.tensor_scale : 1.0f;
  return w;
}

}  // namespace

extern "C" {

size_t ufp4_moe_tokens_workspace_bytes(int64_t T, int32_t E, int32_t top_k, int64_t H, int64_t F) {
  if (moe_sizes(T, E, top_k, H, F) || T == 0) return 0;
  MoeLaunch p;
  std::memset(&p, 0, sizeof(p));
  p.T = T;
  p.E = E;
  p.k = top_k;
  p.H = H;
  p.F = F;
  return (size_t)moe_plan(p, nullptr);
}

int ufp4_moe_tokens(const void* x, int64_t ldx, int64_t T, const float* logits, int64_t ldl,
                    int32_t E, int32_t top_k, int32_t renorm, int32_t act, const ufp4_qtensor* Wg,
                    const ufp4_qtensor* Wu, const ufp4_qtensor* Wd, void* y, int64_t ldy,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!act_ok(act) || !Wg || !Wu || !Wd || E < 1) return UFP4_ERR_INVALID_ARG;
  int st;
  if ((st = check_operand(Wg)) || (st = check_operand(Wu)) || (st = check_operand(Wd))) return st;
  if (Wg->P % E || Wd->P % E) return UFP4_ERR_SHAPE;
  const int64_t H = Wg->K, F = Wg->P / E;
  if ((st = moe_sizes(T, E, top_k, H, F))) return st;
  const ufp4_quant_cfg &a = Wg->cfg, &b = Wu->cfg;
  if (Wu->K != H || a.grid != b.grid || a.scale_mode != b.scale_mode ||
      a.block_rows != b.block_rows || a.block_cols != b.block_cols || a.rht_n != b.rht_n ||
      (a.rht_n > 1 && a.sign_seed != b.sign_seed))
    return UFP4_ERR_MISMATCH;
  if (Wu->P != Wg->P || Wd->P != E * H || Wd->K != F) return UFP4_ERR_SHAPE;
  if (a.grid == UFP4_E4M3 || Wd->cfg.grid == UFP4_E4M3) return UFP4_ERR_UNSUPPORTED;
  if (T == 0) return UFP4_OK;
  if (!x || !logits || !y || !workspace) return UFP4_ERR_INVALID_ARG;
  if (ldx < H || ldx % 8 || ldl < E || ldy < H || ldy % 2) return UFP4_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(logits, 4) || !aligned(y, 4) || !aligned(workspace, 256) ||
      !aligned(Wg->codes, 16) || !aligned(Wu->codes, 16) || !aligned(Wd->codes, 16))
    return UFP4_ERR_INVALID_ARG;
  if (workspace_bytes < ufp4_moe_tokens_workspace_bytes(T, E, top_k, H, F))
    return UFP4_ERR_INVALID_ARG;
  MoeLaunch p;
  std::memset(&p, 0, sizeof(p));
  p.x = static_cast<const uint16_t*>(x);
  p.logits = logits;
  p.y = static_cast<uint16_t*>(y);
  p.ldx = ldx;
  p.ldl = ldl;
  p.ldy = ldy;
  p.T = T;
  p.H = H;
  p.F = F;
  p.E = E;
  p.k = top_k;
  p.renorm = renorm != 0;
  p.act = act;
  p.wg = moe_weight(Wg);
  p.wu = moe_weight(Wu);
  p.wd = moe_weight(Wd);
  p.nx = a.rht_n;
  p.nh = Wd->cfg.rht_n;
  p.cnx = (float)(1.0 / std::sqrt((double)p.nx));   // as the quantizer's c_n
  p.cnh = (float)(1.0 / std::sqrt((double)p.nh));
  sign_bits128(&a, p.sign_x);
  sign_bits128(&Wd->cfg, p.sign_h);
  moe_plan(p, static_cast<uint8_t*>(workspace));
  return hip_status(launch_moe_tokens(p, (hipStream_t)stream));
}

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
