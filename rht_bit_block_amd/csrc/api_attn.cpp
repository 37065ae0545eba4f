// C ABI of the attention operators: argument validation and launch planning.
// As in api.cpp every check runs before any HIP call, so a rejected call has no
// side effect and needs no GPU.
#include <cmath>
#include <cstring>

#include "../../include/ufp4.h"
#include "attn_internal.h"

using namespace ufp4;

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? UFP4_OK : UFP4_ERR_HIP; }

// The kernels compute powers of 2: a factor of the scores has to be finite times log2(e) as well.
bool factor_ok(float scale) { return std::isfinite(scale * 1.4426950408889634f); }

// Sizes of packed rows with heads.
int packed_sizes(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t D) {
  if (T < 0 || B < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads || D < 1)
    return UFP4_ERR_INVALID_ARG;
  if (D % 8) return UFP4_ERR_SHAPE;
  if (D > kAttnMaxWidth || T > kAttnMaxRows || B > kAttnMaxSeqs || heads > kAttnMaxHeads)
    return UFP4_ERR_UNSUPPORTED;
  return UFP4_OK;
}

// A bf16 tensor of rows with `heads` heads.
int rows_of(const void* p, int64_t ld, int64_t heads, int64_t D) {
  if (!p || ld < heads * D || ld % 8 || !aligned(p, 16)) return UFP4_ERR_INVALID_ARG;
  return ld > kAttnMaxPitch ? UFP4_ERR_UNSUPPORTED : UFP4_OK;
}

int attn_inputs(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                const int32_t* starts, int32_t heads, int32_t kv_heads, int32_t D, float scale) {
  int st;
  if ((st = rows_of(q, ldq, heads, D)) || (st = rows_of(k, ldk, kv_heads, D)) ||
      (st = rows_of(v, ldv, kv_heads, D)))
    return st;
  if (!starts || !aligned(starts, 4) || !factor_ok(scale)) return UFP4_ERR_INVALID_ARG;
  return UFP4_OK;
}

void attn_fill(AttnLaunch& p, const void* q, int64_t ldq, const void* k, int64_t ldk,
               const void* v, int64_t ldv, const int32_t* starts, int32_t B, int64_t T,
               int32_t heads, int32_t kv_heads, int32_t D, float scale) {
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.ldq = ldq;
  p.ldk = ldk;
  p.ldv = ldv;
  p.starts = starts;
  p.B = B;
  p.T = T;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.group = heads / kv_heads;
  p.D = D;
  p.by_heads = make_fastdiv((uint32_t)heads);
  p.by_kv_heads = make_fastdiv((uint32_t)kv_heads);
  p.scale = scale;
}

bool page_ok(int32_t n) { return n > 0 && n <= (1 << 16) && (n & (n - 1)) == 0; }

// A cache and where its tokens lie; everything but the rows themselves.
int cache_inputs(const ufp4_kv_cache* c, const int32_t* starts, int64_t B, int64_t T,
                 const int32_t* lens, const int32_t* table, int64_t ldt, int64_t width) {
  if (!c || T < 0 || B < 0 || width < 0 || c->pages < 0 || c->kv_heads < 1 || c->D < 1 ||
      !page_ok(c->page_tokens))
    return UFP4_ERR_INVALID_ARG;
  // the configuration's own rules, on an operand without rows
  ufp4_qtensor t;
  std::memset(&t, 0, sizeof(t));
  t.K = c->D;
  t.cfg = c->cfg;
  const int st = check_operand(&t);
  if (st) return st;
  if (c->cfg.grid == UFP4_E4M3 || c->cfg.block_rows != 1 || c->cfg.rounding != UFP4_RTNE ||
      c->cfg.tensor_scale != 0.0f)
    return UFP4_ERR_UNSUPPORTED;
  if (c->D > kAttnMaxWidth || T > kAttnMaxRows || B > kAttnMaxSeqs || width > kAttnMaxPitch ||
      ldt > kAttnMaxPitch || c->kv_heads > kAttnMaxHeads || c->pages > ((int64_t)1 << 31) - 1)
    return UFP4_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return UFP4_OK;
  if (!starts || !lens || !aligned(starts, 4) || !aligned(lens, 4) || !aligned(table, 4) ||
      (width > 0 && !table) || (B > 1 && ldt < width))
    return UFP4_ERR_INVALID_ARG;
  if (c->pages > 0 && (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales))
    return UFP4_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) ||
      !aligned(c->v_scales, 16))
    return UFP4_ERR_INVALID_ARG;
  return UFP4_OK;
}

KvPlace place(const ufp4_kv_cache* c, const int32_t* starts, int32_t B, int64_t T,
              const int32_t* lens, const int32_t* table, int64_t ldt, int64_t width) {
  KvPlace a;
  std::memset(&a, 0, sizeof(a));
  a.starts = starts;
  a.lens = lens;
  a.table = table;
  a.ldt = ldt;
  a.width = width;
  a.T = T;
  a.pages = c->pages;
  a.B = B;
  while ((1 << a.page_shift) < c->page_tokens) ++a.page_shift;
  a.kv_heads = c->kv_heads;
  a.D = c->D;
  return a;
}

KvRows rows_launch(const ufp4_kv_cache* c, const KvPlace& at, const void* k, int64_t ldk,
                   const void* v, int64_t ldv) {
  KvRows p;
  std::memset(&p, 0, sizeof(p));
  p.at = at;
  p.k = static_cast<uint16_t*>(const_cast<void*>(k));
  p.v = static_cast<uint16_t*>(const_cast<void*>(v));
  p.ldk = ldk;
  p.ldv = ldv;
  p.codes[0] = c->k_codes;
  p.codes[1] = c->v_codes;
  p.scales[0] = c->k_scales;
  p.scales[1] = c->v_scales;
  // a lane's 16 or 32 elements carry the signs of their places in the chunk: words
  // 0 .. 3 of the n-periodic pattern; for n <= 32 they are all alike
  sign_bits128(&c->cfg, p.sign_pat);
  p.cn = (float)(1.0 / std::sqrt((double)c->cfg.rht_n));
  p.n = c->cfg.rht_n;
  p.grid = c->cfg.grid;
  p.scale_mode = c->cfg.scale_mode;
  p.bc = c->cfg.block_cols;
  p.tmul = 1.0f;
  return p;
}

}  // namespace

extern "C" {

size_t ufp4_attn_workspace_bytes(int64_t T, int32_t heads) {
  if (T <= 0 || packed_sizes(T, 1, heads, heads, 8)) return 0;
  return (size_t)attn_workspace(T, heads);
}

int ufp4_attn_fwd(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                  int64_t ldv, const int32_t* starts, int32_t B, int64_t T, int32_t heads,
                  int32_t kv_heads, int32_t D, float scale, void* o, int64_t ldo, float* lse,
                  void* stream) {
  int st = packed_sizes(T, B, heads, kv_heads, D);
  if (st) return st;
  if (T == 0 || B == 0) return UFP4_OK;
  if ((st = attn_inputs(q, ldq, k, ldk, v, ldv, starts, heads, kv_heads, D, scale)) ||
      (st = rows_of(o, ldo, heads, D)))
    return st;
  if (!aligned(lse, 4)) return UFP4_ERR_INVALID_ARG;
  AttnLaunch p;
  attn_fill(p, q, ldq, k, ldk, v, ldv, starts, B, T, heads, kv_heads, D, scale);
  p.o = static_cast<uint16_t*>(o);
  p.ldo = ldo;
  p.lse = lse;
  return hip_status(launch_attn_fwd(p, (hipStream_t)stream));
}

int ufp4_attn_bwd(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                  int64_t ldv, const int32_t* starts, int32_t B, int64_t T, int32_t heads,
                  int32_t kv_heads, int32_t D, float scale, const void* o, int64_t ldo,
                  const float* lse, const void* dout, int64_t lddo, void* dq, int64_t lddq,
                  void* dk, int64_t lddk, void* dv, int64_t lddv, void* workspace,
                  size_t workspace_bytes, void* stream) {
  int st = packed_sizes(T, B, heads, kv_heads, D);
  if (st) return st;
  if (T == 0 || B == 0) return UFP4_OK;
  if ((st = attn_inputs(q, ldq, k, ldk, v, ldv, starts, heads, kv_heads, D, scale)) ||
      (st = rows_of(o, ldo, heads, D)) || (st = rows_of(dout, lddo, heads, D)) ||
      (st = rows_of(dq, lddq, heads, D)) || (st = rows_of(dk, lddk, kv_heads, D)) ||
      (st = rows_of(dv, lddv, kv_heads, D)))
    return st;
  if (!lse || !aligned(lse, 4) || !workspace || !aligned(workspace, 256) ||
      workspace_bytes < ufp4_attn_workspace_bytes(T, heads))
    return UFP4_ERR_INVALID_ARG;
  AttnLaunch p;
  attn_fill(p, q, ldq, k, ldk, v, ldv, starts, B, T, heads, kv_heads, D, scale);
  p.o = static_cast<uint16_t*>(const_cast<void*>(o));
  p.ldo = ldo;
  p.lse = const_cast<float*>(lse);
  p.dout = static_cast<const uint16_t*>(dout);
  p.lddo = lddo;
  p.dq = static_cast<uint16_t*>(dq);
  p.dk = static_cast<uint16_t*>(dk);
  p.dv = static_cast<uint16_t*>(dv);
  p.lddq = lddq;
  p.lddk = lddk;
  p.lddv = lddv;
  p.lw = static_cast<float*>(workspace);
  p.delta = p.lw + (int64_t)heads * T;
  return hip_status(launch_attn_bwd(p, (hipStream_t)stream));
}

int ufp4_kv_write(const void* k, int64_t ldk, const void* v, int64_t ldv, const int32_t* starts,
                  int32_t B, int64_t T, const int32_t* lens, const int32_t* table, int64_t ldt,
                  int64_t width, const ufp4_kv_cache* cache, void* stream) {
  int st = cache_inputs(cache, starts, B, T, lens, table, ldt, width);
  if (st) return st;
  if (T == 0 || B == 0) return UFP4_OK;
  if ((st = rows_of(k, ldk, cache->kv_heads, cache->D)) ||
      (st = rows_of(v, ldv, cache->kv_heads, cache->D)))
    return st;
  const KvPlace at = place(cache, starts, B, T, lens, table, ldt, width);
  return hip_status(launch_kv_write(rows_launch(cache, at, k, ldk, v, ldv), (hipStream_t)stream));
}

int ufp4_kv_read(const ufp4_kv_cache* cache, const int32_t* starts, int32_t B, int64_t T,
                 const int32_t* lens, const int32_t* table, int64_t ldt, int64_t width, void* k,
                 int64_t ldk, void* v, int64_t ldv, void* stream) {
  int st = cache_inputs(cache, starts, B, T, lens, table, ldt, width);
  if (st) return st;
  if (T == 0 || B == 0) return UFP4_OK;
  if ((st = rows_of(k, ldk, cache->kv_heads, cache->D)) ||
      (st = rows_of(v, ldv, cache->kv_heads, cache->D)))
    return st;
  const KvPlace at = place(cache, starts, B, T, lens, table, ldt, width);
  return hip_status(launch_kv_read(rows_launch(cache, at, k, ldk, v, ldv), (hipStream_t)stream));
}

size_t ufp4_kv_attn_workspace_bytes(int64_t T, int32_t B, int32_t heads, int32_t kv_heads,
                                    int32_t D) {
  if (T <= 0 || B <= 0 || packed_sizes(T, B, heads, kv_heads, D)) return 0;
  return (size_t)kv_attn_workspace(T, B, heads, kv_heads, D);
}

int ufp4_kv_attn(const void* q, int64_t ldq, const int32_t* starts, int32_t B, int64_t T,
                 int32_t heads, const int32_t* lens, const int32_t* table, int64_t ldt,
                 int64_t width, const ufp4_kv_cache* cache, float scale, void* o, int64_t ldo,
                 void* workspace, size_t workspace_bytes, void* stream) {
  int st = cache_inputs(cache, starts, B, T, lens, table, ldt, width);
  if (st) return st;
  if ((st = packed_sizes(T, B, heads, cache->kv_heads, cache->D))) return st;
  if (T == 0 || B == 0) return UFP4_OK;
  if ((st = rows_of(q, ldq, heads, cache->D)) || (st = rows_of(o, ldo, heads, cache->D))) return st;
  if (!factor_ok(scale) || !workspace || !aligned(workspace, 256) ||
      workspace_bytes < ufp4_kv_attn_workspace_bytes(T, B, heads, cache->kv_heads, cache->D))
    return UFP4_ERR_INVALID_ARG;
  KvAttn p;
  std::memset(&p, 0, sizeof(p));
  p.at = place(cache, starts, B, T, lens, table, ldt, width);
  p.q = static_cast<const uint16_t*>(q);
  p.o = static_cast<uint16_t*>(o);
  p.ldq = ldq;
  p.ldo = ldo;
  p.k_codes = cache->k_codes;
  p.v_codes = cache->v_codes;
  p.k_scales = static_cast<const uint8_t*>(cache->k_scales);
  p.v_scales = static_cast<const uint8_t*>(cache->v_scales);
  sign_bits128(&cache->cfg, p.sign);
  p.n = cache->cfg.rht_n;
  p.cn = (float)(1.0 / std::sqrt((double)p.n));
  p.scale = scale;
  p.grid = cache->cfg.grid;
  p.kind = cache->cfg.scale_mode == UFP4_SCALE_POW2 ? 2 : cache->cfg.block_cols == 16 ? 1 : 0;
  p.heads = heads;
  p.group = heads / cache->kv_heads;
  p.rows16 = kv_attn_rows16(T, B, p.group);
  p.partial = static_cast<float*>(workspace);
  return hip_status(launch_kv_attn(p, (hipStream_t)stream));
}

}  // extern "C"
