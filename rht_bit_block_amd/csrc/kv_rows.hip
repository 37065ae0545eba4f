// Rows of a 4-bit cache read back, and the dispatch of writes by codebook (see
// kv_rows.h).
#include "kv_rows.h"

namespace ufp4 {

namespace kv {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// The eight codes of a word as fp32 levels times 2^e of `scale`, two to a conversion: E2M1
// directly, E1M2 and INT4 by way of E4M3 bytes from tables.
template <int GRID>
__device__ __forceinline__ void levels8(uint32_t c, float scale, float* y) {
  if constexpr (GRID == 2) {
    f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0);
    y[0] = v[0]; y[1] = v[1];
    v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1);
    y[2] = v[0]; y[3] = v[1];
    v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2);
    y[4] = v[0]; y[5] = v[1];
    v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3);
    y[6] = v[0]; y[7] = v[1];
  } else {
    uint32_t b[2];   // of the even and of the odd nibbles
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = c >> (4 * i), low = x & 0x07070707u;
      if constexpr (GRID == 0) {
        b[i] = __builtin_amdgcn_perm(0x3E3C3A38u, 0x34302800u, low) | ((x << 4) & 0x80808080u);
      } else {
        const uint32_t pos = __builtin_amdgcn_perm(0x4E4C4A48u, 0x44403800u, low);
        const uint32_t neg = __builtin_amdgcn_perm(0xB8C0C4C8u, 0xCACCCED0u, low);
        b[i] = __builtin_amdgcn_perm(neg, pos, ((x >> 1) & 0x04040404u) | 0x03020100u);
      }
      f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(b[i], scale, false);
      y[i] = v[0]; y[2 + i] = v[1];
      v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(b[i], scale, true);
      y[4 + i] = v[0]; y[6 + i] = v[1];
    }
  }
}

// Codes and scales of W elements of an item's row.
template <int W, int B, bool E8>
__device__ __forceinline__ void load_codes(const KvRows& p, const Lane& l, const Where& at, int item,
                                           uint32_t (&c)[W / 8], float (&s)[W / B]) {
  const bool is_v = item >= p.at.kv_heads;
  const uint64_t row = cache_row(p.at, at, is_v ? item - p.at.kv_heads : item);
  const uint32_t* codes =
      reinterpret_cast<const uint32_t*>((is_v ? p.codes[1] : p.codes[0]) + (row * p.at.D + l.k0) / 2);
  const uint64_t s0 = row * (uint32_t)(p.at.D / B) + l.k0 / B;
  const void* scales = is_v ? p.scales[1] : p.scales[0];
#pragma unroll
  for (int i = 0; i < W / 8; ++i) c[i] = codes[i];
#pragma unroll
  for (int b = 0; b < W / B; ++b) {
    if constexpr (E8) s[b] = __uint_as_float(reinterpret_cast<const uint8_t*>(scales)[s0 + b]);   // still the byte
    else s[b] = reinterpret_cast<const float*>(scales)[s0 + b];
  }
}

template <int W, int B, int N, int GRID, bool E8>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvRows p, FastDiv segs) {
  __shared__ int32_t starts[kSeqLds];
  const bool in_lds = starts_to_lds(p.at, starts);
  constexpr int lpc = N > W ? N / W : 1;
  const Lane l = lane_of<W, lpc>(p, segs);
  const Where at = locate(p.at, starts, in_lds, l.t);
  if (at.seq < 0) return;
  uint32_t pm[W / 2];
  qk::sign_masks<W>(qk::select_pattern(p, l.qpos), pm);
  uint32_t c[W / 8];
  float s[W / B];
  if (at.page >= 0) load_codes<W, B, E8>(p, l, at, l.item, c, s);
  for (int item = l.item; item < l.end; ++item) {
    const bool is_v = item >= p.at.kv_heads;
    const int h = is_v ? item - p.at.kv_heads : item;
    uint16_t* dst = (is_v ? p.v + l.t * p.ldv : p.k + l.t * p.ldk) + (int64_t)h * p.at.D + l.k0;
    if (at.page < 0) {
#pragma unroll
      for (int i = 0; i < W / 8; ++i) reinterpret_cast<uint4*>(dst)[i] = make_uint4(0, 0, 0, 0);
      continue;
    }
    float y[W];
#pragma unroll
    for (int i = 0; i < W / 8; ++i)   // an E8M0 byte is the exponent of the conversion's factor
      levels8<GRID>(c[i], E8 ? __uint_as_float(__float_as_uint(s[8 * i / B]) << 23) : 1.0f, y + 8 * i);
    if constexpr (!E8) {
#pragma unroll
      for (int i = 0; i < W; ++i) y[i] = __fmul_rn(y[i], s[i / B]);
    }
    if (item + 1 < l.end) load_codes<W, B, E8>(p, l, at, item + 1, c, s);
    const uint32_t sig = qk::fwht<W, N>(y, (l.qpos & 1u) ? 0x80000000u : 0u,
                                        (l.qpos & 2u) ? 0x80000000u : 0u, false);
    if constexpr (N > 1) qk::scale_by<W>(y, p.cn);
    const uint32_t both = sig | (sig >> 16);   // the signs of a pair that came out negated
#pragma unroll
    for (int i = 0; i < W; i += 8) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = i + 2 * j;
        const f32x2 v = {y[e], y[e + 1]};
        o[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2)) ^ pm[e / 2] ^ both;
      }
      *reinterpret_cast<u32x4*>(dst + i) = o;
    }
  }
}

template <int W, int B, int N, int GRID, bool E8>
hipError_t read_n(const KvRows& p, hipStream_t s) {
  return over_rows(k_kv_read<W, B, N, GRID, E8>, p, W, s);
}

template <int B, int GRID, bool E8>
hipError_t read_b(const KvRows& p, hipStream_t s) {
  constexpr int W = B == 32 ? 32 : 16;
  switch (p.n) {
    case 1: return read_n<W, B, 1, GRID, E8>(p, s);
    case 2: return read_n<W, B, 2, GRID, E8>(p, s);
    case 4: return read_n<W, B, 4, GRID, E8>(p, s);
    case 8: return read_n<W, B, 8, GRID, E8>(p, s);
    case 16: return read_n<W, B, 16, GRID, E8>(p, s);
    case 32: return read_n<32, B, 32, GRID, E8>(p, s);
    case 64: return read_n<32, B, 64, GRID, E8>(p, s);
    default: return read_n<32, B, 128, GRID, E8>(p, s);
  }
}

template <int GRID>
hipError_t read_grid(const KvRows& p, hipStream_t s) {
  if (p.scale_mode == UFP4_SCALE_POW2) return read_b<32, GRID, true>(p, s);
  return p.bc == 32 ? read_b<32, GRID, false>(p, s) : read_b<16, GRID, false>(p, s);
}

}  // namespace
}  // namespace kv

hipError_t launch_kv_read(const KvRows& p, hipStream_t s) {
  switch (p.grid) {
    case 0: return kv::read_grid<0>(p, s);
    case 1: return kv::read_grid<1>(p, s);
    default: return kv::read_grid<2>(p, s);
  }
}

hipError_t launch_kv_write(const KvRows& p, hipStream_t s) {
  switch (p.grid) {
    case 0: return kv_write_e1m2(p, s);
    case 1: return kv_write_int4(p, s);
    default: return kv_write_e2m1(p, s);
  }
}

}  // namespace ufp4
