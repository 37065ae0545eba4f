// Rows of a 4-bit cache read back, and the dispatch of writes by codebook (see
// kv_rows.h).
#include "kv_rows.h"

namespace ufp4 {

namespace kv {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Levels of the eight codes of a word.
template <int GRID>
__device__ __forceinline__ void levels8(uint32_t c, float* y) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (GRID == 1) {
      y[i] = (float)((int)(c << (28 - 4 * i)) >> 28);
    } else {
      const uint32_t m = (c >> (4 * i)) & 7u, sign = (c << (28 - 4 * i)) & 0x80000000u;
      float v;
      if constexpr (GRID == 0) v = 0.25f * (float)m;
      else v = m < 4 ? 0.5f * (float)m : (float)((2u + (m & 1u)) << ((m >> 1) - 2u));
      y[i] = __uint_as_float(__float_as_uint(v) | sign);
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
    for (int i = 0; i < W / 8; ++i) levels8<GRID>(c[i], y + 8 * i);
#pragma unroll
    for (int b = 0; b < W / B; ++b) {
      float f = s[b];
      if constexpr (E8) f = ldexpf(1.0f, (int)__float_as_uint(s[b]) - 127);
#pragma unroll
      for (int i = 0; i < B; ++i) y[b * B + i] = __fmul_rn(y[b * B + i], f);
    }
    if (item + 1 < l.end) load_codes<W, B, E8>(p, l, at, item + 1, c, s);
    const uint32_t sig = qk::fwht<W, N>(y, (l.qpos & 1u) ? 0x80000000u : 0u,
                                        (l.qpos & 2u) ? 0x80000000u : 0u, false);
    if constexpr (N > 1) qk::scale_by<W>(y, p.cn);
    const uint32_t pat = qk::select_pattern(p, l.qpos) ^ (sig ? 0xFFFFFFFFu : 0u);
#pragma unroll
    for (int i = 0; i < W; i += 8) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = i + 2 * j;
        const f32x2 v = {y[e], y[e + 1]};
        o[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2)) ^
               (((pat >> e) & 1u) << 15) ^ (((pat >> (e + 1)) & 1u) << 31);
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
