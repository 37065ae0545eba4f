// Gated activation between an expert's two products, its inputs kept as MXFP8
// checkpoints, and the backward pass that starts from those.
//
//   forward   h = r act(g) u                      r: a factor per row, or 1
//             g~ = Q8(g), u~ = Q8(u)              kept for the backward pass
//   backward  dg = r dh u~ act'(g~)    du = r dh act(g~)
//             dr = sum over the row of dh act(g~) u~
//             h~ = r act(g~) u~                   recomputed on request
//
// Both activations are g times a logistic function s = 1 / (1 + e^-y):
//   SiLU           y = g                            y' = 1
//   GELU (tanh)    y = 2 c (g + b g^3)              y' = 2 c (1 + 3 b g^2)
// with c = sqrt(2 / pi), b = 0.044715, since (1 + tanh(y / 2)) / 2 = s(y); so
// act = g s and act' = s (1 + g (1 - s) y').  All of it in fp32.
//
// Q8 is the package's MXFP8 rule ([2DFP4] = "Stable FP4 Training via
// Transposition-Invariant Block Quantization", its power-of-two scale
// equation): 1 x 32 blocks, the least 2^e with absmax <= 448 2^e (e >= -127),
// E4M3 codes rounded to nearest even.  A NaN stays a NaN code; a block that
// holds an infinity keeps it (448 2^120 reads back as infinity), its other
// elements are rounded at that scale.
//
// Every element is read and written once and costs some tens of fp32
// operations against 7 to 16 bytes of HBM traffic, so the kernels are bound by
// HBM.  A thread takes 8 neighbouring elements of a row (16-byte loads), four
// neighbouring lanes hold one 32-element block, and a row is padded to whole
// blocks, so that the block's absmax is two lane exchanges and no block ever
// straddles two rows.
#include <type_traits>

#include "lm_internal.h"

namespace ufp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;      // elements per thread

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
// the same at the alignment of their elements (the hardware takes any)
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight elements at p (n of them inside the row; the others read as 0).  VEC:
// p is 16-byte aligned and n is 8 or <= 0; else whole eights are still one or
// two wide accesses, at the elements' own alignment, and only a row's end goes
// element by element.  What a whole wave reads line by line, here and in read8, is
// loaded non-temporally: the backward pass of 262144 x 1536 rows with fp32 dh
// takes 742 us instead of 760, with bf16 inputs 1 to 5 % more (forward 541 instead of
// 536).  Stores past the caches gained nothing at any size (forward 884 us either way).
template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void* base, int64_t at, int n, float (&v)[kPer]) {
  if constexpr (VEC) {
    if constexpr (F32) {
      const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + at);
      const f32x4 a = p[0], b = p[1];   // halves of one line: it has to stay for the second
#pragma unroll
      for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
    } else {
      const u32x4 a = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + at));
#pragma unroll
      for (int i = 0; i < 4; ++i) { v[2 * i] = bf16_lo(a[i]); v[2 * i + 1] = bf16_hi(a[i]); }
    }
  } else if (n >= kPer) {
    if constexpr (F32) {
      const f32x4u* p = reinterpret_cast<const f32x4u*>(static_cast<const float*>(base) + at);
      const f32x4u a = p[0], b = p[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
    } else {
      const u32x4u a = *reinterpret_cast<const u32x4u*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) { v[2 * i] = bf16_lo(a[i]); v[2 * i + 1] = bf16_hi(a[i]); }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] = 0.0f;
      if (i < n) {
        if constexpr (F32) v[i] = static_cast<const float*>(base)[at + i];
        else v[i] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(base)[at + i] << 16);
      }
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void store8_bf16(uint16_t* base, int64_t at, int n,
                                            const float (&v)[kPer]) {
  const u32x4 w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                   pack_bf16(v[6], v[7])};
  if constexpr (VEC) {
    *reinterpret_cast<u32x4*>(base + at) = w;
  } else if (n >= kPer) {
    *reinterpret_cast<u32x4u*>(base + at) = w;
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < n) base[at + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}

// s, act(g) = g s and, if asked for, act'(g).
template <int ACT, bool GRAD>
__device__ __forceinline__ void activation(float g, float& a, float& da) {
  float y = g, dy = 1.0f;
  if constexpr (ACT == 1) {
    // past +-1e4 the logistic function is 0 or 1 to the last bit; the bound
    // keeps the cube finite, so that 0 is not multiplied by infinity
    const float c = fminf(fmaxf(g, -1e4f), 1e4f), q = c * c;
    constexpr float k = 1.5957691216057308f, b = 0.044715f;   // 2 sqrt(2 / pi)
    y = k * __builtin_fmaf(b * q, c, c);
    dy = k * __builtin_fmaf(3.0f * b, q, 1.0f);
  }
  // s = 1 / (1 + t) and 1 - s = t / (1 + t) for y >= 0 with t = e^-|y| <= 1,
  // the other way round below 0: neither overflows nor cancels, and t keeps
  // its subnormals (the compiler's exp2 scales around the instruction's flush)
  const float t = __builtin_exp2f(-1.4426950408889634f * fabsf(y));
  const float p = __builtin_amdgcn_rcpf(1.0f + t), tp = t * p;
  const float s = y < 0.0f ? tp : p;
  a = g * s;
  if constexpr (GRAD) da = s * __builtin_fmaf(g * (y < 0.0f ? p : tp), dy, 1.0f);
}

// Largest |v| of the block that four neighbouring lanes hold (quad permutes).
__device__ __forceinline__ float block_absmax(const float (&v)[kPer]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) m = fmaxf(m, fabsf(v[i]));   // a NaN is passed over
  m = fmaxf(m, __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp(
                   (int)__float_as_uint(m), 0xB1, 0xF, 0xF, true)));   // lanes 1 0 3 2
  m = fmaxf(m, __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp(
                   (int)__float_as_uint(m), 0x4E, 0xF, 0xF, true)));   // lanes 2 3 0 1
  return m;
}

// Least e >= -127 with m <= 448 2^e, 448 = 1.75 * 2^8: from the bits of
// m = 1.f * 2^E (a subnormal m is below 448 * 2^-127).
__device__ __forceinline__ int scale_exponent(float m) {
  const uint32_t b = __float_as_uint(m);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e > -127 ? e : -127;
}

// Codes and scale of a thread's 8 elements (n inside the row).
template <bool VEC>
__device__ __forceinline__ void save8(uint8_t* codes, int64_t at, uint8_t* scales, int64_t sat,
                                      int n, bool first, const float (&x)[kPer]) {
  const float m = block_absmax(x);
  const int e = scale_exponent(m);
  float v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = __builtin_ldexpf(x[i], -e);   // exact
  if (m > 3.4028234e38f) {   // an infinity in the block: it becomes the largest code
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (fabsf(v[i]) > 448.0f) v[i] = copysignf(448.0f, v[i]);
  }
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    i16x2 o = {0, 0};
    o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, v[4 * i], v[4 * i + 1], 1.0f, false);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, v[4 * i + 2], v[4 * i + 3], 1.0f, true);
    uint32_t b = __builtin_bit_cast(uint32_t, o);
    const uint32_t mag = b & 0x7F7F7F7Fu;   // zero is stored as 0x00, never 0x80
    w[i] = mag | (b & ((mag + 0x7F7F7F7Fu) & 0x80808080u));
  }
  if constexpr (VEC) {
    if (n > 0) *reinterpret_cast<u32x2*>(codes + at) = w;
  } else if (n >= kPer) {
    *reinterpret_cast<u32x2u*>(codes + at) = w;
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < n) codes[at + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
  if (first && n > 0) scales[sat] = (uint8_t)(e + 127);
}

// The 8 values that a thread's codes stand for.
template <bool VEC>
__device__ __forceinline__ void read8(const uint8_t* codes, int64_t at, const uint8_t* scales,
                                      int64_t sat, int n, float (&v)[kPer]) {
  u32x2 w = {0, 0};
  if constexpr (VEC) {
    w = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(codes + at));
  } else if (n >= kPer) {
    w = *reinterpret_cast<const u32x2u*>(codes + at);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < n) w[i >> 2] |= (uint32_t)codes[at + i] << (8 * (i & 3));
  }
  const int e = (int)scales[sat] - 127;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 p = (i & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i >> 1], true)
                            : __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i >> 1], false);
    v[2 * i] = __builtin_ldexpf(p[0], e);
    v[2 * i + 1] = __builtin_ldexpf(p[1], e);
  }
}

// One thread per 8 elements; chunks: 8-element chunks per row, a multiple of
// four (whole blocks).  Threads past the last row take part in the lane
// exchanges with zeros and write nothing.
template <bool F32, bool VEC, int ACT, bool SAVE>
__global__ __launch_bounds__(kThreads) void k_glu_fwd(GluLaunch g, FastDiv chunks, uint32_t total) {
  const uint32_t i = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
  const uint32_t q = (uint32_t)(((uint64_t)__umulhi(chunks.m, i) + i) >> chunks.l);
  const int64_t row = q;
  const uint32_t c = i - q * chunks.d;
  const int64_t col = (int64_t)c * kPer;
  int n = i < total ? (g.cols - col < kPer ? (int)(g.cols - col) : kPer) : 0;
  float a[kPer] = {}, u[kPer] = {};
  if (n > 0) {
    load8<F32, VEC>(g.gate, row * g.ld + col, n, a);
    load8<F32, VEC>(g.up, row * g.ld + col, n, u);
  }
  if constexpr (SAVE) {
    const int64_t at = row * g.cols + col, sat = row * (chunks.d / 4) + c / 4;
    save8<VEC>(g.gate_codes, at, g.gate_scales, sat, n, (c & 3) == 0, a);
    save8<VEC>(g.up_codes, at, g.up_scales, sat, n, (c & 3) == 0, u);
  }
  if (n <= 0) return;
  const float r = g.row_scale ? g.row_scale[row] : 1.0f;
  float h[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    float s, unused;
    activation<ACT, false>(a[k], s, unused);
    h[k] = s * u[k] * r;
  }
  store8_bf16<VEC>(g.h, row * g.ldh + col, n, h);
}

// One chunk of the backward pass; returns its part of dr.
template <bool F32, bool VEC, int ACT, bool AGAIN>
__device__ __forceinline__ float bwd_chunk(const GluLaunch& g, int64_t row, uint32_t c,
                                           uint32_t chunks, float r) {
  const int64_t col = (int64_t)c * kPer;
  const int n = g.cols - col < kPer ? (int)(g.cols - col) : kPer;
  if (n <= 0) return 0.0f;
  const int64_t at = row * g.cols + col, sat = row * (chunks / 4) + c / 4;
  float a[kPer], u[kPer], d[kPer], og[kPer], ou[kPer], oh[kPer];
  load8<F32, VEC>(g.dh, row * g.lddh + col, n, d);
  read8<VEC>(g.gate_codes, at, g.gate_scales, sat, n, a);
  read8<VEC>(g.up_codes, at, g.up_scales, sat, n, u);
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    float s, ds;
    activation<ACT, true>(a[k], s, ds);
    const float dr = d[k] * r;
    og[k] = dr * u[k] * ds;
    ou[k] = dr * s;
    if constexpr (AGAIN) oh[k] = s * u[k] * r;
    sum = __builtin_fmaf(d[k] * s, u[k], sum);   // past the row everything is 0
  }
  store8_bf16<VEC>(g.dgate, row * g.ldd + col, n, og);
  store8_bf16<VEC>(g.dup, row * g.ldd + col, n, ou);
  if constexpr (AGAIN) store8_bf16<VEC>(g.h, row * g.ldh + col, n, oh);
  return sum;
}

template <bool F32, bool VEC, int ACT, bool AGAIN>
__global__ __launch_bounds__(kThreads) void k_glu_bwd(GluLaunch g, FastDiv chunks, uint32_t total) {
  const uint32_t i = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
  if (i >= total) return;
  const uint32_t q = (uint32_t)(((uint64_t)__umulhi(chunks.m, i) + i) >> chunks.l);
  const float r = g.row_scale ? g.row_scale[q] : 1.0f;
  bwd_chunk<F32, VEC, ACT, AGAIN>(g, q, i - q * chunks.d, chunks.d, r);
}

// With the row factor's gradient: one wave per row, its lanes' sums added by
// lane exchanges in a fixed order.
template <bool F32, bool VEC, int ACT, bool AGAIN>
__global__ __launch_bounds__(kThreads) void k_glu_bwd_row(GluLaunch g, uint32_t chunks) {
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= g.rows) return;
  const uint32_t lane = threadIdx.x & 63;
  const float r = g.row_scale[row];
  float sum = 0.0f;
  for (uint32_t c = lane; c < chunks; c += 64)
    sum += bwd_chunk<F32, VEC, ACT, AGAIN>(g, row, c, chunks, r);
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
  if (lane == 0) g.drow[row] = sum;
}

bool vec_ok(const void* p, int64_t ld, int64_t elem) {
  return (reinterpret_cast<uintptr_t>(p) % 16) == 0 && (ld * elem) % 16 == 0;
}

template <typename F> auto pick2(bool a, bool b, F f) {
  return a ? (b ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{}))
           : (b ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{}));
}

// Launches of at most 2^30 threads each (HIP takes fewer than 2^32), `threads` for
// a row: some rows at a time.
template <typename F>
hipError_t in_slices(const GluLaunch& g, uint32_t chunks, uint32_t threads, F one) {
  const int64_t step = ((int64_t)1 << 30) / threads;   // chunks <= 2^27
  const int64_t es = g.dtype == UFP4_BF16 ? 2 : 4, blocks = chunks / 4;
  for (int64_t r = 0; r < g.rows; r += step) {
    GluLaunch p = g;
    p.rows = g.rows - r < step ? g.rows - r : step;
    auto bytes = [&](const void* b, int64_t off) {
      return b ? static_cast<const void*>(static_cast<const uint8_t*>(b) + off) : nullptr;
    };
    p.gate = bytes(g.gate, r * g.ld * es);
    p.up = bytes(g.up, r * g.ld * es);
    p.dh = bytes(g.dh, r * g.lddh * es);
    if (g.row_scale) p.row_scale = g.row_scale + r;
    if (g.h) p.h = g.h + r * g.ldh;
    if (g.gate_codes) {
      p.gate_codes = g.gate_codes + r * g.cols;
      p.up_codes = g.up_codes + r * g.cols;
      p.gate_scales = g.gate_scales + r * blocks;
      p.up_scales = g.up_scales + r * blocks;
    }
    if (g.dgate) p.dgate = g.dgate + r * g.ldd;
    if (g.dup) p.dup = g.dup + r * g.ldd;
    if (g.drow) p.drow = g.drow + r;
    one(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_glu_fwd(const GluLaunch& g, hipStream_t s) {
  const uint32_t chunks = 4 * (uint32_t)((g.cols + 31) / 32);
  const int64_t es = g.dtype == UFP4_BF16 ? 2 : 4;
  const bool save = g.gate_codes != nullptr;
  const bool vec = g.cols % kPer == 0 && vec_ok(g.gate, g.ld, es) && vec_ok(g.up, g.ld, es) &&
                   vec_ok(g.h, g.ldh, 2) &&
                   (!save || ((uintptr_t)g.gate_codes % 8 == 0 && (uintptr_t)g.up_codes % 8 == 0));
  const FastDiv div = make_fastdiv(chunks);
  return in_slices(g, chunks, chunks, [&](const GluLaunch& p) {
    const uint32_t total = (uint32_t)(p.rows * chunks);
    const dim3 grid((total + kThreads - 1) / kThreads);
    pick2(g.dtype != UFP4_BF16, vec, [&](auto f32, auto v) {
      pick2(g.act == UFP4_ACT_GELU, save, [&](auto gelu, auto sv) {
        hipLaunchKernelGGL((k_glu_fwd<decltype(f32)::value, decltype(v)::value,
                                      decltype(gelu)::value ? 1 : 0, decltype(sv)::value>),
                           grid, dim3(kThreads), 0, s, p, div, total);
      });
    });
  });
}

hipError_t launch_glu_bwd(const GluLaunch& g, hipStream_t s) {
  const uint32_t chunks = 4 * (uint32_t)((g.cols + 31) / 32);
  const int64_t es = g.dtype == UFP4_BF16 ? 2 : 4;
  const bool vec = g.cols % kPer == 0 && vec_ok(g.dh, g.lddh, es) && vec_ok(g.dgate, g.ldd, 2) &&
                   vec_ok(g.dup, g.ldd, 2) && (!g.h || vec_ok(g.h, g.ldh, 2)) &&
                   (uintptr_t)g.gate_codes % 8 == 0 && (uintptr_t)g.up_codes % 8 == 0;
  const FastDiv div = make_fastdiv(chunks > 0 ? chunks : 1);
  return in_slices(g, chunks, g.drow ? 64 : chunks, [&](const GluLaunch& p) {
    const uint32_t total = (uint32_t)(p.rows * chunks);   // unused with a wave per row
    pick2(g.dtype != UFP4_BF16, vec, [&](auto f32, auto v) {
      pick2(g.act == UFP4_ACT_GELU, g.h != nullptr, [&](auto gelu, auto ag) {
        constexpr bool F = decltype(f32)::value, V = decltype(v)::value, A = decltype(ag)::value;
        constexpr int ACT = decltype(gelu)::value ? 1 : 0;
        if (g.drow)
          hipLaunchKernelGGL((k_glu_bwd_row<F, V, ACT, A>),
                             dim3((unsigned)((p.rows + kThreads / 64 - 1) / (kThreads / 64))),
                             dim3(kThreads), 0, s, p, chunks);
        else
          hipLaunchKernelGGL((k_glu_bwd<F, V, ACT, A>), dim3((total + kThreads - 1) / kThreads),
                             dim3(kThreads), 0, s, p, div, total);
      });
    });
  });
}

}  // namespace ufp4
