// A whole mixture-of-experts layer for a few tokens on 4-bit weights.
//
//   chosen(t) = the k largest router logits of token t (ties: lowest index;
//               -inf and NaN never), p_te = their softmax, over the chosen
//               experts or over all
//   y_t = sum over e in chosen(t) of Wd_e R( p_te act(Wg_e R x_t) (Wu_e R x_t) )
//
// R is the rotation S H of the weights' quantization along the contracted
// dimension ([UFP4] Method: it cancels in the product); the activations stay
// in high precision.  Few tokens mean that reading the chosen experts' codes
// and scales is all that costs: the kernels stream them once, 16 bytes per
// lane, straight from HBM into registers, and everything else is sized to
// hide behind that.
//
// Three launches:
//   k_moe_route  one workgroup per token: routing, and R x
//   k_moe_up     one workgroup per chosen expert and run of max(32, n) columns:
//                both products, the activation, the weight p and the rotation
//                of the run for the down product
//   k_moe_down   one workgroup per 16 output columns (and a share of the
//                experts): the down product summed over the experts
//
// Products: v_mfma_f32_16x16x32_bf16 with 16 tokens as rows and 16 weight rows
// as columns.  A code's level is exact in bf16; an activation is split into
// two bf16 pieces (16 bits of mantissa, off by at most 2^-16 of itself: far
// below the output's rounding, and the matrix cores idle here anyway); the
// level product of one scale block is accumulated in fp32 and then multiplied
// by the block's scale, which is the same for a lane's four values (one weight
// row), so that scales never enter the bf16 operands.
//
// A lane loads 16 bytes = 32 codes of one weight row: lanes l, l + 16, l + 32,
// l + 48 hold four consecutive 32-element blocks of row l % 16.  The matrix
// instruction wants 8 codes of ONE block from each of the four, so the 4 x 4
// words of the four lanes are transposed in registers (two lane-half swaps and
// two row swaps).
#include <type_traits>

#include "lm_internal.h"

namespace ufp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32u __attribute__((aligned(1)));
typedef unsigned long long u64u __attribute__((aligned(1)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kRouteThreads = 256;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// --- codes -> bf16 levels ------------------------------------------------------
// E4M3 bytes of the level magnitudes 0..7 (INT4: of the nibbles 0..7 and 8..15).
template <int GRID> struct Lut;
template <> struct Lut<0> { static constexpr uint32_t lo = 0x34302800u, hi = 0x3E3C3A38u; };
template <> struct Lut<2> { static constexpr uint32_t lo = 0x3C383000u, hi = 0x4C484440u; };
template <> struct Lut<1> {
  static constexpr uint32_t lo = 0x44403800u, hi = 0x4E4C4A48u;
  static constexpr uint32_t nlo = 0xCACCCED0u, nhi = 0xB8C0C4C8u;
};

// Nibbles in the low half of each byte of v -> E4M3 bytes.
template <int GRID>
__device__ __forceinline__ uint32_t nib_to_e4m3(uint32_t v) {
  const uint32_t m = v & 0x07070707u;
  const uint32_t pos = __builtin_amdgcn_perm(Lut<GRID>::hi, Lut<GRID>::lo, m);
  if constexpr (GRID == 1) {
    const uint32_t neg = __builtin_amdgcn_perm(Lut<1>::nhi, Lut<1>::nlo, m);
    return __builtin_amdgcn_perm(neg, pos, ((v >> 1) & 0x04040404u) | 0x03020100u);
  } else {
    return pos | ((v & 0x08080808u) << 4);
  }
}

// The bf16 levels of 8 codes in the order 0 2 4 6 1 3 5 7 (activations are
// stored in the same order).
template <int GRID>
__device__ __forceinline__ u32x4 levels8(uint32_t w) {
  const uint32_t ev = nib_to_e4m3<GRID>(w & 0x0F0F0F0Fu);
  const uint32_t od = nib_to_e4m3<GRID>((w >> 4) & 0x0F0F0F0Fu);
  auto two = [](bf16x2 v) { return __builtin_bit_cast(uint32_t, v); };
  return u32x4{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(ev, 1.0f, false)),
               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(ev, 1.0f, true)),
               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(od, 1.0f, false)),
               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(od, 1.0f, true))};
}

// Position of element i of an 8-group in that order.
__device__ __forceinline__ int slot8(int i) { return 4 * (i & 1) + (i >> 1); }

// --- scales ---------------------------------------------------------------------
// Scale kinds: fp32 or E8M0, 32- or 16-element blocks along K.
enum { kF32b32 = 0, kF32b16 = 1, kE8b32 = 2, kE8b16 = 3 };
template <int SK> struct Sk {
  static constexpr bool e8 = SK >= 2;
  static constexpr int per = (SK & 1) ? 2 : 1;   // scales per 32 elements
};

__device__ __forceinline__ float e8m0(uint32_t byte) {
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);   // 0 is 2^-127
}

// One 16-row tile's codes and scales of four 32-element blocks (128 of K).
template <int SK>
struct Tile {
  u32x4 codes;               // this lane's block: row l % 16, block l / 16
  float s[4 * Sk<SK>::per];  // the row's scales of all four blocks
};

// crow, srow: this lane's row; b0: first of the four blocks, nb: blocks of K.
template <int SK>
__device__ __forceinline__ void load_tile(Tile<SK>& t, const uint8_t* crow, const uint8_t* srow,
                                          int b0, int nb, int g) {
  constexpr int P = Sk<SK>::per;
  t.codes = u32x4{0, 0, 0, 0};
  if (b0 + g < nb)   // each byte is read once: past the caches' keeping
    t.codes = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(crow + 16 * (int64_t)(b0 + g)));
  if (b0 + 4 <= nb) {
    if constexpr (Sk<SK>::e8) {
      if constexpr (P == 1) {
        const uint32_t w = *reinterpret_cast<const u32u*>(srow + b0);
#pragma unroll
        for (int j = 0; j < 4; ++j) t.s[j] = e8m0((w >> (8 * j)) & 255u);
      } else {
        const unsigned long long w = *reinterpret_cast<const u64u*>(srow + 2 * b0);
#pragma unroll
        for (int j = 0; j < 8; ++j) t.s[j] = e8m0((uint32_t)(w >> (8 * j)) & 255u);
      }
    } else {
#pragma unroll
      for (int q = 0; q < P; ++q) {
        const f32x4u v = reinterpret_cast<const f32x4u*>(srow + 4 * P * (int64_t)b0)[q];
#pragma unroll
        for (int j = 0; j < 4; ++j) t.s[4 * q + j] = v[j];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4 * P; ++j) {
      const int64_t at = (int64_t)P * b0 + j;
      t.s[j] = 0.0f;
      if (at < (int64_t)P * nb)
        t.s[j] = Sk<SK>::e8 ? e8m0(srow[at]) : reinterpret_cast<const float*>(srow)[at];
    }
  }
}

// Transposes the 4 x 4 words that lanes l, l + 16, l + 32, l + 48 hold: lane
// group g then holds word g of blocks 0..3.
__device__ __forceinline__ void turn4(u32x4& c) {
  const u32x2 a = __builtin_amdgcn_permlane32_swap(c[0], c[2], false, false);
  const u32x2 b = __builtin_amdgcn_permlane32_swap(c[1], c[3], false, false);
  const u32x2 x = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const u32x2 y = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  c = u32x4{x[0], x[1], y[0], y[1]};
}

// Adds four blocks of NM weight tiles against TT 16-token tiles.  act[tt]:
// this lane's token row (null: no token), at K element 0: 32 bytes per
// 8 elements, the upper bf16 pieces and then the lower ones.
template <int GRID, int SK, int NM, int TT>
__device__ __forceinline__ void add_blocks(f32x4 (&acc)[NM][TT], Tile<SK> (&w)[NM],
                                           const uint8_t* const (&act)[TT], int b0, int nb, int g) {
  constexpr int P = Sk<SK>::per;
#pragma unroll
  for (int m = 0; m < NM; ++m) turn4(w[m].codes);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (b0 + j >= nb) break;
    bf16x8 hi[TT], lo[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      u32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
      if (act[t]) {
        const u32x4* p = reinterpret_cast<const u32x4*>(act[t] + 128 * (int64_t)(b0 + j) + 32 * g);
        a = p[0];
        b = p[1];
      }
      hi[t] = __builtin_bit_cast(bf16x8, a);
      lo[t] = __builtin_bit_cast(bf16x8, b);
    }
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const u32x4 lv = levels8<GRID>(w[m].codes[j]);
#pragma unroll
      for (int q = 0; q < P; ++q) {
        u32x4 l = lv;
        if constexpr (P == 2) {   // lane groups 0, 1 hold the first 16 of the 32, 2, 3 the others
          const uint32_t keep = (g >> 1) == q ? 0xFFFFFFFFu : 0u;
#pragma unroll
          for (int i = 0; i < 4; ++i) l[i] &= keep;
        }
        const bf16x8 b = __builtin_bit_cast(bf16x8, l);
        const float s = w[m].s[P * j + q];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
          c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo[t], b, c, 0, 0, 0);
          c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi[t], b, c, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][t][r] = __builtin_fmaf(c[r], s, acc[m][t][r]);
        }
      }
    }
  }
}

template <int ACT>
__device__ __forceinline__ float activation(float g) {
  float y = g;
  if constexpr (ACT == 1) {   // GELU, tanh form: g times the logistic function of y
    const float c = fminf(fmaxf(g, -1e4f), 1e4f);
    y = 1.5957691216057308f * __builtin_fmaf(0.044715f * c * c, c, c);
  }
  const float t = __builtin_exp2f(-kLog2e * fabsf(y));
  const float p = __builtin_amdgcn_rcpf(1.0f + t);
  return g * (y < 0.0f ? t * p : p);
}

// Order-preserving key of a float, 0 for what is never chosen.
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t b = __float_as_uint(l);
  return l > -INFINITY ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto step = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  v = step(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));    // quad 1 0 3 2
  v = step(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));    // quad 2 3 0 1
  v = step(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));   // half-row mirror
  v = step(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));   // row mirror
  const uint32_t a = step(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16));
  const uint32_t b = step(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48));
  return step(a, b);
}

// --- routing and the rotation of x -----------------------------------------------
__global__ __launch_bounds__(kRouteThreads) void k_moe_route(MoeLaunch p) {
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  if (t == 0) {
    for (int i = tid; i < p.E; i += kRouteThreads) p.count[i] = 0;
    for (int64_t i = tid; i < p.H / 16; i += kRouteThreads) p.done[i] = 0;
  }
  if (tid < 64) {
    // expert lane + 64 q in register q
    constexpr int Q = kMoeMaxExperts / 64;
    uint32_t key[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = lane + 64 * q;
      key[q] = e < p.E ? logit_key(p.logits[(int64_t)t * p.ldl + e]) : 0u;
    }
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) top = key[q] > top ? key[q] : top;
    top = wave_max(top);
    const float first = key_logit(top);
    float den = 0.0f;
    if (!p.renorm) {
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (key[q]) den += __builtin_amdgcn_exp2f((key_logit(key[q]) - first) * kLog2e);
#pragma unroll
      for (int m = 32; m > 0; m >>= 1) den += __shfl_xor(den, m);
    }
    int id = -1;        // lane r: the r-th choice and its share
    float share = 0.0f;
    for (int r = 0; r < p.k; ++r) {
      uint32_t best = 0;
#pragma unroll
      for (int q = 0; q < Q; ++q) best = key[q] > best ? key[q] : best;
      best = wave_max(best);
      if (best == 0) break;
      int e = -1;
#pragma unroll
      for (int q = 0; q < Q; ++q) {   // ascending: the lowest index of a tie
        const uint64_t has = __ballot(key[q] == best);
        if (e < 0 && has) {
          const int l = __builtin_ctzll(has);
          e = l + 64 * q;
          if (lane == l) key[q] = 0;
        }
      }
      const float x = __builtin_amdgcn_exp2f((key_logit(best) - first) * kLog2e);
      if (p.renorm) den += x;
      if (lane == r) { id = e; share = x; }
    }
    if (lane < p.k) {
      p.ids[(int64_t)t * p.k + lane] = id;
      p.share[(int64_t)t * p.k + lane] = id >= 0 ? share / den : 0.0f;
    }
  }
  // rotation, 8 elements per thread: y = c_n (x S) H, split into two bf16 pieces
  const int n = p.nx;
  const float cn = p.cnx;
  const int64_t groups = p.H / 8;
  for (int64_t i0 = 0; i0 < groups; i0 += kRouteThreads) {
    const int64_t i = i0 + tid;
    float v[8] = {};
    if (i < groups) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(p.x + (int64_t)t * p.ldx + 8 * i);
      const int o = (int)(8 * i) & 127;
      const uint32_t sg = p.sign_x[o >> 5] >> (o & 31);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b = (j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16;
        v[j] = __uint_as_float(b ^ ((sg >> j) << 31));
      }
    }
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) {
      if (n > h) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!(j & h)) {
            const float a = v[j], b = v[j + h];
            v[j] = a + b;
            v[j + h] = a - b;
          }
      }
    }
    for (int h = 8; h < n; h <<= 1) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float o = __shfl_xor(v[j], h >> 3);
        v[j] = (lane & (h >> 3)) ? o - v[j] : v[j] + o;
      }
    }
    if (i < groups) {
      u32x4 hi, lo;
      constexpr int order[8] = {0, 2, 4, 6, 1, 3, 5, 7};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = v[order[2 * j]] * cn, b = v[order[2 * j + 1]] * cn;
        hi[j] = pack_bf16(a, b);
        lo[j] = pack_bf16(a - __uint_as_float(hi[j] << 16),
                          b - __uint_as_float(hi[j] & 0xFFFF0000u));
      }
      u32x4* o = reinterpret_cast<u32x4*>(p.xr + ((int64_t)t * p.H + 8 * i) * 4);
      o[0] = hi;
      o[1] = lo;
    }
  }
}

// --- gate and up products, activation ---------------------------------------------
// NF: columns of the intermediate that a workgroup computes, max(32, n).
template <int GRID, int SK, int NF, int TT>
__device__ __forceinline__ void moe_up_body(const MoeLaunch& p, int e, int f0, int m,
                                            const int* tok, const float* share, float* part) {
  constexpr int PT = NF / 16, KS = kWaves / PT;   // 16-row pairs, shares of K
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int pt = wave % PT, ks = wave / PT, g = lane >> 4, r16 = lane & 15;
  const int nb = (int)(p.H / 32);
  const int64_t row = (int64_t)e * p.F + f0 + pt * 16 + r16;
  const uint8_t* crow[2];
  const uint8_t* srow[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const MoeWeight& w = q ? p.wu : p.wg;
    crow[q] = w.codes + row * (p.H / 2);
    srow[q] = w.scales + (row >> w.row_shift) * w.scale_pitch;
  }
  const uint8_t* act[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int i = t * 16 + r16;
    act[t] = i < m ? p.xr + (int64_t)tok[i] * p.H * 4 : nullptr;
  }
  f32x4 acc[2][TT];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[q][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  Tile<SK> cur[2], nxt[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) load_tile<SK>(cur[q], crow[q], srow[q], 4 * ks < nb ? 4 * ks : 0, nb, g);
  for (int b0 = 4 * ks; b0 < nb; b0 += 4 * KS) {
    const int bn = b0 + 4 * KS < nb ? b0 + 4 * KS : b0;   // past the end: this one again, unused
#pragma unroll
    for (int q = 0; q < 2; ++q) load_tile<SK>(nxt[q], crow[q], srow[q], bn, nb, g);
    add_blocks<GRID, SK, 2, TT>(acc, cur, act, b0, nb, g);
#pragma unroll
    for (int q = 0; q < 2; ++q) cur[q] = nxt[q];
  }

  // the shares of K added in order: part[matrix][token][column]
  constexpr int ROWS = TT * 16;
  for (int s = 0; s < KS; ++s) {
    if (ks == s) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float* d = part + (q * ROWS + t * 16 + 4 * g + r) * NF + pt * 16 + r16;
            *d = s == 0 ? acc[q][t][r] : *d + acc[q][t][r];
          }
    }
    __syncthreads();
  }

  // h = p act(gate) up, rotated along the run, as two bf16 pieces; 128
  // neighbouring elements of [token][column] per wave and pass
  const int n = p.nh, total = m * NF;
  for (int i0 = wave * 128; i0 < total; i0 += kWaves * 128) {
    float v[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = i0 + 64 * q + lane;
      v[q] = 0.0f;
      if (i < total) {
        const float a = part[i] * p.wg.factor, b = part[ROWS * NF + i] * p.wu.factor;
        const float s = p.act == UFP4_ACT_GELU ? activation<1>(a) : activation<0>(a);
        const int o = (f0 + i % NF) & 127;
        v[q] = s * b * share[i / NF];
        v[q] = __uint_as_float(__float_as_uint(v[q]) ^ ((p.sign_h[o >> 5] >> (o & 31)) << 31));
      }
    }
    for (int h = 1; h < n && h < 64; h <<= 1) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float o = __shfl_xor(v[q], h);
        v[q] = (lane & h) ? o - v[q] : v[q] + o;
      }
    }
    if (n == 128) {
      const float a = v[0], b = v[1];
      v[0] = a + b;
      v[1] = a - b;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = i0 + 64 * q + lane;
      if (i < total) {
        const int f = f0 + i % NF;
        const float y = v[q] * p.cnh;
        const uint32_t hi = pack_bf16(y, 0.0f) & 0xFFFFu;
        const uint32_t lo = pack_bf16(y - __uint_as_float(hi << 16), 0.0f);
        uint16_t* o = reinterpret_cast<uint16_t*>(
                          p.hr + (((int64_t)e * p.T + i / NF) * p.F + (f & ~7)) * 4) + slot8(f & 7);
        o[0] = (uint16_t)hi;
        o[8] = (uint16_t)lo;
      }
    }
  }
}

template <int GRID, int SK, int NF>
__global__ __launch_bounds__(kThreads) void k_moe_up(MoeLaunch p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int tok[kMoeMaxTokens];
  __shared__ float share[kMoeMaxTokens];
  __shared__ int found[2];   // expert, tokens
  const int tid = threadIdx.x, lane = tid & 63;
  const int fc = blockIdx.x, slot = blockIdx.y;
  if (tid < 64) {
    const int pairs = (int)(p.T * p.k);
    // by_pair: slot s stands for the s-th choice, unless the same expert
    // was chosen before it; else for expert s
    int e = slot;
    bool mine = true;
    if (p.by_pair) {
      e = p.ids[slot];
      if (e < 0) {
        mine = false;
      } else {
        bool before = false;
        for (int i0 = 0; i0 < slot; i0 += 64) {
          const int i = i0 + lane;
          before |= __any(i < slot && p.ids[i < slot ? i : 0] == e);
        }
        mine = !before;
      }
    }
    int m = 0;
    if (mine) {
      for (int i0 = 0; i0 < pairs; i0 += 64) {
        const int i = i0 + lane;
        const bool hit = i < pairs && p.ids[i < pairs ? i : 0] == e;
        const uint64_t mask = __ballot(hit);
        if (hit) {
          const int at = m + __builtin_popcountll(mask & (((uint64_t)1 << lane) - 1));
          tok[at] = i / p.k;
          share[at] = p.share[i];
        }
        m += __builtin_popcountll(mask);
      }
    }
    if (lane == 0) {
      found[0] = e;
      found[1] = m;
    }
  }
  __syncthreads();
  const int e = found[0], m = found[1];
  if (m == 0) return;
  if (fc == 0) {   // for the down product
    if (tid < m) p.list[(int64_t)e * p.T + tid] = tok[tid];
    if (tid == 0) p.count[e] = m;
  }
  float* part = reinterpret_cast<float*>(lds);
  if (m <= 16) moe_up_body<GRID, SK, NF, 1>(p, e, fc * NF, m, tok, share, part);
  else if (m <= 32) moe_up_body<GRID, SK, NF, 2>(p, e, fc * NF, m, tok, share, part);
  else moe_up_body<GRID, SK, NF, 4>(p, e, fc * NF, m, tok, share, part);
}

// --- down product --------------------------------------------------------------------
// A wave's run of (expert, 128 of F) items against one expert's tokens.
template <int GRID, int SK, int TT>
__device__ __forceinline__ void moe_down_run(const MoeLaunch& p, int e, int m, int s0, int s1,
                                             int64_t col0, float* y) {
  const int lane = threadIdx.x & 63, g = lane >> 4, r16 = lane & 15;
  const int nb = (int)(p.F / 32);
  const int64_t row = (int64_t)e * p.H + col0 + r16;
  const uint8_t* crow = p.wd.codes + row * (p.F / 2);
  const uint8_t* srow = p.wd.scales + (row >> p.wd.row_shift) * p.wd.scale_pitch;
  const uint8_t* act[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int i = t * 16 + r16;
    act[t] = i < m ? p.hr + ((int64_t)e * p.T + i) * p.F * 4 : nullptr;
  }
  f32x4 acc[1][TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[0][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  Tile<SK> cur[1], nxt[1];
  load_tile<SK>(cur[0], crow, srow, 4 * s0, nb, g);
  for (int s = s0; s < s1; ++s) {
    load_tile<SK>(nxt[0], crow, srow, 4 * (s + 1 < s1 ? s + 1 : s), nb, g);
    add_blocks<GRID, SK, 1, TT>(acc, cur, act, 4 * s, nb, g);
    cur[0] = nxt[0];
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = t * 16 + 4 * g + r;
      if (i < m) y[p.list[(int64_t)e * p.T + i] * 16 + r16] += acc[0][t][r];
    }
}

template <int GRID, int SK>
__global__ __launch_bounds__(kThreads) void k_moe_down(MoeLaunch p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];   // [wave][token][16]
  __shared__ int active[kMoeMaxExperts];
  __shared__ int tokens[kMoeMaxExperts];
  __shared__ int nactive, last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tile = blockIdx.x, split = blockIdx.y, S = gridDim.y;
  const int T = (int)p.T, cells = T * 16;
  float* all = reinterpret_cast<float*>(lds);
  for (int i = tid; i < kWaves * cells; i += kThreads) all[i] = 0.0f;
  if (tid < 64) {
    int n = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const int e = e0 + lane;
      const int m = e < p.E ? p.count[e] : 0;
      const uint64_t mask = __ballot(m > 0);
      if (m > 0) {
        const int at = n + __builtin_popcountll(mask & (((uint64_t)1 << lane) - 1));
        active[at] = e;
        tokens[at] = m;
      }
      n += __builtin_popcountll(mask);
    }
    if (lane == 0) nactive = n;
  }
  __syncthreads();
  // items 0 .. n steps - 1 in equal runs over the splits' waves
  const int steps = (int)((p.F + 127) / 128), items = nactive * steps;
  const int parts = S * kWaves, me = split * kWaves + wave;
  const int lo = (int)((int64_t)items * me / parts), hi = (int)((int64_t)items * (me + 1) / parts);
  float* y = all + wave * cells;
  for (int it = lo; it < hi;) {
    const int a = it / steps, s0 = it - a * steps;
    const int s1 = s0 + (hi - it) < steps ? s0 + (hi - it) : steps;
    const int e = __builtin_amdgcn_readfirstlane(active[a]);
    const int m = __builtin_amdgcn_readfirstlane(tokens[a]);
    const int64_t col0 = (int64_t)tile * 16;
    if (m <= 16) moe_down_run<GRID, SK, 1>(p, e, m, s0, s1, col0, y);
    else if (m <= 32) moe_down_run<GRID, SK, 2>(p, e, m, s0, s1, col0, y);
    else moe_down_run<GRID, SK, 4>(p, e, m, s0, s1, col0, y);
    it += s1 - s0;
  }
  __syncthreads();
  // the waves' sums in order; several splits leave theirs in the workspace and
  // the last workgroup of a tile to get there adds them, in order as well
  for (int i = tid; i < cells; i += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += all[w * cells + i];
    if (S == 1) all[i] = v;   // only this thread reads cell i of any wave
    else p.partial[((int64_t)tile * S + split) * cells + i] = v;
  }
  if (S > 1) {
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(&p.done[tile], 1) == S - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    for (int i = tid; i < cells; i += kThreads) {
      float v = 0.0f;
      for (int s = 0; s < S; ++s)
        v += __hip_atomic_load(&p.partial[((int64_t)tile * S + s) * cells + i], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
      all[i] = v;
    }
  }
  __syncthreads();
  for (int i = tid; i < cells / 2; i += kThreads) {
    const int t = i / 8, c = 2 * (i % 8);
    *reinterpret_cast<uint32_t*>(p.y + (int64_t)t * p.ldy + (int64_t)tile * 16 + c) =
        pack_bf16(all[t * 16 + c] * p.wd.factor, all[t * 16 + c + 1] * p.wd.factor);
  }
}

template <int GRID, int SK, int NF>
hipError_t launch_up_n(const MoeLaunch& p, hipStream_t s) {
  const int tt = p.T <= 16 ? 1 : p.T <= 32 ? 2 : 4;
  const int bytes = 2 * tt * 16 * NF * 4;
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t e = set_lds_limit((const void*)k_moe_up<GRID, SK, NF>, 2 * 64 * NF * 4, lds_set);
  if (e != hipSuccess) return e;
  const unsigned slots = (unsigned)(p.by_pair ? p.T * p.k : p.E);
  hipLaunchKernelGGL((k_moe_up<GRID, SK, NF>), dim3((unsigned)(p.F / NF), slots), dim3(kThreads),
                     bytes, s, p);
  return hipGetLastError();
}

template <int GRID, int SK>
hipError_t launch_up(const MoeLaunch& p, hipStream_t s) {
  if (p.nh <= 32) return launch_up_n<GRID, SK, 32>(p, s);
  if (p.nh == 64) return launch_up_n<GRID, SK, 64>(p, s);
  return launch_up_n<GRID, SK, 128>(p, s);
}

template <int GRID, int SK>
hipError_t launch_down(const MoeLaunch& p, hipStream_t s) {
  hipLaunchKernelGGL((k_moe_down<GRID, SK>), dim3((unsigned)(p.H / 16), (unsigned)p.splits),
                     dim3(kThreads), kWaves * (size_t)p.T * 16 * 4, s, p);
  return hipGetLastError();
}

template <typename F>
hipError_t by_format(const MoeWeight& w, F f) {
  auto scales = [&](auto grid) {
    constexpr int G = decltype(grid)::value;
    switch (w.kind) {
      case kF32b32: return f(std::integral_constant<int, G>{}, std::integral_constant<int, kF32b32>{});
      case kF32b16: return f(std::integral_constant<int, G>{}, std::integral_constant<int, kF32b16>{});
      case kE8b32: return f(std::integral_constant<int, G>{}, std::integral_constant<int, kE8b32>{});
      default: return f(std::integral_constant<int, G>{}, std::integral_constant<int, kE8b16>{});
    }
  };
  switch (w.grid) {
    case 0: return scales(std::integral_constant<int, 0>{});
    case 1: return scales(std::integral_constant<int, 1>{});
    default: return scales(std::integral_constant<int, 2>{});
  }
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// Workspace parts, in this order, each 256-byte aligned.
int64_t moe_plan(MoeLaunch& p, uint8_t* ws) {
  // the down product: splits of the experts until two workgroups per compute
  // unit are there, each wave at least two 128-element steps
  const int64_t met = p.T * p.k < p.E ? p.T * p.k : p.E;
  const int64_t items = met * ((p.F + 127) / 128);
  int64_t splits = 512 / (p.H / 16 > 0 ? p.H / 16 : 1);
  if (splits > items / (2 * kWaves)) splits = items / (2 * kWaves);
  p.splits = (int32_t)(splits < 1 ? 1 : splits > 16 ? 16 : splits);
  p.by_pair = p.T * p.k < p.E;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* q = ws ? ws + at : nullptr;
    at += up256(bytes);
    return q;
  };
  p.ids = reinterpret_cast<int*>(take(4 * p.T * p.k));
  p.share = reinterpret_cast<float*>(take(4 * p.T * p.k));
  p.count = reinterpret_cast<int*>(take(4 * p.E));
  p.list = reinterpret_cast<int*>(take(4 * p.E * p.T));
  p.done = reinterpret_cast<int*>(take(4 * (p.H / 16)));
  p.xr = take(4 * p.T * p.H);
  p.hr = take(4 * (int64_t)p.E * p.T * p.F);
  p.partial = reinterpret_cast<float*>(take(p.splits > 1 ? 4 * p.splits * p.T * p.H : 0));
  return at;
}

hipError_t launch_moe_tokens(const MoeLaunch& p, hipStream_t s) {
  hipLaunchKernelGGL(k_moe_route, dim3((unsigned)p.T), dim3(kRouteThreads), 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  e = by_format(p.wg, [&](auto g, auto k) {
    return launch_up<decltype(g)::value, decltype(k)::value>(p, s);
  });
  if (e != hipSuccess) return e;
  return by_format(p.wd, [&](auto g, auto k) {
    return launch_down<decltype(g)::value, decltype(k)::value>(p, s);
  });
}

}  // namespace ufp4
