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
// lane, straight from HBM into shared memory, and everything else is sized to
// hide behind that.
//
// Launches:
//   k_moe_up     one workgroup per chosen expert and run of columns: both
//                products, the activation and the weight p.  For a handful of
//                tokens the routing and the rotation of x run in front, in
//                every workgroup; otherwise k_moe_route has done both once.
//   k_moe_down   one workgroup per chosen expert and run of output columns,
//                behind the rotation of its tokens' intermediate
//   k_moe_join   a token's experts added up
//
// Products: v_mfma_f32_16x16x32_bf16 with 16 tokens as rows and 16 weight rows
// as columns.  A code's level is exact in bf16; an activation is split into
// two bf16 pieces (16 bits of mantissa, off by at most 2^-16 of itself: far
// below the output's rounding, and the matrix cores idle here anyway); the
// level product of one scale block is accumulated in fp32 and then multiplied
// by the block's scale, which is the same for a lane's four values (one weight
// row), so that scales never enter the bf16 operands.
//
// The weights go HBM -> LDS (buffer_load ... lds) in steps of 128 of K, two
// steps per wave in a ring of its own, so that no barrier or register holds a
// load back: a lane copies 16 bytes and four neighbouring lanes a row's 64.
// Straight into registers in the layout of the instruction (neighbouring lanes
// in different rows) every lane's 16 bytes were a cache access of their own,
// and the address unit, not HBM, set the pace (200 us against 66 for the up
// product of 16 tokens, four pairs of tiles to a workgroup).  The activations of the workgroup's tokens lie in LDS,
// 28 KB of them at a time.
//
// What bounds them (16 tokens, 16 experts of 5120 x 1536 with 1 x 16 scales: up 62 us,
// 3.0 TB/s; down 43): the copies alone took 49 and 31, the arithmetic alone, with
// four pairs to a workgroup, 54 and 38; neither is hidden whole behind the other.
// With four pairs and no copies of scales, whose requests are as many as the codes',
// they took 56 and 38 instead of 65 and 42.  Half the decoding's instructions (INT4 as
// unsigned levels, the offset in the accumulator) gave 1 %, a third step in the ring
// nothing.
#include <cmath>
#include <type_traits>

#include "lds_copy.h"
#include "lm_internal.h"

namespace ufp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kBf16Max = 0x1.FEp127f;
constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kRouteThreads = 256;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// --- codes -> bf16 levels ------------------------------------------------------
// E4M3 bytes of the level magnitudes 0..7 of E1M2, and of INT4's nibbles 0..7
// and 8..15.
template <int GRID> struct Lut;
template <> struct Lut<0> { static constexpr uint32_t lo = 0x34302800u, hi = 0x3E3C3A38u; };
template <> struct Lut<1> {
  static constexpr uint32_t lo = 0x44403800u, hi = 0x4E4C4A48u;
  static constexpr uint32_t nlo = 0xCACCCED0u, nhi = 0xB8C0C4C8u;
};

// Nibbles in the low half of each byte of v (the high halves are not looked at)
// -> E4M3 bytes.
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

// The bf16 levels of 8 codes as four pairs.  E2M1 codes are FP4 values, which
// convert by themselves, two neighbours at a time: (0 1) (2 3) (4 5) (6 7); the
// uniform grids go through E4M3 bytes: (0 2) (4 6) (1 3) (5 7).
template <int GRID>
__device__ __forceinline__ u32x4 levels8(uint32_t w) {
  auto two = [](bf16x2 v) { return __builtin_bit_cast(uint32_t, v); };
  if constexpr (GRID == 2) {
    return u32x4{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0)),
                 two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1)),
                 two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2)),
                 two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3))};
  } else {
    const uint32_t ev = nib_to_e4m3<GRID>(w), od = nib_to_e4m3<GRID>(w >> 4);
    return u32x4{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(ev, 1.0f, false)),
                 two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(ev, 1.0f, true)),
                 two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(od, 1.0f, false)),
                 two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(od, 1.0f, true))};
  }
}

// The same with the codes 0..3 in the first two words and 4..7 in the others.
template <int GRID>
__device__ __forceinline__ u32x4 levels4x2(uint32_t w) {
  const u32x4 l = levels8<GRID>(w);
  if constexpr (GRID == 2) return l;
  else return u32x4{l[0], l[2], l[1], l[3]};   // (0 2) (1 3), (4 6) (5 7)
}

// --- weights in LDS -----------------------------------------------------------
// Scale kinds: fp32 or E8M0, 32- or 16-element blocks along K.
enum { kF32b32 = 0, kF32b16 = 1, kE8b32 = 2, kE8b16 = 3 };
template <int SK> struct Sk {
  static constexpr bool e8 = SK >= 2;
  static constexpr int per = (SK & 1) ? 2 : 1;   // scales per 32 elements
};

// A wave's ring: kRing steps of two 16-row tiles, each 1 KB of codes and the
// scales of 16 rows.  Two steps and 28 KB of activations let two workgroups
// share a compute unit: while one waits for its tokens' activations or adds
// up, the other one reads.
constexpr int kRing = 2;
template <int SK> constexpr int scale_bytes() { return (Sk<SK>::e8 ? 128 : 256) * Sk<SK>::per; }
template <int SK> constexpr int tile_bytes() { return 1024 + scale_bytes<SK>(); }
template <int SK> constexpr int ring_bytes() { return kRing * 2 * tile_bytes<SK>(); }
constexpr int kCopies = 4;   // loads per wave and step
constexpr int kActBytes = 28 * 1024;

// Where a 16-row tile comes from.
struct TileSource {
  sgpr4 codes, scales;
  uint32_t vcodes, vscales;   // this lane's offsets at step 0
  uint32_t shift;             // E8M0: where in its word this lane's row starts
};

// row0: the tile's first row (a multiple of 16) in the stacked matrix of K
// columns.  Past the tile's end the loads give zeros; between rows they give
// the next row's bytes, which no block below K / 32 meets.
template <int SK>
__device__ __forceinline__ TileSource tile_source(const MoeWeight& w, int64_t row0, int64_t K,
                                                  int lane) {
  constexpr int P = Sk<SK>::per;
  TileSource t;
  const uint32_t half = (uint32_t)(K / 2);
  t.codes = rsrc4(w.codes + row0 * half, 16 * half);
  // lane l: row l / 4, its 16-byte chunk in the place l % 4 of the row's 64
  // bytes; places are exchanged by row / 4 so that the 64 lanes' word reads
  // below fall on 64 banks
  const int r = lane >> 2;
  t.vcodes = (uint32_t)r * half + 16u * (uint32_t)((lane & 3) ^ (r >> 2));
  const uint8_t* s = w.scales + (row0 >> w.row_shift) * w.scale_pitch;
  const uint32_t pitch = w.row_shift ? 0u : (uint32_t)w.scale_pitch;   // square blocks: one row
  t.shift = 0;
  if constexpr (!Sk<SK>::e8) {
    t.scales = rsrc4(s, 15 * pitch + (uint32_t)w.scale_pitch);
    // 16 bytes of fp32 scales per lane, one (b32) or two (b16) lanes per row
    t.vscales = (uint32_t)(lane / P) * pitch + 16u * (uint32_t)(lane % P);
  } else {
    // bytes at any alignment: whole words around them, two (b32) or four (b16)
    // per row
    const uint32_t off = (uint32_t)((uintptr_t)s & 3);
    t.scales = rsrc4(s - off, (off + 15 * pitch + (uint32_t)w.scale_pitch + 3) & ~3u);
    constexpr int W = 2 * P;
    t.vscales = ((off + (uint32_t)(lane / W) * pitch) & ~3u) + 4u * (uint32_t)(lane % W);
    t.shift = (off + (uint32_t)(lane & 15) * pitch) & 3;
  }
  return t;
}

// Copies step `step` (elements 128 step ..) of a tile to LDS address `to`.
template <int SK>
__device__ __forceinline__ void copy_tile(const TileSource& t, uint32_t to, int step, int lane) {
  constexpr int P = Sk<SK>::per;
  lds_load16(to, t.codes, t.vcodes, 64u * (uint32_t)step);
  if constexpr (!Sk<SK>::e8) {
    if (lane < 16 * P) lds_load16(to + 1024, t.scales, t.vscales, 16u * P * (uint32_t)step);
  } else {
    if (lane < 32 * P) lds_load4(to + 1024, t.scales, t.vscales, 4u * P * (uint32_t)step);
  }
}

// The four blocks' scales of this lane's row (column of the instruction).
template <int SK>
__device__ __forceinline__ void read_scales(const uint8_t* tile, uint32_t shift, int r16,
                                            float (&s)[4 * Sk<SK>::per]) {
  constexpr int P = Sk<SK>::per;
  if constexpr (!Sk<SK>::e8) {
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(tile + 1024 + 16 * (P * r16 + q));
#pragma unroll
      for (int i = 0; i < 4; ++i) s[4 * q + i] = v[i];
    }
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(tile + 1024 + 8 * P * r16);
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const uint32_t b = __builtin_amdgcn_alignbyte(w[q + 1], w[q], shift);
#pragma unroll
      for (int i = 0; i < 4; ++i)   // 2^(byte - 127)
        s[4 * q + i] = __builtin_ldexpf(1.0f, (int)__builtin_amdgcn_ubfe(b, 8 * i, 8) - 127);
    }
  }
}

// --- activations in LDS ---------------------------------------------------------
// Row i, 32 bytes per 8 elements: the upper bf16 pieces and then the lower ones
// of what lane group g of the instruction takes of a 32-element block: its
// elements 8 g .. 8 g + 7 where the block has one scale (MFMA over 32 of K);
// 4 g .. 4 g + 3 of the first 16 and of the second 16 where it has two (two
// MFMAs over 16).  The 16-byte chunks of a row are exchanged by its number, so
// that 16 rows read at one place fall on all banks (row_bytes is a multiple
// of 16 chunks).
__device__ __forceinline__ uint32_t act_chunk(int row, int row_bytes, int chunk) {
  return (uint32_t)(row * row_bytes + 16 * (chunk ^ (row & 15)));
}

// Where this lane reads, of its row of token tile t: [t][parity of the block]
// [upper, lower], without the step's 512 bytes and the block pair's 256.
template <int TT>
struct ActReads {
  uint32_t at[TT][2][2];
};
template <int TT>
__device__ __forceinline__ ActReads<TT> act_reads(const int (&arow)[TT], int row_bytes, int g) {
  ActReads<TT> a;
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int b = 0; b < 2; ++b) a.at[t][q][b] = act_chunk(arow[t], row_bytes, 8 * q + 2 * g + b);
  return a;
}

// One step of both tiles against TT tiles of 16 tokens.  acts: LDS, at the
// step's activations.  WHOLE: all four blocks are inside K.
template <int GRID, int SK, int TT, bool WHOLE>
__device__ __forceinline__ void add_step(f32x4 (&acc)[2][TT], const uint8_t* ring,
                                         const TileSource (&src)[2], const uint8_t* acts,
                                         const ActReads<TT>& reads, int blocks, int lane) {
  constexpr int P = Sk<SK>::per;
  const int g = lane >> 4, r16 = lane & 15;
  uint32_t code[2][4];
  float s[2][4 * P];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const uint8_t* t = ring + m * tile_bytes<SK>();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t* w =
          reinterpret_cast<const uint32_t*>(t + 64 * r16 + 16 * (j ^ (r16 >> 2)));
      if constexpr (P == 1) code[m][j] = w[g];
      else   // half of a word of each 16: codes 4 g .. 4 g + 3 of both
        code[m][j] = __builtin_amdgcn_perm(w[2 + (g >> 1)], w[g >> 1],
                                           (g & 1) ? 0x07060302u : 0x05040100u);
    }
    read_scales<SK>(t, src[m].shift, r16, s[m]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!WHOLE && j >= blocks) break;
    // several token tiles: one block's activations at a time fit the registers
    if constexpr (TT > 1) __builtin_amdgcn_sched_barrier(0);
    u32x4 hi[TT], lo[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const uint8_t* a = acts + 256 * (j >> 1);
      hi[t] = *reinterpret_cast<const u32x4*>(a + reads.at[t][j & 1][0]);
      lo[t] = *reinterpret_cast<const u32x4*>(a + reads.at[t][j & 1][1]);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if constexpr (P == 1) {
        const bf16x8 b = __builtin_bit_cast(bf16x8, levels8<GRID>(code[m][j]));
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
          x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, lo[t]), b, x, 0, 0,
                                                      0);
          x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, hi[t]), b, x, 0, 0,
                                                      0);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][t][r] = __builtin_fmaf(x[r], s[m][j], acc[m][t][r]);
        }
      } else {
        const u32x4 l = levels4x2<GRID>(code[m][j]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          auto half = [q](const u32x4& v) {
            return __builtin_bit_cast(i16x4, u32x2{v[2 * q], v[2 * q + 1]});
          };
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
            x = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(half(lo[t]), half(l), x, 0, 0, 0);
            x = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(half(hi[t]), half(l), x, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[m][t][r] = __builtin_fmaf(x[r], s[m][2 * j + q], acc[m][t][r]);
          }
        }
      }
    }
  }
}

// LDS address of a pointer into LDS.
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p;
}

// What a wave of a workgroup with `pairs` pairs of tiles does: of pair pt the
// steps ks, ks + shares, .. of K.  Waves that are left over only help to fill.
struct Share {
  int pt, ks, shares;
  bool works;
};
__device__ __forceinline__ Share share_of(int wave, int pairs) {
  // kWaves / pairs and wave / pairs, by tables of the quotients and of 64 / pairs
  // rounded up
  const int shares = (int)(0x11112248u >> (4 * (pairs - 1)) & 15);
  const int ks = wave * (int)(0x080A0B0D10162040ull >> (8 * (pairs - 1)) & 255) >> 6;
  return Share{wave - ks * pairs, ks, shares, ks < shares};
}

// acc += the product over K of a workgroup's two tiles per wave (src) with its
// tokens.  fill(first block, blocks) puts the activations of a range of K into
// `acts`, one range after another (what kActBytes hold).
template <int GRID, int SK, int TT, class Fill>
__device__ __forceinline__ void product(f32x4 (&acc)[2][TT], const TileSource (&src)[2],
                                        uint8_t* acts, uint8_t* ring, const int (&arow)[TT],
                                        int row_bytes, int range, int nb, const Share& w, Fill fill) {
  const int lane = threadIdx.x & 63;
  const int steps = (nb + 3) / 4;
  const uint32_t ring0 = lds_addr(ring);
  const ActReads<TT> reads = act_reads<TT>(arow, row_bytes, lane >> 4);
  // the i-th step of this wave; past the last one the copies give zeros or
  // bytes that nothing reads, and keep the count of loads in flight
  auto copy = [&](int i) {
    const uint32_t to = ring0 + (uint32_t)(i % kRing) * (2 * tile_bytes<SK>());
    int step = w.ks + i * w.shares;
    if (step >= steps) step = steps - 1;
#pragma unroll
    for (int m = 0; m < 2; ++m) copy_tile<SK>(src[m], to + m * tile_bytes<SK>(), step, lane);
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i)
    if (w.works) copy(i);
  int i = 0;
  for (int b0 = 0; b0 < nb; b0 += range) {
    const int bn = nb - b0 < range ? nb - b0 : range;
    if (b0) __syncthreads();   // everyone has read the range before
    fill(b0, bn);
    __syncthreads();
    for (; w.works && w.ks + i * w.shares < (b0 + bn + 3) / 4; ++i) {
      copy(i + kRing - 1);
      wait_vmcnt<(kRing - 1) * kCopies>();   // step i is there; later ones need not be
      const int step = w.ks + i * w.shares;
      const uint8_t* from = ring + (i % kRing) * (2 * tile_bytes<SK>());
      const uint8_t* a = acts + 512 * (step - b0 / 4);
      if (4 * step + 4 <= nb)
        add_step<GRID, SK, TT, true>(acc, from, src, a, reads, 4, lane);
      else
        add_step<GRID, SK, TT, false>(acc, from, src, a, reads, nb - 4 * step, lane);
      // the ring's next copy overwrites what was just read
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  }
  wait_vmcnt<0>();   // nothing may arrive after the ring is used for something else
  __syncthreads();
}

// The shares of K added in order: part[pair][matrix][token][16 columns].
template <int TT>
__device__ __forceinline__ void join_shares(const f32x4 (&acc)[2][TT], float* part, const Share& w) {
  const int lane = threadIdx.x & 63, g = lane >> 4, r16 = lane & 15;
  constexpr int ROWS = TT * 16;
  for (int s = 0; s < w.shares; ++s) {
    if (w.ks == s) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float* d = part + ((w.pt * 2 + q) * ROWS + t * 16 + 4 * g + r) * 16 + r16;
            *d = s == 0 ? acc[q][t][r] : *d + acc[q][t][r];
          }
    }
    __syncthreads();
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

// Order-preserving key of a float, 0 for what is never chosen; equal logits have
// equal keys (the sum turns -0 into +0).
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  return l > -INFINITY ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// --- routing and the rotation of x -----------------------------------------------
// One wave: the choices of token t into ids[r], share[r], r < k (-1: none).  An
// expert's rank is the number of experts before it: larger logits, and equal
// ones of lower index.  Every lane counts it for its experts against all others
// at once.  The code runs once per wave, so its size counts as much as its
// length: unrolled over 64 experts the instruction fetches took longer than
// taking the largest k times over.  Q: experts per lane.
template <int Q>
__device__ __forceinline__ void route_token(const MoeLaunch& p, int t, int* ids, float* shares) {
  const int lane = threadIdx.x & 63;   // expert lane + 64 q in register q
  uint32_t key[Q];
  int rank[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int e = lane + 64 * q;
    key[q] = e < p.E ? logit_key(p.logits[(int64_t)t * p.ldl + e]) : 0u;
    rank[q] = 0;
  }
#pragma unroll
  for (int qo = 0; qo < Q; ++qo) {
#pragma unroll 8
    for (int j = 0; j < 64; ++j) {
      const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)key[qo], j);
#pragma unroll
      for (int q = 0; q < Q; ++q)
        rank[q] += other > key[q] || (other == key[q] && j + 64 * qo < lane + 64 * q) ? 1 : 0;
    }
  }
  // the largest logit is in the lane that holds rank 0
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const uint64_t has = __ballot(rank[q] == 0);
    if (has) top = (uint32_t)__builtin_amdgcn_readlane((int)key[q], __builtin_ctzll(has));
  }
  const float first = key_logit(top);
  float x[Q], den = 0.0f;
  int chosen = 0;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const bool in = key[q] != 0 && rank[q] < p.k;
    x[q] = 0.0f;
    if (key[q] != 0) {
      x[q] = __builtin_amdgcn_exp2f((key_logit(key[q]) - first) * kLog2e);
      if (in || !p.renorm) den += x[q];
    }
    chosen += __builtin_popcountll(__ballot(in));
  }
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) den += __shfl_xor(den, m);
#pragma unroll
  for (int q = 0; q < Q; ++q)
    if (key[q] != 0 && rank[q] < p.k) {
      ids[rank[q]] = lane + 64 * q;
      shares[rank[q]] = x[q] / den;
    }
  if (lane >= chosen && lane < p.k) {
    ids[lane] = -1;
    shares[lane] = 0.0f;
  }
}

__device__ __forceinline__ void route(const MoeLaunch& p, int t, int* ids, float* shares) {
  if (p.E <= 64) route_token<1>(p, t, ids, shares);
  else route_token<kMoeMaxExperts / 64>(p, t, ids, shares);
}

// One butterfly of eight values with the lane whose number differs in bit M:
// the lower lane gets the sum, the upper one the difference.
template <int M>
__device__ __forceinline__ void butterfly(float (&v)[8], int lane) {
  const float sign = (lane & M) ? -1.0f : 1.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    int o = (int)__float_as_uint(v[j]);
    if constexpr (M == 1) o = __builtin_amdgcn_mov_dpp(o, 0xB1, 0xF, 0xF, true);
    if constexpr (M == 2) o = __builtin_amdgcn_mov_dpp(o, 0x4E, 0xF, 0xF, true);
    if constexpr (M == 4)   // 7 - l, then 3 - l inside four
      o = __builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(o, 0x141, 0xF, 0xF, true), 0x1B, 0xF,
                                   0xF, true);
    if constexpr (M == 8) o = __builtin_amdgcn_mov_dpp(o, 0x128, 0xF, 0xF, true);   // l + 8 of 16
    v[j] = __builtin_fmaf(sign, v[j], __uint_as_float((uint32_t)o));   // exact product
  }
}

// Eight neighbouring elements of a row rotated, y = c_n (v S) H, and split into
// two bf16 pieces in the order of the weights' codebook and scales (per 32
// elements).  i: which eight of the
// row; every lane of the wave takes part, and lane l holds an i that is
// congruent to l modulo 64, so a chunk's neighbours are neighbouring lanes.
__device__ __forceinline__ void rotate8(float (&v)[8], int64_t i, int n, float cn,
                                        const uint32_t (&signs)[4], int grid, int per, u32x4& hi,
                                        u32x4& lo) {
  const int lane = threadIdx.x & 63;
  const int o = (int)(8 * i) & 127;
  const uint32_t sg = signs[o >> 5] >> (o & 31);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = __uint_as_float(__float_as_uint(v[j]) ^ ((sg >> j) << 31));
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
  if (n > 8) butterfly<1>(v, lane);
  if (n > 16) butterfly<2>(v, lane);
  if (n > 32) butterfly<4>(v, lane);
  if (n > 64) butterfly<8>(v, lane);
  // the pairs of levels8 or levels4x2
  constexpr int order8[8] = {0, 2, 4, 6, 1, 3, 5, 7}, order4[8] = {0, 2, 1, 3, 4, 6, 5, 7};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a = v[2 * j], b = v[2 * j + 1];
    if (grid != 2) {
      a = per == 1 ? v[order8[2 * j]] : v[order4[2 * j]];
      b = per == 1 ? v[order8[2 * j + 1]] : v[order4[2 * j + 1]];
    }
    a *= cn;
    b *= cn;
    // the upper piece is held to bf16's largest, so that an infinity stays one in the
    // lower piece and a float above that largest does not become one
    hi[j] = pack_bf16(__builtin_amdgcn_fmed3f(a, -kBf16Max, kBf16Max),
                      __builtin_amdgcn_fmed3f(b, -kBf16Max, kBf16Max));
    lo[j] = pack_bf16(a - __uint_as_float(hi[j] << 16), b - __uint_as_float(hi[j] & 0xFFFF0000u));
  }
}

// The pieces of the i-th eight elements of a row into the activations' layout;
// at(chunk) is the address of a 16-byte chunk of the row.
template <class At>
__device__ __forceinline__ void put8(const u32x4& hi, const u32x4& lo, int64_t i, int per, At at) {
  if (per == 1) {
    *reinterpret_cast<u32x4*>(at(2 * i)) = hi;
    *reinterpret_cast<u32x4*>(at(2 * i + 1)) = lo;
  } else {
    // elements 0..3 go to lane group g, 4..7 to g + 1, the first or second half
    const int64_t c = 8 * (i >> 2) + 4 * (i & 1);   // chunk of lane group 2 (i & 1)
    const int h = 8 * (int)(i >> 1 & 1);
    *reinterpret_cast<u32x2*>(at(c) + h) = u32x2{hi[0], hi[1]};
    *reinterpret_cast<u32x2*>(at(c + 1) + h) = u32x2{lo[0], lo[1]};
    *reinterpret_cast<u32x2*>(at(c + 2) + h) = u32x2{hi[2], hi[3]};
    *reinterpret_cast<u32x2*>(at(c + 3) + h) = u32x2{lo[2], lo[3]};
  }
}

__device__ __forceinline__ void load_x8(const uint16_t* x, bool in, int64_t i, float (&v)[8]) {
  u32x4 w = {0, 0, 0, 0};
  if (in) w = *reinterpret_cast<const u32x4*>(x + 8 * i);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// Routing and rotation once for all: token blockIdx.x, 2048 elements of it.
__global__ __launch_bounds__(kRouteThreads) void k_moe_route(MoeLaunch p) {
  const int64_t t = blockIdx.x, i = (int64_t)blockIdx.y * kRouteThreads + threadIdx.x;
  if (blockIdx.y == 0 && threadIdx.x < 64)
    route(p, (int)t, p.ids + t * p.k, p.share + t * p.k);
  const bool in = i < p.H / 8;
  float v[8];
  load_x8(p.x + t * p.ldx, in, i, v);
  u32x4 hi, lo;
  const int per = 1 + (p.wg.kind & 1);
  rotate8(v, i, p.nx, p.cnx, p.sign_x, p.wg.grid, per, hi, lo);
  if (in) put8(hi, lo, i, per, [&](int64_t c) { return p.xr + t * p.H * 4 + 16 * c; });
}

// Bytes of a row of x in LDS where all of K is there.
__host__ __device__ inline int fused_row(int64_t H) { return (int)((H * 4 + 255) / 256 * 256); }

// Blocks of 32 columns of m tokens that fit the activations' LDS, whole steps.
__device__ __forceinline__ int range_of(int m, int nb) {
  const int fit = kActBytes / (m * 128) & ~3, all = (nb + 3) & ~3;
  return fit < all ? fit : all;
}

// --- gate and up products, activation ---------------------------------------------
// A workgroup computes `pairs` times 16 columns of the intermediate from f0 on,
// each a pair of a gate and an up tile, for m of the expert's tokens, whose rows of the
// intermediate start at hrow; FUSED: x is in LDS already, row t for token t.
template <int GRID, int SK, int TT, bool FUSED>
__device__ __forceinline__ void moe_up_body(const MoeLaunch& p, int64_t hrow, int e, int f0,
                                            int pairs, int m, const int* tok, const float* share,
                                            uint8_t* lds) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15;
  const Share w = share_of(wave, pairs);
  const int nb = (int)(p.H / 32);
  const int64_t row0 = (int64_t)e * p.F + f0 + w.pt * 16;
  const TileSource src[2] = {tile_source<SK>(p.wg, row0, p.H, lane),
                             tile_source<SK>(p.wu, row0, p.H, lane)};
  uint8_t* acts = lds;
  uint8_t* ring = lds + kActBytes + wave * ring_bytes<SK>();
  int arow[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int i = t * 16 + r16;   // rows past the tokens give rows that nobody takes
    arow[t] = i < m ? (FUSED ? tok[i] : i) : 0;
  }
  f32x4 acc[2][TT];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[q][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (FUSED) {
    product<GRID, SK, TT>(acc, src, acts, ring, arow, fused_row(p.H), nb, nb, w,
                          [](int, int) {});
  } else {
    const int range = range_of(m, nb);
    const sgpr4 xr = rsrc4(p.xr, (uint32_t)(p.T * p.H * 4));
    const uint32_t to = lds_addr(acts);
    product<GRID, SK, TT>(acc, src, acts, ring, arow, range * 128, range, nb, w, [&](int b0, int) {
      // rows of 128 range bytes, 512 bytes per half wave; past K nothing is read
      const int per_row = range / 4, halves = m * per_row, hl = lane & 31;
      for (int c = 2 * wave; c < halves; c += 2 * kWaves) {
        const int h = c + (lane >> 5), i = h / per_row, part = h % per_row;
        if (h < halves)
          lds_load16(to + (uint32_t)c * 512u, xr,
                     (uint32_t)tok[i] * (uint32_t)(p.H * 4) + (uint32_t)b0 * 128u +
                         16u * (uint32_t)((part * 32 + hl) ^ (i & 15)), 0);
      }
      wait_vmcnt<0>();
    });
  }
  float* part = reinterpret_cast<float*>(lds);
  join_shares<TT>(acc, part, w);
  constexpr int ROWS = TT * 16;
  const int col = tid % (16 * kWaves);   // of 16 pairs columns
  for (int row = tid / (16 * kWaves); row < m; row += kThreads / (16 * kWaves)) {
    if (col >= 16 * pairs) continue;
    const float* at = part + ((col >> 4) * 2 * ROWS + row) * 16 + (col & 15);
    const float a = at[0] * p.wg.factor, b = at[ROWS * 16] * p.wu.factor;
    const float s = p.act == UFP4_ACT_GELU ? activation<1>(a) : activation<0>(a);
    p.h[(hrow + row) * p.F + f0 + col] = s * b * share[row];
  }
  if constexpr (TT > 1) __syncthreads();   // the next tokens' activations go where `part` is
}

// FUSED: routing and rotation here, for a few tokens.  WIDE: an expert may have
// more than 16 tokens.
enum { kFused = 0, kNarrow = 1, kWide = 2 };
template <int GRID, int SK, int MODE>
__global__ __launch_bounds__(kThreads, 4) void k_moe_up(MoeLaunch p) {
  constexpr bool FUSED = MODE == kFused;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int tok[kMoeMaxTokens];
  __shared__ float share[kMoeMaxTokens];
  __shared__ int choice[kMoeMaxTokens];
  __shared__ int ids_here[FUSED ? kMoeFusedTokens * kMoeMaxChoices : 1];
  __shared__ float share_here[FUSED ? kMoeFusedTokens * kMoeMaxChoices : 1];
  __shared__ int found[3];   // expert, tokens, their first row
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fc = blockIdx.x, slot = blockIdx.y;
  const int* ids = p.ids;
  const float* shares = p.share;
  if constexpr (FUSED) {
    for (int t = wave; t < p.T; t += kWaves)
      route(p, t, ids_here + t * p.k, share_here + t * p.k);
    // the waves that route take the last part of x
    const int bytes = fused_row(p.H);
    for (int t = 0; t < p.T; ++t)
      for (int64_t i0 = (kWaves - 1 - wave) * 64; i0 < p.H / 8; i0 += kThreads) {
        const int64_t i = i0 + lane;
        const bool in = i < p.H / 8;
        float v[8];
        load_x8(p.x + t * p.ldx, in, i, v);
        u32x4 hi, lo;
        rotate8(v, i, p.nx, p.cnx, p.sign_x, p.wg.grid, Sk<SK>::per, hi, lo);
        if (in)
          put8(hi, lo, i, Sk<SK>::per, [&](int64_t c) { return lds + act_chunk(t, bytes, (int)c); });
      }
    ids = ids_here;
    shares = share_here;
    __syncthreads();
  }
  if (tid < 64) {
    const int pairs = (int)(p.T * p.k);
    // by_pair: slot s stands for the s-th choice, unless the same expert
    // was chosen before it; else for expert s
    int e = slot;
    bool mine = true;
    if (p.by_pair) {
      e = ids[slot];
      if (e < 0) {
        mine = false;
      } else {
        bool before = false;
        for (int i0 = 0; i0 < slot; i0 += 64) {
          const int i = i0 + lane;
          before |= __any(i < slot && ids[i < slot ? i : 0] == e);
        }
        mine = !before;
      }
    }
    // the rows of the intermediate go by experts: those of lower ones come first
    int m = 0, row0 = 0;
    for (int i0 = 0; i0 < pairs; i0 += 64) {
      const int i = i0 + lane;
      const int id = ids[i < pairs ? i : 0];
      const bool hit = mine && i < pairs && id == e;
      const uint64_t mask = __ballot(hit);
      if (hit) {
        const int at = m + __builtin_popcountll(mask & (((uint64_t)1 << lane) - 1));
        tok[at] = i / p.k;
        share[at] = shares[i];
        choice[at] = i;
      }
      if (fc == 0 && slot == 0 && i < pairs && id < 0) p.place[i] = -1;
      m += __builtin_popcountll(mask);
      row0 += __builtin_popcountll(__ballot(i < pairs && id >= 0 && id < e));
    }
    if (lane == 0) {
      found[0] = e;
      found[1] = m;
      found[2] = row0;
      if (fc == 0) {   // for the down product
        p.expert[slot] = e;
        p.count[slot] = m;
        p.row0[slot] = row0;
      }
    }
  }
  __syncthreads();
  const int e = __builtin_amdgcn_readfirstlane(found[0]);
  const int m = __builtin_amdgcn_readfirstlane(found[1]);
  const int row0 = __builtin_amdgcn_readfirstlane(found[2]);
  if (m == 0) return;
  if (fc == 0 && tid < m) p.place[choice[tid]] = row0 + tid;   // for the join
  const int pair0 = fc * p.run_up, left = (int)(p.F / 16) - pair0;
  const int pairs = left < p.run_up ? left : p.run_up;
  auto body = [&](auto tt, int first, int n) {
    moe_up_body<GRID, SK, decltype(tt)::value, FUSED>(p, row0 + first, e, 16 * pair0, pairs, n,
                                                      tok + first, share + first, lds);
  };
  if (MODE != kWide || m <= 16) {
    body(std::integral_constant<int, 1>{}, 0, m);
  } else if constexpr (MODE == kWide) {
    for (int i = 0; i < m; i += 32) body(std::integral_constant<int, 2>{}, i, m - i < 32 ? m - i : 32);
  }
}

// --- down product --------------------------------------------------------------------
// A workgroup computes `pairs` times 32 output columns from col0 on, each a pair of
// tiles.  hrow: the tokens' first row of the intermediate and of the results.
template <int GRID, int SK, int TT>
__device__ __forceinline__ void moe_down_body(const MoeLaunch& p, int64_t hrow, int e, int m,
                                              int64_t col0, int pairs, uint8_t* lds) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15;
  const Share w = share_of(wave, pairs);
  const int nb = (int)(p.F / 32);
  const int64_t row0 = (int64_t)e * p.H + col0 + w.pt * 32;
  const TileSource src[2] = {tile_source<SK>(p.wd, row0, p.F, lane),
                             tile_source<SK>(p.wd, row0 + 16, p.F, lane)};
  uint8_t* acts = lds;
  uint8_t* ring = lds + kActBytes + wave * ring_bytes<SK>();
  int arow[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int i = t * 16 + r16;
    arow[t] = i < m ? i : 0;
  }
  f32x4 acc[2][TT];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[q][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int range = range_of(m, nb);
  product<GRID, SK, TT>(acc, src, acts, ring, arow, range * 128, range, nb, w, [&](int b0, int bn) {
    // one row after another, 64 times 8 neighbouring elements per wave
    const int groups = 4 * bn, runs = (groups + 63) / 64;
    for (int c = wave; c < m * runs; c += kWaves) {
      const int row = c / runs, i = (c % runs) * 64 + lane;
      float v[8] = {};
      if (i < groups) {
        const f32x4* h = reinterpret_cast<const f32x4*>(
            p.h + (hrow + row) * p.F + 32 * (int64_t)b0 + 8 * i);
        const f32x4 a = h[0], b = h[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[4 + j] = b[j]; }
      }
      u32x4 hi, lo;
      rotate8(v, 4 * (int64_t)b0 + i, p.nh, p.cnh, p.sign_h, p.wd.grid, Sk<SK>::per, hi, lo);
      if (i < groups)
        put8(hi, lo, i, Sk<SK>::per,
             [&](int64_t c) { return acts + act_chunk(row, range * 128, (int)c); });
    }
  });
  float* part = reinterpret_cast<float*>(lds);
  constexpr int ROWS = TT * 16;
  join_shares<TT>(acc, part, w);
  const int col = tid % (32 * kWaves);   // of 32 pairs columns
  for (int row = tid / (32 * kWaves); row < m; row += kThreads / (32 * kWaves))
    if (col < 32 * pairs)
      p.partial[(hrow + row) * p.H + col0 + col] = part[((col >> 4) * ROWS + row) * 16 + (col & 15)];
  if constexpr (TT > 1) __syncthreads();   // the next tokens' activations go where `part` is
}

template <int GRID, int SK, bool WIDE>
__global__ __launch_bounds__(kThreads, 4) void k_moe_down(MoeLaunch p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int slot = blockIdx.y;
  const int m = p.count[slot], e = p.expert[slot], row0 = p.row0[slot];
  if (m == 0) return;
  const int pair0 = (int)blockIdx.x * p.run_down, left = (int)(p.H / 32) - pair0;
  const int pairs = left < p.run_down ? left : p.run_down;
  auto body = [&](auto tt, int first, int n) {
    moe_down_body<GRID, SK, decltype(tt)::value>(p, row0 + first, e, n,
                                                 32 * (int64_t)pair0, pairs, lds);
  };
  if (!WIDE || m <= 16) {
    body(std::integral_constant<int, 1>{}, 0, m);
  } else if constexpr (WIDE) {
    for (int i = 0; i < m; i += 32) body(std::integral_constant<int, 2>{}, i, m - i < 32 ? m - i : 32);
  }
}

// y_t: its choices' sums in their order; two columns per thread.
__global__ __launch_bounds__(kRouteThreads) void k_moe_join(MoeLaunch p) {
  const int64_t col = 2 * ((int64_t)blockIdx.x * kRouteThreads + threadIdx.x), t = blockIdx.y;
  if (col >= p.H) return;
  f32x2 v = {0.0f, 0.0f};
  for (int r0 = 0; r0 < p.k; r0 += 8) {   // eight rows in flight
    int at[8];
    f32x2 part[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) at[r] = r0 + r < p.k ? p.place[t * p.k + r0 + r] : -1;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      part[r] = f32x2{0.0f, 0.0f};
      if (at[r] >= 0)
        part[r] = *reinterpret_cast<const f32x2*>(p.partial + (int64_t)at[r] * p.H + col);
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) v += part[r];
  }
  *reinterpret_cast<uint32_t*>(p.y + t * p.ldy + col) =
      pack_bf16(v[0] * p.wd.factor, v[1] * p.wd.factor);
}

// LDS of a product: activations and rings; the shares of K of two tiles by 128
// columns and 32 tokens take their place at the end.
template <int SK> constexpr int lds_bytes() { return kActBytes + kWaves * ring_bytes<SK>(); }
static_assert(lds_bytes<kE8b32>() >= 2 * 128 * 32 * 4, "the shares of K fit");
static_assert(kActBytes >= 32 * 512, "one step of 32 tokens fits");

template <int GRID, int SK>
hipError_t launch_up(const MoeLaunch& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.F / 16 + p.run_up - 1) / p.run_up), (unsigned)p.slots);
  auto go = [&](auto mode) {
    constexpr int MODE = decltype(mode)::value;
    static std::atomic<uint64_t> lds_set{0};
    const hipError_t e =
        set_lds_limit((const void*)k_moe_up<GRID, SK, MODE>, lds_bytes<SK>(), lds_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_moe_up<GRID, SK, MODE>), grid, dim3(kThreads), lds_bytes<SK>(), s, p);
    return hipGetLastError();
  };
  if (p.fused) return go(std::integral_constant<int, kFused>{});
  return p.T <= 16 ? go(std::integral_constant<int, kNarrow>{})
                   : go(std::integral_constant<int, kWide>{});
}

template <int GRID, int SK>
hipError_t launch_down(const MoeLaunch& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.H / 32 + p.run_down - 1) / p.run_down), (unsigned)p.slots);
  auto go = [&](auto wide) {
    constexpr bool WIDE = decltype(wide)::value;
    static std::atomic<uint64_t> lds_set{0};
    const hipError_t e =
        set_lds_limit((const void*)k_moe_down<GRID, SK, WIDE>, lds_bytes<SK>(), lds_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_moe_down<GRID, SK, WIDE>), grid, dim3(kThreads), lds_bytes<SK>(), s,
                       p);
    return hipGetLastError();
  };
  return p.T <= 16 ? go(std::false_type{}) : go(std::true_type{});
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

// Pairs of tiles per workgroup, of `pairs` of each expert, where `experts` of them
// have `tokens` each, in the mean.  The cost, in the time that a compute unit
// takes for a pair: the fullest unit's workgroups, each with its pairs (half of one
// more where there are three: two waves have nothing to do) and a fixed part for
// routing, joining and the tokens' activations; and once the time that a wave
// takes for its share of K with the unit to itself.  Workgroups of up to 4 % of the
// units more than a round share a unit with another and cost no round of their own
// (one token, 264 workgroups of two pairs: up product 14.6 us, 15.1 with 132 of four).
// Three pairs have the two shares of four, and pay for K long enough that the first
// copies' latency does not count: of K = 1408 the down product of one token takes 10.6
// with 3 and 8.7 with 2, of two tokens 15.4 and 11.4; of K = 5120 the up product below
// gains.  The border lies between: from K = 1408 to 2944 three pairs would still gain
// 2 to 7 % over four in the up product of 16 experts and 16 tokens, and lose 4 to 25 %
// against two in the down product (K = 1536) of 64 experts and 4 tokens.  Of equals the
// most pairs.
// Measured, in us with 2 / 3 / 4 / 8 pairs: up product, 16 experts of 5120 x 1536
// and 16 tokens: 65.7 / 61.4 / 67.2 / 69.8; 64 of 2048 x 1408, 16 tokens: 56.0 / 60.4 /
// 55.1 / 68.1; 61 tokens: 74.8 / 68.5 / 62.0 / 58.4, and its down product 49.9 /
// 46.1 / 39.0 / 35.6.
int32_t run_pairs(int64_t pairs, int64_t K, double experts, double tokens) {
  constexpr double kUnits = 256;
  int32_t best = 1;
  double least = 1e300;
  for (int32_t w : {1, 2, 3, 4, 8}) {
    if (w == 3 && K < 24 * 128) continue;
    const double per_unit = std::ceil((double)((pairs + w - 1) / w) * experts / kUnits - 0.04);
    const double cost = per_unit * (w + (w == 3 ? 0.5 : 0.0) + 1.5 + tokens / 8) + 4.0 / (kWaves / w);
    if (cost <= least) {
      least = cost;
      best = w;
    }
  }
  return best;
}

// Workspace parts, in this order, each 256-byte aligned.
int64_t moe_plan(MoeLaunch& p, uint8_t* ws) {
  const int64_t pairs = p.T * p.k;
  p.by_pair = pairs < p.E;
  p.slots = (int32_t)(p.by_pair ? pairs : p.E);
  p.fused = p.T <= kMoeFusedTokens && p.T * fused_row(p.H) <= kActBytes;
  // distinct experts that T evenly spread choices of k meet
  double miss = 1.0;
  for (int64_t t = 0; t < p.T; ++t) miss *= 1.0 - (double)p.k / (double)p.E;
  const double experts = (1.0 - miss) * (double)p.E;
  const double tokens = experts > 0.0 ? (double)pairs / experts : 0.0;
  p.run_up = run_pairs(p.F / 16, p.H, experts, tokens);
  p.run_down = run_pairs(p.H / 32, p.F, experts, tokens);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* q = ws ? ws + at : nullptr;
    at += up256(bytes);
    return q;
  };
  p.ids = reinterpret_cast<int*>(take(p.fused ? 0 : 4 * pairs));
  p.share = reinterpret_cast<float*>(take(p.fused ? 0 : 4 * pairs));
  p.expert = reinterpret_cast<int*>(take(4 * p.slots));
  p.count = reinterpret_cast<int*>(take(4 * p.slots));
  p.row0 = reinterpret_cast<int*>(take(4 * p.slots));
  p.place = reinterpret_cast<int*>(take(4 * pairs));
  p.xr = take(p.fused ? 0 : 4 * p.T * p.H);
  p.h = reinterpret_cast<float*>(take(4 * pairs * p.F));
  p.partial = reinterpret_cast<float*>(take(4 * pairs * p.H));
  return at;
}

hipError_t launch_moe_tokens(const MoeLaunch& p, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (!p.fused) {
    const unsigned runs = (unsigned)((p.H / 8 + kRouteThreads - 1) / kRouteThreads);
    hipLaunchKernelGGL(k_moe_route, dim3((unsigned)p.T, runs), dim3(kRouteThreads), 0, s, p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  e = by_format(p.wg, [&](auto g, auto k) {
    return launch_up<decltype(g)::value, decltype(k)::value>(p, s);
  });
  if (e != hipSuccess) return e;
  e = by_format(p.wd, [&](auto g, auto k) {
    return launch_down<decltype(g)::value, decltype(k)::value>(p, s);
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_moe_join,
                     dim3((unsigned)((p.H / 2 + kRouteThreads - 1) / kRouteThreads), (unsigned)p.T),
                     dim3(kRouteThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace ufp4
