// Softmax cross entropy of a linear layer over a large vocabulary, and its
// gradients, in pieces of the vocabulary: the logits are never stored.
//
//   z = h W^T                        h [T][D], W [V][D] bf16; fp32 sums
//   lse_t = log sum_v e^z_tv         loss_t = lse_t - z_t,target
//   G_tv = a_t e^(z_tv - lse_t) - b_t [v = target_t]
//   dh = G W        dW = G^T h
// with b = dloss (0 where the target is no class) and a = b + dlse.
//
// Forward: one product whose 256 x 256 tiles end in a running maximum and sum
// of exponentials per token instead of a store; a small kernel joins the tiles.
// Backward, for one piece of the vocabulary after another: the product again,
// whose tiles end in G / s (bf16: the operand type of the two products that
// follow; half a step of rounding per element, averaged over the long sums),
// then dh += G W in fp32 and dW = G^T h, both times s where they are rounded.
// s is the largest |dloss|: with the usual equal dloss G / s is p - [v =
// target], whose heavy entries near -1 round to almost nothing, while the
// rounding of dloss itself would be the same in every one of them (measured on
// 8192 tokens: 3.4e-3 of the norm without, 1.8e-3 with s).  Every product runs as C[m][n] = sum_k
// A[m][k] B[n][k] with both operands K-contiguous, so h, the piece of W and G
// are also laid out transposed (plain tiled copies: 16 us for h and 65 for each of four
// pieces of W in a step of 4096 tokens, 65536 classes, 5120 wide, 2.6 % of its
// 10.4 ms; G leaves its tiles in both orders).
//
// The products are bound by the matrix cores: v_mfma_f32_32x32x16_bf16, 256 x
// 256 tiles, eight waves of 128 x 64 (two to a SIMD: while one of them waits to
// issue a copy or an LDS read, the other one feeds the matrix core), operands
// copied HBM -> LDS by buffer_load ... lds in 128-byte rows with XOR-swizzled
// 16-byte chunks.  The output's contiguous dimension is m, because a lane of the
// instruction holds four consecutive m of one n: 8- and 16-byte stores, and
// the softmax statistics of a token (an n) are almost all inside one lane.
#include "gemm_epilogue.h"
#include "lds_copy.h"
#include "lm_internal.h"

namespace ufp4 {

namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Byte offset of 16-byte chunk c of tile row `row` in LDS (128-byte rows,
// chunks XOR-swizzled so that 16 consecutive rows reading one chunk fill all
// 64 banks).
__device__ __forceinline__ uint32_t off128(int row, int c) {
  return (uint32_t)(row * 128 + 16 * (c ^ ((row >> 1) & 7)));
}

// What a tile ends in.
enum { kStats = 0, kGrad = 1, kSlab = 2, kOut = 3 };

// Operands [rows][ld] of a product with m over A's rows and n over B's.
struct Prod {
  const uint16_t* a;
  const uint16_t* b;
  int64_t M, N, K;          // K: elements contracted (a multiple of 8)
  int64_t lda, ldb;         // row pitches in elements
  int32_t tiles_m, tiles_n, tiles, splits;
  int64_t k_per_split;      // a multiple of 64
  // kStats: partials [WM tiles_m][part_ld] (maximum, sum), logits of the targets
  float2* part;
  int64_t part_ld;
  float* zt;
  // kStats, kGrad
  const int64_t* targets;   // class of n; m + m0 is the class of m
  int64_t m0, classes;
  const float* lse;
  const float* dloss;
  const float* dlse;
  const float* scale;       // kGrad, kOut: s
  // kGrad, kOut: bf16 [N][ldo], m contiguous, m < m_store written
  uint16_t* out;
  int64_t ldo, m_store, n_store;
  uint16_t* out_t;          // kGrad: the same turned, [m_store][ldt], columns n < ldt
  int64_t ldt;
  // kSlab: fp32 [splits][N][M], added to unless `first`
  float* slab;
  int32_t first;
};

// Tile shape: WM x WN waves of (32 NI) x (32 NJ), ST stages of 64 k in LDS.
template <int WM_, int WN_, int NI_, int NJ_, int ST_>
struct Shape {
  static constexpr int WM = WM_, WN = WN_, NI = NI_, NJ = NJ_, ST = ST_;
  static constexpr int TM = WM * NI * 32, TN = WN * NJ * 32;
  static constexpr int STAGE = (TM + TN) * 128;
  static constexpr int W = WM * WN, THREADS = 64 * W;
  static constexpr int LA = TM / 8 / W, LB = TN / 8 / W;   // 8-row copies per wave and step
  static_assert(LA * 8 * W == TM && LB * 8 * W == TN, "the waves share the rows evenly");
};
using Big = Shape<2, 4, 4, 2, 2>;
// For up to 32 or 64 tokens, where reading W is all that counts: 128 classes per
// workgroup and four stages, so that 60 KB of every compute unit's share are
// in flight (the 256 x 256 tile on 7 tokens, 32003 classes, 2048 wide: 48 us)
using Thin32 = Shape<4, 1, 1, 1, 4>;
using Thin64 = Shape<4, 1, 1, 2, 4>;

// The swizzle's part that differs between a wave's 8-row loads.
__device__ __forceinline__ uint32_t chunk_flip(int row8) { return (uint32_t)(row8 & 1) << 6; }

template <class S>
struct Ctx {
  sgpr4 ra, rb;
  uint32_t lds0;
  uint32_t va[S::LA], vb[S::LB];
  uint32_t kbytes, cbyte;    // bytes of K in this split, this lane's chunk within a step
  int wave, nsteps;
};

// The q-th of a wave's LA + LB copies of step `step` (64 k) into stage `st`.
// Past the last step the last one is copied again, and not read; chunks past
// K read as zeros.
template <class S>
__device__ __forceinline__ void issue_one(const Ctx<S>& c, int step, int st, int q) {
  const int s = step < c.nsteps ? step : c.nsteps - 1;
  const uint32_t koff = (uint32_t)s * 128u;
  const bool in_a = q < S::LA;
  const int row8 = in_a ? c.wave * S::LA + q : c.wave * S::LB + (q - S::LA);
  uint32_t v = in_a ? c.va[in_a ? q : 0] : c.vb[in_a ? 0 : q - S::LA];
  if (koff + 128u > c.kbytes && koff + (c.cbyte ^ chunk_flip(row8)) >= c.kbytes)
    v = 0x7FFFFF00u;   // outside every buffer: zeros
  const uint32_t to =
      c.lds0 + (uint32_t)st * S::STAGE + (uint32_t)(in_a ? row8 : S::TM / 8 + row8) * 1024u;
  if (in_a) lds_load16(to, c.ra, v, koff);
  else lds_load16(to, c.rb, v, koff);
}

template <class S>
struct Frags {
  bf16x8 a[S::NI], b[S::NJ];
};

// The q-th fragment of quarter s of a stage: the first row tile of A and all of
// B, which the first MFMAs need, come first.
template <class S>
__device__ __forceinline__ void read_one(Frags<S>& f, const uint8_t* stage, int s, int q, int lane,
                                         int wm, int wn) {
  const int c = 2 * s + (lane >> 5), r = lane & 31;
  if (q >= 1 && q <= S::NJ) {
    f.b[q - 1] = *reinterpret_cast<const bf16x8*>(
        stage + S::TM * 128 + off128(wn * S::NJ * 32 + (q - 1) * 32 + r, c));
  } else {
    const int i = q == 0 ? 0 : q - S::NJ;
    f.a[i] = *reinterpret_cast<const bf16x8*>(stage + off128(wm * S::NI * 32 + i * 32 + r, c));
  }
}

// A quarter's MFMAs on `f`, and among them the reads of the next quarter's
// fragments (quarter s of `stage`) and COUNT copies from number FIRST on.
template <class S, int FIRST, int COUNT>
__device__ __forceinline__ void quarter(floatx16 (&acc)[S::NI][S::NJ], const Frags<S>& f,
                                        Frags<S>& next, const uint8_t* stage, int s,
                                        const Ctx<S>& c, int step, int st, int lane, int wm,
                                        int wn) {
  constexpr int M = S::NI * S::NJ, R = S::NI + S::NJ;
#pragma unroll
  for (int m = 0; m < M; ++m) {
#pragma unroll
    for (int q = 0; q < R; ++q)
      if (q * M / R == m) read_one<S>(next, stage, s, q, lane, wm, wn);
    if constexpr (COUNT > 0) {
#pragma unroll
      for (int q = 0; q < COUNT; ++q)
        if (q * M / COUNT == m) issue_one<S>(c, step, st, FIRST + q);
    }
    acc[m / S::NJ][m % S::NJ] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
        f.a[m / S::NJ], f.b[m % S::NJ], acc[m / S::NJ][m % S::NJ], 0, 0, 0);
  }
}

// The tile as bf16 in LDS and from there to memory in whole rows.  store_nm:
// rows n of m (a lane holds four neighbouring m of one n); store_mn: rows m of
// n.  dst is the tile's first element; only m < m_end and n < n_end are written
// (multiples of 8 along a row).  16-byte chunks of a row are exchanged by its
// number, so that both the writes and the row reads spread over the banks.
template <class S, int ROWS, int COLS>
__device__ __forceinline__ void rows_out(const uint8_t* lds, uint16_t* dst, int64_t ld,
                                         int64_t row_end, int64_t col_end) {
  constexpr int C = COLS / 8;   // chunks of a row
  for (int i = threadIdx.x; i < ROWS * C; i += S::THREADS) {
    const int r = i / C, c = i % C;
    if (r < row_end && 8 * c < col_end)
      *reinterpret_cast<u32x4*>(dst + r * ld + 8 * c) =
          *reinterpret_cast<const u32x4*>(lds + r * (COLS * 2) + 16 * (c ^ (r & (C - 1))));
  }
}

template <class S>
__device__ __forceinline__ void store_nm(const floatx16 (&acc)[S::NI][S::NJ], uint8_t* lds,
                                         uint16_t* dst, int64_t ld, int64_t m_end, int64_t n_end,
                                         int wm, int wn) {
  const int lane = threadIdx.x & 63;
  constexpr int C = S::TM / 8;
#pragma unroll
  for (int j = 0; j < S::NJ; ++j) {
    const int n = wn * S::NJ * 32 + j * 32 + (lane & 31);
#pragma unroll
    for (int i = 0; i < S::NI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = (wm * S::NI * 32 + i * 32 + 8 * q) / 8;
        const u32x2 w = {pack_bf16(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                         pack_bf16(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3])};
        *reinterpret_cast<u32x2*>(lds + n * (S::TM * 2) + 16 * (c ^ (n & (C - 1))) +
                                  8 * (lane >> 5)) = w;
      }
  }
  __syncthreads();
  rows_out<S, S::TN, S::TM>(lds, dst, ld, n_end, m_end);
}

template <class S>
__device__ __forceinline__ void store_mn(const floatx16 (&acc)[S::NI][S::NJ], uint8_t* lds,
                                         uint16_t* dst, int64_t ld, int64_t m_end, int64_t n_end,
                                         int wm, int wn) {
  const int lane = threadIdx.x & 63;
  constexpr int C = S::TN / 8;
#pragma unroll
  for (int j = 0; j < S::NJ; ++j) {
    const int n = wn * S::NJ * 32 + j * 32 + (lane & 31);
#pragma unroll
    for (int i = 0; i < S::NI; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int m = wm * S::NI * 32 + i * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        *reinterpret_cast<uint16_t*>(lds + m * (S::TN * 2) + 16 * ((n >> 3) ^ (m & (C - 1))) +
                                     2 * (n & 7)) =
            (uint16_t)pack_bf16(acc[i][j][r], 0.0f);
      }
  }
  __syncthreads();
  rows_out<S, S::TM, S::TN>(lds, dst, ld, m_end, n_end);
}

template <class S, int EPI>
__global__ __launch_bounds__(S::THREADS) void k_prod(Prod p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN, h = lane >> 5;
  const int split = blockIdx.x / p.tiles, b = blockIdx.x % p.tiles;
  int tm, tn;
  tile_order(b, p.tiles, p.tiles_m, p.tiles_n, tm, tn);
  const int64_t row0 = (int64_t)tm * S::TM, col0 = (int64_t)tn * S::TN;
  const int64_t k0 = (int64_t)split * p.k_per_split;
  const int64_t kn = p.K - k0 < p.k_per_split ? p.K - k0 : p.k_per_split;
  const int64_t rows = p.M - row0 < S::TM ? p.M - row0 : S::TM;
  const int64_t cols = p.N - col0 < S::TN ? p.N - col0 : S::TN;

  Ctx<S> c;
  c.wave = wave;
  c.kbytes = (uint32_t)(2 * kn);
  c.nsteps = (int)((kn + 63) / 64);
  c.ra = rsrc4(p.a + row0 * p.lda + k0, (uint32_t)(2 * ((rows - 1) * p.lda + kn)));
  c.rb = rsrc4(p.b + col0 * p.ldb + k0, (uint32_t)(2 * ((cols - 1) * p.ldb + kn)));
  c.lds0 = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)lds;
  // lane i of a wave load covers row i / 8 of its eight and the chunk whose
  // swizzled slot is i % 8
  c.cbyte = 16u * (uint32_t)((lane & 7) ^ (lane >> 4));
#pragma unroll
  for (int q = 0; q < S::LA; ++q) {
    const int row8 = wave * S::LA + q;
    c.va[q] = (uint32_t)(2 * (row8 * 8 + (lane >> 3)) * p.lda) + (c.cbyte ^ chunk_flip(row8));
  }
#pragma unroll
  for (int q = 0; q < S::LB; ++q) {
    const int row8 = wave * S::LB + q;
    c.vb[q] = (uint32_t)(2 * (row8 * 8 + (lane >> 3)) * p.ldb) + (c.cbyte ^ chunk_flip(row8));
  }

  floatx16 acc[S::NI][S::NJ];
#pragma unroll
  for (int i = 0; i < S::NI; ++i)
#pragma unroll
    for (int j = 0; j < S::NJ; ++j) acc[i][j] = floatx16{};

  if constexpr (S::ST == 2) {
    // Step i computes from stage i % 2.  Its last fragments are read before its
    // last quarter; there every wave has read the stage, so behind one barrier
    // the copies of step i + 2 start into it: three quarters of them in that last
    // quarter, the rest in the first quarter of step i + 1, and both have the two
    // quarters after that to land.
    constexpr int L = S::LA + S::LB, L3 = L * 3 / 4, L0 = L - L3;
#pragma unroll
    for (int q = 0; q < L; ++q) issue_one<S>(c, 0, 0, q);
#pragma unroll
    for (int q = 0; q < L3; ++q) issue_one<S>(c, 1, 1, q);
    wait_vmcnt<L3>();
    __syncthreads();
    Frags<S> f0, f1;
#pragma unroll
    for (int q = 0; q < S::NI + S::NJ; ++q) read_one<S>(f0, lds, 0, q, lane, wm, wn);
    for (int step = 0; step < c.nsteps; ++step) {
      const int st = step & 1;
      const uint8_t* cur = lds + st * S::STAGE;
      quarter<S, L3, L0>(acc, f0, f1, cur, 1, c, step + 1, st ^ 1, lane, wm, wn);
      quarter<S, 0, 0>(acc, f1, f0, cur, 2, c, 0, 0, lane, wm, wn);
      quarter<S, 0, 0>(acc, f0, f1, cur, 3, c, 0, 0, lane, wm, wn);
      wait_vmcnt<0>();
      __syncthreads();
      quarter<S, 0, L3>(acc, f1, f0, lds + (st ^ 1) * S::STAGE, 0, c, step + 2, st, lane, wm, wn);
    }
    wait_vmcnt<0>();
  } else {
    // Memory-bound: step i + ST - 1 is copied while step i is computed.
    constexpr int L = S::LA + S::LB;
#pragma unroll
    for (int i = 0; i < S::ST - 1; ++i)
#pragma unroll
      for (int q = 0; q < L; ++q) issue_one<S>(c, i, i, q);
    for (int step = 0, st = 0; step < c.nsteps; ++step) {
      wait_vmcnt<(S::ST - 2) * L>();
      __syncthreads();   // the step is there, and the one before has been read
      const int prev = st == 0 ? S::ST - 1 : st - 1;
#pragma unroll
      for (int q = 0; q < L; ++q) issue_one<S>(c, step + S::ST - 1, prev, q);
      Frags<S> f[4];
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int q = 0; q < S::NI + S::NJ; ++q)
          read_one<S>(f[s], lds + st * S::STAGE, s, q, lane, wm, wn);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < S::NI; ++i)
#pragma unroll
          for (int j = 0; j < S::NJ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[s].a[i], f[s].b[j], acc[i][j], 0,
                                                                0, 0);
      st = st + 1 == S::ST ? 0 : st + 1;
    }
    wait_vmcnt<0>();
  }

  // acc[i][j][r]: n = j 32 + lane % 32, m = i 32 + 8 (r / 4) + 4 (lane / 32) + r % 4
  const int mw = wm * S::NI * 32 + 4 * h, nw = wn * S::NJ * 32 + (lane & 31);
  if constexpr (EPI == kStats) {
    const bool edge = rows < S::TM;
#pragma unroll
    for (int j = 0; j < S::NJ; ++j) {
      const int64_t n = col0 + nw + j * 32;
      const bool live = n < p.N;
      if (edge) {
#pragma unroll
        for (int i = 0; i < S::NI; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (mw + i * 32 + 8 * (r >> 2) + (r & 3) >= rows) acc[i][j][r] = -INFINITY;
      }
      // the target's logit, if this lane holds it
      const int64_t t = live ? p.targets[n] : -1;
      const int64_t at = t - (p.m0 + row0) - mw;
      const bool here = t >= 0 && t < p.classes && at >= 0 && at < S::NI * 32 && (at & 4) == 0;
      if (__any(here)) {
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < S::NI; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (at == i * 32 + 8 * (r >> 2) + (r & 3)) z = acc[i][j][r];
        if (here) p.zt[n] = z;
      }
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < S::NI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) m = fmaxf(m, acc[i][j][r]);
      m = fmaxf(m, __shfl_xor(m, 32));
      // a maximum of -inf leaves nothing to sum; NaNs pass fmaxf and reach the sum
      // (the difference first: exact near the maximum however large the logits)
      const float base = m == -INFINITY ? 0.0f : m;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < S::NI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          s += __builtin_amdgcn_exp2f((acc[i][j][r] - base) * kLog2e);
      s += __shfl_xor(s, 32);
      if (live && h == 0)
        p.part[(int64_t)(tm * S::WM + wm) * p.part_ld + n] = make_float2(m, s);
    }
  } else if constexpr (EPI == kGrad) {
#pragma unroll
    for (int j = 0; j < S::NJ; ++j) {
      const int64_t n = col0 + nw + j * 32;
      const bool live = n < p.N;
      float a = 0.0f, bt = 0.0f, l = 0.0f;
      int64_t at = -1;
      if (live) {
        const int64_t t = p.targets[n];
        if (t >= 0 && t < p.classes) {
          bt = p.dloss[n];
          at = t - (p.m0 + row0) - mw;
        }
        a = (bt + (p.dlse ? p.dlse[n] : 0.0f)) / p.scale[0];
        bt /= p.scale[0];
        l = p.lse[n];
      }
      const bool none = a == 0.0f && bt == 0.0f;   // whatever its logits hold
#pragma unroll
      for (int i = 0; i < S::NI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int m = i * 32 + 8 * (r >> 2) + (r & 3);
          float g = a * __builtin_amdgcn_exp2f((acc[i][j][r] - l) * kLog2e);
          if (at == m) g -= bt;
          acc[i][j][r] = none || mw + m >= rows ? 0.0f : g;
        }
    }
    __syncthreads();   // the stages are done with
    store_nm<S>(acc, lds, p.out + col0 * p.ldo + row0, p.ldo, p.m_store - row0, p.n_store - col0, wm,
                wn);
    __syncthreads();
    store_mn<S>(acc, lds, p.out_t + row0 * p.ldt + col0, p.ldt, p.m_store - row0, p.ldt - col0, wm,
                wn);
  } else if constexpr (EPI == kOut) {
    const float sc = p.scale[0];
#pragma unroll
    for (int i = 0; i < S::NI; ++i)
#pragma unroll
      for (int j = 0; j < S::NJ; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] *= sc;
    __syncthreads();
    store_nm<S>(acc, lds, p.out + col0 * p.ldo + row0, p.ldo, p.M - row0, p.N - col0, wm, wn);
  } else {
#pragma unroll
    for (int j = 0; j < S::NJ; ++j) {
      const int64_t n = col0 + nw + j * 32;
      if (n >= p.N) continue;
#pragma unroll
      for (int i = 0; i < S::NI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t m = row0 + mw + i * 32 + 8 * q;
          if (m >= p.M) continue;   // M is a multiple of 8: four at a time are in or out
          f32x4* o = reinterpret_cast<f32x4*>(p.slab + ((int64_t)split * p.N + n) * p.M + m);
          f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                     acc[i][j][4 * q + 3]};
          if (!p.first) v += *o;
          *o = v;
        }
    }
  }
}

// Joins the tiles' statistics: TB tokens per workgroup, 256 / TB threads each,
// their partial results joined in a fixed order.
template <int TB>
__global__ __launch_bounds__(kThreads) void k_xent_join(const float2* part, const float* zt,
                                                        const int64_t* targets, int64_t T,
                                                        int64_t classes, int parts, float* loss,
                                                        float* lse) {
  constexpr int SL = kThreads / TB;
  __shared__ float2 red[SL][TB];
  const int tl = threadIdx.x % TB, sl = threadIdx.x / TB;
  const int64_t t = (int64_t)blockIdx.x * TB + tl;
  auto add = [](float2 a, float2 b) {   // of two (maximum, sum)
    const float m = fmaxf(a.x, b.x);
    if (m == -INFINITY) return make_float2(m, a.y + b.y);   // nothing yet (a NaN stays)
    return make_float2(m, a.y * __builtin_amdgcn_exp2f((a.x - m) * kLog2e) +
                              b.y * __builtin_amdgcn_exp2f((b.x - m) * kLog2e));
  };
  float2 v = make_float2(-INFINITY, 0.0f);
  if (t < T)
    for (int q = sl; q < parts; q += SL) v = add(v, part[(int64_t)q * T + t]);
  red[sl][tl] = v;
  for (int h = SL / 2; h > 0; h /= 2) {
    __syncthreads();
    if (sl < h) red[sl][tl] = add(red[sl][tl], red[sl + h][tl]);
  }
  if (sl == 0 && t < T) {
    const float l = red[0][tl].x + __builtin_amdgcn_logf(red[0][tl].y) * kLn2;   // log2
    lse[t] = l;
    const int64_t c = targets[t];
    loss[t] = c >= 0 && c < classes ? l - zt[t] : 0.0f;
  }
}

// dst[c][r] = src[r][c] for bf16, 64 x 64 tiles; rows r >= R and columns
// c >= C of the padded destination [Cp][Rp] are zeros, and so are source rows
// whose gradient factors are both zero (what they hold is not looked at).
__global__ __launch_bounds__(kThreads) void k_turn(const uint16_t* src, int64_t R, int64_t C,
                                                   int64_t ld, uint16_t* dst, int64_t Rp,
                                                   int64_t Cp, const int64_t* targets,
                                                   int64_t classes, const float* dloss,
                                                   const float* dlse) {
  __shared__ uint16_t t[64][66];
  const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3;   // 8 columns of 8, 32 rows
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t r = r0 + y + 32 * k, c = c0 + 8 * x;
    u32x4 v = {0, 0, 0, 0};
    bool take = r < R && c < C;
    if (take && targets) {
      const int64_t q = targets[r];
      const float b = q >= 0 && q < classes ? dloss[r] : 0.0f;
      const float a = b + (dlse ? dlse[r] : 0.0f);
      take = a != 0.0f || b != 0.0f;
    }
    if (take) v = *reinterpret_cast<const u32x4*>(src + r * ld + c);   // C is a multiple of 8
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[8 * x + 2 * i][y + 32 * k] = (uint16_t)v[i];
      t[8 * x + 2 * i + 1][y + 32 * k] = (uint16_t)(v[i] >> 16);
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t c = c0 + y + 32 * k, r = r0 + 8 * x;
    if (c >= Cp || r >= Rp) continue;
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = (uint32_t)t[y + 32 * k][8 * x + 2 * i] |
             ((uint32_t)t[y + 32 * k][8 * x + 2 * i + 1] << 16);
    *reinterpret_cast<u32x4*>(dst + c * Rp + r) = v;
  }
}

// s: the largest finite |b| over the tokens, or where that is nothing next to
// the largest |a| (or 0) that one, or 1; one workgroup.
__global__ __launch_bounds__(kThreads) void k_xent_scale(const int64_t* targets, int64_t classes,
                                                         const float* dloss, const float* dlse,
                                                         int64_t T, float* scale) {
  __shared__ float red[2][kThreads];
  float mb = 0.0f, ma = 0.0f;
  for (int64_t t = threadIdx.x; t < T; t += kThreads) {
    const int64_t c = targets[t];
    const float b = c >= 0 && c < classes ? dloss[t] : 0.0f, a = b + (dlse ? dlse[t] : 0.0f);
    if (fabsf(b) < INFINITY) mb = fmaxf(mb, fabsf(b));
    if (fabsf(a) < INFINITY) ma = fmaxf(ma, fabsf(a));
  }
  red[0][threadIdx.x] = mb;
  red[1][threadIdx.x] = ma;
  for (int h = kThreads / 2; h > 0; h /= 2) {
    __syncthreads();
    if ((int)threadIdx.x < h)
      for (int k = 0; k < 2; ++k)
        red[k][threadIdx.x] = fmaxf(red[k][threadIdx.x], red[k][threadIdx.x + h]);
  }
  if (threadIdx.x == 0) {
    mb = red[0][0];
    ma = red[1][0];
    scale[0] = mb > 0.0f && mb >= ma * 0x1p-20f ? mb : ma > 0.0f ? ma : 1.0f;
  }
}

// out[n][m] = s times the sum of the slabs, rounded to bf16; 4 elements per
// thread and round of the grid.
__global__ __launch_bounds__(kThreads) void k_slab_sum(const float* slab, int64_t N, int64_t M,
                                                       int splits, const float* scale,
                                                       uint16_t* out, int64_t ldo) {
  int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
  for (; i < N * M; i += (int64_t)gridDim.x * kThreads * 4) {
    f32x4 v = *reinterpret_cast<const f32x4*>(slab + i);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(slab + s * N * M + i);
    const int64_t n = i / M, m = i - n * M;
    v *= scale[0];
    const u32x2 w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    *reinterpret_cast<u32x2*>(out + n * ldo + m) = w;
  }
}

__global__ __launch_bounds__(kThreads) void k_zero_rows(uint16_t* out, int64_t N, int64_t M,
                                                        int64_t ldo) {
  int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8;
  for (; i < N * M; i += (int64_t)gridDim.x * kThreads * 8) {
    const int64_t n = i / M, m = i - n * M;
    *reinterpret_cast<u32x4*>(out + n * ldo + m) = u32x4{0, 0, 0, 0};
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up(int64_t a, int64_t b) { return cdiv(a, b) * b; }

// HIP takes fewer than 2^32 threads in a launch: tiles of a product (of 512
// threads), and workgroups of an elementwise kernel, which then goes round.
constexpr int64_t kMaxTiles = (int64_t)1 << 22;
dim3 grid_for(int64_t threads) {
  const int64_t g = cdiv(threads, kThreads);
  return dim3((unsigned)(g < kMaxTiles ? g : kMaxTiles));
}

template <class S, int EPI>
hipError_t launch_prod(Prod p, hipStream_t s) {
  constexpr int bytes = S::ST * S::STAGE;
  static std::atomic<uint64_t> lds_set{0};
  const hipError_t e = set_lds_limit((const void*)k_prod<S, EPI>, bytes, lds_set);
  if (e != hipSuccess) return e;
  p.tiles_m = (int32_t)cdiv(p.M, S::TM);
  p.tiles_n = (int32_t)cdiv(p.N, S::TN);
  p.tiles = p.tiles_m * p.tiles_n;
  if (p.splits < 1) p.splits = 1;
  p.k_per_split = p.splits == 1 ? p.K : up(cdiv(p.K, p.splits), 64);
  p.splits = (int32_t)cdiv(p.K, p.k_per_split);
  hipLaunchKernelGGL((k_prod<S, EPI>), dim3((unsigned)(p.tiles * p.splits)), dim3(S::THREADS),
                     bytes, s, p);
  return hipGetLastError();
}

// The product of the logits: by tokens, see the shapes.  Statistics of more tiles
// than a launch takes (T V > 2^38) some tokens at a time; a piece of the backward
// pass has at most 2^13 tiles.
template <int EPI>
hipError_t launch_logits(const Prod& p, hipStream_t s) {
  if (p.N <= 32) return launch_prod<Thin32, EPI>(p, s);
  if (p.N <= 64) return launch_prod<Thin64, EPI>(p, s);
  if constexpr (EPI == kStats) {
    const int64_t step = kMaxTiles / cdiv(p.M, Big::TM) * Big::TN;   // M <= 2^30: one tile or more
    for (int64_t n = 0; n < p.N; n += step) {
      Prod q = p;
      q.N = p.N - n < step ? p.N - n : step;
      q.b = p.b + n * p.ldb;
      q.targets = p.targets + n;
      q.part = p.part + n;
      q.zt = p.zt + n;
      const hipError_t e = launch_prod<Big, EPI>(q, s);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  } else {
    return launch_prod<Big, EPI>(p, s);
  }
}
// Rows of the forward statistics for V classes and T tokens.
int64_t stat_rows(int64_t T, int64_t V) {
  return T <= 64 ? Thin32::WM * cdiv(V, Thin32::TM) : Big::WM * cdiv(V, Big::TM);
}
static_assert(Thin32::TM == Thin64::TM && Thin32::WM == Thin64::WM, "one count for both");

hipError_t launch_turn(const uint16_t* src, int64_t R, int64_t C, int64_t ld, uint16_t* dst,
                       int64_t Rp, int64_t Cp, const XentLaunch* dead, hipStream_t s) {
  hipLaunchKernelGGL(k_turn, dim3((unsigned)cdiv(Cp, 64), (unsigned)cdiv(Rp, 64)), dim3(kThreads),
                     0, s, src, R, C, ld, dst, Rp, Cp, dead ? dead->targets : nullptr,
                     dead ? dead->V : 0, dead ? dead->dloss : nullptr,
                     dead ? dead->dlse : nullptr);
  return hipGetLastError();
}

}  // namespace

// Backward plan: classes per piece, splits of the dh product, workspace parts.
XentPlan xent_plan(int64_t T, int64_t V, int64_t D) {
  XentPlan p;
  p.parts = stat_rows(T, V);
  p.fwd_bytes = up(8 * p.parts * T, 256) + up(4 * T, 256);
  // one piece holds at most 2^26 elements of G, whole tiles of classes
  int64_t piece = up(V, 256);
  const int64_t most = ((int64_t)1 << 26) / up(T, 256) / 256 * 256;
  if (piece > most) piece = most < 256 ? 256 : most;
  p.pieces = cdiv(V, piece);
  p.piece = piece;
  p.Tp = up(T, 8);
  // the dh product has few tiles and a long K: split it until the chip is
  // covered, at least 512 of K each
  const int64_t tiles = cdiv(D, 256) * cdiv(T, 256);
  int64_t splits = cdiv(256, tiles);
  if (splits > piece / 512) splits = piece / 512;
  if (splits < 1) splits = 1;
  p.splits = (int32_t)cdiv(piece, up(cdiv(piece, splits), 64));
  int64_t at = 0;
  auto take = [&](int64_t bytes) { const int64_t o = at; at += up(bytes, 256); return o; };
  p.g = take(2 * T * piece);
  p.gt = take(2 * piece * p.Tp);
  p.wt = take(2 * D * piece);
  p.ht = take(2 * D * p.Tp);
  p.slab = take(4 * (int64_t)p.splits * T * D);
  p.scale = take(4);
  p.bwd_bytes = at;
  return p;
}

hipError_t launch_xent_fwd(const XentLaunch& x, hipStream_t s) {
  const XentPlan pl = xent_plan(x.T, x.V, x.D);
  Prod p = {};
  p.a = x.w; p.lda = x.ldw; p.M = x.V;
  p.b = x.h; p.ldb = x.ldh; p.N = x.T;
  p.K = x.D;
  p.part = reinterpret_cast<float2*>(x.ws);
  p.part_ld = x.T;
  p.zt = reinterpret_cast<float*>(x.ws + up(8 * pl.parts * x.T, 256));
  p.targets = x.targets;
  p.classes = x.V;
  hipError_t e = launch_logits<kStats>(p, s);
  if (e != hipSuccess) return e;
  // up to 512 tokens a workgroup each (7 tokens, 1004 rows: 12 us with eight
  // tokens to a workgroup, whose threads then walk 31 rows), else eight
  if (x.T <= 512)
    hipLaunchKernelGGL((k_xent_join<1>), dim3((unsigned)x.T), dim3(kThreads), 0, s, p.part, p.zt,
                       x.targets, x.T, x.V, (int)pl.parts, x.loss, x.lse_out);
  else
    hipLaunchKernelGGL((k_xent_join<8>), dim3((unsigned)cdiv(x.T, 8)), dim3(kThreads), 0, s, p.part,
                       p.zt, x.targets, x.T, x.V, (int)pl.parts, x.loss, x.lse_out);
  return hipGetLastError();
}

hipError_t launch_xent_bwd(const XentLaunch& x, hipStream_t s) {
  if (x.T == 0) {   // no token: dW is zero
    hipLaunchKernelGGL(k_zero_rows, grid_for(cdiv(x.V * x.D, 8)), dim3(kThreads), 0, s, x.dw,
                       x.V, x.D, x.lddw);
    return hipGetLastError();
  }
  const XentPlan pl = xent_plan(x.T, x.V, x.D);
  uint16_t* G = reinterpret_cast<uint16_t*>(x.ws + pl.g);
  uint16_t* GT = reinterpret_cast<uint16_t*>(x.ws + pl.gt);
  uint16_t* WT = reinterpret_cast<uint16_t*>(x.ws + pl.wt);
  uint16_t* HT = reinterpret_cast<uint16_t*>(x.ws + pl.ht);
  float* slab = reinterpret_cast<float*>(x.ws + pl.slab);
  float* scale = reinterpret_cast<float*>(x.ws + pl.scale);
  hipLaunchKernelGGL(k_xent_scale, dim3(1), dim3(kThreads), 0, s, x.targets, x.V, x.dloss, x.dlse,
                     x.T, scale);
  hipError_t e = launch_turn(x.h, x.T, x.D, x.ldh, HT, pl.Tp, x.D, &x, s);
  if (e != hipSuccess) return e;
  int32_t splits = 1;
  for (int64_t c = 0; c < pl.pieces; ++c) {
    const int64_t v0 = c * pl.piece, vn = x.V - v0 < pl.piece ? x.V - v0 : pl.piece;
    const int64_t vp = up(vn, 64);   // padded with zeros, in G and in W^T
    const uint16_t* W = x.w + v0 * x.ldw;
    Prod p = {};
    p.a = W; p.lda = x.ldw; p.M = vn;
    p.b = x.h; p.ldb = x.ldh; p.N = x.T;
    p.K = x.D;
    p.targets = x.targets;
    p.m0 = v0;
    p.classes = x.V;
    p.lse = x.lse;
    p.dloss = x.dloss;
    p.dlse = x.dlse;
    p.scale = scale;
    p.out = G;
    p.ldo = vp;
    p.m_store = vp;
    p.n_store = x.T;
    p.out_t = GT;
    p.ldt = pl.Tp;
    if ((e = launch_logits<kGrad>(p, s)) != hipSuccess) return e;
    if ((e = launch_turn(W, vn, x.D, x.ldw, WT, vp, x.D, nullptr, s)) != hipSuccess) return e;
    Prod d = {};
    d.a = WT; d.lda = vp; d.M = x.D;
    d.b = G; d.ldb = vp; d.N = x.T;
    d.K = vp;
    d.splits = pl.splits;
    d.slab = slab;
    d.first = c == 0;
    if ((e = launch_prod<Big, kSlab>(d, s)) != hipSuccess) return e;
    Prod w = {};
    w.a = HT; w.lda = pl.Tp; w.M = x.D;
    w.b = GT; w.ldb = pl.Tp; w.N = vn;
    w.K = pl.Tp;
    w.scale = scale;
    w.out = x.dw + v0 * x.lddw;
    w.ldo = x.lddw;
    if ((e = launch_prod<Big, kOut>(w, s)) != hipSuccess) return e;
    if (c == 0) splits = (int32_t)cdiv(vp, pl.splits == 1 ? vp : up(cdiv(vp, pl.splits), 64));
  }
  hipLaunchKernelGGL(k_slab_sum, grid_for(cdiv(x.T * x.D, 4)), dim3(kThreads), 0, s, slab,
                     x.T, x.D, splits, scale, x.dh, x.lddh);
  return hipGetLastError();
}

}  // namespace ufp4
