// Pieces that the attention kernels share: how a workgroup finds its sequence,
// copies of K or V tiles into LDS, and the fragments that the matrix
// instructions read from them.
//
// Everything is built on v_mfma_f32_32x32x16_bf16, C[m][n] = sum_k A[m][k]
// B[n][k]: lane l holds A's row (B's row) l % 32 with k = 8 (l / 32) .. + 7, and
// of C the column n = l % 32 with rows m = 8 (r / 4) + 4 (l / 32) + r % 4 in
// registers r = 0 .. 15.  A product's registers 8 t .. 8 t + 7 therefore are a
// fragment of the next product, which contracts over m, as long as the other
// operand's lane holds the same sixteen m in the same order: rows 16 t + 4 (l /
// 32) + {0 .. 3} and those + 8.  The transposing LDS read gives just that from
// row-major tiles (16 lanes read 4 rows of 16 elements and each gets a column), so
// neither the weights nor V, nor the gradients' operands, are ever exchanged
// between lanes or stored turned.
#pragma once

#include "attn_internal.h"
#include "lds_copy.h"

namespace ufp4 {
namespace attn {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kOutside = 0x7FFFFF00u;   // an offset past every buffer: reads as zeros

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p;
}

// The larger of x in lanes l and l ^ 32; their sum.
__device__ __forceinline__ float both_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float both_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Rows of sequence b, clipped to the arrays whatever starts holds.
__device__ __forceinline__ void rows_of(const int32_t* starts, int b, int64_t T, int64_t& row0,
                                        int& n) {
  const int64_t a = max(starts[b], 0), e = min((int64_t)starts[b + 1], T);
  row0 = a;
  n = e > a ? (int)(e - a) : 0;
}

// Tile number `x` of all sequences' tiles of kAttnTile rows, those with the most work first:
// its sequence's first row and length, and the tile's number in it; false past the
// last one.  A sequence of N tiles has one of each work 1 .. N (its tile t attends to t +
// 1 tiles of keys, and is attended to from N - t of queries: FROM_END).  Up to 64
// sequences, a lane each: of the tiles with more work than w there are sum of max(0, N -
// w), and the work of number x is found by trying 64 w at once, a lane each.  More
// sequences: one after another, from the last one, whatever their lengths.
template <bool FROM_END>
__device__ __forceinline__ bool find_tile(const int32_t* starts, int B, int64_t T, int tiles, int x,
                                          int64_t& row0, int& n, int& t) {
  const int lane = threadIdx.x & 63;
  if (B <= 64) {
    int64_t r0 = 0;
    int rows = 0;
    if (lane < B) rows_of(starts, lane, T, r0, rows);
    const int own = (rows + kAttnTile - 1) / kAttnTile;
    int all = 0, most = 0;
    for (int b = 0; b < B; ++b) {
      const int N = __builtin_amdgcn_readlane(own, b);
      all += N;
      most = max(most, N);
    }
    if (x >= all) return false;
    // tiles with more work than lo: more than x; than hi: `beyond`, not more than x
    int lo = 0, hi = most, beyond = 0;
    while (hi - lo > 1) {
      const int step = (hi - lo + 63) >> 6, w = min(lo + (lane + 1) * step, hi);
      int c = 0;
      for (int b = 0; b < B; ++b) c += max(__builtin_amdgcn_readlane(own, b) - w, 0);
      const int l = __builtin_ctzll(__ballot(c <= x));   // lane 63 has w = hi
      lo += l * step;
      hi = min(hi, lo + step);
      beyond = __builtin_amdgcn_readlane(c, l);
    }
    // work hi: the (x - beyond)-th sequence of that many tiles or more
    uint64_t in = __ballot(own >= hi);
    for (int skip = x - beyond; skip > 0; --skip) in &= in - 1;
    const int l = __builtin_ctzll(in);
    t = FROM_END ? __builtin_amdgcn_readlane(own, l) - hi : hi - 1;
    n = __builtin_amdgcn_readlane(rows, l);
    row0 = __builtin_amdgcn_readlane((int)r0, l);
    return true;
  }
  const int tile = FROM_END ? x : tiles - 1 - x;
  int before = 0;
  for (int b0 = 0; b0 < B; b0 += 64) {
    int64_t r0 = 0;
    int rows = 0;
    if (b0 + lane < B) rows_of(starts, b0 + lane, T, r0, rows);
    const int own = (rows + kAttnTile - 1) / kAttnTile;
    int upto = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(upto, d);
      if (lane >= d) upto += y;
    }
    const uint64_t past = __ballot(before + upto > tile);
    if (past) {
      const int l = __builtin_ctzll(past);
      t = __builtin_amdgcn_readfirstlane(tile - before - __shfl(upto - own, l));
      n = __builtin_amdgcn_readfirstlane(__shfl(rows, l));
      const int r = __shfl((int)r0, l);
      row0 = __builtin_amdgcn_readfirstlane(r);
      return true;
    }
    before += __shfl(upto, 63);
  }
  return false;
}

// Which tile and head a workgroup takes.  All heads of a tile follow one another, so that
// workgroups that start late have little work (one head after another, a head's
// longest tiles started last: 32768 tokens 2.76 ms instead of 2.33, as the kernel was then).  Key heads
// alternate first, then the heads of a group: workgroups go to the XCDs in turn, so
// with eight key heads each XCD keeps one of them in its cache.
struct Share {
  int tile, head, kv_head;
};
__device__ __forceinline__ uint32_t over(uint32_t x, FastDiv f) {
  return (uint32_t)(((uint64_t)__umulhi(x, f.m) + x) >> f.l);
}
__device__ __forceinline__ Share share_of(uint32_t id, FastDiv by_heads, FastDiv by_kv, int group) {
  const uint32_t tile = over(id, by_heads), r = id - tile * by_heads.d;
  const uint32_t in_group = over(r, by_kv);
  return Share{(int)tile, (int)((r - in_group * by_kv.d) * group + in_group), (int)(r - in_group * by_kv.d)};
}

// Whether a launch of so many workgroups (at most) takes them in two parts, of which each
// has every other step of its tile: eight waves instead of four, joined at the end.
// The last tile to finish is then what a launch takes, and half as long; with more
// workgroups than fit at once the waves' common barriers cost more.  Forward and
// backward, four waves and eight: 2048 tokens of 4 heads (68 workgroups) 173 and 137 us, 2
// x 1500 of 16 (400) 156 and 135; 3001 tokens of 20 heads (540) 123 and 130, 4 x
// 4096 of 40 (5280) 3.16 and 3.41 ms.  Sequences of one tile of keys have nothing for a
// second part to do (19 tokens, forward: 5.6 and 6.4 us).
inline bool in_parts(const AttnLaunch& p, int64_t workgroups) {
  return workgroups <= kInParts && p.T > 64 * (int64_t)p.B;
}

// The second part's sums of a wave's 32 x 32 N accumulators pass through LDS to the first
// part: `sums` is the wave's, 4096 N bytes.
template <int N>
__device__ __forceinline__ void leave_sums(float* sums, const floatx16 (&x)[N], int lane) {
#pragma unroll
  for (int b = 0; b < N; ++b)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *reinterpret_cast<f32x4*>(sums + 256 * (4 * b + r / 4) + 4 * lane) =
          f32x4{x[b][r], x[b][r + 1], x[b][r + 2], x[b][r + 3]};
}
template <int N>
__device__ __forceinline__ void take_sums(const float* sums, floatx16 (&x)[N], float mine, float theirs, int lane) {
#pragma unroll
  for (int b = 0; b < N; ++b)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const f32x4 y = *reinterpret_cast<const f32x4*>(sums + 256 * (4 * b + r / 4) + 4 * lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[b][r + e] = x[b][r + e] * mine + y[e] * theirs;
    }
}

// Launches over `tiles` tiles of `heads` heads, fewer than 2^24 workgroups at a time; f(first
// tile, workgroups).
template <class F>
void over_tiles(int64_t tiles, int heads, F&& f) {
  const int64_t slice = ((int64_t)1 << 23) / heads;
  for (int64_t t0 = 0; t0 < tiles; t0 += slice)
    f((int)t0, (unsigned)((tiles - t0 < slice ? tiles - t0 : slice) * heads));
}

// A tile in LDS has rows of DP elements whose 16-byte chunks are exchanged by the
// row's number so that both kinds of reads fill all 64 banks: sixteen rows
// reading one chunk each (sixteen different places of a 256-byte line), and the turned reads'
// four rows reading four neighbouring chunks each (four different quarters of
// the line; with the row's own low bits instead, the four rows meet in one quarter:
// 60 % of the LDS cycles of the forward pass were conflicts).
template <int DP>
__device__ __forceinline__ uint32_t swz(int row) {
  return DP == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
}
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  return (uint32_t)(row * (DP * 2)) + 16u * ((uint32_t)c ^ swz<DP>(row));
}

// Copies of a tile of R rows: instruction i of wave w carries rows (w PER + i) ROWS
// .. + ROWS - 1, ROWS = 512 / DP.
template <int DP, int R, int WAVES>
struct TileCopy {
  static constexpr int CH = DP / 8, ROWS = 64 / CH, PER = R / ROWS / WAVES;
  static_assert(PER * ROWS * WAVES == R, "the waves share the rows evenly");
  uint32_t row, col;   // this lane's row within an instruction's, byte in its row

  __device__ __forceinline__ void init(int lane) { row = lane / CH; }

  // Rows j0 .. of a sequence of n rows at `base` (row 0), pitch ld elements.
  __device__ __forceinline__ void issue(uint32_t lds, const uint16_t* base, int64_t ld, int j0,
                                        int n, int D, int wave, int lane) const {
    const int rows = min(n - j0, R);
    const sgpr4 r = rsrc4(base + (int64_t)j0 * ld,
                          rows > 0 ? (uint32_t)(((int64_t)(rows - 1) * ld + D) * 2) : 0u);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int first = (wave * PER + i) * ROWS;
      const int at = first + (int)row;
      const uint32_t c = (uint32_t)(lane % CH) ^ swz<DP>(at);
      uint32_t v = (uint32_t)at * (uint32_t)(ld * 2) + 16u * c;
      if (8 * (int)c >= D) v = kOutside;
      lds_load16(lds + (uint32_t)first * (DP * 2), r, v, 0u);
    }
  }
};

// Fragment s (16 elements of D) of 32 rows of a tile, as A's or B's rows: at(lane) is the
// lane's part of the address, which the fragment's number changes by an exclusive or.
template <int DP>
struct RowFrag {
  uint32_t lane_at;
  __device__ __forceinline__ explicit RowFrag(int lane) {
    lane_at = chunk_at<DP>(lane & 31, lane >> 5);
  }
  __device__ __forceinline__ bf16x8 read(const uint8_t* tile, int row0, int s) const {
    return *reinterpret_cast<const bf16x8*>(tile + row0 * (DP * 2) + (lane_at ^ (uint32_t)(32 * s)));
  }
};

// The turned fragment: lane l holds column d0 + l % 32 of the sixteen rows row0 + 4
// (l / 32) + {0 .. 3, 8 .. 11} (row0 and d0 multiples of 16 and 32).
template <int DP>
struct TurnedFrag {
  uint32_t lane_at[2];   // of the first and of the second four rows
  __device__ __forceinline__ explicit TurnedFrag(int lane) {
    const int i = lane & 15, row = 4 * (lane >> 5) + (i >> 2), d = (lane & 16) + 4 * (i & 3);
    lane_at[0] = chunk_at<DP>(row, d >> 3) + 2 * (d & 7);
    lane_at[1] = chunk_at<DP>(row + 8, d >> 3) + 2 * (d & 7);
  }
  __device__ __forceinline__ bf16x8 read(const uint8_t* tile, int row0, int d0) const {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4*)(tile + row0 * (DP * 2) + (lane_at[0] ^ (uint32_t)(2 * d0))));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4*)(tile + row0 * (DP * 2) + (lane_at[1] ^ (uint32_t)(2 * d0))));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const s16x8 v = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return __builtin_bit_cast(bf16x8, v);
  }
};

// Fragments of 32 rows straight from memory (rows past n and elements past D: 0).
template <int S>
__device__ __forceinline__ void load_rows(bf16x8 (&f)[S], const uint16_t* base, int64_t ld,
                                          int row0, int n, int D, int lane) {
  const int row = row0 + (lane & 31);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int d = 16 * s + 8 * (lane >> 5);
    u32x4 x = {0u, 0u, 0u, 0u};
    if (row < n && d < D) x = *reinterpret_cast<const u32x4*>(base + (int64_t)row * ld + d);
    f[s] = __builtin_bit_cast(bf16x8, x);
  }
}

// The factor of the scores in base 2.  Its size multiplies the products, so it is kept above 0 (-inf
// marks a key that is not seen); its sign, or that it is 0, goes into the operand held in
// registers.
__device__ __forceinline__ float score_factor(float scale) {
  return scale == 0.0f ? 1.0f : fabsf(scale) * kLog2e;
}
template <int S>
__device__ __forceinline__ void apply_sign(bf16x8 (&f)[S], float scale) {
  if (scale > 0.0f) return;
  const uint32_t flip = scale < 0.0f ? 0x80008000u : 0u, keep = scale < 0.0f ? 0xFFFFFFFFu : 0u;
#pragma unroll
  for (int s = 0; s < S; ++s)
    f[s] = __builtin_bit_cast(bf16x8, (__builtin_bit_cast(u32x4, f[s]) & keep) ^ flip);
}

// Waits for fragments that load_rows asked for.  Left to their first use inside a loop, the
// compiler's wait stands there in every pass, and with it one for all copies in flight
// (701 + 1300 + 17 + 983 tokens of 80 elements, forward and backward: 142 us instead of 122).
template <int S>
__device__ __forceinline__ void arrived(bf16x8 (&f)[S]) {
#pragma unroll
  for (int s = 0; s < S; ++s) asm volatile("" : "+v"(f[s]));
}

// Registers 8 t .. 8 t + 7 of a product as a fragment, rounded to bf16: pairs w[4 t] .. w[4 t + 3].
__device__ __forceinline__ bf16x8 frag_of(const uint32_t (&w)[8], int t) {
  return __builtin_bit_cast(bf16x8, (u32x4{w[4 * t], w[4 * t + 1], w[4 * t + 2], w[4 * t + 3]}));
}
__device__ __forceinline__ void round_pairs(const floatx16& x, uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
}

__device__ __forceinline__ floatx16 mfma(const bf16x8& a, const bf16x8& b, const floatx16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Multiplies a run of COUNT fragments in order, each read from LDS LEAD places before its
// MFMA: mul(i, fragment) after read(i), held in that order (left alone, the compiler
// reads a fragment right before its MFMA and waits).  The first LEAD are read by
// `begin`, before whatever code stands between.
template <int COUNT, int LEAD, class F>
struct Run {
  F f[LEAD + 1];
  template <class R>
  __device__ __forceinline__ void begin(R&& read) {
#pragma unroll
    for (int i = 0; i < LEAD; ++i) f[i] = read(i);
  }
  template <class R, class M>
  __device__ __forceinline__ void go(R&& read, M&& mul) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      if (i + LEAD < COUNT) f[(i + LEAD) % (LEAD + 1)] = read(i + LEAD);
      __builtin_amdgcn_sched_barrier(0);
      mul(i, f[i % (LEAD + 1)]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// a b, and 0 where either is 0, whatever the other (v_mul_legacy_f32).
extern "C" __device__ float ufp4_llvm_fmul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float mul_legacy(float a, float b) { return ufp4_llvm_fmul_legacy(a, b); }

__device__ __forceinline__ floatx16 zero16() {
  floatx16 z;
#pragma unroll
  for (int r = 0; r < 16; ++r) z[r] = 0.0f;
  return z;
}

}  // namespace attn
}  // namespace ufp4
