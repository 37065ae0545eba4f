// Attention of a few new tokens over a paged cache held in 4 bits.
//
//   q' = c_n FWHT(S q)    z_t = scale q' . K_t      K_t, V_t: level * block scale,
//   o' = sum_t e^(z_t - lse) V_t                    in the basis of the rotation
//   o = S c_n FWHT(o')
//
// The rotation is orthogonal, so the few queries and outputs are rotated and the
// many keys and values never are.  Every code is read once from HBM for all the
// queries of a key head (the heads of its group, times the sequence's new
// tokens): the bytes of the codes and scales are the bound, with the decoding of
// the codes on the vector units close behind.
//
// A wave takes 64 tokens a step, by itself: codes and scales come straight into
// its own part of the LDS, one step ahead.  s = K q' runs on
// v_mfma_f32_16x16x32_bf16 with 16 tokens as rows and 16 queries as columns: a
// lane ends with the scores of four tokens of one query in each of four
// products, and those sixteen are, scaled and rounded, the fragments of o' = V^T p
// without an exchange, because the transposing 4-bit LDS read lets every lane
// pick which sixteen tokens it gets of a column of V: just those.
//
// Levels are exact in bf16.  E2M1 codes are converted in pairs by
// v_cvt_scalef32_pk_bf16_fp4; INT4 and E1M2 codes become E4M3 bytes through byte
// tables and are then converted in pairs.  E8M0 scales of keys are applied by
// that conversion (exact); fp32 scales of keys multiply the products of one block, in
// fp32; scales of values multiply the weights, which are then rounded to bf16 (half a
// step each: the size of o's own rounding, and random over the sum).  q' enters as
// two bf16 pieces, 16 bits of mantissa.
//
// Bound: HBM first, 4 sequences of 131072 tokens on 8 key heads of 128 (E1M2, fp32 scales of 32)
// 130 us for 670 MB, 5.2 TB/s, with the vector instructions next (719 a step, two thirds of the
// cycles; the same in E2M1 with E8M0 scales 111 us); 64 sequences of 1 to 16384 tokens (E2M1, E8M0)
// 80 us for 385 MB.  Two tiles of queries (16 sequences of about 5900 tokens, 5 rows of 5
// heads) take 76 us for 146 MB: twice the arithmetic on the same bytes, all registers, and 11 to 22
// spilled, whose reloads in the steps wait for the copies issued before them.  Pages below 64 tokens
// and heads other than 64 and 128 (the 64 sequences in pages of 16: 139 us with the join)
// take their addresses lane by lane, with two tiles and 45 to 87 spilled.  Tried and slower at 131072 tokens: three workgroups to a compute unit with
// two buffers a wave (162 us instead of 141 with the join), two or four times as many
// workgroups (141 and 158 instead of 131); with two tiles, one wave to a SIMD (107 instead
// of 81) and scales read two at a time (95 instead of 79).
//
// The work is cut evenly, not by sequence: with u = 64-token steps of every (sequence,
// tile of queries, key head) laid end to end, and a few for each as such, workgroup w
// takes steps w / W .. (w + 1) / W of all.  Whole items are finished where they are computed; parts of one
// leave (o', m, l) in the workspace and a second launch joins them in order.
#include "attn_internal.h"

namespace ufp4 {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kStep = 64;       // tokens of a wave's step
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p;
}

__device__ __forceinline__ int64_t uniform64(int64_t x) {
  return ((int64_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32) |
         (uint32_t)__builtin_amdgcn_readfirstlane((int)x);
}

// a b, and 0 where either is 0, whatever the other (v_mul_legacy_f32).
extern "C" __device__ float ufp4_llvm_fmul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float mul_legacy(float a, float b) { return ufp4_llvm_fmul_legacy(a, b); }

// HBM -> LDS without registers, lane i's bytes at lds + 16 i (4 i); waited for with
// wait_copies.  Lanes that are switched off leave their place as it is.
__device__ __forceinline__ void copy16(uint32_t lds, const void* src) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off"
               : : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t lds, const void* src) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, off"
               : : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src) : "memory");
}
// The same from a wave-uniform address and a lane's offset.
__device__ __forceinline__ void copy16(uint32_t lds, uint64_t base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2"
               : : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t lds, uint64_t base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, %2"
               : : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" : : : "memory"); }
template <int N>
__device__ __forceinline__ void wait_all_but() { asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory"); }
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

// Maximum and sum over the lanes that hold one query (l % 16).
__device__ __forceinline__ float query_max(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float query_sum(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Eight codes as bf16 values, in the order of `order`: levels times 2^e of `scale`.  SPLIT: the codes of
// two 1 x 16 blocks, nibbles 0 .. 3 of the first in registers 0, 1, nibbles 4 .. 7 of the
// second in 2, 3.  (INT4 as 136 + n, n ^ 8 in the low mantissa bits of 128, is two
// instructions for two codes where tables and a conversion take four, and 5 to 10 % faster with one
// tile of queries; but taking 136 times the sum of the other operand off again leaves the
// rounding of that sum, however small the codes are.)
template <int GRID, bool SPLIT>
__device__ __forceinline__ u32x4 decode8(uint32_t x, float scale) {
  u32x4 v;
  if constexpr (GRID == 2) {
    v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 0));
    v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 1));
    v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 2));
    v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 3));
  } else {
    // E4M3 bytes of the even and of the odd nibbles
    const uint32_t y = x >> 4;
    uint32_t a, b;
    if constexpr (GRID == 0) {   // k / 4, k = 0 .. 7, and the sign
      a = __builtin_amdgcn_perm(0x3E3C3A38u, 0x34302800u, x & 0x07070707u) | ((x << 4) & 0x80808080u);
      b = __builtin_amdgcn_perm(0x3E3C3A38u, 0x34302800u, y & 0x07070707u) | (x & 0x80808080u);
    } else {   // 0 .. 7 and -8 .. -1, chosen by the nibble's top bit
      const uint32_t sa = x & 0x07070707u, sb = y & 0x07070707u;
      const uint32_t pa = __builtin_amdgcn_perm(0x4E4C4A48u, 0x44403800u, sa);
      const uint32_t na = __builtin_amdgcn_perm(0xB8C0C4C8u, 0xCACCCED0u, sa);
      const uint32_t pb = __builtin_amdgcn_perm(0x4E4C4A48u, 0x44403800u, sb);
      const uint32_t nb = __builtin_amdgcn_perm(0xB8C0C4C8u, 0xCACCCED0u, sb);
      a = __builtin_amdgcn_perm(na, pa, ((x >> 1) & 0x04040404u) | 0x03020100u);
      b = __builtin_amdgcn_perm(nb, pb, ((y >> 1) & 0x04040404u) | 0x03020100u);
    }
    v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false));
    v[SPLIT ? 2 : 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true));
    v[SPLIT ? 1 : 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false));
    v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true));
  }
  return v;
}
// Which nibble is the i-th value.
template <int GRID, bool SPLIT>
__device__ constexpr int order(int i) {
  if (GRID == 2) return i;
  if (SPLIT) return (i & 4) | ((i & 1) << 1) | ((i >> 1) & 1);
  return i < 4 ? 2 * i : 2 * i - 7;
}

// Butterflies over N rows of D elements, two neighbours to a lane.
template <int N>
__device__ __forceinline__ void rotate_rows(float (&a)[N], float (&b)[N], int n, int lane) {
  if (n > 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float s = a[k] + b[k], d = a[k] - b[k];
      a[k] = s;
      b[k] = d;
    }
  }
  for (int h = 2; h < n; h <<= 1) {
    const int m = h >> 1;
    const uint32_t neg = (lane & m) ? 0x80000000u : 0u;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float pa = __shfl_xor(a[k], m), pb = __shfl_xor(b[k], m);
      a[k] = pa + __uint_as_float(__float_as_uint(a[k]) ^ neg);
      b[k] = pb + __uint_as_float(__float_as_uint(b[k]) ^ neg);
    }
  }
}
// Signs of elements 2 lane, 2 lane + 1 of a row.
__device__ __forceinline__ float signed_by(const uint32_t (&sign)[4], int e, float x) {
  const uint32_t lo = (e & 32) ? sign[1] : sign[0], hi = (e & 32) ? sign[3] : sign[2];
  const uint32_t w = (e & 64) ? hi : lo;
  return __uint_as_float(__float_as_uint(x) ^ ((w >> (e & 31)) << 31));
}

// What an item (a tile of queries of one key head) costs besides its steps, in steps:
// rotating its queries, filling and joining its waves.  Without it a workgroup that
// drew the short sequences of a batch took 88 of them one after another, 590 us where
// the others were done after 100; 4 steps: 160 us, 8: 105, 12: 83.
constexpr int kItem = 12;

// Sequence b's share of the work.
struct Seq {
  int row0, rows;     // packed rows
  int len;            // tokens in the cache
  int64_t tiles, units;
  __device__ int64_t cost(int heads) const { return tiles * heads * (units + kItem); }
};
__device__ __forceinline__ Seq sequence(const KvAttn& p, int b) {
  Seq q;
  const int64_t a = max(p.at.starts[b], 0), e = min((int64_t)p.at.starts[b + 1], p.at.T);
  q.row0 = (int)a;
  q.rows = e > a ? (int)(e - a) : 0;
  const int64_t room = p.at.width << p.at.page_shift;
  const int64_t len = p.at.lens[b];
  q.len = (int)len;
  const int per = 16 * p.rows16;
  q.tiles = ((int64_t)q.rows * p.group + per - 1) / per;
  const int64_t seen = min(len, room);
  q.units = seen > 0 ? (seen + kStep - 1) / kStep : 1;
  return q;
}

// Inclusive sums of x over the workgroup's threads, and the total.
struct ScanLds {
  int64_t sum[kWaves];
};
__device__ __forceinline__ int64_t scan(int64_t x, ScanLds& s, int64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up((long long)x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) s.sum[wave] = x;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) x += s.sum[w];
    total += s.sum[w];
  }
  return x;
}

struct Found {
  int b;              // the sequence, B: none
  int64_t before;     // units before it
};
struct PlanLds {
  ScanLds scan;
  Found found;
};

// Units of a workgroup; whole steps of all its waves where there are many.
__device__ __forceinline__ int64_t quota_of(int64_t total, int groups) {
  const int64_t q = (total + groups - 1) / groups;
  return q >= 4 * kWaves ? (q + kWaves - 1) / kWaves * kWaves : q;
}

// The quota, and the sequence that holds unit w quota.
__device__ __forceinline__ int64_t plan(const KvAttn& p, int groups, int w, PlanLds& s, Found& f) {
  const int B = p.at.B;
  if (B <= 64) {   // every wave by itself
    const int lane = threadIdx.x & 63;
    int64_t mine = 0;
    if (lane < B) mine = sequence(p, lane).cost(p.at.kv_heads);
    int64_t sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t y = __shfl_up((long long)sum, d);
      if (lane >= d) sum += y;
    }
    const int64_t quota = quota_of(__shfl((long long)sum, 63), groups), u = (int64_t)w * quota;
    const uint64_t here = __ballot(u < sum && u >= sum - mine);
    f.b = here ? __builtin_ctzll(here) : B;
    f.before = uniform64(__shfl((long long)(sum - mine), f.b & 63));
    f.b = __builtin_amdgcn_readfirstlane(f.b);
    return uniform64(quota);
  }
  int64_t total = 0, own = 0, upto = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + (int)threadIdx.x;
    own = 0;
    if (b < B) {
      const Seq q = sequence(p, b);
      own = q.cost(p.at.kv_heads);
    }
    int64_t part;
    upto = scan(own, s.scan, part);
    total += part;
  }
  const int64_t quota = quota_of(total, groups), u = (int64_t)w * quota;
  if (threadIdx.x == 0) s.found = Found{B, total};
  __syncthreads();
  int64_t before = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    if (B > kThreads) {   // else the one block's sums are still here
      const int b = b0 + (int)threadIdx.x;
      own = 0;
      if (b < B) {
        const Seq q = sequence(p, b);
        own = q.cost(p.at.kv_heads);
      }
      int64_t part;
      upto = scan(own, s.scan, part);
      if (u < before + upto && u >= before + upto - own) s.found = Found{b, before + upto - own};
      before += part;
    } else if (u < upto && u >= upto - own) {
      s.found = Found{(int)threadIdx.x, upto - own};
    }
  }
  __syncthreads();
  f = s.found;
  f.b = __builtin_amdgcn_readfirstlane(f.b);
  f.before = uniform64(f.before);
  return uniform64(quota);
}

// Rows at, at + kWaves, .. (of `nrows`) of o', divided by l and out of the basis of the rotation,
// to memory.
template <int N>
__device__ __forceinline__ void store_rows(const KvAttn& p, float (&a)[N], float (&b)[N],
                                           const float (&l)[N], int row0, int64_t at,
                                           int64_t nrows, int hk, int lane) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float inv = l[k] == 0.0f ? 0.0f : 1.0f / l[k];   // nothing to attend to: 0
    a[k] *= inv;
    b[k] *= inv;
  }
  rotate_rows<N>(a, b, p.n, lane);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (p.n > 1) {
      a[k] *= p.cn;
      b[k] *= p.cn;
    }
    const int64_t r = at + k * kWaves;
    if (r < nrows && 2 * lane < p.at.D) {
      const int64_t i = r / p.group;
      const int h = hk * p.group + (int)(r - i * p.group);
      *reinterpret_cast<uint32_t*>(p.o + (row0 + i) * p.ldo + (int64_t)h * p.at.D + 2 * lane) =
          pack_bf16(signed_by(p.sign, 2 * lane, a[k]), signed_by(p.sign, 2 * lane + 1, b[k]));
    }
  }
}

// LDS of one wave: three buffers that K and V take in turn, each the codes of 64
// tokens (rows of ROW bytes, 16-byte chunks exchanged by the token) and their
// scales as memory has them, SC bytes a token; KIND 2 also the current values' scales in fp32.
template <int KIND, int NB>
struct Lay {
  static constexpr int ROW = 16 * NB, CODES = kStep * ROW;
  static constexpr int SC = KIND == 2 ? NB : KIND == 1 ? 8 * NB : 4 * NB;
  static constexpr int NS = SC / 4;   // words of a token (KIND 2, NB = 2: half a word)
  static constexpr int UNIT = CODES + kStep * SC;
  // copies of a step's keys or values (whole pages)
  static constexpr int COPIES = CODES / 1024 + (kStep * SC > 1024 ? 2 : 1);
  static constexpr int WIDE = KIND == 2 ? kStep * 4 * NB : 0;   // a step's value scales in fp32
  static constexpr int PAIR = 2 * UNIT + WIDE;                  // a wave's part but the third buffer
  __device__ static uint32_t flip(int tok) {
    return NB == 4 ? ((tok >> 2) ^ (tok >> 4)) & 3 : ((tok >> 3) ^ (tok >> 4)) & 1;
  }
};

// (Elements past D: any codes, which stand for something finite, against q' = 0, and scales of 0.)

// N floats of an LDS row that starts at a multiple of 8 bytes.
template <int N>
__device__ __forceinline__ void read_scales(float (&x)[N], const float* at) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(at + i);
      x[i] = v[0]; x[i + 1] = v[1]; x[i + 2] = v[2]; x[i + 3] = v[3];
    }
  } else {
    const f32x2 v = *reinterpret_cast<const f32x2*>(at);
    x[0] = v[0]; x[1] = v[1];
  }
}

// NB: 32-element blocks of a row in LDS (2 or 4), MT: tiles of 16 queries.  FAST: D = 32 NB
// and pages of 64 tokens or more, so that a step's codes and scales are one run of memory
// each and its page one scalar: its copies need no address arithmetic (otherwise a
// step's addresses cost as many instructions as half of its arithmetic).
template <int GRID, int KIND, int NB, int MT, bool FAST>
__global__ __launch_bounds__(kThreads, 2) void k_kv_attn(KvAttn p) {
  using L = Lay<KIND, NB>;
  constexpr int DP = 32 * NB, QP = DP + 4;
  constexpr bool SPLIT = KIND == 1;
  constexpr int NBLK = SPLIT ? 2 * NB : NB;   // blocks of a row
  constexpr int GB = NBLK < 4 ? NBLK : 4;     // blocks whose scales are read together
  constexpr int kRows = kWaves * L::PAIR;   // where the waves' third buffers lie, and `rows`
  constexpr int kThird = kWaves * L::UNIT > 16 * MT * QP * 4 ? kWaves * L::UNIT : 16 * MT * QP * 4;
  constexpr int kParts = kWaves * 16 * MT * QP * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kRows + kThird > kParts ? kRows + kThird : kParts];
  __shared__ PlanLds plan_lds;
  __shared__ float stat[2][kWaves][16 * MT];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, li = lane & 15;
  const int D = FAST ? DP : p.at.D;
  Found f;
  const int64_t quota = plan(p, gridDim.x, blockIdx.x, plan_lds, f);
  int64_t u = (int64_t)blockIdx.x * quota;
  const int64_t u_end = u + quota;
  const int64_t u_first = u;
  const float c = p.scale * kLog2e;
  float* rows = reinterpret_cast<float*>(lds + kRows);   // [16 MT][QP], before the steps
  uint8_t* const wide = lds + wave * L::PAIR + 2 * L::UNIT;
  auto buffer = [&](int b) -> uint8_t* {
    return b < 2 ? lds + wave * L::PAIR + b * L::UNIT : lds + kRows + wave * L::UNIT;
  };
  // a lane's 16 bytes within the 1024 of a copy; NB = 4: and 16 bytes times the copy's number
  const uint32_t run = NB == 4 ? 64u * (lane >> 2) + 16u * ((lane & 3) ^ ((lane >> 4) & 3))
                               : 32u * (lane >> 1) + 16u * ((lane & 1) ^ (((lane >> 4) ^ (lane >> 5)) & 1));

  while (f.b < p.at.B && u < u_end) {
    const Seq q = sequence(p, f.b);
    const int64_t cost = q.cost(p.at.kv_heads);
    if (u >= f.before + cost) {   // this sequence is done
      f.before += cost;
      ++f.b;
      continue;
    }
    const int64_t item = (u - f.before) / (q.units + kItem);
    const int64_t from = (u - f.before) - item * (q.units + kItem);
    const int64_t to = min(q.units + kItem, from + (u_end - u));
    const bool leading = u == u_first;   // the workgroup's first item
    u += to - from;
    if (to <= kItem) continue;           // none of its steps
    const int64_t first = max(from - kItem, (int64_t)0);
    const int count = (int)(to - kItem - first);
    const int hk = (int)(item % p.at.kv_heads);
    const int64_t r0 = item / p.at.kv_heads * (16 * MT);   // first (token, head of the group) row
    const int64_t nrows = (int64_t)q.rows * p.group;

    __syncthreads();   // the item before is done with the buffers
    const int t_first = (int)first * kStep;
    const int32_t* pages = p.at.table + f.b * p.at.ldt;

    // Where the tokens of a step lie.  FAST: the page of all of them; else the row of token
    // 64 step + lane among all rows, or -1.
    auto place = [&](int step) -> int64_t {
      if constexpr (FAST) {
        const int t = t_first + step * kStep;
        const int slot = t >> p.at.page_shift;
        if (step >= count || t >= q.len || slot >= (int)p.at.width) return -1;
        // the table does not change while the kernel runs: a scalar load
        const int page = reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(
            (uint64_t)pages)[slot];
        return page >= 0 && page < p.at.pages ? page : -1;
      } else {
        const int t = t_first + step * kStep + lane;
        const int slot = t >> p.at.page_shift;
        if (step >= count || t >= q.len || slot >= (int)p.at.width) return -1;
        const int page = pages[slot];
        if (page < 0 || page >= p.at.pages) return -1;
        return (((int64_t)page * p.at.kv_heads + hk) << p.at.page_shift) +
               (t & ((1 << p.at.page_shift) - 1));
      }
    };
    // Which of a step's tokens have a place.
    auto places = [&](int64_t at) -> uint64_t {
      return FAST ? (at >= 0 ? ~(uint64_t)0 : 0) : __ballot(at >= 0);
    };
    // Codes and scales of a step into buffer `buf`.  Not FAST: the scales of token lane come
    // back in registers, and are stored when the step begins.
    float held[2][L::NS > 0 ? L::NS : 1];   // of keys and values (KIND 2: a word)
    auto issue = [&](int buf, int step, int64_t at, uint64_t valid, int is_v) {
      const uint8_t* codes = is_v ? p.v_codes : p.k_codes;
      const uint8_t* scales = is_v ? p.v_scales : p.k_scales;
      const uint32_t dst = lds_address(buffer(buf)), ds = dst + L::CODES;
      if constexpr (FAST) {
        const uint64_t row = (((uint64_t)at * p.at.kv_heads + hk) << p.at.page_shift) +
                             (uint64_t)((t_first + step * kStep) & ((1 << p.at.page_shift) - 1));
        const uint64_t cb = (uint64_t)codes + row * L::ROW, sb = (uint64_t)scales + row * L::SC;
#pragma unroll
        for (int i = 0; i < L::CODES / 1024; ++i)
          copy16(dst + 1024u * i, cb + 1024u * i, NB == 4 ? run ^ (16u * i) : run);
        constexpr int SB = kStep * L::SC;   // 128 .. 2048 bytes
        if constexpr (SB >= 1024) {
#pragma unroll
          for (int i = 0; i < SB / 1024; ++i) copy16(ds + 1024u * i, sb + 1024u * i, 16u * lane);
        } else if constexpr (SB >= 256) {
          if (16 * lane < SB) copy16(ds, sb, 16u * lane);
        } else {
          if (4 * lane < SB) copy4(ds, sb, 4u * lane);
        }
      } else {
        // a token without a place: any row that has one, and a mask
        const int some = __builtin_ctzll(valid);
        const uint32_t lo = at >= 0 ? (uint32_t)at : (uint32_t)__shfl((int)at, some);
        const uint32_t hi = at >= 0 ? (uint32_t)(at >> 32) : (uint32_t)__shfl((int)(at >> 32), some);
        const int64_t row = ((int64_t)hi << 32) | lo;
        const int row_bytes = D / 2;
        if ((D & 31) == 0) {
          constexpr int PER = 64 / NB;   // tokens of an instruction
#pragma unroll
          for (int i = 0; i < kStep / PER; ++i) {
            const int tok = PER * i + lane / NB;
            const int64_t r = ((int64_t)(uint32_t)__shfl((int)hi, tok) << 32) | (uint32_t)__shfl((int)lo, tok);
            const int ch = (lane % NB) ^ (int)L::flip(tok);
            if (32 * ch < D) copy16(dst + 1024u * i, codes + r * row_bytes + 16 * ch);
          }
        } else {   // rows that end inside a chunk, by words
          constexpr int PER = 16 / NB;
          for (int i = 0; i < kStep / PER; ++i) {
            const int tok = PER * i + lane / (4 * NB);
            const int64_t r = ((int64_t)(uint32_t)__shfl((int)hi, tok) << 32) | (uint32_t)__shfl((int)lo, tok);
            const int word = lane % (4 * NB);
            const int ch = (word >> 2) ^ (int)L::flip(tok);
            if (32 * ch + 8 * (word & 3) < D)
              copy4(dst + 256u * i, codes + r * row_bytes + 16 * ch + 4 * (word & 3));
          }
        }
        if constexpr (KIND == 2) {
          uint32_t w = 0;
#pragma unroll
          for (int i = 0; i < NB; ++i)
            if (32 * i < D) w |= (uint32_t)scales[row * (D / 32) + i] << (8 * i);
          held[is_v][0] = __uint_as_float(w);
        } else {
          const int ns = SPLIT ? D / 16 : D / 32;
#pragma unroll
          for (int i = 0; i < L::NS; ++i)
            held[is_v][i] = i < ns ? reinterpret_cast<const float*>(scales)[row * ns + i] : 0.0f;
        }
      }
    };
    auto settle = [&](int buf, int is_v) {   // the held scales of a step into its buffer
      if constexpr (!FAST) {
        uint8_t* to = buffer(buf) + L::CODES + lane * L::SC;
        if constexpr (KIND == 2) {
          if constexpr (NB == 4) *reinterpret_cast<uint32_t*>(to) = __float_as_uint(held[is_v][0]);
          else *reinterpret_cast<uint16_t*>(to) = (uint16_t)__float_as_uint(held[is_v][0]);
        } else {
#pragma unroll
          for (int i = 0; i < L::NS; ++i) reinterpret_cast<float*>(to)[i] = held[is_v][i];
        }
      }
    };
    auto scale_word = [&](const uint8_t* ss, int tok) -> uint32_t {
      if constexpr (NB == 4) return reinterpret_cast<const uint32_t*>(ss)[tok];
      else return reinterpret_cast<const uint16_t*>(ss)[tok];
    };

    int kb = 0, vb = 1, nb = 2;   // buffers of the step's keys, its values, and the free one
    int64_t at = place(wave), next_at = place(wave + kWaves);
    uint64_t valid = places(at);
    if (valid) {
      issue(kb, wave, at, valid, 0);
      issue(vb, wave, at, valid, 1);
    }
    // q' of the tile's rows in fp32, times the factor of the scores
    uint32_t raw[16 * MT / kWaves];
#pragma unroll
    for (int k = 0; k < 16 * MT / kWaves; ++k) {
      const int64_t row = r0 + wave + k * kWaves;
      raw[k] = 0;
      if (row < nrows && 2 * lane < D) {
        const int64_t i = row / p.group;
        const int h = hk * p.group + (int)(row - i * p.group);
        raw[k] = *reinterpret_cast<const uint32_t*>(p.q + (q.row0 + i) * p.ldq + (int64_t)h * D + 2 * lane);
      }
    }
    {
      constexpr int PER = 16 * MT / kWaves;
      float a[PER], b[PER];
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        a[k] = signed_by(p.sign, 2 * lane, __uint_as_float(raw[k] << 16));
        b[k] = signed_by(p.sign, 2 * lane + 1, __uint_as_float(raw[k] & 0xFFFF0000u));
      }
      rotate_rows<PER>(a, b, p.n, lane);
      const float f = p.n > 1 ? p.cn : 1.0f;
#pragma unroll
      for (int k = 0; k < PER; ++k)
        if (2 * lane < DP)
          *reinterpret_cast<f32x2*>(rows + (wave + k * kWaves) * QP + 2 * lane) = f32x2{a[k] * f * c, b[k] * f * c};
    }
    __syncthreads();
    // its fragments, in two bf16 pieces; value i of a lane is element `order`
    u32x4 qh[MT][NB], ql[MT][NB];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int s = 0; s < NB; ++s) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          float x[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int nib = order<GRID, SPLIT>(i + e);
            const int d = SPLIT ? 32 * s + 16 * (nib >> 2) + 4 * g + (nib & 3) : 32 * s + 8 * g + nib;
            x[e] = rows[(16 * mt + li) * QP + d];
          }
          const uint32_t hi = pack_bf16(x[0], x[1]);
          qh[mt][s][i / 2] = hi;
          // an infinite piece leaves nothing
          const float l0 = x[0] - __uint_as_float(hi << 16), l1 = x[1] - __uint_as_float(hi & 0xFFFF0000u);
          ql[mt][s][i / 2] = pack_bf16(fabsf(x[0]) < INFINITY ? l0 : 0.0f, fabsf(x[1]) < INFINITY ? l1 : 0.0f);
        }
      }
    wait_lds();
    __syncthreads();   // `rows` has been read: the steps may overwrite it

    f32x4 o[MT][2 * NB];
    float m[MT], l[MT];
    int last[MT];      // the last token that this lane's query sees
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int d = 0; d < 2 * NB; ++d) o[mt][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      m[mt] = -INFINITY;
      l[mt] = 0.0f;
      const int64_t at = r0 + 16 * mt + li;
      last[mt] = at < nrows ? q.len - q.rows + (int)(at / p.group) : -1;
    }
    // the earliest last token of any row: steps up to there need no mask
    const int sure = q.len - q.rows + (int)(r0 / p.group);
    for (int step = wave; step < count; step += kWaves) {
      const int64_t after_at = place(step + 2 * kWaves);
      const uint64_t next_valid = places(next_at);
      // the keys are there; the values, copied after them, may still be on their way
      if constexpr (FAST) wait_all_but<L::COPIES>();
      else wait_copies();
      settle(kb, 0);
      if (next_valid) issue(nb, step + kWaves, next_at, next_valid, 0);
      f32x4 s[MT][4];
      if (valid) {
        const uint8_t* kt = buffer(kb);
        const uint8_t* ss = kt + L::CODES;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int tok = 16 * j + li;
          uint32_t sw = 0;
          float sc[4][GB];   // scales of the lane's four tokens, of the blocks in work
          if constexpr (KIND == 2) sw = scale_word(ss, tok);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) s[mt][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            constexpr int PER = SPLIT ? GB / 2 : GB;   // blocks or pairs of them in a group
            if constexpr (KIND != 2) {
              if (b % PER == 0) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  read_scales<GB>(sc[r], reinterpret_cast<const float*>(ss + (16 * j + 4 * g + r) * L::SC) + b / PER * GB);
              }
            }
            const uint8_t* at_k = kt + tok * L::ROW + 16 * (b ^ (int)L::flip(tok));
            if constexpr (SPLIT) {
              const uint32_t x = (uint32_t)*reinterpret_cast<const uint16_t*>(at_k + 2 * g) |
                                 (uint32_t)*reinterpret_cast<const uint16_t*>(at_k + 8 + 2 * g) << 16;
              const u32x4 v = decode8<GRID, true>(x, 1.0f);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const s16x4 k = __builtin_bit_cast(s16x4, (u32x2{v[2 * e], v[2 * e + 1]}));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
                  y = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(k, __builtin_bit_cast(s16x4, (u32x2{qh[mt][b][2 * e], qh[mt][b][2 * e + 1]})), y, 0, 0, 0);
                  y = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(k, __builtin_bit_cast(s16x4, (u32x2{ql[mt][b][2 * e], ql[mt][b][2 * e + 1]})), y, 0, 0, 0);
#pragma unroll
                  for (int r = 0; r < 4; ++r) s[mt][j][r] = __builtin_fmaf(y[r], sc[r][(2 * b + e) % GB], s[mt][j][r]);
                }
              }
            } else {
              const uint32_t x = *reinterpret_cast<const uint32_t*>(at_k + 4 * g);
              float scale = 1.0f;
              if constexpr (KIND == 2) scale = __uint_as_float(((sw >> (8 * b)) & 0xFFu) << 23);
              const bf16x8 k8 = __builtin_bit_cast(bf16x8, decode8<GRID, false>(x, scale));
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                f32x4 y = KIND == 2 ? s[mt][j] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8, __builtin_bit_cast(bf16x8, qh[mt][b]), y, 0, 0, 0);
                y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8, __builtin_bit_cast(bf16x8, ql[mt][b]), y, 0, 0, 0);
                if constexpr (KIND == 2) {   // the conversion has applied the scale
                  s[mt][j] = y;
                } else {
#pragma unroll
                  for (int r = 0; r < 4; ++r) s[mt][j][r] = __builtin_fmaf(y[r], sc[r][b % GB], s[mt][j][r]);
                }
              }
            }
          }
        }
      }
      // the keys have been read: the next step's values take their place
      wait_lds();
      if (FAST && next_valid) wait_all_but<L::COPIES>();   // this step's values are there
      else wait_copies();
      if (valid) settle(vb, 1);   // before the next ones are loaded
      if (next_valid) issue(kb, step + kWaves, next_at, next_valid, 1);
      if (valid) {
        if constexpr (KIND == 2) {   // the scales of values in fp32
          const uint32_t w = scale_word(buffer(vb) + L::CODES, lane);
          float* vs = reinterpret_cast<float*>(wide) + lane * NB;
#pragma unroll
          for (int i = 0; i < NB; ++i)   // 2^(byte - 127); of byte 0 that is below the exponents' range
            vs[i] = __uint_as_float(max(((w >> (8 * i)) & 0xFFu) << 23, 0x00400000u));
        }
        const int t0 = t_first + step * kStep;
        if (valid != ~(uint64_t)0 || t0 + kStep - 1 > sure) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int tok = 16 * j + 4 * g + r;
                if (t0 + tok > last[mt] || !((valid >> tok) & 1)) s[mt][j][r] = -INFINITY;
              }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) top = fmaxf(top, s[mt][j][r]);
          top = query_max(top);
          if (__any(top > m[mt] + 8.0f)) {
            const float next = top > m[mt] + 8.0f ? top : m[mt];
            const float fac = next == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[mt] - next);
            m[mt] = next;
            l[mt] *= fac;
#pragma unroll
            for (int d = 0; d < 2 * NB; ++d)
#pragma unroll
              for (int r = 0; r < 4; ++r) o[mt][d][r] *= fac;
          }
          const float base = m[mt] == -INFINITY ? 0.0f : m[mt];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              s[mt][j][r] = __builtin_amdgcn_exp2f(s[mt][j][r] - base);
              l[mt] += s[mt][j][r];
            }
        }
        const uint8_t* vt = buffer(vb);
        const uint8_t* vs = KIND == 2 ? wide : vt + L::CODES;
        const int vtok = 16 * (li >> 2) + 4 * g + (li & 3);
        constexpr int VSC = KIND == 2 ? 4 * NB : L::SC;   // bytes of a token's fp32 scales
        constexpr int BD = SPLIT ? 1 : 2;                 // 16-element columns of a block
#pragma unroll
        for (int k0 = 0; k0 < NBLK; k0 += GB) {           // blocks of the values
          i32x2 vc[GB * BD];   // columns of 16 values: eight codes of each half of the step
#pragma unroll
          for (int e = 0; e < GB * BD; ++e) {
            const int d = BD * k0 + e;
            const uint8_t* at_v = vt + vtok * L::ROW + 16 * ((d >> 1) ^ (int)L::flip(vtok)) + 8 * (d & 1);
            typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
            vc[e] = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_i32x2*)at_v);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {                   // half of the step
            u32x4 w[MT][GB];                              // weights times scales
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e0 = order<GRID, false>(2 * i), e1 = order<GRID, false>(2 * i + 1);
              float a[GB], b[GB];
              read_scales<GB>(a, reinterpret_cast<const float*>(vs + (32 * x + 16 * (e0 >> 2) + 4 * g + (e0 & 3)) * VSC) + k0);
              read_scales<GB>(b, reinterpret_cast<const float*>(vs + (32 * x + 16 * (e1 >> 2) + 4 * g + (e1 & 3)) * VSC) + k0);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int k = 0; k < GB; ++k)
                  // 0 times whatever the scale of a token that is not seen holds is 0
                  w[mt][k][i] = pack_bf16(mul_legacy(s[mt][2 * x + (e0 >> 2)][e0 & 3], a[k]),
                                          mul_legacy(s[mt][2 * x + (e1 >> 2)][e1 & 3], b[k]));
            }
#pragma unroll
            for (int e = 0; e < GB * BD; ++e) {
              const bf16x8 v = __builtin_bit_cast(bf16x8, decode8<GRID, false>((uint32_t)vc[e][x], 1.0f));
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                o[mt][BD * k0 + e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    v, __builtin_bit_cast(bf16x8, w[mt][e / BD]), o[mt][BD * k0 + e], 0, 0, 0);
            }
          }
        }
      }
      wait_lds();   // the values have been read
      const int free_now = vb;
      vb = kb;
      kb = nb;
      nb = free_now;
      at = next_at;
      next_at = after_at;
      valid = next_valid;
    }
    wait_copies();

    // every wave's part, [16 MT][QP] each, and what a row's parts come to
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      l[mt] = query_sum(l[mt]);
      if (g == 0) {
        stat[0][wave][16 * mt + li] = m[mt];
        stat[1][wave][16 * mt + li] = l[mt];
      }
    }
    __syncthreads();   // all steps are done with the buffers
    float* parts = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int d = 0; d < 2 * NB; ++d)
        *reinterpret_cast<f32x4*>(parts + (wave * 16 * MT + 16 * mt + li) * QP + 16 * d + 4 * g) = o[mt][d];
    __syncthreads();
    const bool whole = first == 0 && count == (int)q.units;
    float* part = p.partial + (int64_t)(2 * blockIdx.x + (leading ? 0 : 1)) * (16 * MT) * (D + 2);
    constexpr int PER = 16 * MT / kWaves;   // rows of a wave
    float ya[PER], yb[PER], top[PER], sum[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int r = wave + k * kWaves;
      top[k] = -INFINITY;
      ya[k] = yb[k] = sum[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top[k] = fmaxf(top[k], stat[0][w][r]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float lw = stat[1][w][r];
        if (lw == 0.0f) continue;   // saw nothing
        const float fac = __builtin_amdgcn_exp2f(stat[0][w][r] - top[k]);
        sum[k] += lw * fac;
        if (2 * lane < DP) {
          const f32x2 x = *reinterpret_cast<const f32x2*>(parts + (w * 16 * MT + r) * QP + 2 * lane);
          ya[k] += x[0] * fac;
          yb[k] += x[1] * fac;
        }
      }
    }
    if (whole) {
      store_rows<PER>(p, ya, yb, sum, q.row0, r0 + wave, nrows, hk, lane);
    } else {
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int r = wave + k * kWaves;
        if (r0 + r >= nrows) continue;
        float* to = part + (int64_t)r * (D + 2);
        if (2 * lane < D) *reinterpret_cast<f32x2*>(to + 2 * lane) = f32x2{ya[k], yb[k]};
        if (lane == 0) *reinterpret_cast<f32x2*>(to + D) = f32x2{top[k], sum[k]};
      }
    }
  }
}

// Joins the parts of the item inside which workgroup w + 1's units begin first;
// blockIdx.y: 4 N rows of its tile, N to a wave, so that all workgroups are on the chip at once
// (16 sequences of 5 tokens, 5 heads to a key head: 8.8 us, with N = 1 in two rounds 10.4).
template <int N>
__global__ __launch_bounds__(kThreads) void k_kv_join(KvAttn p) {
  __shared__ PlanLds plan_lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = blockIdx.x + 1, D = p.at.D;
  Found f;
  const int64_t quota = plan(p, kKvGroups, w, plan_lds, f);
  if (f.b >= p.at.B) return;
  const Seq q = sequence(p, f.b);
  const int64_t u = (int64_t)w * quota, item = (u - f.before) / (q.units + kItem);
  const int64_t a0 = f.before + item * (q.units + kItem);  // the item's place, and its steps'
  const int64_t s0 = a0 + kItem;
  if (s0 >= u || s0 < u - quota) return;                   // not split here, or before
  const int hk = (int)(item % p.at.kv_heads);
  const int r = 4 * N * blockIdx.y + wave;                 // and r + kWaves, ..
  const int64_t at = item / p.at.kv_heads * (16 * p.rows16) + r, nrows = (int64_t)q.rows * p.group;
  if (at >= nrows) return;
  const int w0 = w - 1, w1 = (int)((s0 + q.units - 1) / quota);
  const int64_t size = (int64_t)16 * p.rows16 * (D + 2);
  // Row k of part x (a row past the last one: the first); an item that begins inside a workgroup's
  // units is its second part.
  auto part = [&](int x, int k) {
    return p.partial + (2 * x + (x == w0 && a0 > (int64_t)w0 * quota ? 1 : 0)) * size +
           (int64_t)(r + (at + k * kWaves < nrows ? k * kWaves : 0)) * (D + 2);
  };
  float top[N], a[N], b[N], l[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    top[k] = -INFINITY;
    a[k] = b[k] = l[k] = 0.0f;
  }
  for (int x = w0 + lane; x <= w1; x += 64)
#pragma unroll
    for (int k = 0; k < N; ++k) top[k] = fmaxf(top[k], part(x, k)[D]);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) top[k] = fmaxf(top[k], __shfl_xor(top[k], d));
  for (int x0 = w0; x0 <= w1; x0 += 64) {
    // lane i: the factors of part x0 + i, and what it adds to l; a part that saw nothing adds nothing
    float fac[N];
#pragma unroll
    for (int k = 0; k < N; ++k) fac[k] = 0.0f;
    if (x0 + lane <= w1) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const f32x2 s = *reinterpret_cast<const f32x2*>(part(x0 + lane, k) + D);
        fac[k] = s[1] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(s[0] - top[k]);
        l[k] += s[1] * fac[k];
      }
    }
    const int n = min(w1 - x0 + 1, 64);
    for (int i = 0; i < n; i += 8) {   // eight parts' loads at once
      f32x2 y[8][N];
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int k = 0; k < N; ++k) {
          y[e][k] = f32x2{0.0f, 0.0f};
          if (i + e < n && 2 * lane < D) y[e][k] = *reinterpret_cast<const f32x2*>(part(x0 + i + e, k) + 2 * lane);
        }
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const float x = __shfl(fac[k], i + e);
          if (x != 0.0f) {
            a[k] += y[e][k][0] * x;
            b[k] += y[e][k][1] * x;
          }
        }
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) l[k] += __shfl_xor(l[k], d);
  store_rows<N>(p, a, b, l, q.row0, at, nrows, hk, lane);
}

template <int GRID, int KIND, int NB, int MT>
void launch_nb(const KvAttn& p, hipStream_t s) {
  if (p.at.D == 32 * NB && p.at.page_shift >= 6)
    k_kv_attn<GRID, KIND, NB, MT, true><<<kKvGroups, kThreads, 0, s>>>(p);
  else
    k_kv_attn<GRID, KIND, NB, MT, false><<<kKvGroups, kThreads, 0, s>>>(p);
}

template <int GRID, int KIND>
void launch(const KvAttn& p, hipStream_t s) {
  const bool narrow = p.at.D <= 64;
  if (p.rows16 == 1) {
    if (narrow) launch_nb<GRID, KIND, 2, 1>(p, s);
    else launch_nb<GRID, KIND, 4, 1>(p, s);
  } else {
    if (narrow) launch_nb<GRID, KIND, 2, 2>(p, s);
    else launch_nb<GRID, KIND, 4, 2>(p, s);
  }
}

template <int GRID>
void launch_grid(const KvAttn& p, hipStream_t s) {
  switch (p.kind) {
    case 0: launch<GRID, 0>(p, s); break;
    case 1: launch<GRID, 1>(p, s); break;
    default: launch<GRID, 2>(p, s); break;
  }
}

}  // namespace

// Tiles of 16 rows that share one decoding: two where the average sequence has more than 16
// (token, head) rows to a key head.
int32_t kv_attn_rows16(int64_t T, int32_t B, int32_t group) {
  return T * group > 16 * (int64_t)B ? 2 : 1;
}

int64_t kv_attn_workspace(int64_t T, int32_t B, int32_t heads, int32_t kv_heads, int32_t D) {
  return (int64_t)2 * kKvGroups * 16 * kv_attn_rows16(T, B, heads / kv_heads) * (D + 2) * 4;
}

hipError_t launch_kv_attn(const KvAttn& p, hipStream_t s) {
  switch (p.grid) {
    case 0: launch_grid<0>(p, s); break;
    case 1: launch_grid<1>(p, s); break;
    default: launch_grid<2>(p, s); break;
  }
  const dim3 rows(kKvGroups - 1, 4);
  if (p.rows16 == 1) k_kv_join<1><<<rows, kThreads, 0, s>>>(p);
  else k_kv_join<2><<<rows, kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace ufp4
