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
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" : : : "memory"); }
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

// Eight codes as bf16 levels times 2^e of `scale`, in the order of kOrder.
template <int GRID>
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
    v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true));
    v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false));
    v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true));
  }
  return v;
}
// Which nibble is the i-th value.
template <int GRID>
__device__ constexpr int order(int i) {
  return GRID == 2 ? i : i < 4 ? 2 * i : 2 * i - 7;
}

// Butterflies over a row of D elements, two neighbours to a lane.
__device__ __forceinline__ void rotate_row(float& a, float& b, int n, int lane) {
  if (n > 1) {
    const float s = a + b, d = a - b;
    a = s;
    b = d;
  }
  for (int h = 2; h < n; h <<= 1) {
    const int m = h >> 1;
    const float pa = __shfl_xor(a, m), pb = __shfl_xor(b, m);
    a = (lane & m) ? pa - a : a + pa;
    b = (lane & m) ? pb - b : b + pb;
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
// the others were done after 100.
constexpr int kItem = 4;

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
  return quota;
}

// One row of o', divided by l and out of the basis of the rotation, to memory.
__device__ __forceinline__ void store_row(const KvAttn& p, float a, float b, float l, int64_t row,
                                          int h, int lane) {
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // nothing to attend to: 0
  a *= inv;
  b *= inv;
  rotate_row(a, b, p.n, lane);
  if (p.n > 1) {
    a *= p.cn;
    b *= p.cn;
  }
  if (2 * lane < p.at.D)
    *reinterpret_cast<uint32_t*>(p.o + row * p.ldo + (int64_t)h * p.at.D + 2 * lane) =
        pack_bf16(signed_by(p.sign, 2 * lane, a), signed_by(p.sign, 2 * lane + 1, b));
}

// LDS of one wave: three buffers that K and V take in turn, each the codes of 64
// tokens (rows of ROW bytes, 16-byte chunks exchanged by the token) and their
// scales, [block][token] (KIND 2: four bytes a token); KIND 2 also the current
// values' scales in fp32.
template <int KIND, int NB>
struct Lay {
  static constexpr int ROW = 16 * NB, CODES = kStep * ROW;
  static constexpr int NS = KIND == 2 ? 1 : KIND == 1 ? 2 * NB : NB;
  static constexpr int UNIT = CODES + NS * 256;
  static constexpr int WAVE = 3 * UNIT + (KIND == 2 ? NB * 256 : 0);
  __device__ static uint32_t flip(int tok) {
    return NB == 4 ? ((tok >> 2) ^ (tok >> 4)) & 3 : ((tok >> 3) ^ (tok >> 4)) & 1;
  }
};

// NB: 32-element blocks of a row in LDS (2 or 4), MT: tiles of 16 queries.
template <int GRID, int KIND, int NB, int MT>
__global__ __launch_bounds__(kThreads, 2) void k_kv_attn(KvAttn p) {
  using L = Lay<KIND, NB>;
  constexpr int DP = 32 * NB, QP = DP + 4;
  constexpr int kArea = kWaves * L::WAVE > 16 * MT * QP * 4 ? kWaves * L::WAVE : 16 * MT * QP * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kArea];
  __shared__ PlanLds plan_lds;
  __shared__ float stat[2][kWaves][16 * MT];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, li = lane & 15;
  const int D = p.at.D;
  Found f;
  const int64_t quota = plan(p, gridDim.x, blockIdx.x, plan_lds, f);
  int64_t u = (int64_t)blockIdx.x * quota;
  const int64_t u_end = u + quota;
  const int64_t u_first = u;
  const float c = p.scale * kLog2e;
  float* rows = reinterpret_cast<float*>(lds);   // [16 MT][QP], before and after the steps
  uint8_t* mine = lds + wave * L::WAVE;
  const uint32_t mine0 = lds_address(mine);

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
    const int64_t first = max(from - kItem, (int64_t)0), count = to - kItem - first;
    const int hk = (int)(item % p.at.kv_heads);
    const int64_t r0 = item / p.at.kv_heads * (16 * MT);   // first (token, head of the group) row
    const int64_t nrows = (int64_t)q.rows * p.group;

    // q' of the tile's rows in fp32
    __syncthreads();   // `rows` is free
    for (int r = wave; r < 16 * MT; r += kWaves) {
      const int64_t at = r0 + r;
      float a = 0.0f, b = 0.0f;
      if (at < nrows) {   // uniform
        const int64_t i = at / p.group;
        const int h = hk * p.group + (int)(at - i * p.group);
        if (2 * lane < D) {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(
              p.q + (q.row0 + i) * p.ldq + (int64_t)h * D + 2 * lane);
          a = signed_by(p.sign, 2 * lane, __uint_as_float(x << 16));
          b = signed_by(p.sign, 2 * lane + 1, __uint_as_float(x & 0xFFFF0000u));
        }
        rotate_row(a, b, p.n, lane);
        if (p.n > 1) {
          a *= p.cn;
          b *= p.cn;
        }
      }
      if (2 * lane < DP) *reinterpret_cast<f32x2*>(rows + r * QP + 2 * lane) = f32x2{a, b};
    }
    __syncthreads();
    // its fragments, in two bf16 pieces; value i of a lane is element `order`
    u32x4 qh[MT][NB], ql[MT][NB];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int s = 0; s < NB; ++s)
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          float x[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int nib = order<GRID>(i + e);
            // 1 x 16 blocks: nibbles 0 .. 3 are of the first block of the step, 4 .. 7 of the second
            const int d = KIND == 1 ? 32 * s + 16 * (nib >> 2) + 4 * g + (nib & 3) : 32 * s + 8 * g + nib;
            x[e] = rows[(16 * mt + li) * QP + d];
          }
          const uint32_t hi = pack_bf16(x[0], x[1]);
          qh[mt][s][i / 2] = hi;
          // an infinite piece leaves nothing
          const float l0 = x[0] - __uint_as_float(hi << 16), l1 = x[1] - __uint_as_float(hi & 0xFFFF0000u);
          ql[mt][s][i / 2] = pack_bf16(fabsf(x[0]) < INFINITY ? l0 : 0.0f, fabsf(x[1]) < INFINITY ? l1 : 0.0f);
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

    // Where token 64 step + lane lies: its row among all, or -1.
    auto place = [&](int64_t step) -> int64_t {
      const int64_t t = (first + step) * kStep + lane;
      if (step >= count || t >= q.len) return -1;
      const int64_t slot = t >> p.at.page_shift;
      if (slot >= p.at.width) return -1;
      const int page = p.at.table[f.b * p.at.ldt + slot];
      if (page < 0 || page >= p.at.pages) return -1;
      return (((int64_t)page * p.at.kv_heads + hk) << p.at.page_shift) +
             (t & (((int64_t)1 << p.at.page_shift) - 1));
    };
    // Codes and scales of the step whose rows are `row` into buffer `buf`.  E8M0 scales
    // that are not a whole word a token come back as its word.
    auto issue = [&](int buf, int64_t row, uint64_t valid, const uint8_t* codes,
                     const uint8_t* scales) -> uint32_t {
      uint32_t tail = 0;
      const uint32_t to = mine0 + buf * L::UNIT;
      // a token without a place: any row that has one, and a mask
      const int some = __builtin_ctzll(valid);
      const uint32_t lo = row >= 0 ? (uint32_t)row : (uint32_t)__shfl((int)row, some);
      const uint32_t hi = row >= 0 ? (uint32_t)(row >> 32) : (uint32_t)__shfl((int)(row >> 32), some);
      const int64_t at = ((int64_t)hi << 32) | lo;
      const int row_bytes = D / 2;
      if ((D & 31) == 0) {
        constexpr int PER = 64 / NB;   // tokens of an instruction
#pragma unroll
        for (int i = 0; i < kStep / PER; ++i) {
          const int tok = PER * i + lane / NB;
          const int64_t r = ((int64_t)(uint32_t)__shfl((int)hi, tok) << 32) | (uint32_t)__shfl((int)lo, tok);
          const int ch = (lane % NB) ^ (int)L::flip(tok);
          if (32 * ch < D) copy16(to + 1024u * i, codes + r * row_bytes + 16 * ch);
        }
      } else {   // rows that end inside a chunk, by words
        constexpr int PER = 16 / NB;
        for (int i = 0; i < kStep / PER; ++i) {
          const int tok = PER * i + lane / (4 * NB);
          const int64_t r = ((int64_t)(uint32_t)__shfl((int)hi, tok) << 32) | (uint32_t)__shfl((int)lo, tok);
          const int word = lane % (4 * NB);
          const int ch = (word >> 2) ^ (int)L::flip(tok);
          if (32 * ch + 8 * (word & 3) < D)
            copy4(to + 256u * i, codes + r * row_bytes + 16 * ch + 4 * (word & 3));
        }
      }
      const uint32_t ts = to + L::CODES;
      if constexpr (KIND == 2) {
        if (D == 128) {
          copy4(ts, scales + at * 4);
        } else {
#pragma unroll
          for (int i = 0; i < NB; ++i)
            if (32 * i < D) tail |= (uint32_t)scales[at * (D / 32) + i] << (8 * i);
        }
      } else {
        const int ns = KIND == 1 ? D / 16 : D / 32;
#pragma unroll
        for (int i = 0; i < L::NS; ++i)
          if (i < ns) copy4(ts + 256u * i, scales + (at * ns + i) * 4);
      }
      return tail;
    };

    uint32_t tail_k = 0, tail_v = 0;
    int kb = 0, vb = 1, nb = 2;   // buffers of the step's keys, its values, and the free one
    int64_t row = place(wave), next_row = place(wave + kWaves);
    uint64_t valid = __ballot(row >= 0);
    if (valid) {
      tail_k = issue(kb, row, valid, p.k_codes, p.k_scales);
      tail_v = issue(vb, row, valid, p.v_codes, p.v_scales);
    }
    for (int64_t step = wave; step < count; step += kWaves) {
      const int64_t after_row = place(step + 2 * kWaves);
      const uint64_t next_valid = __ballot(next_row >= 0);
      wait_copies();
      if constexpr (KIND == 2) {
        // the scales of values in fp32, and words where they came by bytes
        uint32_t* ks = reinterpret_cast<uint32_t*>(mine + kb * L::UNIT + L::CODES);
        uint32_t w = reinterpret_cast<uint32_t*>(mine + vb * L::UNIT + L::CODES)[lane];
        if (D != 128) {
          ks[lane] = tail_k;
          w = tail_v;
        }
        float* vs = reinterpret_cast<float*>(mine + 3 * L::UNIT);
#pragma unroll
        for (int i = 0; i < NB; ++i) vs[64 * i + lane] = __uint_as_float(((w >> (8 * i)) & 0xFFu) << 23);
      }
      if (next_valid) tail_k = issue(nb, next_row, next_valid, p.k_codes, p.k_scales);
      f32x4 s[MT][4];
      if (valid) {
        const uint8_t* kt = mine + kb * L::UNIT;
        const float* ks = reinterpret_cast<const float*>(kt + L::CODES);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int tok = 16 * j + li;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) s[mt][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          uint32_t sw = 0;
          if constexpr (KIND == 2) sw = reinterpret_cast<const uint32_t*>(ks)[tok];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint8_t* at = kt + tok * L::ROW + 16 * (b ^ (int)L::flip(tok));
            if constexpr (KIND == 1) {
              const uint32_t x = (uint32_t)*reinterpret_cast<const uint16_t*>(at + 2 * g) |
                                 (uint32_t)*reinterpret_cast<const uint16_t*>(at + 8 + 2 * g) << 16;
              const u32x4 v = decode8<GRID>(x, 1.0f);
              // values 0 .. 3 of the order above lie in registers 0, 1 (E2M1) or 0, 2
              constexpr int A1 = GRID == 2 ? 1 : 2, B0 = GRID == 2 ? 2 : 1;
              const s16x4 ka = __builtin_bit_cast(s16x4, (u32x2{v[0], v[A1]}));
              const s16x4 kc = __builtin_bit_cast(s16x4, (u32x2{v[B0], v[3]}));
              const f32x4 s0 = *reinterpret_cast<const f32x4*>(ks + 64 * (2 * b) + 16 * j + 4 * g);
              const f32x4 s1 = *reinterpret_cast<const f32x4*>(ks + 64 * (2 * b + 1) + 16 * j + 4 * g);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                const u32x4 h = qh[mt][b], w = ql[mt][b];
                f32x4 x0 = {0.0f, 0.0f, 0.0f, 0.0f}, x1 = x0;
                x0 = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(ka, __builtin_bit_cast(s16x4, (u32x2{h[0], h[A1]})), x0, 0, 0, 0);
                x1 = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(kc, __builtin_bit_cast(s16x4, (u32x2{h[B0], h[3]})), x1, 0, 0, 0);
                x0 = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(ka, __builtin_bit_cast(s16x4, (u32x2{w[0], w[A1]})), x0, 0, 0, 0);
                x1 = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(kc, __builtin_bit_cast(s16x4, (u32x2{w[B0], w[3]})), x1, 0, 0, 0);
                const bool second = 32 * b + 16 < D;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  if (32 * b < D) s[mt][j][r] = __builtin_fmaf(x0[r], s0[r], s[mt][j][r]);
                  if (second) s[mt][j][r] = __builtin_fmaf(x1[r], s1[r], s[mt][j][r]);
                }
              }
            } else {
              const uint32_t x = *reinterpret_cast<const uint32_t*>(at + 4 * g);
              float scale = 1.0f;
              if constexpr (KIND == 2) scale = __uint_as_float(((sw >> (8 * b)) & 0xFFu) << 23);
              const bf16x8 k8 = __builtin_bit_cast(bf16x8, decode8<GRID>(x, scale));
              f32x4 sc = {1.0f, 1.0f, 1.0f, 1.0f};
              if constexpr (KIND == 0) sc = *reinterpret_cast<const f32x4*>(ks + 64 * b + 16 * j + 4 * g);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                f32x4 y = KIND == 2 ? s[mt][j] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8, __builtin_bit_cast(bf16x8, qh[mt][b]), y, 0, 0, 0);
                y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8, __builtin_bit_cast(bf16x8, ql[mt][b]), y, 0, 0, 0);
                if constexpr (KIND == 2) {
                  if (32 * b < D) s[mt][j] = y;
                } else if (32 * b < D) {
#pragma unroll
                  for (int r = 0; r < 4; ++r) s[mt][j][r] = __builtin_fmaf(y[r], sc[r], s[mt][j][r]);
                }
              }
            }
          }
        }
      }
      // the keys have been read: the next step's values take their place
      wait_lds();
      if (next_valid) tail_v = issue(kb, next_row, next_valid, p.v_codes, p.v_scales);
      if (valid) {
        const int64_t t0 = (first + step) * kStep;
        const bool masked = valid != ~(uint64_t)0 || t0 + kStep - 1 > sure;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float z = s[mt][j][r] * c;
              if (masked) {
                const int tok = 16 * j + 4 * g + r;
                if (t0 + tok > last[mt] || !((valid >> tok) & 1)) z = -INFINITY;
              }
              s[mt][j][r] = z;
              top = fmaxf(top, z);
            }
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
        const uint8_t* vt = mine + vb * L::UNIT;
        const float* vs = reinterpret_cast<const float*>(KIND == 2 ? mine + 3 * L::UNIT : vt + L::CODES);
        constexpr int BD = KIND == 1 ? 1 : 2;   // 16-element columns of a block
        const int vtok = 16 * (li >> 2) + 4 * g + (li & 3);
#pragma unroll
        for (int b = 0; b < 2 * NB / BD; ++b) {
          if (16 * BD * b >= D) continue;
          bf16x8 w[MT][2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(vs + 64 * b + 32 * x + 4 * g);
            const f32x4 e = *reinterpret_cast<const f32x4*>(vs + 64 * b + 32 * x + 16 + 4 * g);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              float y[8];
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                y[r] = s[mt][2 * x][r] * a[r];
                y[4 + r] = s[mt][2 * x + 1][r] * e[r];
                if (masked) {   // whatever the scale of a token that is not seen
                  y[r] = s[mt][2 * x][r] == 0.0f ? 0.0f : y[r];
                  y[4 + r] = s[mt][2 * x + 1][r] == 0.0f ? 0.0f : y[4 + r];
                }
              }
              u32x4 v;
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = pack_bf16(y[order<GRID>(2 * i)], y[order<GRID>(2 * i + 1)]);
              w[mt][x] = __builtin_bit_cast(bf16x8, v);
            }
          }
#pragma unroll
          for (int e = 0; e < BD; ++e) {
            const int d = BD * b + e;
            const uint8_t* at = vt + vtok * L::ROW + 16 * ((d >> 1) ^ (int)L::flip(vtok)) + 8 * (d & 1);
            typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
            const i32x2 x = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_i32x2*)at);
            const bf16x8 v0 = __builtin_bit_cast(bf16x8, decode8<GRID>((uint32_t)x[0], 1.0f));
            const bf16x8 v1 = __builtin_bit_cast(bf16x8, decode8<GRID>((uint32_t)x[1], 1.0f));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              o[mt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, w[mt][0], o[mt][d], 0, 0, 0);
              o[mt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, w[mt][1], o[mt][d], 0, 0, 0);
            }
          }
        }
      }
      wait_lds();   // the values have been read
      const int free_now = vb;
      vb = kb;
      kb = nb;
      nb = free_now;
      row = next_row;
      next_row = after_row;
      valid = next_valid;
    }
    wait_copies();

    // the waves' parts, one after another into `rows`
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      l[mt] = query_sum(l[mt]);
      if (g == 0) {
        stat[0][wave][16 * mt + li] = m[mt];
        stat[1][wave][16 * mt + li] = l[mt];
      }
    }
    __syncthreads();   // and all steps are done with the buffers
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stat[0][w][16 * mt + li]);
      const float fac = l[mt] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m[mt] - top);
#pragma unroll
      for (int d = 0; d < 2 * NB; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[mt][d][r] = l[mt] == 0.0f ? 0.0f : o[mt][d][r] * fac;
    }
    for (int w = 0; w < kWaves; ++w) {
      if (w == wave) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int d = 0; d < 2 * NB; ++d) {
            f32x4* to = reinterpret_cast<f32x4*>(rows + (16 * mt + li) * QP + 16 * d + 4 * g);
            *to = w ? *to + o[mt][d] : o[mt][d];
          }
      }
      __syncthreads();
    }
    const bool whole = first == 0 && count == q.units;
    float* part = p.partial + (int64_t)(2 * blockIdx.x + (leading ? 0 : 1)) * (16 * MT) * (D + 2);
    for (int r = wave; r < 16 * MT; r += kWaves) {
      const int64_t at = r0 + r;
      if (at >= nrows) break;
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stat[0][w][r]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float lw = stat[1][w][r];
        if (lw != 0.0f) sum += lw * __builtin_amdgcn_exp2f(stat[0][w][r] - top);
      }
      float a = 0.0f, b = 0.0f;
      if (2 * lane < D) {
        const f32x2 x = *reinterpret_cast<const f32x2*>(rows + r * QP + 2 * lane);
        a = x[0];
        b = x[1];
      }
      if (whole) {
        const int64_t i = at / p.group;
        store_row(p, a, b, sum, q.row0 + i, hk * p.group + (int)(at - i * p.group), lane);
      } else {
        float* to = part + (int64_t)r * (D + 2);
        if (2 * lane < D) *reinterpret_cast<f32x2*>(to + 2 * lane) = f32x2{a, b};
        if (lane == 0) *reinterpret_cast<f32x2*>(to + D) = f32x2{top, sum};
      }
    }
  }
}

// Joins the parts of the item inside which workgroup w + 1's units begin first;
// blockIdx.y: four rows of its tile.
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
  const int r = 4 * blockIdx.y + wave;
  const int64_t at = item / p.at.kv_heads * (16 * p.rows16) + r, nrows = (int64_t)q.rows * p.group;
  if (at >= nrows) return;
  const int w0 = w - 1, w1 = (int)((s0 + q.units - 1) / quota);
  const int64_t size = (int64_t)16 * p.rows16 * (D + 2);
  auto part = [&](int x) {   // an item that begins inside a workgroup's units is its second part
    return p.partial + (2 * x + (x == w0 && a0 > (int64_t)w0 * quota ? 1 : 0)) * size + (int64_t)r * (D + 2);
  };
  float top = -INFINITY;
  for (int x = w0 + lane; x <= w1; x += 64) top = fmaxf(top, part(x)[D]);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  float a = 0.0f, b = 0.0f, l = 0.0f;
  for (int x = w0; x <= w1; ++x) {
    const float* from = part(x);
    const f32x2 s = *reinterpret_cast<const f32x2*>(from + D);
    f32x2 y = {0.0f, 0.0f};
    if (2 * lane < D) y = *reinterpret_cast<const f32x2*>(from + 2 * lane);
    if (s[1] == 0.0f) continue;   // saw nothing
    const float fac = __builtin_amdgcn_exp2f(s[0] - top);
    a += y[0] * fac;
    b += y[1] * fac;
    l += s[1] * fac;
  }
  const int64_t i = at / p.group;
  store_row(p, a, b, l, q.row0 + i, hk * p.group + (int)(at - i * p.group), lane);
}

template <int GRID, int KIND>
void launch(const KvAttn& p, hipStream_t s) {
  const bool narrow = p.at.D <= 64;
  if (p.rows16 == 1) {
    if (narrow) k_kv_attn<GRID, KIND, 2, 1><<<kKvGroups, kThreads, 0, s>>>(p);
    else k_kv_attn<GRID, KIND, 4, 1><<<kKvGroups, kThreads, 0, s>>>(p);
  } else {
    if (narrow) k_kv_attn<GRID, KIND, 2, 2><<<kKvGroups, kThreads, 0, s>>>(p);
    else k_kv_attn<GRID, KIND, 4, 2><<<kKvGroups, kThreads, 0, s>>>(p);
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
  k_kv_join<<<dim3(kKvGroups - 1, 4 * (unsigned)p.rows16), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace ufp4
