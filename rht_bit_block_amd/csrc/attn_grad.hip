// Gradients of causal attention over packed sequences with shared key heads.
//
//   p_ij = e^(z_ij - lse_i)        delta_i = do_i . o_i
//   dv_j = sum_i p_ij do_i         ds_ij = p_ij (do_i . v_j - delta_i)
//   dk_j = scale sum_i ds_ij q_i   dq_i = scale sum_j ds_ij k_j
//
// The scores are computed again, twice: one kernel goes over the keys for 128 queries
// and sums dq (and leaves their delta and lse log2(e) for the other); another goes
// over the queries for 128 keys and sums dk and dv, over all heads of the group, in
// registers.  Eight products instead of five,
// but no sum is shared between workgroups: no atomics, no order that changes,
// nothing in memory that is not an output.  p and ds are rounded to bf16 for the
// products that they enter, half a step each in long sums.
//
// Bound as the forward pass is: 4 sequences of 4096 tokens, 40 heads on 8 key heads, D =
// 128, on cards of 3.16 .. 3.37 ms for forward and backward: forward 0.69 .. 0.72 ms
// (0.95 .. 1.0 PFLOP/s), dq 1.20 .. 1.30 and dk/dv 1.26 .. 1.36 ms (four products
// each: 1.06 .. 1.15 and 1.01 .. 1.09 PFLOP/s).
//
// As in the forward pass a product's registers are the next one's fragments: with
// s = q k^T (a key per lane) p and ds enter dv = p^T do and dk = ds^T q, with s^T =
// k q^T (a query per lane) ds enters dq^T = k^T ds^T.
#include "attn_core.h"

namespace ufp4 {

namespace {

using namespace attn;

// x plus both bf16 values of a pair, in fp32.
__device__ __forceinline__ float add_pair(uint32_t pair, float x) {
  const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), one, x, false);
}

// dk and dv of 128 keys of one key head, 32 to a wave: two waves to a SIMD, whose
// registers hold the sums and K; V's rows stay in LDS.
template <int DP, int S, int NB, int PARTS>
__global__ __launch_bounds__(256 * PARTS, 2) void k_attn_dkv(AttnLaunch p, int first, int tiles_in_all) {
  constexpr int TILE = 32 * DP * 2;
  constexpr int STAGE = 2 * TILE;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * TILE + PARTS * 2 * STAGE];
  __shared__ __attribute__((aligned(16))) float all_stat[PARTS][2][64];   // stage; lse log2(e) and delta of 32 queries
  int64_t row0;
  int n, t;
  const Share me = share_of(blockIdx.x, p.by_kv_heads, p.by_kv_heads, 1);
  if (!find_tile<true>(p.starts, p.B, p.T, tiles_in_all, first + me.tile, row0, n, t)) return;
  const int lane = threadIdx.x & 63, any_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = any_wave & 3, part = any_wave >> 2;
  float (&stat)[2][64] = all_stat[part];
  const int hk = me.head;
  const int k0 = t * kAttnTile, kw = k0 + 32 * wave;
  const int key = kw + (lane & 31);
  const float c = score_factor(p.scale);

  bf16x8 k[S];
  load_rows<S>(k, p.k + row0 * p.ldk + (int64_t)hk * p.D, p.ldk, kw, n, p.D, lane);
  apply_sign(k, p.scale);
  floatx16 dk[NB], dv[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) dk[b] = dv[b] = zero16();

  // the queries from the first key on, 32 a step, head after head of the group
  const int per_head = (n - k0 + 31) / 32;
  uint8_t* const stages = lds + 4 * TILE + part * 2 * STAGE;
  const uint32_t lds0 = lds_address(lds), steps0 = lds_address(stages);
  {
    TileCopy<DP, 128, 4 * PARTS> copy;
    copy.init(lane);
    copy.issue(lds0, p.v + row0 * p.ldv + (int64_t)hk * p.D, p.ldv, k0, n, p.D, any_wave, lane);
  }
  TileCopy<DP, 32, 4> copy;
  copy.init(lane);
  // queries past the sequence: q, do, lse and delta are 0
  auto issue = [&](int h, int i0, int st) {
    copy.issue(steps0 + st * STAGE, p.q + row0 * p.ldq + (int64_t)h * p.D, p.ldq, i0, n, p.D, wave, lane);
    copy.issue(steps0 + st * STAGE + TILE, p.dout + row0 * p.lddo + (int64_t)h * p.D, p.lddo, i0, n, p.D,
               wave, lane);
    if (wave < 2 && lane < 32)
      lds_load4(lds_address(&stat[st][32 * wave]),
                rsrc4((wave ? p.delta : p.lw) + h * p.T + row0 + i0, 4u * (uint32_t)min(n - i0, 32)),
                4u * lane, 0u);
  };
  arrived(k);
  const RowFrag<DP> rows(lane);
  const TurnedFrag<DP> turned(lane);
  const int h_end = (hk + 1) * p.group;
  int h = hk * p.group, step = part;   // of the step in work
  auto settle = [&] {
    while (step >= per_head) {   // at most PARTS times
      step -= per_head;
      ++h;
    }
  };
  settle();
  if (h < h_end) issue(h, k0 + 32 * step, 0);
  const int passes = ((int)p.group * per_head + PARTS - 1) / PARTS;
  for (int x = 0; x < passes; ++x) {
    const int st = x & 1;
    const uint8_t* qt = stages + st * STAGE;
    const uint8_t* ot = qt + TILE;
    const int i0 = k0 + 32 * step;
    const bool live = h < h_end;   // a part may have a step less
    wait_vmcnt<0>();
    __syncthreads();   // the step is there, and the one before has been read
    step += PARTS;
    settle();
    if (h < h_end) issue(h, k0 + 32 * step, st ^ 1);
    if (!live || i0 + 31 < kw || kw >= n) continue;   // every query lies before the wave's keys
    floatx16 s = zero16(), dp = zero16();
    {
      struct Three {
        bf16x8 q, g, v;
      };
      auto read = [&](int x) {
        return Three{rows.read(qt, 0, x), rows.read(ot, 0, x), rows.read(lds, 32 * wave, x)};
      };
      Run<S, 1, Three> run;
      run.begin(read);
      run.go(read, [&](int x, const Three& f) {
        s = mfma(f.q, k[x], s);
        dp = mfma(f.g, f.v, dp);
      });
    }
    // do for dv, q for dk, in turn
    auto read_t = [&](int i) {
      return turned.read((i & 1) ? qt : ot, 16 * (i / (2 * NB)), 32 * ((i >> 1) % NB));
    };
    Run<4 * NB, 3, bf16x8> run;
    run.begin(read_t);
    // queries before the key, and past the sequence: their score may be 0 times an infinite
    // element of the key
    if (i0 < kw + 31 || i0 + 32 > n) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int i = i0 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        if (key > i || i >= n) s[r] = -INFINITY;
      }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int at = 8 * g + 4 * (lane >> 5);
      const f32x4 lw = *reinterpret_cast<const f32x4*>(&stat[st][at]);
      const f32x4 de = *reinterpret_cast<const f32x4*>(&stat[st][32 + at]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 4 * g + e;
        s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c, -lw[e]));
        dp[r] = mul_legacy(s[r], dp[r] - de[e]);   // 0 for a key that is not seen
      }
    }
    uint32_t pw[8], pd[8];
    round_pairs(s, pw);
    round_pairs(dp, pd);
    const bf16x8 w[2] = {frag_of(pw, 0), frag_of(pw, 1)}, ds[2] = {frag_of(pd, 0), frag_of(pd, 1)};
    run.go(read_t, [&](int i, const bf16x8& f) {
      const int x = i / (2 * NB), b = (i >> 1) % NB;
      if (i & 1) dk[b] = mfma(ds[x], f, dk[b]);
      else dv[b] = mfma(w[x], f, dv[b]);
    });
  }
  wait_vmcnt<0>();
  if constexpr (PARTS == 2) {
    static_assert(sizeof(lds) >= 4 * NB * 4096, "the sums of four waves");
    float* sums = reinterpret_cast<float*>(lds) + wave * NB * 1024;
    __syncthreads();   // all steps have been read
    if (part) leave_sums(sums, dk, lane);
    __syncthreads();
    if (!part) take_sums(sums, dk, 1.0f, 1.0f, lane);
    __syncthreads();
    if (part) leave_sums(sums, dv, lane);
    __syncthreads();
    if (part) return;
    take_sums(sums, dv, 1.0f, 1.0f, lane);
  }
  // a lane holds element 32 b + l % 32 of keys kw + 8 (r / 4) + 4 (l / 32) + r % 4
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int d = 32 * b + (lane & 31);
    if (d >= p.D) continue;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int at = kw + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
      if (at >= n) continue;
      const int64_t row = row0 + at;
      const uint32_t x = pack_bf16(dk[b][r] * p.scale, dv[b][r]);
      p.dk[row * p.lddk + (int64_t)hk * p.D + d] = (uint16_t)x;
      p.dv[row * p.lddv + (int64_t)hk * p.D + d] = (uint16_t)(x >> 16);
    }
  }
}

// dq of 128 queries of one head, 32 to a wave.  The forward pass' o is rounded, and
// with it delta, which enters every ds of a row: it would be the largest error of both
// gradients (4.3e-3 of the norm, where the outputs' rounding is 1.7e-3).  But the ds
// of a row add to 0, so that from a near delta0
//   dq = scale (sum_j ds0_j k_j - (sum_j ds0_j) (sum_j p_j k_j))     ds0 = p (dp - delta0)
// holds for whatever is summed: with the rounded ds0 in both sums the roundings' common
// part goes as well (2.2e-3).  It takes one product more, on fragments of K that are
// there.  The row's sum of the ds0 themselves is what delta lacks, for dk.
template <int DP, int S, int NB, int PARTS>
__global__ __launch_bounds__(256 * PARTS, 2) void k_attn_dq(AttnLaunch p, int first, int tiles_in_all) {
  constexpr int TILE = 32 * DP * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[(4 + 4 * PARTS) * TILE];
  int64_t row0;
  int n, t;
  const Share me = share_of(blockIdx.x, p.by_heads, p.by_kv_heads, p.group);
  if (!find_tile<false>(p.starts, p.B, p.T, tiles_in_all, first + me.tile, row0, n, t)) return;
  const int lane = threadIdx.x & 63, any_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = any_wave & 3, part = any_wave >> 2;
  const int h = me.head, hk = me.kv_head;
  const int q0 = t * kAttnTile, qw = q0 + 32 * wave;
  const int qi = qw + (lane & 31);
  const uint16_t* kb = p.k + row0 * p.ldk + (int64_t)hk * p.D;
  const uint16_t* vb = p.v + row0 * p.ldv + (int64_t)hk * p.D;
  const uint16_t* gb = p.dout + row0 * p.lddo + (int64_t)h * p.D;
  const int tiles = (min(n, q0 + kAttnTile) + 31) / 32;
  uint8_t* const stages = lds + (4 + 4 * part) * TILE;
  const uint32_t lds0 = lds_address(lds), steps0 = lds_address(stages);
  {
    TileCopy<DP, 128, 4 * PARTS> copy;   // the rows of do
    copy.init(lane);
    copy.issue(lds0, gb, p.lddo, q0, n, p.D, any_wave, lane);
  }
  TileCopy<DP, 32, 4> copy;
  copy.init(lane);
  copy.issue(steps0, kb, p.ldk, 32 * part, n, p.D, wave, lane);
  copy.issue(steps0 + TILE, vb, p.ldv, 32 * part, n, p.D, wave, lane);
  // delta0 is the diagonal of o do^T, by the instructions that v do^T comes from: where a
  // query has one key, o is that v and do . v - delta0 exactly 0
  float lw = INFINITY, delta = 0.0f;
  {
    bf16x8 o[S], g[S];
    load_rows<S>(o, p.o + row0 * p.ldo + (int64_t)h * p.D, p.ldo, qw, n, p.D, lane);
    load_rows<S>(g, gb, p.lddo, qw, n, p.D, lane);
    floatx16 x = zero16();
#pragma unroll
    for (int s = 0; s < S; ++s) x = mfma(o[s], g[s], x);
    // element (i, i) is register i % 4 + 4 (i / 8) of lane i or i + 32
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if ((lane & 31) == 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) delta = x[r];
    delta = both_sum(delta);
    if (qi < n) lw = p.lse[(row0 + qi) * p.heads + h] * kLog2e;
  }
  bf16x8 q[S];
  load_rows<S>(q, p.q + row0 * p.ldq + (int64_t)h * p.D, p.ldq, qw, n, p.D, lane);
  const float c = score_factor(p.scale);
  apply_sign(q, p.scale);
  arrived(q);
  asm volatile("" : "+v"(lw));
  const RowFrag<DP> rows(lane);
  const TurnedFrag<DP> turned(lane);
  floatx16 dq[NB], pk[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) dq[b] = pk[b] = zero16();
  float lacks = 0.0f, rounded = 0.0f;   // this lane's half of the sums of ds0

  for (int step = 0; PARTS * step < tiles; ++step) {
    const int j = PARTS * step + part;
    const uint8_t* kt = stages + (step & 1) * 2 * TILE;
    const uint8_t* vt = kt + TILE;
    wait_vmcnt<0>();
    __syncthreads();   // tile j is there, and the one before has been read
    if (j + PARTS < tiles) {
      const uint32_t to = steps0 + ((step + 1) & 1) * 2 * TILE;
      copy.issue(to, kb, p.ldk, 32 * (j + PARTS), n, p.D, wave, lane);
      copy.issue(to + TILE, vb, p.ldv, 32 * (j + PARTS), n, p.D, wave, lane);
    }
    const int j0 = 32 * j;
    if (j0 > qw + 31 || qw >= n) continue;
    floatx16 s = zero16(), dp = zero16();
    {
      struct Three {
        bf16x8 k, v, g;
      };
      auto read = [&](int x) {
        return Three{rows.read(kt, 0, x), rows.read(vt, 0, x), rows.read(lds, 32 * wave, x)};
      };
      Run<S, 1, Three> run;
      run.begin(read);
      run.go(read, [&](int x, const Three& f) {
        s = mfma(f.k, q[x], s);
        dp = mfma(f.v, f.g, dp);
      });
    }
    auto read_k = [&](int i) { return turned.read(kt, 16 * (i / NB), 32 * (i % NB)); };
    Run<2 * NB, 2, bf16x8> run;
    run.begin(read_k);
    if (j0 + 31 > qw) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (j0 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3) > qi) s[r] = -INFINITY;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c, -lw));
      dp[r] = mul_legacy(s[r], dp[r] - delta);   // 0 for a key that is not seen
      lacks += dp[r];
    }
    uint32_t pw[8], pd[8];
    round_pairs(s, pw);
    round_pairs(dp, pd);
    const bf16x8 w[2] = {frag_of(pw, 0), frag_of(pw, 1)}, ds[2] = {frag_of(pd, 0), frag_of(pd, 1)};
#pragma unroll
    for (int i = 0; i < 8; ++i) rounded = add_pair(pd[i], rounded);
    run.go(read_k, [&](int i, const bf16x8& f) {
      dq[i % NB] = mfma(f, ds[i / NB], dq[i % NB]);
      pk[i % NB] = mfma(f, w[i / NB], pk[i % NB]);
    });
  }
  wait_vmcnt<0>();
  rounded = both_sum(rounded);
  lacks = both_sum(lacks);
  float* sums = reinterpret_cast<float*>(lds) + wave * (NB * 1024);
  if constexpr (PARTS == 2) {
    __shared__ float both[2][2][4][64];   // part; rounded and lacks, of both parts in the end
    both[part][0][wave][lane] = rounded;
    both[part][1][wave][lane] = lacks;
    __syncthreads();   // and all tiles have been read
    rounded = both[0][0][wave][lane] + both[1][0][wave][lane];
    lacks = both[0][1][wave][lane] + both[1][1][wave][lane];
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) dq[b][r] = __builtin_fmaf(-rounded, pk[b][r], dq[b][r]);
  if constexpr (PARTS == 2) {
    static_assert(sizeof(lds) >= 4 * NB * 4096, "the sums of four waves");
    if (part) leave_sums(sums, dq, lane);
    __syncthreads();
    if (part) return;
    take_sums(sums, dq, 1.0f, 1.0f, lane);
  }
  if (qi >= n) return;
  if (lane < 32) {
    p.delta[h * p.T + row0 + qi] = delta + lacks;
    // finite for a row whose every score is -inf, so that its weights are 0 and keys that it does not
    // see keep theirs
    p.lw[h * p.T + row0 + qi] = lw == -INFINITY ? -3.0e38f : lw;
  }
  uint16_t* out = p.dq + (row0 + qi) * p.lddq + (int64_t)h * p.D;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int d = 32 * b + 2 * r + 4 * (lane >> 5);
      if (d < p.D) {
        const u32x2 v = {pack_bf16(dq[b][r] * p.scale, dq[b][r + 1] * p.scale),
                         pack_bf16(dq[b][r + 2] * p.scale, dq[b][r + 3] * p.scale)};
        *reinterpret_cast<u32x2*>(out + d) = v;
      }
    }
}

template <int DP, int S, int NB>
void launch(const AttnLaunch& p, hipStream_t s) {
  const int64_t tiles = p.T / kAttnTile + p.B;
  over_tiles(tiles, p.heads, [&](int t0, unsigned blocks) {
    if (in_parts(p, tiles * p.heads)) k_attn_dq<DP, S, NB, 2><<<blocks, 512, 0, s>>>(p, t0, (int)tiles);
    else k_attn_dq<DP, S, NB, 1><<<blocks, 256, 0, s>>>(p, t0, (int)tiles);
  });
  over_tiles(tiles, p.kv_heads, [&](int t0, unsigned blocks) {   // reads what dq's left
    if (in_parts(p, tiles * p.kv_heads)) k_attn_dkv<DP, S, NB, 2><<<blocks, 512, 0, s>>>(p, t0, (int)tiles);
    else k_attn_dkv<DP, S, NB, 1><<<blocks, 256, 0, s>>>(p, t0, (int)tiles);
  });
}

}  // namespace

int64_t attn_workspace(int64_t T, int32_t heads) { return 2 * (int64_t)heads * T * 4; }

hipError_t launch_attn_bwd(const AttnLaunch& p, hipStream_t s) {
  if (p.D <= 32) launch<64, 2, 1>(p, s);
  else if (p.D <= 64) launch<64, 4, 2>(p, s);
  else if (p.D <= 96) launch<128, 6, 3>(p, s);
  else launch<128, 8, 4>(p, s);
  return hipGetLastError();
}

}  // namespace ufp4
