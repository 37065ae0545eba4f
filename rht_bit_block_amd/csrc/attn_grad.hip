// Gradients of causal attention over packed sequences with shared key heads.
//
//   p_ij = e^(z_ij - lse_i)        delta_i = do_i . o_i
//   dv_j = sum_i p_ij do_i         ds_ij = p_ij (do_i . v_j - delta_i)
//   dk_j = scale sum_i ds_ij q_i   dq_i = scale sum_j ds_ij k_j
//
// The scores are computed again, twice: one kernel goes over the queries for
// 128 keys and sums dk and dv, over all heads of the group, in registers; another
// goes over the keys for 128 queries and sums dq.  Seven products instead of five,
// but no sum is shared between workgroups: no atomics, no order that changes,
// nothing in memory that is not an output.  p and ds are rounded to bf16 for the
// products that they enter, half a step each in long sums.
//
// As in the forward pass a product's registers are the next one's fragments: with
// s = q k^T (a key per lane) p and ds enter dv = p^T do and dk = ds^T q, with s^T =
// k q^T (a query per lane) ds enters dq^T = k^T ds^T.
#include "attn_core.h"

namespace ufp4 {

namespace {

using namespace attn;

// delta and lse log2(e), [heads][T]: sixteen lanes a row of a head.
__global__ __launch_bounds__(256) void k_attn_delta(AttnLaunch p) {
  const int part = threadIdx.x & 15, h = blockIdx.y;
  for (int64_t t = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); t < p.T;
       t += (int64_t)gridDim.x * 16) {
    float s = 0.0f;
    if (8 * part < p.D) {
      const u32x4 a = *reinterpret_cast<const u32x4*>(p.o + t * p.ldo + (int64_t)h * p.D + 8 * part);
      const u32x4 b =
          *reinterpret_cast<const u32x4*>(p.dout + t * p.lddo + (int64_t)h * p.D + 8 * part);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s = __builtin_fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), s);
        s = __builtin_fmaf(__uint_as_float(a[i] & 0xFFFF0000u), __uint_as_float(b[i] & 0xFFFF0000u), s);
      }
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) s += __shfl_xor(s, d);
    if (part == 0) {
      p.delta[h * p.T + t] = s;
      p.lw[h * p.T + t] = p.lse[t * p.heads + h] * kLog2e;
    }
  }
}

// dk and dv of 128 keys of one key head, 32 to a wave.
template <int DP>
__global__ __launch_bounds__(256, 1) void k_attn_dkv(AttnLaunch p) {
  constexpr int S = DP / 16, NB = DP / 32;
  constexpr int TILE = 64 * DP * 2;
  constexpr int STAGE = 2 * TILE;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];
  __shared__ __attribute__((aligned(16))) float stat[2][2][64];   // stage; lse log2(e), delta
  int64_t row0;
  int n, t;
  if (!find_tile(p.starts, p.B, p.T, (int)blockIdx.x, row0, n, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = blockIdx.y;
  const int k0 = t * kAttnTile, kw = k0 + 32 * wave;
  const int key = kw + (lane & 31);
  const float c = p.scale * kLog2e;

  bf16x8 k[S], v[S];
  load_rows<DP>(k, p.k + row0 * p.ldk + (int64_t)hk * p.D, p.ldk, kw, n, p.D, lane);
  load_rows<DP>(v, p.v + row0 * p.ldv + (int64_t)hk * p.D, p.ldv, kw, n, p.D, lane);
  floatx16 dk[NB], dv[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) dk[b] = dv[b] = zero16();

  // the queries from the first key on, 64 a step, head after head of the group
  const int per_head = (n - k0 + 63) / 64, steps = per_head * p.group;
  TileCopy<DP, 4> copy;
  copy.init(lane);
  const uint32_t lds0 = lds_address(lds);
  auto issue = [&](int i, int st) {
    const int h = hk * p.group + i / per_head, i0 = k0 + 64 * (i % per_head);
    copy.issue(lds0 + st * STAGE, p.q + row0 * p.ldq + (int64_t)h * p.D, p.ldq, i0, n, p.D, wave, lane);
    copy.issue(lds0 + st * STAGE + TILE, p.dout + row0 * p.lddo + (int64_t)h * p.D, p.lddo, i0, n, p.D,
               wave, lane);
    // queries past the sequence: q, do, lse and delta are 0, and so is what they add
    if (wave < 2)
      lds_load4(lds_address(&stat[st][wave][0]),
                rsrc4((wave ? p.delta : p.lw) + h * p.T + row0 + i0, 4u * (uint32_t)min(n - i0, 64)),
                4u * lane, 0u);
  };
  issue(0, 0);
  for (int i = 0; i < steps; ++i) {
    const int st = i & 1;
    const uint8_t* qt = lds + st * STAGE;
    const uint8_t* ot = qt + TILE;
    wait_vmcnt<0>();
    __syncthreads();   // step i is there, and step i - 1 has been read
    if (i + 1 < steps) issue(i + 1, st ^ 1);
    const int i0 = k0 + 64 * (i % per_head);
    if (i0 + 63 < kw || kw >= n) continue;   // every query lies before the wave's keys
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (i0 + 32 * u + 31 < kw) continue;
      floatx16 s = zero16(), dp = zero16();
#pragma unroll
      for (int x = 0; x < S; ++x) {
        s = mfma(frag_rows<DP>(qt, 32 * u, x, lane), k[x], s);
        dp = mfma(frag_rows<DP>(ot, 32 * u, x, lane), v[x], dp);
      }
      const bool edge = i0 + 32 * u < kw + 31;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int at = 32 * u + 8 * g + 4 * (lane >> 5);
        const f32x4 lw = *reinterpret_cast<const f32x4*>(&stat[st][0][at]);
        const f32x4 de = *reinterpret_cast<const f32x4*>(&stat[st][1][at]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 4 * g + e;
          float w = __builtin_amdgcn_exp2f(s[r] * c - lw[e]);
          if (edge && key > i0 + at + e) w = 0.0f;
          s[r] = w;
          dp[r] = w == 0.0f ? 0.0f : w * (dp[r] - de[e]);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bf16x8 w = frag_of(s, x), ds = frag_of(dp, x);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          dv[b] = mfma(w, frag_turned<DP>(ot, 32 * u + 16 * x, 32 * b, lane), dv[b]);
          dk[b] = mfma(ds, frag_turned<DP>(qt, 32 * u + 16 * x, 32 * b, lane), dk[b]);
        }
      }
    }
  }
  wait_vmcnt<0>();
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

// dq of 128 queries of one head, 32 to a wave.
template <int DP>
__global__ __launch_bounds__(256, 1) void k_attn_dq(AttnLaunch p) {
  constexpr int S = DP / 16, NB = DP / 32;
  constexpr int TILE = 64 * DP * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * TILE];
  int64_t row0;
  int n, t;
  if (!find_tile(p.starts, p.B, p.T, (int)(gridDim.x - 1 - blockIdx.x), row0, n, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.y, hk = h / p.group;
  const int q0 = t * kAttnTile, qw = q0 + 32 * wave;
  const int qi = qw + (lane & 31);
  const uint16_t* kb = p.k + row0 * p.ldk + (int64_t)hk * p.D;
  const uint16_t* vb = p.v + row0 * p.ldv + (int64_t)hk * p.D;
  const int tiles = (min(n, q0 + kAttnTile) + 63) / 64;
  TileCopy<DP, 4> copy;
  copy.init(lane);
  const uint32_t lds0 = lds_address(lds);
  copy.issue(lds0, kb, p.ldk, 0, n, p.D, wave, lane);
  copy.issue(lds0 + TILE, vb, p.ldv, 0, n, p.D, wave, lane);
  bf16x8 q[S], g[S];
  load_rows<DP>(q, p.q + row0 * p.ldq + (int64_t)h * p.D, p.ldq, qw, n, p.D, lane);
  load_rows<DP>(g, p.dout + row0 * p.lddo + (int64_t)h * p.D, p.lddo, qw, n, p.D, lane);
  const float lw = qi < n ? p.lw[h * p.T + row0 + qi] : INFINITY;
  const float delta = qi < n ? p.delta[h * p.T + row0 + qi] : 0.0f;
  const float c = p.scale * kLog2e;
  floatx16 dq[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) dq[b] = zero16();

  for (int j = 0; j < tiles; ++j) {
    const uint8_t* kt = lds + (j & 1) * 2 * TILE;
    const uint8_t* vt = kt + TILE;
    wait_vmcnt<0>();
    __syncthreads();   // tile j is there, and tile j - 1 has been read
    if (j + 1 < tiles) {
      const uint32_t to = lds0 + ((j + 1) & 1) * 2 * TILE;
      copy.issue(to, kb, p.ldk, 64 * (j + 1), n, p.D, wave, lane);
      copy.issue(to + TILE, vb, p.ldv, 64 * (j + 1), n, p.D, wave, lane);
    }
    const int j0 = 64 * j;
    if (j0 > qw + 31 || qw >= n) continue;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (j0 + 32 * u > qw + 31) continue;
      floatx16 s = zero16(), dp = zero16();
#pragma unroll
      for (int x = 0; x < S; ++x) {
        s = mfma(frag_rows<DP>(kt, 32 * u, x, lane), q[x], s);
        dp = mfma(frag_rows<DP>(vt, 32 * u, x, lane), g[x], dp);
      }
      const bool edge = j0 + 32 * u + 31 > qw;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int key = j0 + 32 * u + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        float w = __builtin_amdgcn_exp2f(s[r] * c - lw);
        if (edge && key > qi) w = 0.0f;
        s[r] = w == 0.0f ? 0.0f : w * (dp[r] - delta);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bf16x8 ds = frag_of(s, x);
#pragma unroll
        for (int b = 0; b < NB; ++b)
          dq[b] = mfma(frag_turned<DP>(kt, 32 * u + 16 * x, 32 * b, lane), ds, dq[b]);
      }
    }
  }
  wait_vmcnt<0>();
  if (qi >= n) return;
  uint16_t* out = p.dq + (row0 + qi) * p.lddq + (int64_t)h * p.D;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int d = 32 * b + 2 * r + 4 * (lane >> 5);
      if (d < p.D) {
        const u32x2 x = {pack_bf16(dq[b][r] * p.scale, dq[b][r + 1] * p.scale),
                         pack_bf16(dq[b][r + 2] * p.scale, dq[b][r + 3] * p.scale)};
        *reinterpret_cast<u32x2*>(out + d) = x;
      }
    }
}

template <int DP>
void launch(const AttnLaunch& p, hipStream_t s) {
  const unsigned tiles = (unsigned)(p.T / kAttnTile + p.B);
  k_attn_dkv<DP><<<dim3(tiles, (unsigned)p.kv_heads), 256, 0, s>>>(p);
  k_attn_dq<DP><<<dim3(tiles, (unsigned)p.heads), 256, 0, s>>>(p);
}

}  // namespace

int64_t attn_workspace(int64_t T, int32_t heads) { return 2 * (int64_t)heads * T * 4; }

hipError_t launch_attn_bwd(const AttnLaunch& p, hipStream_t s) {
  const int64_t blocks = (p.T + 15) / 16;
  k_attn_delta<<<dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20), (unsigned)p.heads), 256, 0, s>>>(p);
  if (p.D <= 64) launch<64>(p, s);
  else launch<128>(p, s);
  return hipGetLastError();
}

}  // namespace ufp4
