// Causal attention over packed sequences with shared key heads.
//
//   z_ij = scale q_i . k_j (j <= i)    o_i = sum_j e^(z_ij - lse_i) v_j
//
// One pass over the keys with a running maximum m and sum l of each query:
// for a tile of keys, with c = scale log2(e), s = q k^T,
//   p = 2^(c s - m)    l = l + sum p    o = o + p v     (o, l first times 2^(m_old - m))
// m moves only when a tile's maximum passes it by more than 8, so that o is
// hardly ever rescaled; p is then at most 2^8, and the result the same up to
// rounding.  lse = (m + log2 l) ln 2.  p is rounded to bf16 for the product with
// v: half a step of each weight, a random sum far below o's own rounding.
//
// A workgroup takes 128 queries of one head, 32 to a wave, in registers; K and V
// pass through LDS in double-buffered tiles of 64 keys, copied by buffer_load
// ... lds while the tile before is computed.  s^T = k q^T comes out with a query per
// lane, so the softmax is in-lane but for one exchange of halves.
#include "attn_core.h"

namespace ufp4 {

namespace {

using namespace attn;

template <int DP>
__global__ __launch_bounds__(256, 2) void k_attn_fwd(AttnLaunch p, int last_tile) {
  constexpr int S = DP / 16, NB = DP / 32;
  constexpr int TILE = 64 * DP * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * TILE];
  int64_t row0;
  int n, t;
  // the last tile of a sequence has the most keys: it goes first
  const Share me = share_of(blockIdx.x, p.kv_heads, p.group);
  if (!find_tile(p.starts, p.B, p.T, last_tile - me.tile, row0, n, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = me.head, hk = h / p.group;
  const int q0 = t * kAttnTile, qw = q0 + 32 * wave;   // the workgroup's and the wave's first query
  const int qi = qw + (lane & 31);
  const uint16_t* kb = p.k + row0 * p.ldk + (int64_t)hk * p.D;
  const uint16_t* vb = p.v + row0 * p.ldv + (int64_t)hk * p.D;
  const int keys = min(n, q0 + kAttnTile);
  const int tiles = (keys + 63) / 64;

  TileCopy<DP, 64, 4> copy;
  copy.init(lane);
  const uint32_t lds0 = lds_address(lds);
  copy.issue(lds0, kb, p.ldk, 0, n, p.D, wave, lane);
  copy.issue(lds0 + TILE, vb, p.ldv, 0, n, p.D, wave, lane);
  bf16x8 q[S];
  load_rows<DP>(q, p.q + row0 * p.ldq + (int64_t)h * p.D, p.ldq, qw, n, p.D, lane);

  floatx16 o[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) o[b] = zero16();
  float m = -INFINITY, l = 0.0f;
  const float c = p.scale * kLog2e;

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
    if (j0 > qw + 31 || qw >= n) continue;   // nothing for this wave in the tile
    floatx16 s[2] = {zero16(), zero16()};
#pragma unroll
    for (int x = 0; x < S; ++x)
#pragma unroll
      for (int u = 0; u < 2; ++u) s[u] = mfma(frag_rows<DP>(kt, 32 * u, x, lane), q[x], s[u]);
    reads_ahead<2 * S, 2 * S, 4>();
    // c is the sign of the factor too: the maximum is of c s
    if (j0 + 63 > qw) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int key = j0 + 32 * u + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
          s[u][r] = key > qi ? -INFINITY : s[u][r] * c;
        }
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[u][r] *= c;
    }
    float top = s[0][0];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[u][r]);
    top = both_max(top);
    if (__any(top > m + 8.0f)) {   // also the first finite one
      const float next = top > m + 8.0f ? top : m;
      const float f = next == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - next);
      m = next;
      l *= f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[b][r] *= f;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[u][r] = __builtin_amdgcn_exp2f(s[u][r] - m);
        l += s[u][r];
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bf16x8 w = frag_of(s[u], x);
#pragma unroll
        for (int b = 0; b < NB; ++b)
          o[b] = mfma(frag_turned<DP>(vt, 32 * u + 16 * x, 32 * b, lane), w, o[b]);
      }
    }
    reads_ahead<4 * NB, 8 * NB, 4>();
  }
  wait_vmcnt<0>();
  if (qi >= n) return;
  l = both_sum(l);
  const float inv = 1.0f / l;
  const int64_t row = row0 + qi;
  if (p.lse && lane < 32) p.lse[row * p.heads + h] = (m + __builtin_amdgcn_logf(l)) * kLn2;
  uint16_t* out = p.o + row * p.ldo + (int64_t)h * p.D;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int d = 32 * b + 2 * r + 4 * (lane >> 5);
      if (d < p.D) {
        const u32x2 v = {pack_bf16(o[b][r] * inv, o[b][r + 1] * inv),
                         pack_bf16(o[b][r + 2] * inv, o[b][r + 3] * inv)};
        *reinterpret_cast<u32x2*>(out + d) = v;
      }
    }
}

}  // namespace

hipError_t launch_attn_fwd(const AttnLaunch& p, hipStream_t s) {
  const int64_t tiles = p.T / kAttnTile + p.B;
  over_tiles(tiles, p.heads, [&](int t0, unsigned blocks) {
    const int last = (int)(tiles - 1) - t0;
    if (p.D <= 64) k_attn_fwd<64><<<blocks, 256, 0, s>>>(p, last);
    else k_attn_fwd<128><<<blocks, 256, 0, s>>>(p, last);
  });
  return hipGetLastError();
}

}  // namespace ufp4
