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
//
// Bound by the matrix cores and the vector units after each other: 32768 tokens, 8 heads on
// one key head, D = 128: 1.97 .. 2.07 ms (1.06 .. 1.11 PFLOP/s), the MFMAs busy 60 % of the
// cycles (at 1.73 GHz, where they alone, busy all the time, run at 1.65), the six vector
// instructions to an MFMA most of the rest, although two workgroups to a compute unit should cover
// one's softmax with the other's products.  Tried and slower: eight waves that share a tile (two sets of keys: 2.17
// ms; 256 queries: 2.03), the next tile's scores multiplied between the exponentials of
// this one (2.05, registers spilled), waves' priorities (no change).
#include "attn_core.h"

namespace ufp4 {

namespace {

using namespace attn;

// DP: elements of a row in LDS; S, NB: 16- and 32-element pieces of a head in use; PARTS: sets of
// four waves that share the tile's keys (in_parts).
template <int DP, int S, int NB, int PARTS>
__global__ __launch_bounds__(256 * PARTS, 2) void k_attn_fwd(AttnLaunch p, int first, int tiles_in_all) {
  constexpr int TILE = 64 * DP * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t all_lds[PARTS * 4 * TILE];
  int64_t row0;
  int n, t;
  const Share me = share_of(blockIdx.x, p.by_heads, p.by_kv_heads, p.group);
  if (!find_tile<false>(p.starts, p.B, p.T, tiles_in_all, first + me.tile, row0, n, t)) return;
  const int lane = threadIdx.x & 63, any_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = any_wave & 3, part = any_wave >> 2;
  uint8_t* const lds = all_lds + part * 4 * TILE;
  const int h = me.head, hk = me.kv_head;
  const int q0 = t * kAttnTile, qw = q0 + 32 * wave;   // the workgroup's and the wave's first query
  const int qi = qw + (lane & 31);
  const uint16_t* kb = p.k + row0 * p.ldk + (int64_t)hk * p.D;
  const uint16_t* vb = p.v + row0 * p.ldv + (int64_t)hk * p.D;
  const int tiles = (min(n, q0 + kAttnTile) + 63) / 64;

  TileCopy<DP, 64, 4> copy;
  copy.init(lane);
  const uint32_t lds0 = lds_address(lds);
  copy.issue(lds0, kb, p.ldk, 64 * part, n, p.D, wave, lane);
  copy.issue(lds0 + TILE, vb, p.ldv, 64 * part, n, p.D, wave, lane);
  bf16x8 q[S];
  load_rows<S>(q, p.q + row0 * p.ldq + (int64_t)h * p.D, p.ldq, qw, n, p.D, lane);
  const float c = score_factor(p.scale);
  apply_sign(q, p.scale);
  arrived(q);
  const RowFrag<DP> rows(lane);
  const TurnedFrag<DP> turned(lane);

  floatx16 o[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) o[b] = zero16();
  float m = -INFINITY, l = 0.0f;   // m: of c s

  for (int step = 0; PARTS * step < tiles; ++step) {
    const int j = PARTS * step + part;
    const uint8_t* kt = lds + (step & 1) * 2 * TILE;
    const uint8_t* vt = kt + TILE;
    wait_vmcnt<0>();
    __syncthreads();   // tile j is there, and the one before has been read
    if (j + PARTS < tiles) {
      const uint32_t to = lds0 + ((step + 1) & 1) * 2 * TILE;
      copy.issue(to, kb, p.ldk, 64 * (j + PARTS), n, p.D, wave, lane);
      copy.issue(to + TILE, vb, p.ldv, 64 * (j + PARTS), n, p.D, wave, lane);
    }
    const int j0 = 64 * j;
    if (j0 > qw + 31 || qw >= n) continue;   // nothing for this wave in the tile
    floatx16 s[2] = {zero16(), zero16()};
    {
      auto read = [&](int i) { return rows.read(kt, 32 * (i & 1), i >> 1); };
      Run<2 * S, 4, bf16x8> run;
      run.begin(read);
      run.go(read, [&](int i, const bf16x8& k) { s[i & 1] = mfma(k, q[i >> 1], s[i & 1]); });
    }
    auto read_v = [&](int i) { return turned.read(vt, 16 * (i / NB), 32 * (i % NB)); };
    Run<4 * NB, 3, bf16x8> run;
    run.begin(read_v);
    if (j0 + 63 > qw) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int key = j0 + 32 * u + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
          if (key > qi) s[u][r] = -INFINITY;
        }
    }
    float top = fmaxf(s[0][0], s[1][0]);
#pragma unroll
    for (int r = 1; r < 16; ++r) top = fmaxf(fmaxf(top, s[0][r]), s[1][r]);
    top = both_max(top) * c;
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
    // a row whose keys so far all score -inf has weights of 0, and m for a later one to move
    const float base = m == -INFINITY ? 0.0f : m;
    bf16x8 w[4];
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[u][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][r], c, -base));
        sum += s[u][r];
      }
      uint32_t pairs[8];
      round_pairs(s[u], pairs);
      w[2 * u] = frag_of(pairs, 0);
      w[2 * u + 1] = frag_of(pairs, 1);
    }
    l += sum;
    run.go(read_v, [&](int i, const bf16x8& v) { o[i % NB] = mfma(v, w[i / NB], o[i % NB]); });
  }
  wait_vmcnt<0>();
  l = both_sum(l);
  if constexpr (PARTS == 2) {
    static_assert(PARTS * 4 * TILE >= 4 * (NB * 4096 + 512), "a lane's sums and two more");
    float* sums = reinterpret_cast<float*>(all_lds) + wave * (NB * 1024 + 128);
    __syncthreads();   // all tiles have been read
    if (part) {
      leave_sums(sums, o, lane);
      sums[NB * 1024 + lane] = m;
      sums[NB * 1024 + 64 + lane] = l;
    }
    __syncthreads();
    if (part) return;
    // a part that has seen no key, or none above -inf, has m = -inf and l = 0
    const float m1 = sums[NB * 1024 + lane], top = fmaxf(m, m1);
    const float base = top == -INFINITY ? 0.0f : top;
    const float f0 = __builtin_amdgcn_exp2f(m - base), f1 = __builtin_amdgcn_exp2f(m1 - base);
    m = top;
    l = l * f0 + sums[NB * 1024 + 64 + lane] * f1;
    take_sums(sums, o, f0, f1, lane);
  }
  if (qi >= n) return;
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

template <int DP, int S, int NB>
void launch(const AttnLaunch& p, hipStream_t s) {
  const int64_t tiles = p.T / kAttnTile + p.B;
  over_tiles(tiles, p.heads, [&](int t0, unsigned blocks) {
    if (in_parts(p, tiles * p.heads)) k_attn_fwd<DP, S, NB, 2><<<blocks, 512, 0, s>>>(p, t0, (int)tiles);
    else k_attn_fwd<DP, S, NB, 1><<<blocks, 256, 0, s>>>(p, t0, (int)tiles);
  });
}

}  // namespace

hipError_t launch_attn_fwd(const AttnLaunch& p, hipStream_t s) {
  if (p.D <= 32) launch<64, 2, 1>(p, s);
  else if (p.D <= 64) launch<64, 4, 2>(p, s);
  else if (p.D <= 96) launch<128, 6, 3>(p, s);
  else launch<128, 8, 4>(p, s);
  return hipGetLastError();
}

}  // namespace ufp4
