// Rows of a 4-bit cache as they are written (included by kv_e1m2.hip,
// kv_int4.hip and kv_e2m1.hip, one translation unit per codebook) and, in
// kv_rows.hip, read back.
//
// A token's row of one head is a row of a quantized operand with K = D, so a
// write is the quantizer's lane function (quant_core.h: signs, butterflies, block
// scales, rounding, packing) between a load from the packed rows and a store to
// wherever the token's page lies, and a read runs it backwards, x = S RN(c_n
// FWHT(level s)).  A lane takes W = 16 or 32 elements; neighbouring lanes take a
// head's row and then the next token's, because a page holds one head's tokens
// one after another: codes and scales of a page are touched in whole lines.
// Bound by HBM: 2 bytes an element on one side, 0.53 to 0.75 on the other: 16381 tokens of
// eight key heads of 128 (E2M1, E8M0 scales, 85 MB in and out) are written in 24 to 25 us and
// read in 25, where the quantizer takes 22 for as many rows without pages.  A lane with one item
// of many rows waits for four loads in a row; a row's items one after another hide
// them.  (Lanes that take a token's heads in turn instead of its elements: 31 us.)
#pragma once

#include "attn_internal.h"
#include "quant_core.h"

namespace ufp4 {
namespace kv {

constexpr int kThreads = 256;
constexpr int kFull = 1024;     // workgroups that fill the chip
constexpr int kSeqLds = 1024;   // starts kept in LDS while a workgroup looks for its rows' sequences

// Where packed row t lies in the cache, as page and row of a page; page < 0: nowhere,
// seq < 0: in no sequence either.
struct Where {
  int seq;
  int64_t page;
  uint32_t row;
};

// The last sequence that starts at or before t.
template <class P>
__device__ __forceinline__ int last_start(const P* starts, int B, int t) {
  int lo = -1, hi = B;   // starts[lo] <= t < starts[hi], for ends that are never read
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ Where locate(const KvPlace& a, const int32_t* lds_starts, bool in_lds,
                                        int64_t t) {
  Where w{-1, -1, 0u};
  if (t >= a.T) return w;
  const int b = in_lds ? last_start(lds_starts, a.B, (int)t) : last_start(a.starts, a.B, (int)t);
  if (b < 0) return w;
  const int s0 = a.starts[b], s1 = a.starts[b + 1];
  if (t >= s1 || s0 < 0) return w;
  w.seq = b;
  const int64_t at = (int64_t)a.lens[b] - s1 + t;
  const int64_t slot = at >> a.page_shift;
  if (at < 0 || slot >= a.width) return w;
  const int page = a.table[b * a.ldt + slot];
  if (page < 0 || page >= a.pages) return w;
  w.page = page;
  w.row = (uint32_t)at & ((1u << a.page_shift) - 1u);
  return w;
}

// starts into LDS where it fits; all threads of the workgroup.
__device__ __forceinline__ bool starts_to_lds(const KvPlace& a, int32_t (&lds)[kSeqLds]) {
  if (a.B > kSeqLds) return false;
  for (int i = threadIdx.x; i < a.B; i += kThreads) lds[i] = a.starts[i];
  __syncthreads();
  return true;
}

// Number of the token's row of head h among all rows of the cache.
__device__ __forceinline__ uint64_t cache_row(const KvPlace& a, const Where& w, int h) {
  return (((uint64_t)w.page * a.kv_heads + h) << a.page_shift) + w.row;
}

// The lane's place in the launch: W elements from k0 on of packed row t, of the heads of k
// and then of v from item blockIdx.y `items` on.
struct Lane {
  int64_t t;
  uint32_t k0, qpos;
  int item, end;
};
template <int W, int LPC>
__device__ __forceinline__ Lane lane_of(const KvRows& p, FastDiv segs) {
  const uint32_t id = blockIdx.x * kThreads + threadIdx.x;
  const uint32_t rel = qk::fdiv_u32(id, segs);
  Lane l;
  l.t = p.t0 + rel;
  l.k0 = (id - rel * segs.d) * W;
  l.qpos = id & (uint32_t)(LPC - 1);
  l.item = (int)blockIdx.y * p.items;
  l.end = min(l.item + p.items, 2 * p.at.kv_heads);
  return l;
}

// W elements of an item of a packed row.
template <int W>
__device__ __forceinline__ void load_row(const KvRows& p, const Lane& l, int item, uint32_t (&w)[W / 2]) {
  const bool is_v = item >= p.at.kv_heads;
  const int h = is_v ? item - p.at.kv_heads : item;
  const uint16_t* src = (is_v ? p.v + l.t * p.ldv : p.k + l.t * p.ldk) + (int64_t)h * p.at.D + l.k0;
#pragma unroll
  for (int i = 0; i < W / 8; ++i) {
    const uint4 x = qk::ld16(reinterpret_cast<const uint4*>(src) + i);
    w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
  }
}

template <int W, int B, int N, int GRID, int RND>
__global__ __launch_bounds__(kThreads) void k_kv_write(KvRows p, FastDiv segs) {
  __shared__ int32_t starts[kSeqLds];
  constexpr int lpc = N > W ? N / W : 1;
  const Lane l = lane_of<W, lpc>(p, segs);
  // the first item is on its way while the row's place is looked up, the next one while
  // an item is quantized
  uint32_t w[W / 2];
  if (l.t < p.at.T) load_row<W>(p, l, l.item, w);
  const bool in_lds = starts_to_lds(p.at, starts);
  const Where at = locate(p.at, starts, in_lds, l.t);
  if (at.page < 0) return;   // a whole row: the lanes of a rotation stay together
  uint32_t pm[W / 2];
  qk::sign_masks<W>(qk::select_pattern(p, l.qpos), pm);
  for (int item = l.item; item < l.end; ++item) {
    float y[W];
    qk::unpack<W>(w, pm, y);
    if (item + 1 < l.end) load_row<W>(p, l, item + 1, w);
    const uint32_t sig = qk::fwht<W, N>(y, (l.qpos & 1u) ? 0x80000000u : 0u,
                                        (l.qpos & 2u) ? 0x80000000u : 0u, false);
    const bool is_v = item >= p.at.kv_heads;
    const uint64_t row = cache_row(p.at, at, is_v ? item - p.at.kv_heads : item);
    uint8_t* codes = is_v ? p.codes[1] : p.codes[0];
    void* scales = is_v ? p.scales[1] : p.scales[0];
    qk::finish_lane<W, B, N, GRID, RND, KvRows>(
        y, sig, p, 0, codes + (row * p.at.D + l.k0) / 2,
        qk::scale_at<RND>(scales, row * (uint32_t)(p.at.D / B) + l.k0 / B));
  }
}

// Launches `kernel` over all rows, 2^30 lanes at a time.  A lane takes several items (heads
// of k and v) of its row where there are rows enough to fill the chip without: looking
// up the row's place is four dependent loads.
template <class K>
hipError_t over_rows(K kernel, const KvRows& p, int W, hipStream_t s) {
  const int64_t per_row = p.at.D / W, slice = ((int64_t)1 << 30) / per_row;
  KvRows q = p;
  const int all = 2 * p.at.kv_heads;
  const int64_t blocks = (p.at.T * per_row + kThreads - 1) / kThreads;
  const int64_t each = blocks * all / kFull;
  q.items = each < 1 ? 1 : each > all ? all : (int)each;
  const unsigned split = (unsigned)((all + q.items - 1) / q.items);
  for (q.t0 = 0; q.t0 < p.at.T; q.t0 += slice) {
    const int64_t rows = p.at.T - q.t0 < slice ? p.at.T - q.t0 : slice;
    kernel<<<dim3((unsigned)((rows * per_row + kThreads - 1) / kThreads), split), kThreads, 0, s>>>(
        q, make_fastdiv((uint32_t)per_row));
  }
  return hipGetLastError();
}

template <int W, int B, int N, int GRID, int RND>
hipError_t write_n(const KvRows& p, hipStream_t s) {
  return over_rows(k_kv_write<W, B, N, GRID, RND>, p, W, s);
}

template <int B, int GRID, int RND>
hipError_t write_b(const KvRows& p, hipStream_t s) {
  constexpr int W = B == 32 ? 32 : 16;
  switch (p.n) {
    case 1: return write_n<W, B, 1, GRID, RND>(p, s);
    case 2: return write_n<W, B, 2, GRID, RND>(p, s);
    case 4: return write_n<W, B, 4, GRID, RND>(p, s);
    case 8: return write_n<W, B, 8, GRID, RND>(p, s);
    case 16: return write_n<W, B, 16, GRID, RND>(p, s);
    case 32: return write_n<32, B, 32, GRID, RND>(p, s);
    case 64: return write_n<32, B, 64, GRID, RND>(p, s);
    default: return write_n<32, B, 128, GRID, RND>(p, s);
  }
}

// RND bit 1: E8M0 scales (1 x 32 blocks)
template <int GRID>
hipError_t write_grid(const KvRows& p, hipStream_t s) {
  if (p.scale_mode == UFP4_SCALE_POW2) return write_b<32, GRID, 2>(p, s);
  return p.bc == 32 ? write_b<32, GRID, 0>(p, s) : write_b<16, GRID, 0>(p, s);
}

}  // namespace kv

hipError_t kv_write_e1m2(const KvRows& p, hipStream_t s);
hipError_t kv_write_int4(const KvRows& p, hipStream_t s);
hipError_t kv_write_e2m1(const KvRows& p, hipStream_t s);

}  // namespace ufp4
