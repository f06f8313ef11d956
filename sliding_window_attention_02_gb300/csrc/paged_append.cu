// A chunk of new keys and values to the pages of their sequences.
//
// Row i of sequence b goes to token lens[b] - T_b + i, row a % P of page
// table[b][a / P], head by head.  A warp moves a row: its first reads of the row
// are on their way while it looks for the row's sequence and page.  Bound by
// HBM for long chunks, by latency (the sequence, its length, its page, each a
// round trip) for single tokens.  Measured: 64 tokens of 8 KV heads 2.5 us in a graph,
// 4.4 a call (the host); 3692 rows of 10 heads, 38 MB to move, 5.3 in a graph (the writes
// stay in L2), 7.2 a call.  A warp for a row and not a CTA: a CTA's four rows are 16 to
// 40 KB in flight, and single tokens have no idle lanes' reads to wait for.
#include <algorithm>

#include "paged.cuh"

namespace rswa {
namespace {

constexpr int kRowsPerCta = 4;                 // a warp each
constexpr int kAhead = 10;                     // 16-byte vectors of a lane in flight

template <int ELT>
__global__ void __launch_bounds__(kRowsPerCta * 32)
paged_append_kernel(PagesView pv, BatchArgs ba, const char* __restrict__ k, int64_t k_stride,
                    const char* __restrict__ v, int64_t v_stride) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0)                         // wrong descriptions without rows are told too
    for (int b = threadIdx.x; b < ba.B; b += blockDim.x) {
      PagedSeq s;
      s.load(pv, ba, b);
    }
  const int row = blockIdx.x * kRowsPerCta + warp;
  if (row >= ba.rows) return;
  const int nv = pv.d * ELT / 16;              // vectors of a head's row (a power of two)
  const int all = 2 * pv.Hkv * nv, half = pv.Hkv * nv;
  const uint4* kr = reinterpret_cast<const uint4*>(k + (int64_t)row * k_stride * ELT);
  const uint4* vr = reinterpret_cast<const uint4*>(v + (int64_t)row * v_stride * ELT);
  uint4 x[kAhead];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int i = i0 + e * 32 + lane;
      if (i < all) x[e] = __ldg(i < half ? kr + i : vr + i - half);
    }
  };
  fetch(0);
  PagedSeq s;
  const int b = find_row(pv, ba, row, s);
  if (s.T == 0) return;                        // nobody's row
  const int a = s.L - s.T + row - s.row0;
  const int page = ba.table[(size_t)b * ba.max_pages + (a >> pv.log2P)];
  if ((unsigned)page >= (unsigned)pv.pages) {
    if (lane == 0) flag_error(pv.err, kErrBadBatch);
    return;
  }
  const size_t at = (size_t)page * pv.Hkv * pv.P + (a & (pv.P - 1));   // of head 0
  uint4* K = static_cast<uint4*>(pv.K);
  uint4* V = static_cast<uint4*>(pv.V);
  for (int i0 = 0; i0 < all; i0 += kAhead * 32) {
    if (i0 > 0) fetch(i0);
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int i = i0 + e * 32 + lane;
      if (i >= all) break;
      const int y = i < half ? i : i - half;
      (i < half ? K : V)[(at + (size_t)(y / nv) * pv.P) * nv + y % nv] = x[e];
    }
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagesView& pv, const BatchArgs& ba, const void* k,
                                int64_t k_stride, const void* v, int64_t v_stride,
                                cudaStream_t s) {
  const dim3 grid((unsigned)(((int64_t)ba.rows + kRowsPerCta - 1) / kRowsPerCta));
  return launch_dependent(pv.dtype == RSWA_F32 ? paged_append_kernel<4> : paged_append_kernel<2>,
                          grid, dim3(kRowsPerCta * 32), 0, s, pv, ba,
                          static_cast<const char*>(k), k_stride, static_cast<const char*>(v),
                          v_stride);
}

}  // namespace rswa
