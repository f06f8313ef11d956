// Attention weights that the cached tokens receive from a chunk:
//   w[b][kvh][j] = decay * w[b][kvh][j] + sum over the chunk's rows i and the G
//   query heads h of the KV head of exp(q_ih . k_j / sqrt(d) - lse_ih), j seen by i.
//
// CUDA-core form.  A CTA takes kKeys tokens of one (sequence, KV head): a lane
// group holds a few of its keys in registers and goes over all rows that may see
// one of them, so that a token's sum is made in one place, in the order of the
// rows, without atomics.  For float32 with few rows and for groups of more than 64
// heads: bound by a lane group's chain of row reads (float32, one sequence of a row of
// 10 heads over 512 keys 3.0 us, tiles of 64 x 64 7.8; 8 of 64 rows 118 and 32).
#include <algorithm>

#include "attend.cuh"
#include "paged.cuh"

namespace rswa {
namespace {

constexpr int kWarps = 8, kU = 2;

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
paged_weigh_kernel(PagesView pv, BatchArgs ba, const T* __restrict__ q, int64_t q_stride,
                   const float* __restrict__ lse, float* __restrict__ weights, float decay) {
  using C = AttendCfg<T, D, kU>;
  constexpr int EPL = C::EPL, LPK = C::LPK, KPW = C::KPW;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = lane / LPK, col = (lane % LPK) * EPL;
  const int G = pv.G, n = ba.window;
  const float sl2 = rsqrtf((float)D) * kLog2e;
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t bh = blockIdx.y; bh < (int64_t)ba.B * pv.Hkv; bh += gridDim.y) {
    const int b = (int)(bh / pv.Hkv), kvh = (int)(bh % pv.Hkv);
    PagedSeq s;
    s.load(pv, ba, b);
    const int t0 = ((int)blockIdx.x * kWarps + warp) * C::KEYS_WARP;   // the warp's first token
    if (t0 >= s.L) continue;
    const int t1 = min(t0 + C::KEYS_WARP, s.L);
    const int tok0 = s.L - s.T;
    float* w = weights + bh * ba.cap;
    // The rows that may see one of the tokens: of tokens a >= t0, and, where none
    // of them is in the prefix, a < t1 - 1 + n.
    const int i0 = max(t0 - tok0, 0);
    const int i1 = t0 < s.m ? s.T : (int)min((int64_t)s.T, (int64_t)t1 - 1 + n - tok0);
    float kf[kU][EPL], sum[kU];
    int t[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      t[u] = t0 + u * KPW + grp;
      sum[u] = 0.f;
      // of the tokens only those that a row sees are read
      const Hull hull(tok0 + i0, tok0 + max(i1, i0 + 1) - 1, s.m, n);
      if (i0 < i1 && t[u] < t1 && hull.has(t[u])) {
        const size_t at = (((size_t)page_at(pv, ba, b, t[u] >> pv.log2P) * pv.Hkv + kvh) * pv.P +
                           (t[u] & (pv.P - 1))) * D + col;
        Elt<T>::widen(ld_stream16(static_cast<const T*>(pv.K) + at), kf[u]);
      } else {
#pragma unroll
        for (int e = 0; e < EPL; ++e) kf[u][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < EPL; ++e) kf[u][e] *= sl2;
    }
    for (int i = i0; i < i1; ++i) {
      const int a = tok0 + i;
      const T* qr = q + (int64_t)(s.row0 + i) * q_stride + (int64_t)kvh * G * D + col;
      const float* lr = lse + (int64_t)(s.row0 + i) * pv.H + (int64_t)kvh * G;
      for (int g = 0; g < G; ++g) {
        float qf[EPL];
        Elt<T>::widen(__ldg(reinterpret_cast<const uint4*>(qr + (int64_t)g * D)), qf);
        const float l2 = __ldg(lr + g) * kLog2e;
        float x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          x[u] = 0.f;
#pragma unroll
          for (int e = 0; e < EPL; ++e) x[u] = fmaf(qf[e], kf[u][e], x[u]);
        }
#pragma unroll
        for (int off = LPK / 2; off > 0; off >>= 1)
#pragma unroll
          for (int u = 0; u < kU; ++u) x[u] += __shfl_xor_sync(0xffffffffu, x[u], off);
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (t[u] <= a && (t[u] < s.m || t[u] > a - n)) sum[u] += fast_exp2(x[u] - l2);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (lane % LPK == 0 && t[u] < t1)
        w[t[u]] = decay == 0.f ? sum[u] : fmaf(decay, w[t[u]], sum[u]);
  }
}

template <typename T, int D>
cudaError_t launch_d(const PagesView& pv, const BatchArgs& ba, const void* q, int64_t q_stride,
                     const float* lse, float* weights, float decay, cudaStream_t s) {
  constexpr int keys = kWarps * AttendCfg<T, D, kU>::KEYS_WARP;
  const dim3 grid((unsigned)((ba.cap + keys - 1) / keys),
                  (unsigned)std::min<int64_t>((int64_t)ba.B * pv.Hkv, 65535));
  return launch_dependent(paged_weigh_kernel<T, D>, grid, dim3(kWarps * 32), 0, s, pv, ba,
                          static_cast<const T*>(q), q_stride, lse, weights, decay);
}

}  // namespace

cudaError_t launch_paged_weigh(const PagesView& pv, const PagesMaps& maps, const BatchArgs& ba,
                               const void* q, int64_t q_stride, const float* lse, float* weights,
                               float decay, cudaStream_t s) {
  if (paged_weigh_tc_supported(pv))
    return launch_paged_weigh_tc(pv, maps, ba, q, q_stride, lse, weights, decay, s);
  // float32 with 16 rows (token, head of the group) of a sequence and more: in tiles of
  // 64 (us here / in tiles at 512 keys: 8 sequences of 10 heads and 8 rows 22.4/28.1, 16
  // rows 36.3/28.5; 64 of 32 / 8 heads and 2 rows 113/146, 4 rows 182/148).
  if (paged_f32_supported(pv, ba) && (int64_t)ba.rows * pv.G >= 16 * (int64_t)ba.B)
    return launch_paged_weigh_f32(pv, ba, q, q_stride, lse, weights, decay, s);
  if (pv.dtype == RSWA_F32)
    return pv.d == 64 ? launch_d<float, 64>(pv, ba, q, q_stride, lse, weights, decay, s)
                      : launch_d<float, 128>(pv, ba, q, q_stride, lse, weights, decay, s);
  return pv.d == 64 ? launch_d<__nv_bfloat16, 64>(pv, ba, q, q_stride, lse, weights, decay, s)
                    : launch_d<__nv_bfloat16, 128>(pv, ba, q, q_stride, lse, weights, decay, s);
}

}  // namespace rswa
