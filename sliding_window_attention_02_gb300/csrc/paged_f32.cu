// float32 paged caches with many rows, on the CUDA cores: attention of a chunk, and the
// weights that cached tokens receive from it, in tiles of 64 query rows (token, head
// of the group) x 64 keys.
//
// The tensor cores have no product of float32's precision, so the bound is the FMA
// rate.  A thread computes 4 x 4 logits from shared memory (8 reads of 16 bytes for 64
// FMAs) and 4 rows x d / 16 columns of the output (d 128: 12 reads for 128 FMAs);
// copies of the next tile run meanwhile (cp.async, two stages).  Rows of 16 threads
// share a query row, so that its softmax statistics and its weights stay within half
// a warp.  Measured: 8 sequences of 256 rows of 10 heads over 512 keys, attention 179 us
// and weights 83; with keys read for every row 800 and 367.
#include <algorithm>

#include "paged.cuh"

namespace rswa {
namespace {

constexpr int BM = 64, BN = 64, kThreads = 256;

// 16 bytes from global to shared memory, or as many zero bytes.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool on) {
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows of shared memory: padded by 16 bytes, so that 16 of them are read without
// conflicts.
template <int D>
struct Tile {
  static constexpr int kRow = D + 4, kFloats = 64 * kRow;
};

// 64 keys (or values) from token x0 on, of those in the hull; the others become zero,
// as they may be any bits.
template <int D>
__device__ __forceinline__ bool load_tokens(const PagesView& pv, const BatchArgs& ba, int b,
                                            int kvh, const Hull& hull, int x0, const float* K,
                                            const float* V, float* sk, float* sv) {
  constexpr int kLanes = D / 4, kPass = kThreads / kLanes;         // threads of a row, rows at once
  const int r0 = threadIdx.x / kLanes, c = threadIdx.x % kLanes * 4;
  bool bad = false;
  int page[64 / kPass];
#pragma unroll
  for (int i = 0; i < 64 / kPass; ++i) {
    const int t = x0 + r0 + i * kPass;
    page[i] = hull.has(t) ? ba.table[(size_t)b * ba.max_pages + (t >> pv.log2P)] : -1;
    bad |= hull.has(t) && (unsigned)page[i] >= (unsigned)pv.pages;
  }
#pragma unroll
  for (int i = 0; i < 64 / kPass; ++i) {
    const int r = r0 + i * kPass, t = x0 + r;
    const bool on = (unsigned)page[i] < (unsigned)pv.pages;
    const size_t at =
        (((size_t)(on ? page[i] : 0) * pv.Hkv + kvh) * pv.P + (t & (pv.P - 1))) * D + c;
    copy16(sk + r * Tile<D>::kRow + c, K + at, on);
    if (V) copy16(sv + r * Tile<D>::kRow + c, V + at, on);
  }
  return bad;
}

// 64 query rows from row f0 of the sequence's on (row f: token f / G of the chunk, head
// f % G of the group); rows past the chunk become zero.
template <int D>
__device__ __forceinline__ void load_queries(const PagesView& pv, const PagedSeq& s, int kvh,
                                             int f0, const float* q, int64_t q_stride, float* sq) {
  constexpr int kLanes = D / 4, kPass = kThreads / kLanes;
  const int r0 = threadIdx.x / kLanes, c = threadIdx.x % kLanes * 4;
#pragma unroll
  for (int i = 0; i < 64 / kPass; ++i) {
    const int r = r0 + i * kPass, f = f0 + r;
    const bool on = f < s.T * pv.G;
    const int64_t row = s.row0 + (on ? f / pv.G : 0);
    copy16(sq + r * Tile<D>::kRow + c,
           q + row * q_stride + (int64_t)(kvh * pv.G + (on ? f % pv.G : 0)) * D + c, on);
  }
}

// x[i][j] = row ty + 16 i of a times row tx + 16 j of b.
template <int D>
__device__ __forceinline__ void products(const float* a, const float* b, int ty, int tx,
                                         float (&x)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
#pragma unroll 4
  for (int k = 0; k < D; k += 4) {
    float4 u[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = *reinterpret_cast<const float4*>(a + (ty + 16 * i) * Tile<D>::kRow + k);
      v[i] = *reinterpret_cast<const float4*>(b + (tx + 16 * i) * Tile<D>::kRow + k);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[i][j] = fmaf(u[i].x, v[j].x, x[i][j]);
        x[i][j] = fmaf(u[i].y, v[j].y, x[i][j]);
        x[i][j] = fmaf(u[i].z, v[j].z, x[i][j]);
        x[i][j] = fmaf(u[i].w, v[j].w, x[i][j]);
      }
  }
}

template <int D>
constexpr size_t attend_smem() {
  return (5 * Tile<D>::kFloats + BM * (BN + 4)) * sizeof(float);   // Q, 2 x (K, V), P
}

// CTA: 64 rows of one (sequence, KV head), all of their keys.  blockIdx.x / Hkv counts
// the blocks of 64 rows of all sequences, and as many as there are sequences more that
// may be nobody's.
template <int D>
__global__ void __launch_bounds__(kThreads)
paged_attend_f32_kernel(PagesView pv, BatchArgs ba, AttendArgs a) {
  extern __shared__ float4 smem4[];
  float* sq = reinterpret_cast<float*>(smem4);
  float* sk = sq + Tile<D>::kFloats;                     // two stages
  float* sv = sk + 2 * Tile<D>::kFloats;
  float* sp = sv + 2 * Tile<D>::kFloats;                 // [64][68]
  constexpr int kPRow = BN + 4, NC = D / 64;
  const int tid = threadIdx.x, lane = tid & 31, ty = tid >> 4, tx = tid & 15;
  const int G = pv.G, n = ba.window;
  const float sl2 = rsqrtf((float)D) * kLog2e;
  griddep_wait();
  griddep_launch_dependents();
  const int kvh = blockIdx.x % pv.Hkv;
  int block = blockIdx.x / pv.Hkv;
  PagedSeq s;
  s.T = 0;
  int b = 0;
  for (int b0 = 0; b0 < ba.B; b0 += 32) {                // every warp looks for itself
    PagedSeq mine;
    mine.row0 = mine.T = mine.L = mine.m = 0;
    if (b0 + lane < ba.B) mine.load(pv, ba, b0 + lane);
    int inc = (mine.T * G + BM - 1) / BM;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += y;
    }
    const int src = __popc(__ballot_sync(0xffffffffu, inc <= block));
    if (src == 32) {
      block -= __shfl_sync(0xffffffffu, inc, 31);
      continue;
    }
    b = b0 + src;
    s.row0 = __shfl_sync(0xffffffffu, mine.row0, src);
    s.T = __shfl_sync(0xffffffffu, mine.T, src);
    s.L = __shfl_sync(0xffffffffu, mine.L, src);
    s.m = __shfl_sync(0xffffffffu, mine.m, src);
    if (src > 0) block -= __shfl_sync(0xffffffffu, inc, src - 1);
    break;
  }
  if (s.T == 0) return;
  const int f0 = block * BM, f1 = min(f0 + BM, s.T * G) - 1, tok0 = s.L - s.T;
  const Hull hull(tok0 + f0 / G, tok0 + f1 / G, s.m, n);
  const HullTiles<BN> tiles(hull);
  const float* K = static_cast<const float*>(pv.K);
  const float* V = static_cast<const float*>(pv.V);
  auto token_of = [&](int j) { return (j < tiles.np ? j : tiles.kb + (j - tiles.np)) * BN; };
  load_queries<D>(pv, s, kvh, f0, static_cast<const float*>(a.q), a.q_stride, sq);
  bool bad = load_tokens<D>(pv, ba, b, kvh, hull, token_of(0), K, V, sk, sv);
  copies_commit();
  int tok[4];
  float m_run[4], l_run[4], acc[4][4 * NC];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    tok[i] = tok0 + min(f0 + ty + 16 * i, f1) / G;
    m_run[i] = -INFINITY;
    l_run[i] = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * NC; ++c) acc[i][c] = 0.f;
  }
  for (int j = 0; j < tiles.nt; ++j) {
    const int st = j & 1;
    if (j + 1 < tiles.nt)
      bad |= load_tokens<D>(pv, ba, b, kvh, hull, token_of(j + 1), K, V,
                            sk + (st ^ 1) * Tile<D>::kFloats, sv + (st ^ 1) * Tile<D>::kFloats);
    copies_commit();
    copies_wait<1>();                                    // this tile's
    __syncthreads();
    float x[4][4];
    products<D>(sq, sk + st * Tile<D>::kFloats, ty, tx, x);
    const int x0 = token_of(j);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = m_run[i];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int t = x0 + tx + 16 * c;
        const bool sees = t <= tok[i] && (t < s.m || t > tok[i] - n);
        x[i][c] = sees ? x[i][c] * sl2 : -INFINITY;
        mx = fmaxf(mx, x[i][c]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float alpha = fast_exp2(m_run[i] - ref);
      m_run[i] = mx;
      l_run[i] *= alpha;
#pragma unroll
      for (int c = 0; c < 4 * NC; ++c) acc[i][c] *= alpha;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = fast_exp2(x[i][c] - ref);
        l_run[i] += p;
        sp[(ty + 16 * i) * kPRow + tx + 16 * c] = p;
      }
    }
    __syncwarp();                                        // a row's weights are its half warp's
    const float* v = sv + st * Tile<D>::kFloats + tx * 4;
#pragma unroll 4
    for (int k = 0; k < BN; k += 4) {
      float4 p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p[i] = *reinterpret_cast<const float4*>(sp + (ty + 16 * i) * kPRow + k);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float4 w = *reinterpret_cast<const float4*>(v + (k + e) * Tile<D>::kRow + 64 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float pe = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
            acc[i][4 * c] = fmaf(pe, w.x, acc[i][4 * c]);
            acc[i][4 * c + 1] = fmaf(pe, w.y, acc[i][4 * c + 1]);
            acc[i][4 * c + 2] = fmaf(pe, w.z, acc[i][4 * c + 2]);
            acc[i][4 * c + 3] = fmaf(pe, w.w, acc[i][4 * c + 3]);
          }
        }
    }
    __syncthreads();                                     // the stage may be filled again
  }
  if (bad) flag_error(pv.err, kErrBadBatch);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float l = l_run[i];
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    const int f = f0 + ty + 16 * i;
    if (f > f1) continue;
    const float inv = 1.f / l;                           // a token sees itself: l > 0
    const int64_t row = (int64_t)(s.row0 + f / G) * pv.H + kvh * G + f % G;
    float* o = static_cast<float*>(a.o) + row * D + tx * 4;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      *reinterpret_cast<float4*>(o + 64 * c) =
          make_float4(acc[i][4 * c] * inv, acc[i][4 * c + 1] * inv, acc[i][4 * c + 2] * inv,
                      acc[i][4 * c + 3] * inv);
    if (tx == 0 && a.lse) a.lse[row] = (m_run[i] + log2f(l)) * kLn2;
  }
}

template <int D>
constexpr size_t weigh_smem() {
  return (3 * Tile<D>::kFloats + 2 * BM + 16 * BN) * sizeof(float);   // K, 2 x Q, 2 x lse, sums
}

// CTA: 64 keys of one (sequence, KV head), all rows that see one of them.
template <int D>
__global__ void __launch_bounds__(kThreads)
paged_weigh_f32_kernel(PagesView pv, BatchArgs ba, const float* __restrict__ q, int64_t q_stride,
                       const float* __restrict__ lse, float* __restrict__ weights, float decay) {
  extern __shared__ float4 smem4[];
  float* sk = reinterpret_cast<float*>(smem4);
  float* sq = sk + Tile<D>::kFloats;                     // two stages
  float* sl = sq + 2 * Tile<D>::kFloats;                 // [2][64]
  float* sum = sl + 2 * BM;                              // [16][64]
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int G = pv.G, n = ba.window;
  const float sl2 = rsqrtf((float)D) * kLog2e;
  griddep_wait();
  griddep_launch_dependents();
  const int x0 = (int)blockIdx.x * BN;
  for (int64_t bh = blockIdx.y; bh < (int64_t)ba.B * pv.Hkv; bh += gridDim.y) {
    const int b = (int)(bh / pv.Hkv), kvh = (int)(bh % pv.Hkv);
    PagedSeq s;
    s.load(pv, ba, b);
    if (x0 >= s.L) continue;
    const int tok0 = s.L - s.T;
    // Tokens that may see one of the keys: a >= x0, and, where none of them is in the
    // prefix, a < x0 + 63 + n; the rows (token, head) of those, in whole blocks.
    const int i0 = max(x0 - tok0, 0);
    const int i1 = x0 < s.m ? s.T : (int)min((int64_t)s.T, (int64_t)x0 + BN - 1 + n - tok0);
    const int lo = i0 * G, hi = max(i1, i0) * G;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    bool bad = false;
    if (lo < hi) {
      const Hull hull(tok0 + i0, tok0 + i1 - 1, s.m, n);
      bad = load_tokens<D>(pv, ba, b, kvh, hull, x0, static_cast<const float*>(pv.K), nullptr, sk,
                           nullptr);
    }
    auto fetch = [&](int f0, int st) {
      load_queries<D>(pv, s, kvh, f0, q, q_stride, sq + st * Tile<D>::kFloats);
      const int f = f0 + tid;
      if (tid < BM)
        sl[st * BM + tid] =
            f < hi ? lse[(int64_t)(s.row0 + f / G) * pv.H + kvh * G + f % G] * kLog2e : 0.f;
    };
    if (lo < hi) fetch(lo, 0);
    copies_commit();
    for (int f0 = lo, st = 0; f0 < hi; f0 += BM, st ^= 1) {
      if (f0 + BM < hi) fetch(f0 + BM, st ^ 1);
      copies_commit();
      copies_wait<1>();
      __syncthreads();
      float x[4][4];
      products<D>(sq + st * Tile<D>::kFloats, sk, ty, tx, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int f = f0 + ty + 16 * i, a = tok0 + f / G;
        const float l = sl[st * BM + ty + 16 * i];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int t = x0 + tx + 16 * c;
          const bool sees = f < hi && t <= a && (t < s.m || t > a - n);
          if (sees) acc[c] += fast_exp2(fmaf(x[i][c], sl2, -l));
        }
      }
      __syncthreads();
    }
    if (bad) flag_error(pv.err, kErrBadBatch);
#pragma unroll
    for (int c = 0; c < 4; ++c) sum[ty * BN + tx + 16 * c] = acc[c];
    __syncthreads();
    if (tid < BN && x0 + tid < s.L) {
      float w = 0.f;
#pragma unroll
      for (int y = 0; y < 16; ++y) w += sum[y * BN + tid];
      float* to = weights + bh * ba.cap + x0 + tid;
      *to = decay == 0.f ? w : fmaf(decay, *to, w);
    }
    __syncthreads();
  }
}

template <int D>
cudaError_t launch_attend(const PagesView& pv, const BatchArgs& ba, const AttendArgs& a,
                          cudaStream_t s) {
  // Per device (the attribute belongs to the current device's context).
  cudaError_t e = cudaFuncSetAttribute(paged_attend_f32_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       attend_smem<D>());
  if (e != cudaSuccess) return e;
  const int64_t blocks = ((int64_t)ba.rows * pv.G + BM - 1) / BM + ba.B;
  return launch_dependent(paged_attend_f32_kernel<D>, dim3((unsigned)(blocks * pv.Hkv)),
                          dim3(kThreads), attend_smem<D>(), s, pv, ba, a);
}

template <int D>
cudaError_t launch_weigh(const PagesView& pv, const BatchArgs& ba, const void* q, int64_t q_stride,
                         const float* lse, float* weights, float decay, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(paged_weigh_f32_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       weigh_smem<D>());
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((ba.cap + BN - 1) / BN),
                  (unsigned)std::min<int64_t>((int64_t)ba.B * pv.Hkv, 65535));
  return launch_dependent(paged_weigh_f32_kernel<D>, grid, dim3(kThreads), weigh_smem<D>(), s, pv,
                          ba, static_cast<const float*>(q), q_stride, lse, weights, decay);
}

}  // namespace

bool paged_f32_supported(const PagesView& pv, const BatchArgs& ba) {
  return pv.dtype == RSWA_F32 &&
         (((int64_t)ba.rows * pv.G + BM - 1) / BM + ba.B) * pv.Hkv < (int64_t(1) << 31);
}

cudaError_t launch_paged_attend_f32(const PagesView& pv, const BatchArgs& ba, const AttendArgs& a,
                                    cudaStream_t s) {
  return pv.d == 64 ? launch_attend<64>(pv, ba, a, s) : launch_attend<128>(pv, ba, a, s);
}

cudaError_t launch_paged_weigh_f32(const PagesView& pv, const BatchArgs& ba, const void* q,
                                   int64_t q_stride, const float* lse, float* weights, float decay,
                                   cudaStream_t s) {
  return pv.d == 64 ? launch_weigh<64>(pv, ba, q, q_stride, lse, weights, decay, s)
                    : launch_weigh<128>(pv, ba, q, q_stride, lse, weights, decay, s);
}

}  // namespace rswa
