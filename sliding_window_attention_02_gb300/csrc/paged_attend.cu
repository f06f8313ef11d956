// Attention of a chunk of tokens over a paged cache, on the CUDA cores: float32
// caches, groups too large for the tensor cores' tiles, and small work, where
// latency counts.
//
//   o = sum_j exp(s_j - lse) v_j,  s_j = q . k_j / sqrt(d),  lse = log sum_j exp(s_j)
// over the tokens j that the row's token sees (paged.cuh).
//
// A unit is up to R rows (token, query head of the group) of one KV head: every
// key and value is loaded once for all of them.  Its keys, packed, are cut into
// tiles that the launch's CTAs share evenly (PagedPlan); the eight warps of a CTA
// take turns on a tile's keys, each lane group with its own running maximum, sum
// and output (online softmax), merged at the end of the unit's part.  Units cut
// over several CTAs leave partials, which the last of the CTAs merges in the
// order of the CTAs, so that a result does not depend on who is last.
#include <algorithm>

#include "attend.cuh"
#include "paged.cuh"

namespace rswa {
namespace {

constexpr int kWarps = 8;
constexpr int kTile = 128;                     // keys

using Plan = PagedPlan<kTile, false, 0, 1>;

constexpr int kMaxPeers = 8;                   // CTAs of a cluster

// Folds U keys of this lane's group (its slices kr, vr of their rows) into the states
// of R query rows.  sees(r, i): whether row r sees key i; a value row that none sees
// has to be finite all the same.
template <typename T, int D, int R, int U, typename F>
__device__ __forceinline__ void fold_keys(const float (&qf)[R][AttendCfg<T, D>::EPL],
                                          const uint4* kr, const uint4* vr, F sees,
                                          SoftmaxState<AttendCfg<T, D>::EPL>* st) {
  constexpr int EPL = AttendCfg<T, D>::EPL, LPK = AttendCfg<T, D>::LPK;
  float s[R][U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float kf[EPL];
    Elt<T>::widen(kr[i], kf);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) x = fmaf(qf[r][e], kf[e], x);
      s[r][i] = x;
    }
  }
#pragma unroll
  for (int off = LPK / 2; off > 0; off >>= 1)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < U; ++i) s[r][i] += __shfl_xor_sync(0xffffffffu, s[r][i], off);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float mx = st[r].m;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (!sees(r, i)) s[r][i] = -INFINITY;
      mx = fmaxf(mx, s[r][i]);
    }
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float alpha = fast_exp2(st[r].m - ref);
    st[r].l *= alpha;
#pragma unroll
    for (int e = 0; e < EPL; ++e) st[r].acc[e] *= alpha;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      s[r][i] = fast_exp2(s[r][i] - ref);
      st[r].l += s[r][i];
    }
    st[r].m = mx;
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float vf[EPL];
    Elt<T>::widen(vr[i], vf);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < EPL; ++e) st[r].acc[e] = fmaf(s[r][i], vf[e], st[r].acc[e]);
  }
}

// A warp's states, its lane groups merged, to shared memory; and a row's column over
// all warps of the CTA.
template <typename T, int D, int R>
__device__ __forceinline__ void publish_warp(SoftmaxState<AttendCfg<T, D>::EPL>* st, int lane,
                                             int warp, float (*s_m)[R], float (*s_l)[R],
                                             float (*s_acc)[R][D]) {
  constexpr int EPL = AttendCfg<T, D>::EPL, LPK = AttendCfg<T, D>::LPK;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    merge_groups<T, D>(st[r]);
    if (lane < LPK) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) s_acc[warp][r][lane * EPL + e] = st[r].acc[e];
      if (lane == 0) {
        s_m[warp][r] = st[r].m;
        s_l[warp][r] = st[r].l;
      }
    }
  }
}
template <int R, int D>
__device__ __forceinline__ void merge_warps(const float (*s_m)[R], const float (*s_l)[R],
                                            const float (*s_acc)[R][D], int r, int c, float& M,
                                            float& L, float& A) {
  M = -INFINITY;
  L = A = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
  const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float sc = fast_exp2(s_m[w][r] - ref);
    L += s_l[w][r] * sc;
    A += s_acc[w][r][c] * sc;
  }
}

// A store to another CTA's shared memory (a cluster address).
__device__ __forceinline__ void store_peer(uint32_t to, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(kWarps * 32)
paged_attend_kernel(PagesView pv, BatchArgs ba, AttendArgs a) {
  constexpr int U = R == 1 ? 8 : 4;
  using C = AttendCfg<T, D, U>;
  constexpr int EPL = C::EPL, LPK = C::LPK, KPW = C::KPW;
  __shared__ PagedUnit s_unit;
  __shared__ int s_more, s_last;
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  __shared__ float s_acc[kWarps][R][D];
  __shared__ float s_M[R], s_L[R];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = lane / LPK, col = (lane % LPK) * EPL;
  const int cta = blockIdx.x, G = pv.G;
  const float sl2 = rsqrtf((float)D) * kLog2e;
  griddep_wait();
  griddep_launch_dependents();
  Plan plan(pv, ba, R);
  if (warp == 0) {
    const bool more = plan.start(cta, gridDim.x);
    if (lane == 0) {
      s_more = more;
      if (more) s_unit = plan.u;
    }
  }
  __syncthreads();
  while (s_more) {
    const PagedUnit& u = s_unit;
    const int rows = min(R, u.seq.T * G - u.f0);
    const int b = u.b, kvh = u.kvh, m = u.seq.m, n = ba.window;
    const int tok0 = u.seq.L - u.seq.T;
    const Hull hull = u.hull;
    const int x0 = u.j0 * kTile, x1 = min(u.j1 * kTile, hull.keys());
    const int skip = hull.w0 - hull.p;
    // Rows of q and o: row f of the unit is query head kvh * G + f % G of chunk
    // row f / G.
    auto row_of = [&](int r, int& head) {
      const int f = u.f0 + r;
      head = kvh * G + f % G;
      return u.seq.row0 + f / G;
    };
    float qf[R][EPL];
    int tok[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      int head;
      const int64_t row = row_of(min(r, rows - 1), head);
      tok[r] = tok0 + (u.f0 + min(r, rows - 1)) / G;
      Elt<T>::widen(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) +
                                                    row * a.q_stride + (int64_t)head * D + col),
                    qf[r]);
#pragma unroll
      for (int e = 0; e < EPL; ++e) qf[r][e] *= sl2;
    }
    SoftmaxState<EPL> st[R];
#pragma unroll
    for (int r = 0; r < R; ++r) st[r].init();
    bool bad = false;                          // a page outside the pool
    for (int base = x0 + warp * C::KEYS_WARP; base < x1; base += kWarps * C::KEYS_WARP) {
      uint4 kr[U], vr[U];
      int t[U], page[U];
      // the pages first, then the rows: reads that do not wait for one another
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int x = base + i * KPW + grp;
        const int y = x < x1 ? x : x0;         // any key of the part
        t[i] = y < hull.p ? y : y + skip;
        page[i] = ba.table[(size_t)b * ba.max_pages + (t[i] >> pv.log2P)];
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        bad |= (unsigned)page[i] >= (unsigned)pv.pages;
        if ((unsigned)page[i] >= (unsigned)pv.pages) page[i] = 0;
        const size_t at = (((size_t)page[i] * pv.Hkv + kvh) * pv.P + (t[i] & (pv.P - 1))) * D + col;
        kr[i] = ld_stream16(static_cast<const T*>(pv.K) + at);
        vr[i] = ld_stream16(static_cast<const T*>(pv.V) + at);
        if (base + i * KPW + grp >= x1) t[i] = INT32_MAX;        // not a key: after every token
      }
      fold_keys<T, D, R, U>(
          qf, kr, vr,
          [&](int r, int i) { return t[i] <= tok[r] && (t[i] < m || t[i] > tok[r] - n); }, st);
    }
    publish_warp<T, D, R>(st, lane, warp, s_m, s_l, s_acc);
    if (bad) flag_error(pv.err, kErrBadBatch);
    __syncthreads();
    // The CTA's result of row r, column c: over the warps.
    const size_t pf = (size_t)R * (D + 2);
    float* part = paged_partial(a.ws, cta, u.first, pf);
    const bool whole = u.whole();
    for (int i = threadIdx.x; i < rows * D; i += kWarps * 32) {
      const int r = i / D, c = i % D;
      float M, L, A;
      merge_warps<R, D>(s_m, s_l, s_acc, r, c, M, L, A);
      if (whole) {
        int head;
        const int64_t row = row_of(r, head), oi = row * pv.H + head;
        static_cast<T*>(a.o)[oi * D + c] = (T)(A / L);   // a token sees itself: L > 0
        if (c == 0 && a.lse) a.lse[oi] = (M + log2f(L)) * kLn2;
      } else {
        part[i] = A;
        if (c == 0) {
          part[R * D + r] = M;
          part[R * D + R + r] = L;
        }
      }
    }
    if (!whole) {
      __syncthreads();
      if (threadIdx.x == 0) {
        int32_t* count = paged_counter(a.ws, u.first);
        s_last = arrive_acq_rel(count) == u.last - u.first;
        if (s_last) *count = 0;                // ready for the next call
      }
      __syncthreads();
      if (s_last) {
        for (int r = warp; r < rows; r += kWarps) {
          float M = -INFINITY;
          for (int p = u.first + lane; p <= u.last; p += 32)
            M = fmaxf(M, __ldcg(paged_partial(a.ws, p, u.first, pf) + R * D + r));
          M = warp_max(M);
          float L = 0.f;
          for (int p = u.first + lane; p <= u.last; p += 32) {
            const float* P = paged_partial(a.ws, p, u.first, pf) + R * D + r;
            L += __ldcg(P + R) * fast_exp2(__ldcg(P) - M);
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
          if (lane == 0) {
            s_M[r] = M;
            s_L[r] = L;
          }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * D; i += kWarps * 32) {
          const int r = i / D, c = i % D;
          const float M = s_M[r], L = s_L[r];
          float A = 0.f;
#pragma unroll 4
          for (int p = u.first; p <= u.last; ++p) {
            const float* P = paged_partial(a.ws, p, u.first, pf);
            A = fmaf(__ldcg(P + i), fast_exp2(__ldcg(P + R * D + r) - M), A);
          }
          int head;
          const int64_t row = row_of(r, head), oi = row * pv.H + head;
          static_cast<T*>(a.o)[oi * D + c] = (T)(A / L);
          if (c == 0 && a.lse) a.lse[oi] = (M + log2f(L)) * kLn2;
        }
      }
    }
    __syncthreads();
    if (warp == 0) {
      const bool more = plan.next();
      if (lane == 0) {
        s_more = more;
        if (more) s_unit = plan.u;
      }
    }
    __syncthreads();
  }
}

// Small work, where latency counts: no list and no plan.  A cluster of CTAs takes R
// query heads of one chunk row and KV head; its CTAs share the row's keys evenly and
// hand their parts to the first through distributed shared memory.  What a call waits
// for is a chain of reads (the row's sequence, its pages, the rows) and the join.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kWarps * 32)
paged_attend_small_kernel(PagesView pv, BatchArgs ba, AttendArgs a) {
  constexpr int U = R <= 2 ? 8 : 4;
  using C = AttendCfg<T, D, U>;
  constexpr int EPL = C::EPL, LPK = C::LPK, KPW = C::KPW;
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  __shared__ float s_acc[kWarps][R][D];
  __shared__ float s_part[kMaxPeers][R][D + 2];          // the first CTA's: everyone's parts
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = lane / LPK, col = (lane % LPK) * EPL;
  const int peers = (int)cluster_size(), rank = (int)cluster_rank();
  const int G = pv.G, groups = (G + R - 1) / R, n = ba.window;
  const float sl2 = rsqrtf((float)D) * kLog2e;
  if (peers > 1) cluster_arrive_relaxed();     // waited for before the first remote store
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.x / peers;
  const int h0 = unit % groups * R, heads = min(R, G - h0);
  const int kvh = unit / groups % pv.Hkv, row = unit / groups / pv.Hkv;
  float qf[R][EPL];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    Elt<T>::widen(*reinterpret_cast<const uint4*>(
                      static_cast<const T*>(a.q) + (int64_t)row * a.q_stride +
                      (int64_t)(kvh * G + h0 + min(r, heads - 1)) * D + col),
                  qf[r]);
#pragma unroll
    for (int e = 0; e < EPL; ++e) qf[r][e] *= sl2;
  }
  // The row's sequence.  Of 32 sequences, every lane reads one: where their rows end
  // and what the one that is found needs, in one go.
  PagedSeq s;
  s.row0 = s.T = s.L = s.m = 0;
  int b = 0;
  if (ba.starts) {
    for (int b0 = 0; b0 < ba.B; b0 += 32) {
      PagedSeq mine;
      mine.row0 = mine.T = mine.L = mine.m = 0;
      const int x = b0 + lane;
      if (x < ba.B) mine.load(pv, ba, x);
      const uint32_t on =
          __ballot_sync(0xffffffffu, row >= mine.row0 && row < mine.row0 + mine.T);
      if (!on) continue;
      const int src = __ffs(on) - 1;
      b = b0 + src;
      s.row0 = __shfl_sync(0xffffffffu, mine.row0, src);
      s.T = __shfl_sync(0xffffffffu, mine.T, src);
      s.L = __shfl_sync(0xffffffffu, mine.L, src);
      s.m = __shfl_sync(0xffffffffu, mine.m, src);
      break;
    }
  } else {
    b = row / ba.each;
    s.load(pv, ba, b);
  }
  if (s.T == 0) return;                        // nobody's row; as do all of the cluster
  const int tok = s.L - s.T + row - s.row0, m = s.m;
  const Hull hull(tok, tok, m, n);
  const int nk = hull.keys(), skip = hull.w0 - hull.p;
  const int x0 = (int)((int64_t)nk * rank / peers), x1 = (int)((int64_t)nk * (rank + 1) / peers);
  SoftmaxState<EPL> st[R];
#pragma unroll
  for (int r = 0; r < R; ++r) st[r].init();
  bool bad = false;                            // a page outside the pool
  for (int base = x0 + warp * C::KEYS_WARP; base < x1; base += kWarps * C::KEYS_WARP) {
    uint4 kr[U], vr[U];
    int t[U], page[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int y = min(base + i * KPW + grp, x1 - 1);
      t[i] = y < hull.p ? y : y + skip;
      page[i] = ba.table[(size_t)b * ba.max_pages + (t[i] >> pv.log2P)];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      bad |= (unsigned)page[i] >= (unsigned)pv.pages;
      if ((unsigned)page[i] >= (unsigned)pv.pages) page[i] = 0;
      const size_t at = (((size_t)page[i] * pv.Hkv + kvh) * pv.P + (t[i] & (pv.P - 1))) * D + col;
      kr[i] = ld_stream16(static_cast<const T*>(pv.K) + at);
      vr[i] = ld_stream16(static_cast<const T*>(pv.V) + at);
    }
    fold_keys<T, D, R, U>(qf, kr, vr, [&](int, int i) { return base + i * KPW + grp < x1; }, st);
  }
  if (bad) flag_error(pv.err, kErrBadBatch);
  publish_warp<T, D, R>(st, lane, warp, s_m, s_l, s_acc);
  if (peers > 1) cluster_wait();               // the first CTA runs
  __syncthreads();
  const int64_t orow = (int64_t)row * pv.H + kvh * G + h0;
  for (int i = threadIdx.x; i < heads * D; i += kWarps * 32) {
    const int r = i / D, c = i % D;
    float M, L, A;
    merge_warps<R, D>(s_m, s_l, s_acc, r, c, M, L, A);
    if (peers == 1) {
      static_cast<T*>(a.o)[(orow + r) * D + c] = (T)(A / L);     // it sees itself: L > 0
      if (c == 0 && a.lse) a.lse[orow + r] = (M + log2f(L)) * kLn2;
    } else {
      float* to = &s_part[rank][r][0];
      store_peer(map_dsmem(to + 2 + c, 0), A);
      if (c == 0) {
        store_peer(map_dsmem(to, 0), M);
        store_peer(map_dsmem(to + 1, 0), L);
      }
    }
  }
  if (peers == 1) return;
  cluster_arrive_release();
  cluster_wait();
  if (rank != 0) return;
  for (int i = threadIdx.x; i < heads * D; i += kWarps * 32) {
    const int r = i / D, c = i % D;
    float M = -INFINITY, L = 0.f, A = 0.f;
    for (int p = 0; p < peers; ++p) M = fmaxf(M, s_part[p][r][0]);
    for (int p = 0; p < peers; ++p) {
      const float sc = fast_exp2(s_part[p][r][0] - M);
      L = fmaf(s_part[p][r][1], sc, L);
      A = fmaf(s_part[p][r][2 + c], sc, A);
    }
    static_cast<T*>(a.o)[(orow + r) * D + c] = (T)(A / L);
    if (c == 0 && a.lse) a.lse[orow + r] = (M + log2f(L)) * kLn2;
  }
}

int grid_of(const PagesView& pv) { return std::min(2 * std::max(pv.sms, 1), kMaxPagedCtas); }

template <typename T, int D>
cudaError_t launch_d(const PagesView& pv, const BatchArgs& ba, const AttendArgs& a,
                     cudaStream_t s) {
  const bool one = (int64_t)ba.rows * pv.G <= ba.B;      // one row to a unit
  return launch_dependent(one ? paged_attend_kernel<T, D, 1> : paged_attend_kernel<T, D, 4>,
                          dim3(grid_of(pv)), dim3(kWarps * 32), 0, s, pv, ba, a);
}

}  // namespace

// How a call is served.
enum class Path { kSmall, kCudaCores, kFewRows, kTiles };
// Query heads that a CTA of the small kernel takes, and the CTAs of a launch without
// sharing keys.
static int small_heads(const PagesView& pv) { return pv.G >= 3 ? 4 : pv.G; }
static int64_t small_units(const PagesView& pv, int64_t rows) {
  const int r = small_heads(pv);
  return rows * pv.Hkv * ((pv.G + r - 1) / r);
}
static Path path_of(const PagesView& pv, int64_t rows, int64_t batch, int64_t keys) {
  // SMALL
  if (small_units(pv, rows) <= 2 * pv.sms && keys <= 2048) return Path::kSmall;
  if (!paged_attend_tc_supported(pv)) return Path::kCudaCores;
  if (rows * pv.G <= 16 * batch) return Path::kFewRows;
  return Path::kTiles;
}

template <typename T, int D>
static cudaError_t launch_small_d(const PagesView& pv, const BatchArgs& ba, const AttendArgs& a,
                                  cudaStream_t s) {
  const int64_t units = small_units(pv, ba.rows);
  // CTAs that share a row's keys: as many as fill the SMs, with 64 keys each at least
  int peers = 1;
  while (peers < kMaxPeers && units * peers * 2 <= 2 * (int64_t)pv.sms && ba.cap >= 128 * peers)
    peers *= 2;
  const int r = small_heads(pv);
  auto kern = r == 1   ? paged_attend_small_kernel<T, D, 1>
              : r == 2 ? paged_attend_small_kernel<T, D, 2>
                       : paged_attend_small_kernel<T, D, 4>;
  return launch_dependent_cluster(kern, dim3((unsigned)(units * peers)), dim3(kWarps * 32), 0, s,
                                  peers, pv, ba, a);
}

size_t paged_attend_workspace(const PagesView& pv, int64_t rows, int batch) {
  size_t need = kPagedCounterBytes + (size_t)grid_of(pv) * 2 * 4 * (pv.d + 2) * sizeof(float);
  if (paged_attend_tc_supported(pv)) {
    need = std::max(need, paged_decode_tc_workspace(pv));
    if (rows * pv.G > 16 * (int64_t)batch) need = std::max(need, paged_attend_tc_workspace(pv));
  }
  return need;
}

cudaError_t launch_paged_attend(const PagesView& pv, const PagesMaps& maps, const BatchArgs& ba,
                                const AttendArgs& a, cudaStream_t s) {
  switch (path_of(pv, ba.rows, ba.B, ba.cap)) {
    case Path::kSmall:
      if (pv.dtype == RSWA_F32)
        return pv.d == 64 ? launch_small_d<float, 64>(pv, ba, a, s)
                          : launch_small_d<float, 128>(pv, ba, a, s);
      return pv.d == 64 ? launch_small_d<__nv_bfloat16, 64>(pv, ba, a, s)
                        : launch_small_d<__nv_bfloat16, 128>(pv, ba, a, s);
    case Path::kTiles: return launch_paged_attend_tc(pv, maps, ba, a, s);
    case Path::kFewRows: return launch_paged_decode_tc(pv, maps, ba, a, s);
    default: break;
  }
  if (pv.dtype == RSWA_F32)
    return pv.d == 64 ? launch_d<float, 64>(pv, ba, a, s) : launch_d<float, 128>(pv, ba, a, s);
  return pv.d == 64 ? launch_d<__nv_bfloat16, 64>(pv, ba, a, s)
                    : launch_d<__nv_bfloat16, 128>(pv, ba, a, s);
}

}  // namespace rswa
