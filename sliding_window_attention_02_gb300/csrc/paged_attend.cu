// Attention of a chunk of tokens over a paged cache, on the CUDA cores: small work,
// where latency counts, float32 caches, and groups too large for the tensor cores'
// tiles.
//
//   o = sum_j exp(s_j - lse) v_j,  s_j = q . k_j / sqrt(d),  lse = log sum_j exp(s_j)
// over the tokens j that the row's token sees (paged.cuh).
//
// No list and no plan: a cluster of CTAs takes R query heads of one chunk row and KV
// head.  Its CTAs share the row's keys evenly, the eight warps of a CTA take turns on
// them, each lane group with its own running maximum, sum and output (online softmax);
// they are merged in shared memory, and the CTAs hand their parts to the first through
// distributed shared memory.  What a small call waits for is a chain of reads (the
// row's sequence, its pages, the rows) and the join; beyond some 50000 pairs of a query
// row and a key it is bound by those, as every CTA reads its keys through L2 for itself.
// Measured: one token of 10 heads over 488 (288 in the prefix) 4.25 us in a graph, 5.3 a
// call; float32, 3 sequences of 4 / 2 heads, d 64, up to 90 rows of 700 tokens, 6.4 (below:
// the rule between the paths, with all three measured).
#include <algorithm>

#include "attend.cuh"
#include "paged.cuh"

namespace rswa {
namespace {

constexpr int kWarps = 8;

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
  PagedSeq s;
  const int b = find_row(pv, ba, row, s);
  if (ba.starts && blockIdx.x == 0)            // wrong descriptions behind it are told too
    for (int x = 32 + threadIdx.x; x < ba.B; x += kWarps * 32) {
      PagedSeq other;
      other.load(pv, ba, x);
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

}  // namespace

// Query heads that a CTA of the CUDA-core kernel takes, and its launch's CTAs before any
// share keys.
static int core_heads(const PagesView& pv) { return pv.G >= 3 ? 4 : pv.G; }
static int64_t core_units(const PagesView& pv, int64_t rows) {
  const int r = core_heads(pv);
  return rows * pv.Hkv * ((pv.G + r - 1) / r);
}

// How a call is served.  The host knows the rows and what the tables can hold, not the
// lengths.  us on the CUDA cores / in units of few rows / of tiles; bf16, d 128:
//   sequences, rows each, heads   keys 512          2048             8192
//    1   1   10                   4.3/9.7/11.2      6.0/10.4/18.7    17.2/14.5/28.8
//    1   4   10                   5.8/10.5/11.5     11.7/11.5/18.3   36.3/16.0/27.3
//    1  16   10                   11.1/12.8/11.8    35.0/15.0/18.3   127/21.6/27.0
//    1   1   32 / 8               5.5/10.4/11.3     9.2/11.3/18.0    23.1/15.2/27.0
//    1   8   32 / 8               9.2/12.9/11.7     23.3/15.6/17.2   76.4/24.1/25.4
//    8   1   32 / 8               9.2/11.5/12.0     30.3/18.8/22.5   112/47.6/61.8
//    8   4   32 / 8               24.2/14.5/12.5    101/25.6/22.7    402/67.8/62.4
//   16  16   10 (512, 1024, 4096) 86/20/20          161/34/27        582/105/71
//   64   1   10                   37.2/33.2/50.5    131/104/130
//   64   4   10                   93/34.8/52.2      317/105/132
//   64  16   10                   332/64.9/52.9     1126/202/134
//   64   1   32 / 8               62.7/31.5/45.0    223/87/108
// The CUDA cores' CTAs have at most so many keys, and all of them so many elements of
// keys, before the tensor cores are ahead; units of few rows read a sequence's keys
// again for every 8 rows, which costs little while all units have CTAs at once.  Over 300
// shapes the path taken is at worst 1.45 times the best one (1 sequence of 4 rows of 16 /
// 2 heads over 4096 keys: 23.2/15.9/18.5).
constexpr int64_t kCoreKeys = 6144, kCoreWork = 10 << 20, kFewRows = 8, kFewUnits = 40;
enum class Path { kCudaCores, kFewRows, kTiles };
static bool few_rows(const PagesView& pv, int64_t rows, int64_t batch) {
  return rows * pv.G <= kFewRows * batch ||
         (rows * pv.G + kFewRows - 1) / kFewRows * pv.Hkv <= kFewUnits;
}
static Path path_of(const PagesView& pv, int64_t rows, int64_t batch, int64_t keys) {
  if (!paged_attend_tc_supported(pv)) return Path::kCudaCores;
  const int64_t units = core_units(pv, rows);
  if (keys <= kCoreKeys && units <= 2 * pv.sms && units * keys * pv.d <= kCoreWork)
    return Path::kCudaCores;
  return few_rows(pv, rows, batch) ? Path::kFewRows : Path::kTiles;
}

template <typename T, int D>
static cudaError_t launch_cores_d(const PagesView& pv, const BatchArgs& ba, const AttendArgs& a,
                                  cudaStream_t s) {
  const int r = core_heads(pv);
  const int64_t units = core_units(pv, ba.rows);
  // CTAs that share a row's keys: as many as are on the SMs together (registers allow
  // two an SM, one with four heads; clusters of 8 do not fill the groups of SMs that
  // they have to lie in: 16 of them, one CTA an SM, take two turns), with 64 keys each
  // at least.
  const int64_t room = (r == 4 ? 1 : 2) * (int64_t)pv.sms;
  int peers = 1;
  while (peers < kMaxPeers && units * peers * 2 <= (peers == 4 ? room * 5 / 8 : room) &&
         ba.cap >= 128 * peers)
    peers *= 2;
  auto kern = r == 1   ? paged_attend_kernel<T, D, 1>
              : r == 2 ? paged_attend_kernel<T, D, 2>
                       : paged_attend_kernel<T, D, 4>;
  return launch_dependent_cluster(kern, dim3((unsigned)(units * peers)), dim3(kWarps * 32), 0, s,
                                  peers, pv, ba, a);
}

// float32 with many rows: tiles of 64 rows, which read keys once for all of them, take
// 0.145 us a key (d 64: 0.083) and turn of CTAs, one an SM (d 64: two); the kernel above
// 90 ps for a pair of row and key (d 64: 45), 55 (26) where four heads share keys.  us
// here / in tiles at 512 keys: 1 sequence of 64 rows of 10 heads 40.6/75.7, of 256 106/75.6,
// 8 of 16 rows 69.5/74.6, of 64 246/75.9, 64 of 8 286/369, of 16 552/370; of 32 / 8
// heads 1 of 64 rows 66/75.7, 8 of 16 127/75.9.
static bool f32_tiles(const PagesView& pv, const BatchArgs& ba) {
  const int64_t rows = ba.rows, room = (pv.d == 64 ? 2 : 1) * (int64_t)pv.sms;
  const int64_t units = std::max((rows * pv.G + 63) / 64, (int64_t)ba.B) * pv.Hkv;
  return rows * pv.H > (pv.G >= 3 ? 2900 : 1700) * ((units + room - 1) / room);
}

size_t paged_attend_workspace(const PagesView& pv, int64_t rows) {
  if (!paged_attend_tc_supported(pv)) return 256;
  // whatever the number of sequences: more rows never need less
  const size_t need = paged_decode_tc_workspace(pv);
  return few_rows(pv, rows, 0) ? need : std::max(need, paged_attend_tc_workspace(pv));
}

cudaError_t launch_paged_attend(const PagesView& pv, const PagesMaps& maps, const BatchArgs& ba,
                                const AttendArgs& a, cudaStream_t s) {
  switch (path_of(pv, ba.rows, ba.B, ba.cap)) {
    case Path::kTiles: return launch_paged_attend_tc(pv, maps, ba, a, s);
    case Path::kFewRows: return launch_paged_decode_tc(pv, maps, ba, a, s);
    default: break;
  }
  if (paged_f32_supported(pv, ba) && f32_tiles(pv, ba)) return launch_paged_attend_f32(pv, ba, a, s);
  if (pv.dtype == RSWA_F32)
    return pv.d == 64 ? launch_cores_d<float, 64>(pv, ba, a, s)
                      : launch_cores_d<float, 128>(pv, ba, a, s);
  return pv.d == 64 ? launch_cores_d<__nv_bfloat16, 64>(pv, ba, a, s)
                    : launch_cores_d<__nv_bfloat16, 128>(pv, ba, a, s);
}

}  // namespace rswa
