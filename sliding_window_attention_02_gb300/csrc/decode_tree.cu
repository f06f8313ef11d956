// R-SWA attention for a tree of drafted tokens per sequence (the cache is only
// read), and the append of the tree's accepted path.
//
// Node i has depth(i) = 0 when its parent is -1, else depth(parent) + 1, and
// stands for output t_b + depth(i).  It attends to
//   the prefix          keys 0..m_b-1
//   cached outputs      j in [max(0, t_b + depth - n + 1), t_b), slot j mod n
//   the tree            itself and its ancestors fewer than n levels above
// which is N(t) = P U D_n(t) of the "Unlimited-OCR deep dive" (R-SWA
// pseudo-code block) along the chain that ends in the node.
#include <algorithm>

#include "attend.cuh"
#include "rswa_device.cuh"

namespace rswa {
namespace {

constexpr int kTreeWarps = 8;

// Live nodes of sequence b; a count outside 0..nodes is flagged and clamped.
__device__ __forceinline__ int live_nodes(const int32_t* counts, int b, int nodes,
                                          int32_t* err) {
  if (!counts) return nodes;
  const int c = counts[b];
  if (c < 0 || c > nodes) flag_error(err, kErrBadTree);
  return min(max(c, 0), nodes);
}

// One CTA of 8 warps per (node, query head, sequence): the warps split every
// key segment between them and merge in shared memory.  A node past the
// sequence's count is left alone.  Bound by latency for a few nodes, a chain of
// reads, merge and store: the walk to the root runs in one lane while the warps
// are at the prefix, whose first rows are requested before the dependency wait
// where the preceding kernel of the stream writes no prefix row (PREFETCH, the
// handle's flag).  Beyond some 50000 pairs of a query row and a key bound by
// those: every CTA reads all keys of its row through L2 for itself, with no reuse
// between nodes or heads, bf16 71 ps a pair at d 128 and 57 at d 64, float32 78 and
// 47, 4.5 to 7 TFLOP/s.  In deep trees by the walk, a load a level.
// 16 nodes of 10 heads over 288 + 128 keys, bf16: 7.8 us (34 MB through L2),
// 0.34 by the 2.3 MB of data.
template <typename T, int D, bool PREFETCH>
__global__ void __launch_bounds__(kTreeWarps * 32)
decode_tree_kernel(CacheView cv, TreeArgs a) {
  using C = AttendCfg<T, D>;
  constexpr int NW = kTreeWarps;
  __shared__ int s_anc[kMaxTreeNodes];         // the node, then its ancestors
  __shared__ int s_len, s_depth;
  __shared__ float s_m[NW], s_l[NW];
  __shared__ float s_acc[NW][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.z * gridDim.y + blockIdx.y;
  if (b >= cv.B) return;
  const int i = blockIdx.x / cv.H, h = blockIdx.x % cv.H;
  const int kvh = h / (cv.H / cv.Hkv);
  const size_t bkv = (size_t)b * cv.Hkv + kvh;
  const T* Kb = static_cast<const T*>(cv.K) + bkv * cv.slab_rows * D;
  const T* Vb = static_cast<const T*>(cv.V) + bkv * cv.slab_rows * D;
  const int64_t first = (int64_t)warp * C::KEYS_WARP, step = (int64_t)NW * C::KEYS_WARP;
  int64_t m_b = 0;
  AttendBatch<T, D> pre;
  bool have_pre = false;
  if (PREFETCH) {
    m_b = cv.m_dev[b];
    if (first < m_b) {
      attend_load<T, D>(Kb, Vb, D, first, 0, m_b, -1, nullptr, nullptr, lane, INT64_MAX, 0,
                        pre);
      have_pre = true;
    }
  }
  griddep_wait();
  griddep_launch_dependents();
  if (!PREFETCH) m_b = cv.m_dev[b];
  const int64_t t_b = cv.t_dev[(size_t)b * cv.H + h];
  const int64_t n = cv.n;
  const size_t qrow = ((size_t)b * a.nodes + i) * cv.H + h;
  if (i >= live_nodes(a.counts, b, a.nodes, cv.err)) return;
  float qf[C::EPL];
  load_q_frag<T, D>(static_cast<const T*>(a.q) + qrow * D, lane, qf);
  if (threadIdx.x == (NW - 1) * 32) {
    // Parents come before their children, so the walk ends; a parent that
    // does not is flagged and taken as none.
    const int32_t* par = a.parents + (size_t)b * a.nodes;
    int len = 0, depth = 0;
    for (int x = i;;) {
      if (len < n) s_anc[len++] = x;
      const int p = par[x];
      if (p < -1 || p >= x) flag_error(cv.err, kErrBadTree);
      if (p < 0 || p >= x) break;
      x = p;
      ++depth;
    }
    s_len = len;
    s_depth = depth;
  }
  __syncwarp();
  SoftmaxState<C::EPL> st;
  st.init();
  if (have_pre) attend_consume<T, D>(qf, pre, st);
  attend_range<T, D>(qf, Kb, Vb, D, 0, m_b, have_pre ? first + step : first, step, -1, nullptr,
                     nullptr, lane, st);
  __syncthreads();
  const int len = s_len;
  const int64_t j_lo = max((int64_t)0, t_b + s_depth - n + 1);
  if (j_lo < t_b) {
    const T* Kr = Kb + cv.m_cap * D;
    const T* Vr = Vb + cv.m_cap * D;
    const int64_t s0 = j_lo % n, cnt = t_b - j_lo;
    attend_range<T, D>(qf, Kr, Vr, D, s0, min(n, s0 + cnt), first, step, -1, nullptr,
                       nullptr, lane, st);
    if (s0 + cnt > n)
      attend_range<T, D>(qf, Kr, Vr, D, 0, s0 + cnt - n, first, step, -1, nullptr, nullptr,
                         lane, st);
  }
  const T* Kt = static_cast<const T*>(a.k) + ((size_t)b * a.nodes * cv.Hkv + kvh) * D;
  const T* Vt = static_cast<const T*>(a.v) + ((size_t)b * a.nodes * cv.Hkv + kvh) * D;
  const int grp = lane / C::LPK, col = (lane % C::LPK) * C::EPL;
  for (int base = warp * C::KPW; base < len; base += NW * C::KPW) {
    AttendBatch<T, D, 1> bt;
    bt.ok[0] = base + grp < len;
    const size_t row = (size_t)s_anc[bt.ok[0] ? base + grp : 0] * cv.Hkv * D;
    bt.k[0] = ld_stream16(Kt + row + col);
    bt.v[0] = ld_stream16(Vt + row + col);
    attend_consume<T, D, 1>(qf, bt, st);
  }
  merge_groups<T, D>(st);
  if (lane < C::LPK) {
#pragma unroll
    for (int e = 0; e < C::EPL; ++e) s_acc[warp][lane * C::EPL + e] = st.acc[e];
    if (lane == 0) {
      s_m[warp] = st.m;
      s_l[warp] = st.l;
    }
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float M = -INFINITY, L = 0.f, A = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w]);
    const float ref = (M == -INFINITY) ? 0.f : M;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float sc = fast_exp2(s_m[w] - ref);
      L += s_l[w] * sc;
      A += s_acc[w][threadIdx.x] * sc;
    }
    static_cast<T*>(a.o)[qrow * D + threadIdx.x] = (T)(A / L);   // self is visible: L > 0
    if (threadIdx.x == 0 && a.lse) a.lse[qrow] = (ref + log2f(L)) * kLn2;
  }
}

// One CTA per KV head of a sequence: the accepted nodes' keys and values go to
// their ring slots, then the group's copies of t_b advance.  Every CTA of a
// sequence checks its whole path and comes to the same answer, so a bad one
// changes nothing.  Bound by latency (t_b and the path, then the rows): one
// sequence of 10 KV heads 2.0 us, 64 of 8 with paths of 0 to 9 nodes 3.3.
template <typename T>
__global__ void __launch_bounds__(128)
commit_tree_kernel(CacheView cv, const T* k, const T* v, int nodes, const int32_t* path,
                   const int32_t* accepted, int max_path) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / cv.Hkv, kvh = blockIdx.x % cv.Hkv;
  const int per_kv = cv.H / cv.Hkv;
  int64_t* t_dev = cv.t_dev + (size_t)b * cv.H + (size_t)kvh * per_kv;
  const int64_t t_b = t_dev[0], n = cv.n;
  const int acc = accepted[b];
  const int32_t* pb = path + (size_t)b * max_path;
  bool bad = acc < 0 || acc > max_path;
  for (int i = threadIdx.x; i < acc && !bad; i += blockDim.x)
    bad = pb[i] < 0 || pb[i] >= nodes;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) flag_error(cv.err, kErrBadTree);
    return;
  }
  const int nv = cv.d * (int)sizeof(T) / 16;            // 16-byte vectors of a row
  const size_t slab = ((size_t)b * cv.Hkv + kvh) * cv.slab_rows + cv.m_cap;
  const int i0 = (int)max((int64_t)0, acc - n);         // earlier ones would be evicted
  for (int x = threadIdx.x; x < (acc - i0) * 2 * nv; x += blockDim.x) {
    const int i = i0 + x / (2 * nv), isv = x / nv & 1, vi = x % nv;
    const T* in = (isv ? v : k) + (((size_t)b * nodes + pb[i]) * cv.Hkv + kvh) * cv.d;
    T* out = static_cast<T*>(isv ? cv.V : cv.K) + (slab + (size_t)((t_b + i) % n)) * cv.d;
    reinterpret_cast<uint4*>(out)[vi] = reinterpret_cast<const uint4*>(in)[vi];
  }
  for (int h = threadIdx.x; h < per_kv; h += blockDim.x) t_dev[h] = t_b + acc;
}

template <typename T, int D>
cudaError_t launch_tree_t(const CacheView& cv, const TreeArgs& a, bool prefetch,
                          cudaStream_t s) {
  const unsigned y = (unsigned)std::min(cv.B, 65535);          // the grid's limit
  return launch_dependent(prefetch ? decode_tree_kernel<T, D, true>
                                   : decode_tree_kernel<T, D, false>,
                          dim3((unsigned)a.nodes * cv.H, y, (unsigned)(cv.B + y - 1) / y),
                          dim3(kTreeWarps * 32), 0, s, cv, a);
}

}  // namespace

// Small work is done sooner on the CUDA cores, whose kernel takes the larger of
// 2.1 us and 7 ns a key (d 64: 2.4 and 3.4 ns) and, once its CTAs fill the SMs, of
// 2.7 us and 71 ps for each pair of a query row and a key (d 64: 2.2 and 57 ps);
// the tensor-core kernel takes 7 us and 1 for a tile of 128 keys while its units
// are few, 13.5 and more where it cuts them, and 3 more for every further unit of
// an SM.  One sequence, bf16, us on the CUDA / tensor cores, d 128 and then d 64,
// at 192 keys (m 64, n 128), 416 and 1184:
//   heads   nodes       192                      416                     1184
//   10        1                         5.0/10.2, 3.9/9.2     10.4/14.7, 6.5/13.0
//   10       16   4.8/7.8, 3.7/7.6      7.0/9.9, 4.7/9.0      16.0/14.2, 8.9/12.6
//   10       32   8.0/8.0, 6.7/8.0     11.2/10.1, 8.3/9.1
//   32 / 8    4   3.7/7.9, 3.3/7.3      5.3/10.2, 4.2/9.2     10.7/14.6, 6.8/12.7
//   32 / 8   16   8.8/7.8, 6.9/7.6     13.9/10.0, 9.1/9.0
//   16 / 2   16   4.9/8.4, 3.9/8.0      7.2/10.6, 4.7/9.5
//   16 / 2   32   9.2/12.6, 7.4/11.4   14.0/15.6, 9.4/13.9
//   40        4   4.6/8.2, 3.7/7.7      7.1/10.6, 4.7/9.6     15.9/17.1, 8.9/14.9
// and 10 heads, d 128: 1 node 34/16 at 4256; 51 sequences of at most 120 keys, 1
// node 7.7/24.6.  At d 64, and with few KV heads, the CUDA cores stay ahead to
// twice the pairs and more; the bound is that of 10 heads at d 128.  The keys are
// the cache's capacity: the host does not know the live ones.
constexpr int64_t kCudaCorePairs = 110000, kCudaCoreKeys = 1200;

static bool small_work(const CacheView& cv, int nodes) {
  const int64_t keys = cv.m_cap + cv.n;
  return keys <= kCudaCoreKeys && (int64_t)cv.B * cv.H * nodes * keys <= kCudaCorePairs;
}

bool decode_tree_use_tc(const CacheView& cv, int nodes) {
  return !small_work(cv, nodes) && decode_tree_tc_supported(cv, nodes);
}

size_t decode_tree_workspace(const CacheView& cv, int nodes) {
  // For any count of nodes that may come, not only those the kernel takes: a
  // workspace for more nodes serves fewer.
  if (small_work(cv, nodes) || cv.dtype != RSWA_BF16 || cv.H / cv.Hkv > 128) return 256;
  return decode_tree_tc_workspace(cv, nodes);
}

cudaError_t launch_decode_tree(const CacheView& cv, const TreeArgs& a, const SlabMaps* maps,
                               bool prefetch, cudaStream_t s) {
  if (decode_tree_use_tc(cv, a.nodes)) return launch_decode_tree_tc(cv, a, *maps, s);
  if (cv.dtype == RSWA_F32)
    return cv.d == 64 ? launch_tree_t<float, 64>(cv, a, prefetch, s)
                      : launch_tree_t<float, 128>(cv, a, prefetch, s);
  return cv.d == 64 ? launch_tree_t<__nv_bfloat16, 64>(cv, a, prefetch, s)
                    : launch_tree_t<__nv_bfloat16, 128>(cv, a, prefetch, s);
}

cudaError_t launch_commit_tree(const CacheView& cv, const void* k, const void* v, int nodes,
                               const int32_t* path, const int32_t* accepted, int max_path,
                               cudaStream_t s) {
  if ((int64_t)cv.B * cv.Hkv > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(cv.B * cv.Hkv));
  if (cv.dtype == RSWA_F32)
    return launch_dependent(commit_tree_kernel<float>, grid, dim3(128), 0, s, cv,
                            (const float*)k, (const float*)v, nodes, path, accepted, max_path);
  return launch_dependent(commit_tree_kernel<__nv_bfloat16>, grid, dim3(128), 0, s, cv,
                          (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, nodes, path,
                          accepted, max_path);
}

}  // namespace rswa
