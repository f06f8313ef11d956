// Eviction from a paged cache: of every (sequence, KV head) the first tokens, the
// last ones and the heaviest of the others stay, up to a budget, in their order.
//
// Two kernels.  The first, a CTA or a cluster of them for each (sequence, KV head),
// finds the least weight that stays: the weights as integers of the same order, a
// radix select of at most four passes over 8 bits each, in shared memory where they
// fit.  Ties of that weight stay from the lowest index on.  Counts of what stays give
// each kept token its place; the weights follow.  The second moves the rows, 64 of them a
// CTA, every read of it in flight at once.
//
// In place a row's place is at or before where it comes from, so a CTA's writes
// may meet only what CTAs of lower rows of the same head read: CTAs take their rows
// in ticket order, read them into registers, say so, and write once the lower ones
// whose reads reach its rows have said so too.  No CTA waits before it has read, so
// the wait ends whatever CTAs run at a time.
#include <algorithm>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace rswa {
namespace {

constexpr int kSelectThreads = 512, kWarps = kSelectThreads / 32;
constexpr int kMoveRows = 64, kMoveThreads = 128;
constexpr uint64_t kWaitLimitNs = 1000000000ull;
// Weights of a CTA's slice that are kept in shared memory between the passes.
constexpr int kSelectSmem = 40 * 1024;

// A float as an unsigned integer of the same order; both zeros alike, NaN lowest.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Tokens of sequence b; a length outside its range is flagged and taken as 0.
__device__ __forceinline__ int length_of(const PagesView& pv, const BatchArgs& ba, int b) {
  const int L = ba.lens[b];
  if (L >= 0 && L <= ba.cap) return L;
  flag_error(pv.err, kErrBadBatch);
  return 0;
}

// The workspace: a ticket, a flag for every CTA of the move, and the kept tokens
// where the caller wants none.
__device__ __forceinline__ int32_t* move_flags(void* ws) { return static_cast<int32_t*>(ws) + 64; }

// Copies of the histogram, by lane: weights share few exponents, and the lanes of a
// warp that add to one word take turns.
constexpr int kCopies = 8;
constexpr int kAhead = 4;                                // weights of a thread in flight

// A word of CTA `rank`'s shared memory at this CTA's address p.
__device__ __forceinline__ uint32_t peer_word(const void* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_dsmem(p, (uint32_t)rank))
               : "memory");
  return v;
}

// A cluster of gridDim-given size for each (sequence, KV head), whose CTAs take a
// slice of its tokens each and add up their counts in one another's shared memory.
// Bound by instruction issue and by the passes' barriers: what is read is small.
template <bool SMEM>
__global__ void __launch_bounds__(kSelectThreads)
evict_select_kernel(PagesView pv, BatchArgs ba, EvictArgs a, int chunks) {
  extern __shared__ float s_w[];                         // the slice's weights
  __shared__ uint32_t s_hist[2][256 * kCopies];
  __shared__ uint32_t s_total[2][256];                   // the slice's counts of a pass
  __shared__ uint32_t s_sum[256];                        // all slices'
  __shared__ uint32_t s_prefix, s_need, s_whole;
  __shared__ int s_warp[2][kWarps], s_slice[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int peers = (int)cluster_size(), rank = (int)cluster_rank();
  griddep_wait();
  griddep_launch_dependents();
  const int64_t bh = blockIdx.x / peers;
  const int b = (int)(bh / pv.Hkv);
  const float* w = a.weights + bh * ba.cap;
  float* wo = a.weights_out + bh * ba.cap;
  int32_t* kept = a.kept + bh * a.budget;
  const int all_tid = rank * kSelectThreads + tid, all_threads = peers * kSelectThreads;
  if (a.in_place) {
    if (blockIdx.x == 0 && tid == 0) *static_cast<int32_t*>(a.ws) = 0;
    for (int i = all_tid; i < chunks; i += all_threads) move_flags(a.ws)[bh * chunks + i] = 0;
  }
  const int L = length_of(pv, ba, b);
  if (L <= a.budget) {
    for (int i = all_tid; i < a.budget; i += all_threads) kept[i] = i < L ? i : -1;
    for (int i = all_tid; i < ba.cap; i += all_threads) {
      if (i >= L)
        wo[i] = 0.f;
      else if (wo != w)
        wo[i] = w[i];
    }
    return;                                              // as do all of the cluster
  }
  auto meet = [&]() {
    if (peers > 1) {
      cluster_arrive_release();
      cluster_wait();
    } else {
      __syncthreads();
    }
  };
  const int lo = a.first, hi = L - a.last;               // the tokens that are weighed
  // the CTA's tokens, and its warps' of them: whole rounds of 32
  const int span = (L + 32 * kWarps * peers - 1) / (32 * kWarps * peers) * 32;
  const int t0 = min(rank * kWarps * span, L), t1 = min(t0 + kWarps * span, L);
  if (SMEM)
    for (int j0 = t0 + tid; j0 < t1; j0 += kAhead * kSelectThreads) {
      float x[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        if (j0 + e * kSelectThreads < t1) x[e] = w[j0 + e * kSelectThreads];
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        if (j0 + e * kSelectThreads < t1) s_w[j0 - t0 + e * kSelectThreads] = x[e];
    }
  const float* from = SMEM ? s_w - t0 : w;
  for (int i = tid; i < 256 * kCopies; i += kSelectThreads) s_hist[0][i] = 0;
  if (tid == 0) {
    s_prefix = 0;
    s_need = (uint32_t)(a.budget - a.first - a.last);
  }
  __syncthreads();
  // Tokens with a key above `least` stay, and the first `ties` with that key.
  uint32_t least = 0xffffffffu;                          // no weight has this key
  int ties = 0;
  if (s_need > 0) {
    for (int pass = 0;; ++pass) {
      const int shift = 24 - 8 * pass;
      const uint32_t prefix = s_prefix, need = s_need;
      uint32_t* hist = s_hist[pass & 1] + (lane & (kCopies - 1));
#pragma unroll 4
      for (int j = max(t0, lo) + tid; j < min(t1, hi); j += kSelectThreads) {
        const uint32_t x = order_key(from[j]);
        if (pass == 0 || (x ^ prefix) >> (shift + 8) == 0)
          atomicAdd(hist + (x >> shift & 255u) * kCopies, 1u);
      }
      for (int i = tid; i < 256 * kCopies; i += kSelectThreads) s_hist[~pass & 1][i] = 0;
      __syncthreads();
      uint32_t* total = s_total[pass & 1];
      if (tid < 256) {
        const uint4* h = reinterpret_cast<const uint4*>(s_hist[pass & 1] + tid * kCopies);
        const uint4 p = h[0], q = h[1];
        total[tid] = ((p.x + p.y) + (p.z + p.w)) + ((q.x + q.y) + (q.z + q.w));
      }
      meet();
      // two passes on, a slice's counts are written again: all have read them by then,
      // as they meet once more in between
      if (tid < 256) {
        uint32_t c[8];                                   // reads on their way together
#pragma unroll
        for (int p = 0; p < 8; ++p)
          c[p] = p >= peers ? 0u : peers > 1 ? peer_word(total + tid, p) : total[tid];
        s_sum[tid] = ((c[0] + c[1]) + (c[2] + c[3])) + ((c[4] + c[5]) + (c[6] + c[7]));
      }
      __syncthreads();
      if (warp == 0) {
        // the digit in which the needed one falls, from the highest down: lane l
        // has digits 255 - 8 l ... 248 - 8 l
        uint32_t c[8], mine = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) mine += c[e] = s_sum[255 - 8 * lane - e];
        uint32_t inc = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, inc, off);
          if (lane >= off) inc += y;
        }
        uint32_t above = inc - mine;
        if (above < need && need <= inc) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (above < need && need <= above + c[e]) {
              s_prefix = prefix | (uint32_t)(255 - 8 * lane - e) << shift;
              s_need = need - above;
              s_whole = need - above == c[e];
            }
            above += c[e];
          }
        }
      }
      __syncthreads();
      // Every weight with these digits stays: the lower ones need not be known.
      if (s_whole && s_prefix != 0) {
        least = s_prefix - 1;
        break;
      }
      if (pass == 3) {
        least = s_prefix;
        ties = (int)s_need;
        break;
      }
    }
  }
  // What stays, in order: a warp looks through a range of tokens, 32 at a time, once
  // for its count and once, behind the counts of the warps before it, for the places.
  const int j0 = min(t0 + warp * span, t1), j1 = min(j0 + span, t1);
  auto look = [&](int j, uint32_t& stays, uint32_t& equal) {
    const bool in = j < j1, end = in && (j < lo || j >= hi);
    const uint32_t x = in ? order_key(from[j]) : 0u;
    stays = __ballot_sync(0xffffffffu, end || (in && x > least));
    equal = __ballot_sync(0xffffffffu, in && !end && x == least);
  };
  int na = 0, ne = 0;
#pragma unroll 4
  for (int j = j0; j < j1; j += 32) {
    uint32_t stays, equal;
    look(j + lane, stays, equal);
    na += __popc(stays);
    ne += __popc(equal);
  }
  if (lane == 0) {
    s_warp[0][warp] = na;
    s_warp[1][warp] = ne;
  }
  __syncthreads();
  if (warp < 2) {
    const int sum = __reduce_add_sync(0xffffffffu, lane < kWarps ? s_warp[warp][lane] : 0);
    if (lane == 0) s_slice[warp] = sum;
  }
  meet();
  {
    int wa = lane < warp ? s_warp[0][lane] : 0, we = lane < warp ? s_warp[1][lane] : 0;
    if (lane < rank) {                                   // at most 8 ranks
      wa += (int)peer_word(&s_slice[0], lane);
      we += (int)peer_word(&s_slice[1], lane);
    }
    na = __reduce_add_sync(0xffffffffu, wa);
    ne = __reduce_add_sync(0xffffffffu, we);
  }
  const uint32_t before = (1u << lane) - 1u;
#pragma unroll 4
  for (int j = j0; j < j1; j += 32) {
    uint32_t stays, equal;
    look(j + lane, stays, equal);
    const int e = ne + __popc(equal & before);           // equals before this token
    if (stays >> lane & 1u || (equal >> lane & 1u && e < ties)) {
      const int at = na + __popc(stays & before) + min(e, ties);
      kept[at] = j + lane;
      // in place too: every slice has been read by now
      if (SMEM) wo[at] = s_w[j + lane - t0];
    }
    na += __popc(stays);
    ne += __popc(equal);
  }
  meet();                                                // peers' counts have been read
  // The weights of a long sequence, by one CTA.  In place too: a batch is read before
  // it is written, and a later batch comes from behind what an earlier one writes.
  if (!SMEM && rank == 0) {
    for (int i0 = 0; i0 < a.budget; i0 += kSelectThreads) {
      const int i = i0 + tid;
      const float x = i < a.budget ? w[__ldcg(kept + i)] : 0.f;
      __syncthreads();
      if (i < a.budget) wo[i] = x;
    }
    __syncthreads();
    for (int i = a.budget + tid; i < ba.cap; i += kSelectThreads) wo[i] = 0.f;
  }
  if (SMEM)
    for (int i = a.budget + all_tid; i < ba.cap; i += all_threads) wo[i] = 0.f;
}

template <int ELT, int D>
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(PagesView pv, BatchArgs ba, EvictArgs a, int chunks) {
  constexpr int NV = D * ELT / 16;                       // vectors of a row
  constexpr int PASS = kMoveThreads / NV;                // rows at a time
  constexpr int N = kMoveRows / PASS;
  static_assert(NV <= kMoveThreads && kMoveRows % PASS == 0, "rows of a CTA");
  __shared__ int s_ticket;
  __shared__ int s_late;
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  int64_t id = blockIdx.x;
  if (a.in_place) {
    if (tid == 0) {
      s_ticket = atomicAdd(static_cast<int32_t*>(a.ws), 1);
      s_late = 0;
    }
    __syncthreads();
    id = s_ticket;
  }
  const int64_t bh = id / chunks;
  const int chunk = (int)(id % chunks), r0 = chunk * kMoveRows;
  const int b = (int)(bh / pv.Hkv), h = (int)(bh % pv.Hkv);
  const int L = length_of(pv, ba, b);
  const int count = min(L, a.budget);
  if (r0 >= count || (a.in_place && L <= a.budget)) return;    // nothing waits for it
  const int32_t* kept = a.kept + bh * a.budget;
  const int32_t* out = a.in_place ? ba.table : a.table_out;
  const int col = tid % NV, row = r0 + tid / NV;
  const uint4* K = static_cast<const uint4*>(pv.K);
  const uint4* V = static_cast<const uint4*>(pv.V);
  // In stages, each of reads that do not wait for one another: the kept tokens, the
  // pages they come from and go to, the rows.
  int j[N], from[N], to[N];
#pragma unroll
  for (int e = 0; e < N; ++e) j[e] = kept[min(row + e * PASS, count - 1)];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    from[e] = ba.table[(size_t)b * ba.max_pages + (j[e] >> pv.log2P)];
    to[e] = out[(size_t)b * ba.max_pages + (min(row + e * PASS, count - 1) >> pv.log2P)];
  }
  uint4 k[N], v[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    bad |= (unsigned)from[e] >= (unsigned)pv.pages || (unsigned)to[e] >= (unsigned)pv.pages;
    const int page = (unsigned)from[e] < (unsigned)pv.pages ? from[e] : 0;
    const size_t at =
        (((size_t)page * pv.Hkv + h) * pv.P + (j[e] & (pv.P - 1))) * NV + col;
    // not through the read-only path: in place, rows are written in this launch
    if (row + e * PASS < count) {
      k[e] = __ldcg(K + at);
      v[e] = __ldcg(V + at);
    }
  }
  if (bad) flag_error(pv.err, kErrBadBatch);
  bool ok = true;
  if (a.in_place) {
    __syncthreads();                                     // the CTA has its rows
    int32_t* flags = move_flags(a.ws) + bh * chunks;
    if (tid == 0)
      asm volatile("st.release.gpu.s32 [%0], 1;" ::"l"(flags + chunk) : "memory");
    // the lower chunks whose last row comes from this one's first row or behind it
    for (int c = chunk - 1 - tid; c >= 0; c -= kMoveThreads) {
      if (kept[c * kMoveRows + kMoveRows - 1] < r0) break;
      const uint64_t t0 = ptx::globaltimer_ns();
      for (;;) {
        int done;
        asm volatile("ld.acquire.gpu.s32 %0, [%1];" : "=r"(done) : "l"(flags + c) : "memory");
        if (done) break;
        if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
          flag_error(pv.err, kErrWaitTimeout);
          s_late = 1;
          break;
        }
      }
    }
    __syncthreads();
    ok = s_late == 0;
  }
  if (!ok) return;
  uint4* Ko = static_cast<uint4*>(pv.K);
  uint4* Vo = static_cast<uint4*>(pv.V);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int r = row + e * PASS;
    if (r >= count) break;
    if ((unsigned)to[e] >= (unsigned)pv.pages) continue;
    const size_t at = (((size_t)to[e] * pv.Hkv + h) * pv.P + (r & (pv.P - 1))) * NV + col;
    Ko[at] = k[e];
    Vo[at] = v[e];
  }
}

// CTAs of the move for each (sequence, KV head).
int move_chunks(int64_t budget) { return (int)((budget + kMoveRows - 1) / kMoveRows); }

template <int ELT, int D>
cudaError_t launch_move(const PagesView& pv, const BatchArgs& ba, const EvictArgs& a, int chunks,
                        cudaStream_t s) {
  return launch_dependent(evict_move_kernel<ELT, D>,
                          dim3((unsigned)((int64_t)ba.B * pv.Hkv * chunks)), dim3(kMoveThreads), 0,
                          s, pv, ba, a, chunks);
}

}  // namespace

size_t paged_evict_workspace(const PagesView& pv, int64_t batch, int64_t budget, bool kept) {
  const size_t heads = (size_t)batch * pv.Hkv;
  return 256 + (heads * move_chunks(budget) + (kept ? 0 : heads * budget)) * sizeof(int32_t);
}

cudaError_t launch_paged_evict(const PagesView& pv, const BatchArgs& ba, const EvictArgs& in,
                               cudaStream_t s) {
  EvictArgs a = in;
  const int chunks = move_chunks(std::min(a.budget, ba.cap));
  const int64_t heads = (int64_t)ba.B * pv.Hkv;
  if (!a.kept) a.kept = static_cast<int32_t*>(a.ws) + 64 + heads * chunks;
  // Few heads have several CTAs each, as many as are on the SMs together, with a
  // round of tokens for every warp at least.
  int peers = 1;
  while (peers < 8 && heads * peers * 2 <= 4 * (int64_t)pv.sms &&
         ba.cap >= 2 * peers * kSelectThreads)
    peers *= 2;
  const int64_t slice = (ba.cap + 32 * kWarps * peers - 1) / (32 * kWarps * peers) * 32 * kWarps;
  const bool smem = slice <= kSelectSmem;
  auto kern = smem ? evict_select_kernel<true> : evict_select_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem ? kSelectSmem * 4 : 0);
  if (e != cudaSuccess) return e;
  e = launch_dependent_cluster(kern, dim3((unsigned)(heads * peers)), dim3(kSelectThreads),
                               smem ? slice * 4 : 0, s, peers, pv, ba, a, chunks);
  if (e != cudaSuccess) return e;
  if (pv.dtype == RSWA_F32)
    return pv.d == 64 ? launch_move<4, 64>(pv, ba, a, chunks, s)
                      : launch_move<4, 128>(pv, ba, a, chunks, s);
  return pv.d == 64 ? launch_move<2, 64>(pv, ba, a, chunks, s)
                    : launch_move<2, 128>(pv, ba, a, chunks, s);
}

}  // namespace rswa
