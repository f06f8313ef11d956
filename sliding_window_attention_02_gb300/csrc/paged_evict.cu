// Eviction from a paged cache: of every (sequence, KV head) the first tokens, the
// last ones and the heaviest of the others stay, up to a budget, in their order.
//
// Two kernels.  The first, a CTA or a cluster of them for each (sequence, KV head),
// finds the least weight that stays: the weights as integers of the same order, a
// radix select of at most three passes over 11 bits each, in registers where they
// fit.  Ties of that weight stay from the lowest index on.  Counts of what stays give
// each kept token its place; the weights follow.  The second moves the rows, every
// read of a CTA in flight at once: bound by HBM (0.95 of a copy's rate for 262 MB).
// Both, one sequence of 10 heads, 10272 tokens to 2048: 13.1 us (a floor of 3.2); 48
// sequences of 8 heads, 400..2300 to 700: 51.5 (38.7).
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
constexpr int kMoveRows = 32;                            // least rows of a move CTA
constexpr uint64_t kWaitLimitNs = 1000000000ull;

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

// The radix select's digits: 11 bits, 11 and 10.
constexpr int kBins = 2048, kGroups = kBins / 32;
// Copies of the histogram, by lane: weights share few exponents, and the lanes of a
// warp that add to one word take turns.
constexpr int kCopies = 2;

// A word of CTA `rank`'s shared memory at this CTA's address p.
__device__ __forceinline__ uint32_t peer_word(const void* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_dsmem(p, (uint32_t)rank))
               : "memory");
  return v;
}
// Stores v there.
__device__ __forceinline__ void push_word(void* p, int rank, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_dsmem(p, (uint32_t)rank)), "r"(v)
               : "memory");
}

// A CTA, or a cluster of them, for each (sequence, KV head): each takes a slice of
// its tokens, each warp a range of the slice.  A cluster finds the digit in which the
// least weight falls in two steps, its group of 32 digits and then the digit: its CTAs
// read 64 + 32 counts of one another and not 2048 (one sequence of 10 heads, 32768
// tokens: 12.8 us; all 2048 counts added to the peers' 25).  Bound by the latency of its
// stages, some 16000 cycles of them: what is read is small.
// R > 0: the R rounds of 32 that a warp's range may have are kept in registers; else
// the weights are read again where they are needed.
template <int R>
__global__ void __launch_bounds__(kSelectThreads, R > 8 ? 1 : 2)
evict_select_kernel(PagesView pv, BatchArgs ba, EvictArgs a, int chunks) {
  constexpr bool REGS = R > 0;
  __shared__ alignas(16) uint32_t s_hist[kCopies][kBins];
  __shared__ uint32_t s_sum[kWarps], s_found[3];
  // The slice's counts by digit and by group, of the even and the odd passes, as a peer
  // may be one pass behind; and the peers'.
  __shared__ alignas(16) uint32_t s_digit[2][kBins];
  __shared__ uint32_t s_group[2][kGroups], s_groups[8][kGroups], s_digits[8][32];
  __shared__ int s_warp[2][kWarps], s_slice[2][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int peers = (int)cluster_size(), rank = (int)cluster_rank();
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto four = [&](uint32_t* bins) { return reinterpret_cast<uint4*>(bins) + tid; };
  static_assert(kBins == 4 * kSelectThreads, "four digits a thread");
#pragma unroll
  for (int p = 0; p < kCopies; ++p) *four(s_hist[p]) = zero;
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
  if (peers > 1) cluster_arrive_relaxed();               // tells only that it has begun
  auto meet = [&]() {
    if (peers > 1) {
      cluster_arrive_release();
      cluster_wait();
    } else {
      __syncthreads();
    }
  };
  const int lo = a.first, hi = L - a.last;               // the tokens that are weighed
  // the CTA's tokens, and this warp's of them: whole rounds of 32
  const int span = (L + 32 * kWarps * peers - 1) / (32 * kWarps * peers) * 32;
  const int j0 = min((rank * kWarps + warp) * span, L), j1 = min(j0 + span, L);
  float x[REGS ? R : 1];
  if (REGS) {
#pragma unroll
    for (int e = 0; e < R; ++e) {
      if (32 * e >= span) break;
      x[e] = j0 + 32 * e + lane < j1 ? w[j0 + 32 * e + lane] : 0.f;
    }
  }
  // f(token, weight), round by round
  auto rounds = [&](auto&& f) {
    if (REGS) {
#pragma unroll
      for (int e = 0; e < R; ++e) {
        if (32 * e >= span) break;
        f(j0 + 32 * e + lane, x[e]);
      }
    } else {
#pragma unroll 8
      for (int j = j0 + lane; j < j0 + span; j += 32) f(j, j < j1 ? w[j] : 0.f);
    }
  };
  auto scan = [&](uint32_t v) {                          // sums up to a lane's
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += y;
    }
    return v;
  };
  uint32_t prefix = 0, need = (uint32_t)(a.budget - a.first - a.last);
  __syncthreads();                                       // the histograms are zero
  if (peers > 1) cluster_wait();                         // and the peers have begun
  // Tokens with a key above `least` stay, and the first `ties` with that key.
  uint32_t least = 0xffffffffu;                          // no weight has this key
  int ties = 0;
  if (need > 0) {
    for (int pass = 0;; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      uint32_t* hist = s_hist[lane & (kCopies - 1)];
      // digits from the highest down
      rounds([&](int j, float weight) {
        const uint32_t k = order_key(weight);
        if (j >= lo && j < min(j1, hi) && (pass == 0 || ((k ^ prefix) >> shift) <= mask))
          atomicAdd(hist + (~k >> shift & mask), 1u);
      });
      __syncthreads();
      // the slice's counts: four digits a thread
      const uint4 c0 = *four(s_hist[0]), c1 = *four(s_hist[1]);
      *four(s_hist[0]) = *four(s_hist[1]) = zero;
      const uint32_t c[4] = {c0.x + c1.x, c0.y + c1.y, c0.z + c1.z, c0.w + c1.w};
      uint32_t sum = (c[0] + c[1]) + (c[2] + c[3]), above;
      bool whole;                                        // all weights with the digit stay
      if (peers == 1) {
        const uint32_t inc = scan(sum);
        if (lane == 31) s_sum[warp] = inc;
        __syncthreads();
        above = __reduce_add_sync(0xffffffffu, lane < warp ? s_sum[lane] : 0u) + inc - sum;
        if (above < need && need <= above + sum) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (above < need && need <= above + c[e]) {
              s_found[0] = prefix | (mask - (uint32_t)(4 * tid + e)) << shift;
              s_found[1] = need - above;
              s_found[2] = need - above == c[e];
            }
            above += c[e];
          }
        }
        __syncthreads();
        prefix = s_found[0];
        need = s_found[1];
        whole = s_found[2] != 0;
      } else {
        // Eight threads have a group of 32 digits.
        const int odd = pass & 1;
        *four(s_digit[odd]) = make_uint4(c[0], c[1], c[2], c[3]);
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if ((lane & 7) == 0) s_group[odd][tid >> 3] = sum;
        cluster_arrive_release();
        cluster_wait();
        // every warp: the group in which the needed one falls, then the digit
        const int p = tid / kGroups, g = tid % kGroups;
        if (p < peers) s_groups[p][g] = peer_word(&s_group[odd][g], p);
        __syncthreads();
        uint32_t g0 = 0, g1 = 0;
        for (int p = 0; p < peers; ++p) {
          g0 += s_groups[p][2 * lane];
          g1 += s_groups[p][2 * lane + 1];
        }
        above = scan(g0 + g1) - g0 - g1;
        const bool second = need > above + g0;
        uint32_t at = __ballot_sync(0xffffffffu, above < need && need <= above + g0 + g1);
        const int src = __ffs(at) - 1;
        const int group = 2 * src + (int)__shfl_sync(0xffffffffu, (uint32_t)second, src);
        need -= __shfl_sync(0xffffffffu, second ? above + g0 : above, src);
        if (warp < peers)
          s_digits[warp][lane] = peer_word(&s_digit[odd][32 * group + lane], warp);
        __syncthreads();
        uint32_t n = 0;
        for (int p = 0; p < peers; ++p) n += s_digits[p][lane];
        above = scan(n) - n;
        at = __ballot_sync(0xffffffffu, above < need && need <= above + n);
        const int digit = __ffs(at) - 1;
        need -= __shfl_sync(0xffffffffu, above, digit);
        whole = need == __shfl_sync(0xffffffffu, n, digit);
        prefix |= (mask - (uint32_t)(32 * group + digit)) << shift;
      }
      // Every weight with these digits stays: the lower ones need not be known.
      if (whole && prefix != 0) {
        least = prefix - 1;
        break;
      }
      if (pass == 2) {
        least = prefix;
        ties = (int)need;
        break;
      }
    }
  }
  // What stays, in order: a warp looks through its tokens once for their count and
  // once, behind the counts of the warps before it, for the places.
  auto look = [&](int j, float weight, uint32_t& stays, uint32_t& equal) {
    const bool in = j < j1, end = in && (j < lo || j >= hi);
    const uint32_t k = order_key(weight);
    stays = __ballot_sync(0xffffffffu, end || (in && k > least));
    equal = __ballot_sync(0xffffffffu, in && !end && k == least);
  };
  int na = 0, ne = 0;
  rounds([&](int j, float weight) {
    uint32_t stays, equal;
    look(j, weight, stays, equal);
    na += __popc(stays);
    ne += __popc(equal);
  });
  if (lane == 0) {
    s_warp[0][warp] = na;
    s_warp[1][warp] = ne;
  }
  __syncthreads();
  if (peers > 1) {
    // the slice's counts, to the peers behind it
    if (warp < 2) {
      const int sum = __reduce_add_sync(0xffffffffu, lane < kWarps ? s_warp[warp][lane] : 0);
      if (lane > rank && lane < peers) push_word(&s_slice[warp][rank], lane, sum);
    }
    meet();
  }
  {
    int wa = lane < warp ? s_warp[0][lane] : 0, we = lane < warp ? s_warp[1][lane] : 0;
    if (lane < rank) {                                   // at most 8 ranks
      wa += s_slice[0][lane];
      we += s_slice[1][lane];
    }
    na = __reduce_add_sync(0xffffffffu, wa);
    ne = __reduce_add_sync(0xffffffffu, we);
  }
  // Weights in place: from registers they may be written, as every slice has been read.
  const bool direct = REGS || wo != w;
  const uint32_t before = (1u << lane) - 1u;
  rounds([&](int j, float weight) {
    uint32_t stays, equal;
    look(j, weight, stays, equal);
    const int e = ne + __popc(equal & before);           // equals before this token
    if (stays >> lane & 1u || (equal >> lane & 1u && e < ties)) {
      const int at = na + __popc(stays & before) + min(e, ties);
      kept[at] = j;
      if (direct) wo[at] = weight;
    }
    na += __popc(stays);
    ne += __popc(equal);
  });
  if (!direct) {
    // By one CTA: a batch is read before it is written, and a later batch comes from
    // behind what an earlier one writes.
    meet();                                              // the kept tokens are written
    for (int i0 = 0; rank == 0 && i0 < a.budget; i0 += kSelectThreads) {
      const int i = i0 + tid;
      const float v = i < a.budget ? w[__ldcg(kept + i)] : 0.f;
      __syncthreads();
      if (i < a.budget) wo[i] = v;
    }
    meet();
  }
  for (int i = a.budget + all_tid; i < ba.cap; i += all_threads) wo[i] = 0.f;
}

template <int ELT, int D, int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS)
evict_move_kernel(PagesView pv, BatchArgs ba, EvictArgs a, int chunks) {
  constexpr int NV = D * ELT / 16;                       // vectors of a row
  constexpr int PASS = THREADS / NV;                // rows at a time
  constexpr int N = ROWS / PASS;
  static_assert(NV <= THREADS && ROWS % PASS == 0, "rows of a CTA");
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
  const int chunk = (int)(id % chunks), r0 = chunk * ROWS;
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
    for (int c = chunk - 1 - tid; c >= 0; c -= THREADS) {
      if (kept[c * ROWS + ROWS - 1] < r0) break;
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

// Most CTAs of the move for each (sequence, KV head).
int move_chunks(int64_t budget) { return (int)((budget + kMoveRows - 1) / kMoveRows); }

// Rows of a move CTA: 64, or 32 where CTAs of 64 would not fill the SMs once, four
// on each (one sequence of 10 heads, 2048 rows: 13.5 and 12.4 us for both kernels;
// 48 sequences of 8 heads, 700 rows: 51.2 and 52.5).
int move_rows(const PagesView& pv, int64_t heads, int64_t budget) {
  return heads * ((budget + 63) / 64) < 4 * (int64_t)pv.sms ? 32 : 64;
}

template <int ELT, int D>
cudaError_t launch_move(const PagesView& pv, const BatchArgs& ba, const EvictArgs& a, int rows,
                        int chunks, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)ba.B * pv.Hkv * chunks));
  return rows == 32 ? launch_dependent(evict_move_kernel<ELT, D, 32, 256>, grid, dim3(256), 0, s,
                                       pv, ba, a, chunks)
                    : launch_dependent(evict_move_kernel<ELT, D, 64, 128>, grid, dim3(128), 0, s,
                                       pv, ba, a, chunks);
}

}  // namespace

size_t paged_evict_workspace(const PagesView& pv, int64_t batch, int64_t budget, bool kept) {
  const size_t heads = (size_t)batch * pv.Hkv;
  return 256 + (heads * move_chunks(budget) + (kept ? 0 : heads * budget)) * sizeof(int32_t);
}

cudaError_t launch_paged_evict(const PagesView& pv, const BatchArgs& ba, const EvictArgs& in,
                               cudaStream_t s) {
  EvictArgs a = in;
  const int64_t heads = (int64_t)ba.B * pv.Hkv, most = std::min(a.budget, ba.cap);
  const int rows = move_rows(pv, heads, most), chunks = (int)((most + rows - 1) / rows);
  if (!a.kept) a.kept = static_cast<int32_t*>(a.ws) + 64 + heads * chunks;
  // A warp's range has `rounds` of 32 tokens.  Few heads have a cluster of CTAs each, as
  // many as are on the SMs together, where one CTA would have more than 8.  10 heads,
  // with the move of 256 rows: 4096 tokens 9.0 us (a bound of 4 rounds 10.9), 10272
  // 11.6 (16 rounds 14.7; 4 rounds 9.6, but with a move of 2048 rows 14.2 for 13.0),
  // 32768 12.8 (16 rounds 16.9); 64 heads of 8192 13.4 (4 rounds 14.9, 16 14.4).  Up to 32
  // rounds stay in registers: 10 heads of 102400 21.0, read again 40.3; 512 heads of 16384
  // 81.6 and 115.
  auto rounds_of = [&](int n) {
    return ((int64_t)ba.cap + 32 * kWarps * n - 1) / (32 * kWarps * n);
  };
  int peers = 1;
  while (peers < 8 && heads * peers * 2 <= 2 * (int64_t)pv.sms && rounds_of(peers) > 8)
    peers *= 2;
  const int64_t rounds = rounds_of(peers);
  auto kern = rounds <= 8    ? evict_select_kernel<8>
              : rounds <= 32 ? evict_select_kernel<32>
                             : evict_select_kernel<0>;
  const cudaError_t e = launch_dependent_cluster(kern, dim3((unsigned)(heads * peers)),
                                                 dim3(kSelectThreads), 0, s, peers, pv, ba, a,
                                                 chunks);
  if (e != cudaSuccess) return e;
  if (pv.dtype == RSWA_F32)
    return pv.d == 64 ? launch_move<4, 64>(pv, ba, a, rows, chunks, s)
                      : launch_move<4, 128>(pv, ba, a, rows, chunks, s);
  return pv.d == 64 ? launch_move<2, 64>(pv, ba, a, rows, chunks, s)
                    : launch_move<2, 128>(pv, ba, a, rows, chunks, s);
}

}  // namespace rswa
