// Attention weights that the cached tokens receive from a chunk, on the 5th-generation
// tensor cores (tcgen05 + TMEM + TMA), bf16, head_dim 64 and 128:
//   w[b][kvh][j] = decay * w[b][kvh][j] + sum over the chunk's rows i and the G
//   query heads h of the KV head of exp(q_ih . k_j / sqrt(d) - lse_ih), j seen by i.
//
// Keys are the products' M and query rows their N: S^T = K Q^T, 128 keys of a tile x
// NR rows (token, head of the group).  Thread t of the softmax warps has key t's row of
// S^T: it sums the exponentials of the columns that see its key, a contiguous range as
// tokens ascend, over all row tiles, and writes the token's weight.  So a token's sum is
// made by one thread in the order of the rows, without atomics, and a key is read once.
//
// The values are not read: the least that a launch reads is the keys.  For single
// tokens that is what bounds it; for chunks of many rows the exponentials, one for
// each pair of a row and a key.
//
// Work: the key tiles of all (sequence, KV head) form one list, cut evenly by cost over
// two CTAs an SM.  A tile costs its load and a turn for each row tile that may see it.
// Tiles that nobody sees are listed only where decay changes their weights.
//
// Roles (256 threads): warps 0-3 softmax, warp 4 TMA producer of keys (a lane for each
// page of a tile), warp 5 TMEM allocator and MMA issuer, warp 6 query rows (TMA) and
// their lse, warp 7 planner.  TMEM: S^T twice.  Every wait is bounded; on a timeout the
// CTA drains its copies and MMAs, frees TMEM and sets the pool's device flag.
//
// Measured: 64 tokens of 32 / 8 heads over 256..4096 (262 MB) 44.5 us, 0.87 of the measured
// copy, the rest start and end (46.2 with a tile's pages looked up when its turn comes);
// on the CUDA cores 231.  64 rows of 10 heads over 10272
// tokens 10.9 (9.6 in a graph) for a floor of 4.0: start, plan and first keys 5, a
// tile's turn 1; on the CUDA cores 174.  NR is 64 where one tile of 16 does not hold a
// chunk's rows.
#include <cuda.h>

#include <algorithm>

#include "paged.cuh"
#include "tc_pipe.cuh"

namespace rswa {
namespace {

using namespace ptx;

constexpr int BN = 128;                        // keys per tile
constexpr int kProducerWarp = 4, kMmaWarp = 5, kQueryWarp = 6, kPlanWarp = 7;
constexpr int kThreads = 256;
constexpr int NSEG = 4;                        // segments handed over at a time
constexpr uint32_t kSub = BN * 64 * 2;         // [128][64] bf16, 128B-swizzled
constexpr uint64_t kWaitLimitNs = 1000000000ull;
// Cost of a tile without its row tiles' turns: a key tile's load takes about as long
// as three of them; of one that nobody sees.
constexpr int kTileCost = 3;

template <int D, int NR>
struct Smem {
  static constexpr int NSUB = D / 64;
  static constexpr uint32_t kTile = NSUB * kSub;
  static constexpr uint32_t kQAtom = NR * 128;                    // [NR][64] bf16
  static constexpr uint32_t kQTile = NSUB * kQAtom;
  static constexpr int NS = (NR == 16 ? 6 : 4) / NSUB;            // key tiles of the ring
  static constexpr uint32_t OFF_RING = 0;
  static constexpr uint32_t OFF_Q = OFF_RING + NS * kTile;        // two row tiles
  static constexpr uint32_t OFF_LSE = OFF_Q + 2 * kQTile;         // [2][NR] floats
  static constexpr uint32_t OFF_SEG = OFF_LSE + 2 * NR * 4;
  static constexpr uint32_t OFF_BAR = OFF_SEG + NSEG * 64;
  static constexpr int B_FULL = 0;             // NS
  static constexpr int B_EMPTY = B_FULL + NS;  // NS
  static constexpr int B_QF = B_EMPTY + NS;    // 2: a row tile and its lse are there
  static constexpr int B_QE = B_QF + 2;        // 2: and no longer needed (1 + 128)
  static constexpr int B_S = B_QE + 2;         // 2: S^T in TMEM
  static constexpr int B_SFREE = B_S + 2;      // 2: S^T read (128)
  static constexpr int B_SEG = B_SFREE + 2;    // NSEG segments handed over
  // NSEG read by the key, MMA and query warps and left by the softmax warps (3 + 128): a
  // segment that nobody sees makes none of them wait for another
  static constexpr int B_SEGFREE = B_SEG + NSEG;
  static constexpr int B_FIN = B_SEGFREE + NSEG;
  static constexpr int NBAR = B_FIN + 1;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr uint32_t kBytes = OFF_MISC + 32 + 1024;        // + alignment slack
  static_assert((kBytes + 1024) * 2 <= 233472, "two CTAs per SM");
  static constexpr uint32_t kTmemCols = 2 * NR < 32 ? 32 : 2 * NR;
};

struct Shape {
  int npt;      // tokens of a row tile
  Divisor by_npt;
  int G;        // query heads of a KV head
  int box;      // rows of a key box: a page's, at most a tile's
  int all;      // 1: tiles that nobody sees are listed as well
  float decay;
};

// Key tiles [j0, j1) of the list of one (sequence, KV head).
struct Segment {
  int b, kvh, row0, T, L, m;
  int np, gap, kb;        // prefix tiles, listed tiles that nobody sees, first band tile
  int nrt;                // row tiles
  int j0, j1;             // j1 = 0: no more segments
  __device__ __forceinline__ int tile(int j) const { return j < np + gap ? j : kb + (j - np - gap); }
};
static_assert(sizeof(Segment) <= 64, "segment");

// Row tiles [lo, hi) that may see a token of the key tile at x0.
__device__ __forceinline__ void row_tiles(const Segment& w, int j, const Divisor& npt, int n, int& lo,
                                          int& hi) {
  if (w.T == 0 || (j >= w.np && j < w.np + w.gap)) {
    lo = hi = 0;
    return;
  }
  const int x0 = w.tile(j) * BN, tok0 = w.L - w.T;
  lo = max(x0 - tok0, 0) / npt;
  hi = x0 < w.m ? w.nrt : min(w.nrt, max(x0 + BN - 1 + n - 1 - tok0, 0) / npt + 1);
  if (x0 >= w.m && x0 + BN - 1 + n - 1 < tok0) hi = lo;
}

// The planner: costs of a sequence's list, and a CTA's walk through all of them.
struct WeighPlan {
  const PagesView& pv;
  const BatchArgs& ba;
  const Shape& sh;
  int lane;
  Segment w;
  int nt, cA, cB;                              // listed tiles; costs of prefix and band tiles
  int64_t base = 0, x0 = 0, x1 = 0;            // where (w.b, w.kvh) begins; the CTA's range
  __device__ WeighPlan(const PagesView& p, const BatchArgs& b, const Shape& s)
      : pv(p), ba(b), sh(s), lane((int)(threadIdx.x & 31)) {}

  __device__ __forceinline__ void take(int row0, int T, int L, int m) {
    w.row0 = row0;
    w.T = T;
    w.L = L;
    w.m = m;
    const int tiles = (L + BN - 1) / BN;
    w.np = 0;
    w.kb = tiles;
    if (T > 0) {
      const Hull h(L - T, L - 1, m, ba.window);
      w.np = (h.p + BN - 1) / BN;
      w.kb = max(h.w0 / BN, w.np);
    }
    w.gap = sh.all ? w.kb - w.np : 0;
    nt = w.np + w.gap + tiles - w.kb;
    w.nrt = T > 0 ? (T - 1) / sh.by_npt + 1 : 0;
    cA = kTileCost + w.nrt;
    // tokens that see a band tile: n + 127 of them at most
    cB = kTileCost + min(w.nrt, (ba.window + BN - 2) / sh.by_npt + 2);
  }
  __device__ __forceinline__ int64_t cost_before(int j) const {
    const int a = min(j, w.np), g = min(j - a, w.gap);
    return (int64_t)a * cA + g + (int64_t)(j - a - g) * cB;
  }
  // The first tile that begins at or after cost x.
  __device__ __forceinline__ int at(int64_t x) const {
    if (x <= 0) return 0;
    const int64_t a = (int64_t)w.np * cA;
    if (x <= a) return (int)quotient(x + cA - 1, cA);
    if (x <= a + w.gap) return w.np + (int)(x - a);
    return (int)min((int64_t)nt, w.np + w.gap + quotient(x - a - w.gap + cB - 1, cB));
  }
  __device__ __forceinline__ PagedSeq lane_seq(int b) const {
    PagedSeq s;
    if (b < ba.B)
      s.load(pv, ba, b);
    else
      s.row0 = s.T = s.L = s.m = 0;
    return s;
  }
  __device__ __forceinline__ int64_t scan(int64_t x) const {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    return x;
  }
  __device__ __forceinline__ void adopt(const PagedSeq& s, int b0, int src) {
    w.b = b0 + src;
    take(__shfl_sync(0xffffffffu, s.row0, src), __shfl_sync(0xffffffffu, s.T, src),
         __shfl_sync(0xffffffffu, s.L, src), __shfl_sync(0xffffffffu, s.m, src));
  }
  __device__ bool start(int cta, int ctas) {
    int64_t total = 0, inc0 = 0;
    PagedSeq s0;
    for (int b0 = 0; b0 < ba.B; b0 += 32) {
      const PagedSeq s = lane_seq(b0 + lane);
      take(s.row0, s.T, s.L, s.m);
      const int64_t inc = scan(cost_before(nt) * pv.Hkv);
      if (b0 == 0) {
        s0 = s;
        inc0 = inc;
      }
      total += __shfl_sync(0xffffffffu, inc, 31);
    }
    x0 = quotient(total * cta, ctas);
    x1 = quotient(total * (cta + 1), ctas);
    if (x0 >= x1) return false;
    for (int b0 = 0;; b0 += 32) {
      if (b0 > 0) {
        s0 = lane_seq(b0 + lane);
        take(s0.row0, s0.T, s0.L, s0.m);
        inc0 = scan(cost_before(nt) * pv.Hkv);
      }
      const uint32_t up = __ballot_sync(0xffffffffu, base + inc0 <= x0);
      if (up == 0xffffffffu) {
        base += __shfl_sync(0xffffffffu, inc0, 31);
        continue;
      }
      const int src = __popc(up);
      if (src > 0) base += __shfl_sync(0xffffffffu, inc0, src - 1);
      adopt(s0, b0, src);
      break;
    }
    const int64_t per = cost_before(nt);
    w.kvh = (int)quotient(x0 - base, per);
    base += w.kvh * per;
    return clip() || next();
  }
  // The next (sequence, KV head) with a tile in the range; false: there is none.
  __device__ bool next() {
    for (;;) {
      base += cost_before(nt);
      if (base >= x1) return false;
      if (++w.kvh == pv.Hkv) {
        w.kvh = 0;
        int b0 = w.b + 1;
        for (; b0 < ba.B; b0 += 32) {          // empty sequences are passed over
          const PagedSeq s = lane_seq(b0 + lane);
          take(s.row0, s.T, s.L, s.m);
          const uint32_t live = __ballot_sync(0xffffffffu, nt > 0);
          if (!live) continue;
          adopt(s, b0, __ffs(live) - 1);
          break;
        }
        if (b0 >= ba.B) return false;
      }
      if (clip()) return true;
    }
  }
  __device__ __forceinline__ bool clip() {
    w.j0 = at(x0 - base);
    w.j1 = at(x1 - base);
    return w.j0 < w.j1;
  }
};

template <int D, int NR>
__global__ void __launch_bounds__(kThreads, 2)
paged_weigh_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK, PagesView pv, BatchArgs ba,
                      const float* __restrict__ lse, float* __restrict__ weights, Shape sh,
                      uint64_t wait_ns) {
  using SM = Smem<D, NR>;
  constexpr int NSUB = SM::NSUB, NS = SM::NS;
  constexpr uint32_t kTile = SM::kTile, kQTile = SM::kQTile, kQAtom = SM::kQAtom;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int k) { return sb + SM::OFF_BAR + 8u * (uint32_t)k; };
  const Segment* segs = reinterpret_cast<const Segment*>(smem + SM::OFF_SEG);
  float* s_lse = reinterpret_cast<float*>(smem + SM::OFF_LSE);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM::OFF_MISC + 4);
  volatile int* never = reinterpret_cast<volatile int*>(smem + SM::OFF_MISC + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  if (tid == 0) {
    for (int k = 0; k < SM::NBAR; ++k)
      mbar_init(bar(k), k >= SM::B_QF && k < SM::B_QE     ? 2u
                        : k >= SM::B_QE && k < SM::B_S    ? 129u
                        : k >= SM::B_SFREE && k < SM::B_SEG  ? 128u
                        : k >= SM::B_SEGFREE && k < SM::B_FIN ? 131u
                                                             : 1u);
    *abort_flag = 0;
    *never = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), SM::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();
  auto wait = [&](int k, uint32_t phase) {
    return wait_for(bar(k), phase & 1, abort_flag, wait_ns);
  };
  auto wait_all = [&](int k, uint32_t phase) { return __all_sync(0xffffffffu, wait(k, phase)); };
  auto has_segment = [&](int k) {
    return wait_all(SM::B_SEG + k % NSEG, k / NSEG) && segs[k % NSEG].j1 > 0;
  };
  // Segment k, copied by a whole warp, which then needs its slot no longer.
  auto take_segment = [&](int k) {
    const Segment w = segs[k % NSEG];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(SM::B_SEGFREE + k % NSEG));
    return w;
  };
  const int n = ba.window;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) prefetch_tmap(&tmK);
    const uint64_t pol = evict_first_policy();
    uint32_t gi = 0;
    bool ok = true;
    for (int k = 0; ok && has_segment(k); ++k) {
      const Segment w = take_segment(k);
      Hull hull(w.L - w.T, w.L - 1, w.m, n);
      if (w.T == 0) hull.p = hull.w0 = hull.end = 0;     // nobody sees a token
      // Whether somebody sees a token of this lane's box of tile j, and its page's entry,
      // read a tile ahead.
      auto seen = [&](int j) {
        const int t0 = w.tile(j) * BN + lane * sh.box;
        return lane * sh.box < BN && hull.meets(t0, t0 + sh.box);
      };
      auto entry = [&](int j) {
        if (j >= w.j1 || !seen(j)) return 0;
        return page_entry(ba, w.b, (w.tile(j) * BN + lane * sh.box) >> pv.log2P);
      };
      int next = entry(w.j0);
      for (int j = w.j0; ok && j < w.j1; ++j) {
        const int at = next;
        next = entry(j + 1);
        int lo, hi;
        row_tiles(w, j, sh.by_npt, n, lo, hi);
        if (lo >= hi) continue;
        const int t0 = w.tile(j) * BN + lane * sh.box;
        const int page = seen(j) ? page_of_entry(pv, at) : -1;
        const int row = (page * pv.Hkv + w.kvh) * pv.P + (t0 & (pv.P - 1));
        const uint32_t bytes =
            __popc(__ballot_sync(0xffffffffu, page >= 0)) * (uint32_t)(sh.box * 128 * NSUB);
        const uint32_t s = gi % NS;
        if (gi >= (uint32_t)NS && !wait_all(SM::B_EMPTY + s, gi / NS - 1)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(bar(SM::B_FULL + s), bytes);
        __syncwarp();
        if (page >= 0) {
          const uint32_t dst = sb + SM::OFF_RING + s * kTile + lane * sh.box * 128;
#pragma unroll
          for (int c = 0; c < NSUB; ++c)
            tma_load_2d_pol(dst + c * kSub, &tmK, c * 64, row, bar(SM::B_FULL + s), pol);
        }
        ++gi;
      }
    }
    // Drain: every copy issued has landed before the CTA may exit.
    if (lane == 0)
      for (uint32_t k = gi > (uint32_t)NS ? gi - NS : 0; k < gi; ++k)
        wait_for(bar(SM::B_FULL + k % NS), (k / NS) & 1, never, kWaitLimitNs);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_bf16(BN, NR, false);
      uint32_t gi = 0, qi = 0, st = 0;         // key tiles, row tiles, steps before
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!wait(SM::B_SEG + k % NSEG, k / NSEG) || segs[k % NSEG].j1 == 0) break;
        const Segment w = segs[k % NSEG];
        mbar_arrive(bar(SM::B_SEGFREE + k % NSEG));
        const bool keep = w.nrt == 1;          // one row tile serves the whole segment
        bool have = false;
        for (int j = w.j0; ok && j < w.j1; ++j) {
          int lo, hi;
          row_tiles(w, j, sh.by_npt, n, lo, hi);
          if (lo >= hi) continue;
          const uint32_t s = gi % NS;
          if (!(ok = wait(SM::B_FULL + s, gi / NS))) break;
          for (int r = lo; r < hi; ++r) {
            if (!have && !(ok = wait(SM::B_QF + (qi & 1), qi >> 1))) break;
            have = true;
            if (st >= 2 && !(ok = wait(SM::B_SFREE + (st & 1), (st >> 1) - 1))) break;
            tc_fence_after();
            const uint32_t kb = sb + SM::OFF_RING + s * kTile;
            const uint32_t qb = sb + SM::OFF_Q + (qi & 1) * kQTile;
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
              mma_bf16_ss(tmem + NR * (st & 1),
                          desc_sw128(kb + (x >> 2) * kSub + (x & 3) * 32, 16, 1024),
                          desc_sw128(qb + (x >> 2) * kQAtom + (x & 3) * 32, 16, 1024), idesc,
                          x > 0);
            mma_commit(bar(SM::B_S + (st & 1)));
            ++st;
            if (!keep) {
              mma_commit(bar(SM::B_QE + (qi & 1)));
              ++qi;
              have = false;
            }
          }
          mma_commit(bar(SM::B_EMPTY + s));
          ++gi;
        }
        if (keep && have) {
          mma_commit(bar(SM::B_QE + (qi & 1)));
          ++qi;
        }
      }
      // Drain: all MMAs of this CTA have finished before TMEM is freed.
      mma_commit(bar(SM::B_FIN));
      wait_for(bar(SM::B_FIN), 0, never, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == kQueryWarp) {
    // ------------------------------------------------- row tiles and their lse
    if (lane == 0) prefetch_tmap(&tmQ);
    uint32_t qi = 0;
    bool ok = true;
    auto load = [&](const Segment& w, int r) {
      const uint32_t s = qi & 1;
      if (qi >= 2 && !wait_all(SM::B_QE + s, (qi >> 1) - 1)) return false;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(SM::B_QF + s), (uint32_t)NSUB * sh.npt * sh.G * 128u);
#pragma unroll
        for (int c = 0; c < NSUB; ++c)
          tma_load_3d(sb + SM::OFF_Q + s * kQTile + c * kQAtom, &tmQ, c * 64, w.kvh * sh.G,
                      w.row0 + r * sh.npt, bar(SM::B_QF + s));
      }
      for (int c = lane; c < NR; c += 32) {
        const int i = r * sh.npt + c / pv.by_G;
        float x = 0.f;
        if (c < sh.npt * sh.G && i < w.T)
          x = lse[(int64_t)(w.row0 + i) * pv.H + w.kvh * sh.G + c % sh.G] * kLog2e;
        s_lse[s * NR + c] = x;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(SM::B_QF + s));
      ++qi;
      return true;
    };
    for (int k = 0; ok && has_segment(k); ++k) {
      const Segment w = take_segment(k);
      bool have = false;
      for (int j = w.j0; ok && j < w.j1; ++j) {
        int lo, hi;
        row_tiles(w, j, sh.by_npt, n, lo, hi);
        for (int r = lo; ok && r < hi; ++r)
          if (w.nrt > 1 || !have) {
            ok = load(w, r);
            have = true;
          }
      }
    }
    if (lane == 0)
      for (uint32_t x = qi > 2 ? qi - 2 : 0; x < qi; ++x)
        wait_for(bar(SM::B_QF + (x & 1)), (x >> 1) & 1, never, kWaitLimitNs);
    __syncwarp();
  } else if (warp == kPlanWarp) {
    // ------------------------------------------------------------ planner
    Segment* out = reinterpret_cast<Segment*>(smem + SM::OFF_SEG);
    WeighPlan plan(pv, ba, sh);
    int k = 0;
    for (bool more = plan.start(blockIdx.x, gridDim.x); more; more = plan.next()) {
      if (k >= NSEG && !wait_all(SM::B_SEGFREE + k % NSEG, k / NSEG - 1)) break;
      if (lane == 0) {
        out[k % NSEG] = plan.w;
        mbar_arrive(bar(SM::B_SEG + k % NSEG));
      }
      __syncwarp();
      ++k;
    }
    if (k >= NSEG) wait_all(SM::B_SEGFREE + k % NSEG, k / NSEG - 1);
    if (lane == 0 && !*abort_flag) {
      out[k % NSEG].j1 = 0;                    // no more segments
      mbar_arrive(bar(SM::B_SEG + k % NSEG));
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const float scale = rsqrtf((float)D) * kLog2e;
    uint32_t qi = 0, st = 0;
    bool ok = true;
    for (int k = 0; ok && has_segment(k); ++k) {
      const Segment w = segs[k % NSEG];
      const bool keep = w.nrt == 1;
      const int tok0 = w.L - w.T;
      bool have = false;
      for (int j = w.j0; ok && j < w.j1; ++j) {
        int lo, hi;
        row_tiles(w, j, sh.by_npt, n, lo, hi);
        const int t = w.tile(j) * BN + tid;
        float* out = weights + ((int64_t)w.b * pv.Hkv + w.kvh) * ba.cap + t;
        float old = 0.f;
        if (t < w.L && sh.decay != 0.f) old = *out;
        // Rows that see this key: tokens t .. t + n - 1, all from t on in the prefix.
        const int i_lo = max(t - tok0, 0);
        const int i_hi = t < w.m ? w.T : min(w.T, max(t - tok0 + n, 0));
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        for (int r = lo; r < hi; ++r) {
          if (!have && !(ok = wait_all(SM::B_QF + (qi & 1), qi >> 1))) break;
          have = true;
          if (!(ok = wait_all(SM::B_S + (st & 1), st >> 1))) break;
          tc_fence_after();
          // columns [c0, c1) of the tile
          const int c0 = max(i_lo - r * sh.npt, 0) * sh.G;
          const int c1 = t < w.L ? min(i_hi - r * sh.npt, sh.npt) * sh.G : 0;
          const float* ls = s_lse + (qi & 1) * NR;
#pragma unroll 1
          for (int c = 0; c < NR; c += 16) {
            if (!__any_sync(0xffffffffu, c0 < c + 16 && c1 > c)) continue;
            uint32_t x[16];
            tmem_ld16(tmem + lane_off + NR * (st & 1) + c, x);
            tmem_wait_ld();
            const bool whole = c0 <= c && c1 >= c + 16;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 l4 = *reinterpret_cast<const float4*>(ls + c + e);
              const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float p = ex2(fmaf(__uint_as_float(x[e + y]), scale, -l[y]));
                if (whole || (c + e + y >= c0 && c + e + y < c1)) sum[y] += p;
              }
            }
          }
          tc_fence_before();
          mbar_arrive(bar(SM::B_SFREE + (st & 1)));
          ++st;
          if (!keep) {
            mbar_arrive(bar(SM::B_QE + (qi & 1)));
            ++qi;
            have = false;
          }
        }
        if (!ok) break;
        if (t < w.L) *out = fmaf(sh.decay, old, (sum[0] + sum[1]) + (sum[2] + sum[3]));
      }
      if (!ok) break;
      if (keep && have) {
        mbar_arrive(bar(SM::B_QE + (qi & 1)));
        ++qi;
      }
      mbar_arrive(bar(SM::B_SEGFREE + k % NSEG));
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, SM::kTmemCols);
  }
  if (tid == 0 && *abort_flag) flag_error(pv.err, kErrWaitTimeout);
}

template <int D, int NR>
cudaError_t launch_r(const PagesView& pv, const PagesMaps& maps, const BatchArgs& ba,
                     const void* q, int64_t q_stride, const float* lse, float* weights,
                     float decay, cudaStream_t s) {
  Shape sh;
  sh.G = pv.G;
  sh.npt = NR / pv.G;
  sh.by_npt = Divisor(sh.npt);
  sh.box = std::min(pv.P, BN);
  sh.all = decay != 1.f;
  sh.decay = decay;
  CUtensorMap mq;
  if (ba.rows == 0) {
    mq = maps.k;                               // not read
  } else {
    const int64_t stride = ba.rows < 2 ? (int64_t)pv.H * D : q_stride;
    if (!make_tmap_heads_bf16(&mq, q, D, pv.H, ba.rows, sh.G, sh.npt, stride))
      return cudaErrorInvalidValue;
  }
  auto kern = paged_weigh_tc_kernel<D, NR>;
  // Per device (the attribute belongs to the current device's context).
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Smem<D, NR>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(2 * std::max(pv.sms, 1)), dim3(kThreads),
                          Smem<D, NR>::kBytes, s, mq, maps.k, pv, ba, lse, weights, sh,
                          phase_wait_limit_ns());
}

}  // namespace

bool paged_weigh_tc_supported(const PagesView& pv) {
  return pv.dtype == RSWA_BF16 && pv.G <= 64;
}

cudaError_t launch_paged_weigh_tc(const PagesView& pv, const PagesMaps& maps, const BatchArgs& ba,
                                  const void* q, int64_t q_stride, const float* lse,
                                  float* weights, float decay, cudaStream_t s) {
  const bool few = pv.G <= 16 && (int64_t)ba.rows * pv.G <= 16 * (int64_t)ba.B;
  if (pv.d == 64)
    return few ? launch_r<64, 16>(pv, maps, ba, q, q_stride, lse, weights, decay, s)
               : launch_r<64, 64>(pv, maps, ba, q, q_stride, lse, weights, decay, s);
  return few ? launch_r<128, 16>(pv, maps, ba, q, q_stride, lse, weights, decay, s)
             : launch_r<128, 64>(pv, maps, ba, q, q_stride, lse, weights, decay, s);
}

}  // namespace rswa
