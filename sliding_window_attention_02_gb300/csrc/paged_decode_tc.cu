// Attention of a few tokens of each sequence over a paged cache on the 5th-generation
// tensor cores (tcgen05 + TMEM + TMA), bf16, head_dim 64 and 128.
//
// What it computes is paged_attend_tc.cu's, for units of at most 8 rows (token, head
// of the group).  So few rows are the MMAs' N: keys fill M, S^T = K Q^T (128 keys of a
// tile x 16 columns, the least at that M) and O^T += V^T P^T (d x 16, K = 128 keys), with
// the accumulators in TMEM.  A key tile is read once for all rows of the unit and takes two short
// products, so the launch runs at the rate at which tiles arrive.
//
// A weight is two bf16 parts, as the product with V wants 16-bit operands: it rounded,
// and what that took off.  Together they are off by 2^-16 of it.  The second parts are the
// columns that 8 rows leave free, so they cost no product (64 tokens of 10 heads 72.9 us with
// and without, of 32 / 8 heads 85.0 and 85.2; where units have 8 rows 62.9 and 61.8).
//
// Keys are fetched in boxes of a page's rows, at most 32, without the boxes in which no
// row sees a token (64 tokens over 2048, 1500 in the prefix and a window of 128, pages of
// 256: 86.6 us, boxes of 128 rows 89.2, of 16 86.1, but 104.9 for 103.6 without a mask); V^T
// P^T takes only the 16-key steps that hold a seen token, and value rows of others
// in such steps are zeroed first (they may be any bits, and 0 x NaN is NaN).
//
// Work: PagedPlan cuts the list of all units' tiles evenly over the CTAs, two an SM,
// each of which streams its range through one TMA ring without draining between units.
// Units cut over several CTAs leave partials (m, l, O), which the last of a unit's
// CTAs merges in the order of the CTAs.
//
// Roles (352 threads): warps 0-3 softmax (thread t owns key t of a tile, TMEM lane t),
// warps 4-7 the ends of segments (thread e owns row d = e of O^T: scales and stores it,
// or publishes and merges; it also stages the queries two segments ahead), warp 8 TMA
// producer (a lane for each box of a tile), warp 9 TMEM allocator and MMA issuer, warp
// 10 planner.  TMEM (64 columns): S^T twice, O^T twice (by segment), so that a
// segment's end runs beside the next one's tiles.  MMA order S(0) S(1) PV(0) S(2)
// PV(1) ...: the softmax of tile j runs beside PV(j - 1).  O^T is rescaled lazily
// (threshold 2^8).  At head_dim 64 the product's upper 64 rows are made of bytes of the
// lower ones' and belong to nobody.  Every wait is bounded; on a timeout the CTA drains
// its copies and MMAs, frees TMEM and sets the pool's device flag.
//
// Bound by HBM and by the launch's start and end: 64 tokens of 10 heads over 300..2300 72.8 us, 429 MB at 0.87 of the measured
// copy; of 32 / 8 heads over 256..4096, 507 MB, 85.0, 0.88.  Rows as M and keys as N, the
// tile kernel, are slower (table of the paths in paged_attend.cu), and so were units of up to
// 16 rows, as the softmax's columns are a thread's serial work.
#include <cuda.h>

#include <algorithm>

#include "paged.cuh"
#include "tc_pipe.cuh"

namespace rswa {
namespace {

using namespace ptx;

constexpr int BN = 128;                        // keys per tile
constexpr int NQ = 16;                         // MMA N
constexpr int kRows = 8;                       // rows of queries and weights that are kept
constexpr int kEpiWarp0 = 4;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kPlanWarp = 10;
constexpr int kThreads = 352;
constexpr int NSEG = 4;                        // segments handed over at a time
constexpr uint32_t kSub = BN * 64 * 2;         // [128][64] bf16, 128B-swizzled
constexpr float kRescaleThreshold = 8.0f;      // log2 units
constexpr uint64_t kWaitLimitNs = 1000000000ull;

// A unit's start and end take about as long as a tile.
using Plan = PagedPlan<BN, 1, 1, 1, 2>;

template <int D>
struct Smem {
  static constexpr int NSUB = D / 64;
  static constexpr uint32_t kTile = NSUB * kSub;
  static constexpr int NS = 6 / NSUB;          // ring slots (a K or a V tile)
  // Queries as the MMAs' N rows: 8 are kept, the other eight are whatever follows them
  // here, with results that nobody reads.  Weights: row g's rounded to bf16, and in row 8 +
  // g what that took off.
  static constexpr uint32_t kNAtom = kRows * 128;                 // [kRows][64] bf16
  static constexpr uint32_t kPAtom = 2 * kNAtom;                  // [NQ][64]
  static constexpr uint32_t OFF_RING = 0;
  static constexpr uint32_t OFF_Q = OFF_RING + NS * kTile;        // two of [kRows][D]
  static constexpr uint32_t OFF_P = OFF_Q + 2 * 2 * kNAtom;       // two of [NQ][128]
  static constexpr int B_FULL = 0;             // NS
  static constexpr int B_EMPTY = B_FULL + NS;  // NS
  static constexpr int B_S = B_EMPTY + NS;     // 2: S^T(j) in TMEM
  static constexpr int B_SFREE = B_S + 2;      // 2: S^T(j) read (128)
  static constexpr int B_P = B_SFREE + 2;      // 2: P^T(j) in smem (128)
  static constexpr int B_PFREE = B_P + 2;      // 2: PV(j) done
  static constexpr int B_QFULL = B_PFREE + 2;  // 2: a segment's queries staged (128)
  static constexpr int B_OREADY = B_QFULL + 2; // 2: a segment's last PV done
  static constexpr int B_OFREE = B_OREADY + 2; // 2: its O^T read out (128)
  static constexpr int B_ML = B_OFREE + 2;     // 2: its m, l written (128)
  static constexpr int B_MLFREE = B_ML + 2;    // 2: m, l read (128)
  static constexpr int B_SYNCS = B_MLFREE + 2; // softmax warps' barrier (128)
  static constexpr int B_SYNCE = B_SYNCS + 1;  // end warps' barrier (128)
  static constexpr int B_SEG = B_SYNCE + 1;    // NSEG segments handed over
  static constexpr int B_SEGFREE = B_SEG + NSEG;   // NSEG left by the end warps (128)
  static constexpr int B_FIN = B_SEGFREE + NSEG;
  static constexpr int NBAR = B_FIN + 1;
  static constexpr uint32_t OFF_BAR = OFF_P + 2 * 2 * kPAtom;
  static constexpr uint32_t OFF_FLAGS = OFF_BAR + 8 * NBAR;       // NS words
  static constexpr uint32_t OFF_SEG = (OFF_FLAGS + 4 * NS + 15) & ~15u;
  static constexpr uint32_t OFF_ML = OFF_SEG + NSEG * 128;        // [2][NQ] m, [2][4][NQ] l
  static constexpr uint32_t OFF_RED = OFF_ML + (2 * NQ + 2 * 4 * NQ) * 4;   // [2][4][NQ] max
  static constexpr uint32_t OFF_MISC = OFF_RED + 2 * 4 * NQ * 4;
  static constexpr uint32_t kBytes = OFF_MISC + 32 + 1024;        // + alignment slack
  // The value operand's second 64 columns: the tile's other atom, or, at head_dim 64,
  // the rows 8 further on (columns of O^T that belong to nobody): 1 KB past the ring
  // at most.
  static constexpr uint32_t kAtomStep = NSUB == 2 ? kSub : 1024;
  static_assert(NSUB == 2 || OFF_Q + 1024 <= OFF_MISC, "inside the CTA's shared memory");
  static_assert((kBytes + 1024) * 2 <= 233472, "two CTAs per SM");
};
constexpr uint32_t TM_S = 0, TM_O = 32, TM_COLS = 64;

// A segment as the planner hands it over.
struct Segment {
  int b, kvh, f0, rows;   // the unit's first row (token f0 / G of the chunk) and rows
  int row0, tok0, m;
  Hull hull;
  int np, kb;
  int j0, j1;             // the tiles inside the range; j1 = 0: no more segments
  int first, last;        // the CTAs that the unit begins and ends in
  int whole;
  __device__ __forceinline__ int tile(int j) const { return j < np ? j : kb + (j - np); }
};
static_assert(sizeof(Segment) <= 128, "segment");

// A partial: for each row O[D], then m and l (and two words, so that rows are aligned to
// 16 bytes).
__host__ __device__ constexpr size_t partial_floats(int D) { return (size_t)kRows * (D + 4); }

struct Shape {
  int G, box;
  Divisor unit;  // rows of a unit
  int64_t q_stride;
};

// N consecutive floats, aligned to as many bytes as they are (16 at most), from L2.
template <int N>
__device__ __forceinline__ void load_columns(const float* p, float* x) {
  if constexpr (N == 1) {
    x[0] = __ldcg(p);
  } else if constexpr (N == 2) {
    const float2 v = __ldcg(reinterpret_cast<const float2*>(p));
    x[0] = v.x;
    x[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p + i));
      x[i] = v.x;
      x[i + 1] = v.y;
      x[i + 2] = v.z;
      x[i + 3] = v.w;
    }
  }
}

// NG: the most rows that a unit has (1, 2, 4 or 8).
template <int D, int NG>
__global__ void __launch_bounds__(kThreads, 2)
paged_decode_tc_kernel(const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, PagesView pv, BatchArgs ba,
                       AttendArgs a, Shape sh, uint64_t wait_ns) {
  using SM = Smem<D>;
  constexpr int NSUB = SM::NSUB, NS = SM::NS;
  constexpr uint32_t kTile = SM::kTile, kNAtom = SM::kNAtom, kPAtom = SM::kPAtom;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int k) { return sb + SM::OFF_BAR + 8u * (uint32_t)k; };
  const Segment* segs = reinterpret_cast<const Segment*>(smem + SM::OFF_SEG);
  volatile uint32_t* slot_flags = reinterpret_cast<volatile uint32_t*>(smem + SM::OFF_FLAGS);
  float* ml_m = reinterpret_cast<float*>(smem + SM::OFF_ML);           // [2][NQ]
  float* ml_l = ml_m + 2 * NQ;                                         // [2][4][NQ]
  float* red_max = reinterpret_cast<float*>(smem + SM::OFF_RED);       // [2][4][NQ]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM::OFF_MISC + 4);
  volatile int* never = reinterpret_cast<volatile int*>(smem + SM::OFF_MISC + 8);
  volatile int* s_last = reinterpret_cast<volatile int*>(smem + SM::OFF_MISC + 12);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int cta = blockIdx.x;

  if (tid == 0) {
    for (int k = 0; k < SM::NBAR; ++k) {
      const bool c128 = (k >= SM::B_SFREE && k < SM::B_PFREE) ||
                        (k >= SM::B_QFULL && k < SM::B_OREADY) ||
                        (k >= SM::B_OFREE && k < SM::B_SEG) ||
                        (k >= SM::B_SEGFREE && k < SM::B_FIN);
      mbar_init(bar(k), c128 ? 128u : 1u);
    }
    *abort_flag = 0;
    *never = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), TM_COLS);
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
  // Whether there is a segment k: waits for the planner's word.
  auto has_segment = [&](int k) {
    return wait_all(SM::B_SEG + k % NSEG, k / NSEG) && segs[k % NSEG].j1 > 0;
  };

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
    const uint64_t pol = evict_first_policy();
    uint32_t gi = 0;
    bool ok = true;
    for (int k = 0; ok && has_segment(k); ++k) {
      const Segment& w = segs[k % NSEG];
      const Hull hull = w.hull;
      const int b = w.b, kvh = w.kvh, np = w.np, kb = w.kb, j1 = w.j1;
      auto tile = [&](int j) { return j < np ? j : kb + (j - np); };
      // This lane's box of tile j: its page, or -1 where no row sees a token of it.
      auto page_of = [&](int j) {
        const int t0 = tile(j) * BN + lane * sh.box;
        if (lane * sh.box >= BN || !hull.meets(t0, t0 + sh.box)) return -1;
        return page_at(pv, ba, b, t0 >> pv.log2P);
      };
      int j = w.j0;
      int page = page_of(j);
      for (; ok && j < j1; ++j) {
        const int next = j + 1 < j1 ? page_of(j + 1) : -1;
        const int x0 = tile(j) * BN, t0 = x0 + lane * sh.box;
        const int row = (page * pv.Hkv + kvh) * pv.P + (t0 & (pv.P - 1));
        const uint32_t bytes =
            __popc(__ballot_sync(0xffffffffu, page >= 0)) * (uint32_t)(sh.box * 128 * NSUB);
        // the 16-key steps that hold a token which some row sees
        const uint32_t flags = __ballot_sync(
            0xffffffffu, lane < BN / 16 && hull.meets(x0 + 16 * lane, x0 + 16 * lane + 16));
#pragma unroll 1
        for (int isv = 0; isv < 2; ++isv, ++gi) {
          const uint32_t s = gi % NS;
          if (gi >= (uint32_t)NS && !wait_all(SM::B_EMPTY + s, gi / NS - 1)) {
            ok = false;
            break;
          }
          const uint32_t dst = sb + SM::OFF_RING + s * kTile + lane * sh.box * 128;
          if (lane == 0) {
            slot_flags[s] = flags;
            mbar_arrive_expect_tx(bar(SM::B_FULL + s), bytes);
          }
          __syncwarp();
          if (page >= 0) {
#pragma unroll
            for (int c = 0; c < NSUB; ++c)
              tma_load_2d_pol(dst + c * kSub, isv ? &tmV : &tmK, c * 64, row,
                              bar(SM::B_FULL + s), pol);
          }
        }
        page = next;
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
      constexpr uint32_t idesc_s = idesc_bf16_ab(BN, NQ, false, false);
      constexpr uint32_t idesc_o = idesc_bf16_ab(128, NQ, true, false);
      // PV of the tile before: its load, segment, and whether it is the segment's
      // first and last.
      int pj = -1, ps = 0;
      bool pfirst = false, plast = false;
      auto pv_prev = [&]() {
        const uint32_t vi = 2 * pj + 1, slot = vi % NS;
        if (!wait(SM::B_FULL + slot, vi / NS)) return false;
        const uint32_t flags = slot_flags[slot];
        // the segment's first product overwrites O^T, once segment ps - 2's is read
        if (pfirst && ps >= 2 && !wait(SM::B_OFREE + (ps & 1), (ps >> 1) - 1)) return false;
        if (!wait(SM::B_P + (pj & 1), pj >> 1)) return false;
        tc_fence_after();
        const uint32_t vb = sb + SM::OFF_RING + slot * kTile;
        const uint32_t pb = sb + SM::OFF_P + (pj & 1) * 2 * kPAtom;
        uint32_t acc = pfirst ? 0u : 1u;
#pragma unroll
        for (int k = 0; k < BN / 16; ++k)
          if (flags >> k & 1u) {
            mma_bf16_ss(tmem + TM_O + 16 * (ps & 1), desc_sw128(vb + k * 2048, SM::kAtomStep, 1024),
                        desc_sw128(pb + (k >> 2) * kPAtom + (k & 3) * 32, 16, 1024), idesc_o,
                        acc);
            acc = 1u;
          }
        mma_commit(bar(SM::B_PFREE + (pj & 1)));
        mma_commit(bar(SM::B_EMPTY + slot));
        if (plast) mma_commit(bar(SM::B_OREADY + (ps & 1)));
        return true;
      };
      int j = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!wait(SM::B_SEG + k % NSEG, k / NSEG) || segs[k % NSEG].j1 == 0) break;
        const int tiles = segs[k % NSEG].j1 - segs[k % NSEG].j0;
        for (int i = 0; i < tiles; ++i, ++j) {
          const uint32_t ki = 2 * j, slot = ki % NS;
          ok = (i > 0 || wait(SM::B_QFULL + (k & 1), k >> 1)) &&
               wait(SM::B_FULL + slot, ki / NS) &&
               (j < 2 || wait(SM::B_SFREE + (j & 1), (j - 2) >> 1));
          if (!ok) break;
          tc_fence_after();
          const uint32_t kb = sb + SM::OFF_RING + slot * kTile;
          const uint32_t qb = sb + SM::OFF_Q + (k & 1) * 2 * kNAtom;
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            mma_bf16_ss(tmem + TM_S + 16 * (j & 1),
                        desc_sw128(kb + (x >> 2) * kSub + (x & 3) * 32, 16, 1024),
                        desc_sw128(qb + (x >> 2) * kNAtom + (x & 3) * 32, 16, 1024), idesc_s,
                        x > 0);
          mma_commit(bar(SM::B_S + (j & 1)));
          mma_commit(bar(SM::B_EMPTY + slot));
          if (pj >= 0 && !(ok = pv_prev())) break;
          pj = j;
          ps = k;
          pfirst = i == 0;
          plast = i + 1 == tiles;
        }
      }
      if (ok && pj >= 0) pv_prev();
      // Drain: all MMAs of this CTA have finished before TMEM is freed.
      mma_commit(bar(SM::B_FIN));
      wait_for(bar(SM::B_FIN), 0, never, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == kPlanWarp) {
    // ------------------------------------------------------------ planner
    Segment* out = reinterpret_cast<Segment*>(smem + SM::OFF_SEG);
    Plan plan(pv, ba, sh.unit);
    int k = 0;
    for (bool more = plan.start(cta, gridDim.x); more; more = plan.next()) {
      if (k >= NSEG && !wait_all(SM::B_SEGFREE + k % NSEG, k / NSEG - 1)) break;
      if (lane == 0) {
        const PagedUnit& u = plan.u;
        Segment& w = out[k % NSEG];
        w.b = u.b;
        w.kvh = u.kvh;
        w.f0 = u.f0;
        w.rows = min(NG, u.seq.T * sh.G - u.f0);
        w.row0 = u.seq.row0;
        w.tok0 = u.seq.L - u.seq.T;
        w.m = u.seq.m;
        w.hull = u.hull;
        w.np = u.np;
        w.kb = u.kb;
        w.j0 = u.j0;
        w.j1 = u.j1;
        w.first = u.first;
        w.last = u.last;
        w.whole = u.whole();
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
  } else if (warp < kEpiWarp0) {
    // ------------------------------------------------------------ softmax
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const float scale = rsqrtf((float)D) * kLog2e;
    int n_sync = 0;
    auto soft_sync = [&]() {
      mbar_arrive(bar(SM::B_SYNCS));
      return wait_all(SM::B_SYNCS, n_sync++);
    };
    bool ok = true;
    int j = 0;
    for (int s = 0; ok && has_segment(s); ++s) {
      const Segment& w = segs[s % NSEG];
      const Hull hull = w.hull;
      const int rows = w.rows, m = w.m, j1 = w.j1;
      const int tok = w.tok0, f0 = w.f0, n = ba.window;
      const int a0 = tok + f0 / pv.by_G, a1 = tok + (f0 + rows - 1) / pv.by_G;
      float m_ref[NG], l_t[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        m_ref[g] = -INFINITY;
        l_t[g] = 0.f;
      }
      for (int i = w.j0; i < j1; ++i, ++j) {
        const int x0 = w.tile(i) * BN, t = x0 + tid;
        // which rows see this thread's key
        uint32_t sees = (1u << rows) - 1u;
        if (!(x0 + BN - 1 <= a0 && (x0 + BN <= m || x0 > a1 - n))) {
          if (a0 == a1) {
            if (!hull.has(t)) sees = 0u;
          } else {
#pragma unroll 1
            for (int g = 0; g < rows; ++g) {
              const int x = tok + (f0 + g) / pv.by_G;
              if (t > x || (t >= m && t <= x - n)) sees &= ~(1u << g);
            }
          }
        }
        if (!wait_all(SM::B_S + (j & 1), j >> 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t r[16];
        tmem_ld16(tmem + lane_off + TM_S + 16 * (j & 1), r);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(bar(SM::B_SFREE + (j & 1)));
        float sc[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g)
          sc[g] = sees >> g & 1u ? __uint_as_float(r[g]) * scale : -INFINITY;
        float* rm = red_max + (j & 1) * 4 * NQ;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float v = warp_max(sc[g]);
          if (lane == 0) rm[warp * NQ + g] = v;
        }
        if (!soft_sync()) {
          ok = false;
          break;
        }
        bool grow = false;
        float mt[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          mt[g] = fmaxf(fmaxf(rm[g], rm[NQ + g]), fmaxf(rm[2 * NQ + g], rm[3 * NQ + g]));
          grow |= mt[g] > m_ref[g] + kRescaleThreshold;          // also where m_ref is -inf
        }
        if (grow) {
          float alpha[NG];
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float mn = fmaxf(m_ref[g], mt[g]);
            alpha[g] = (mn == -INFINITY) ? 1.f : fast_exp2(m_ref[g] - mn);
            m_ref[g] = mn;
            l_t[g] *= alpha[g];
          }
          if (i > w.j0) {
            // O^T holds PV of this segment's earlier tiles: rescaled once PV(j - 1)
            // has completed.
            if (!wait_all(SM::B_PFREE + ((j - 1) & 1), (j - 1) >> 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
            uint32_t ov[16];
            tmem_ld16(tmem + lane_off + TM_O + 16 * (s & 1), ov);
            tmem_wait_ld();
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              ov[g] = __float_as_uint(__uint_as_float(ov[g]) * alpha[g]);
              ov[kRows + g] = __float_as_uint(__uint_as_float(ov[kRows + g]) * alpha[g]);
            }
            tmem_st16(tmem + lane_off + TM_O + 16 * (s & 1), ov);
            tmem_wait_st();
          }
        }
        // P^T(j): buffer j & 1 is free once PV(j - 2) has completed.
        if (j >= 2 && !wait_all(SM::B_PFREE + (j & 1), (j - 2) >> 1)) {
          ok = false;
          break;
        }
        uint8_t* pbuf = smem + SM::OFF_P + (j & 1) * 2 * kPAtom;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float ref = (m_ref[g] == -INFINITY) ? 0.f : m_ref[g];
          const float p = fast_exp2(sc[g] - ref);
          l_t[g] += p;
          const __nv_bfloat16 hi = __float2bfloat16(p);
          uint8_t* to = pbuf + sw128_off(g, tid, kPAtom);
          *reinterpret_cast<__nv_bfloat16*>(to) = hi;
          *reinterpret_cast<__nv_bfloat16*>(to + kNAtom) =
              __float2bfloat16(p - __bfloat162float(hi));
        }
        // A value row that no row of the unit sees, in a step that holds others that
        // one does: zero, as 0 x NaN is NaN.
        const bool mine = hull.has(t);
        const uint32_t on = __ballot_sync(0xffffffffu, mine);
        const uint32_t lo = on & 0xffffu, hi = on >> 16;
        if ((lo != 0 && lo != 0xffffu) || (hi != 0 && hi != 0xffffu)) {
          const uint32_t vi = 2 * (uint32_t)j + 1;
          if (!wait_all(SM::B_FULL + vi % NS, vi / NS)) {
            ok = false;
            break;
          }
          if (!mine && (lane < 16 ? lo : hi) != 0) {
            uint4* v = reinterpret_cast<uint4*>(smem + SM::OFF_RING + (vi % NS) * kTile + tid * 128);
#pragma unroll
            for (int c = 0; c < NSUB; ++c)
#pragma unroll
              for (int x = 0; x < 8; ++x) v[c * (kSub / 16) + x] = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(SM::B_P + (j & 1)));
      }
      if (!ok) break;
      // The segment's reference maxima and per-warp sums for its end.
      if (s >= 2 && !wait_all(SM::B_MLFREE + (s & 1), (s >> 1) - 1)) break;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float v = l_t[g];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (lane == 0) ml_l[((s & 1) * 4 + warp) * NQ + g] = v;
        if (tid == 0) ml_m[(s & 1) * NQ + g] = m_ref[g];
      }
      mbar_arrive(bar(SM::B_ML + (s & 1)));
    }
  } else {
    // ----------------------------------------------------- ends of segments
    const int e = tid - kEpiWarp0 * 32;               // row d of O^T
    const uint32_t lane_off = (uint32_t)((warp - kEpiWarp0) * 32) << 16;
    const bool mine = e < D;                          // head_dim 64: half of them
    int n_sync = 0;
    auto end_sync = [&]() {
      mbar_arrive(bar(SM::B_SYNCE));
      return wait_all(SM::B_SYNCE, n_sync++);
    };
    // Queries of segment s as the S MMA's B operand: row g of [kRows][D], column e.
    auto stage_q = [&](int s) {
      const Segment& w = segs[s % NSEG];
      __nv_bfloat16 qv[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int f = w.f0 + g;
        qv[g] = __float2bfloat16(0.f);
        if (mine && g < w.rows)
          qv[g] = static_cast<const __nv_bfloat16*>(
              a.q)[(int64_t)(w.row0 + f / pv.by_G) * sh.q_stride +
                   (int64_t)(w.kvh * sh.G + f % pv.by_G) * D + e];
      }
      if (mine)
#pragma unroll
        for (int g = 0; g < kRows; ++g)
          *reinterpret_cast<__nv_bfloat16*>(smem + SM::OFF_Q + (s & 1) * 2 * kNAtom +
                                            sw128_off(g, e, kNAtom)) =
              g < NG ? qv[g < NG ? g : 0] : __float2bfloat16(0.f);
      fence_proxy_async_smem();
      mbar_arrive(bar(SM::B_QFULL + (s & 1)));
    };
    for (int s = 0; s < 2 && has_segment(s); ++s) stage_q(s);
    for (int s = 0; has_segment(s); ++s) {
      const Segment& w = segs[s % NSEG];
      const int rows = w.rows;
      if (!wait_all(SM::B_OREADY + (s & 1), s >> 1)) break;
      tc_fence_after();
      uint32_t ov[16];
      tmem_ld16(tmem + lane_off + TM_O + 16 * (s & 1), ov);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(bar(SM::B_OFREE + (s & 1)));
      if (!wait_all(SM::B_ML + (s & 1), s >> 1)) break;
      float mg[NG], lg[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        mg[g] = ml_m[(s & 1) * NQ + g];
        const float* lw = ml_l + (s & 1) * 4 * NQ;
        lg[g] = (lw[g] + lw[NQ + g]) + (lw[2 * NQ + g] + lw[3 * NQ + g]);
      }
      mbar_arrive(bar(SM::B_MLFREE + (s & 1)));
      float og[NG];                                     // both parts of the weights
#pragma unroll
      for (int g = 0; g < NG; ++g)
        og[g] = __uint_as_float(ov[g]) + __uint_as_float(ov[kRows + g]);
      // Row g of the unit is chunk row f / G, query head kvh * G + f % G.
      auto out_row = [&](int g) {
        const int f = w.f0 + g;
        return (int64_t)(w.row0 + f / pv.by_G) * pv.H + w.kvh * sh.G + f % pv.by_G;
      };
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o);
      if (w.whole) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (g >= rows) break;
          const int64_t row = out_row(g);
          if (mine) o[row * D + e] = __float2bfloat16(og[g] / lg[g]);
          if (e == 0 && a.lse) a.lse[row] = (mg[g] + log2f(lg[g])) * kLn2;
        }
      } else {
        float* P = paged_partial(a.ws, cta, w.first, partial_floats(D));
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (g >= rows) break;
          if (mine) P[g * (D + 4) + e] = og[g];
          if (e == 0) {
            P[g * (D + 4) + D] = mg[g];
            P[g * (D + 4) + D + 1] = lg[g];
          }
        }
        if (!end_sync()) break;
        if (e == 0) {
          int32_t* count = paged_counter(a.ws, w.first);
          const bool last = arrive_acq_rel(count) == w.last - w.first;
          if (last) *count = 0;                       // ready for the next call
          *s_last = last;
        }
        if (!end_sync()) break;
        if (*s_last) {
          // Each thread has some columns of one row; of that row, the reads of kParts
          // parts, in the order of their CTAs, are on their way together.
          constexpr int kPer = 128 / NG, kCols = D * NG / 128 > 0 ? D * NG / 128 : 1;
          constexpr int kParts = kCols >= 8 ? 4 : 8;
          const int g = e / kPer, c0 = e % kPer * kCols;
          if (g < rows && c0 < D) {
            float M = -INFINITY, L = 0.f, A[kCols];
#pragma unroll
            for (int c = 0; c < kCols; ++c) A[c] = 0.f;
#pragma unroll 1
            for (int p0 = w.first; p0 <= w.last; p0 += kParts) {
              float mk[kParts], lk[kParts], ak[kParts][kCols];
#pragma unroll
              for (int x = 0; x < kParts; ++x) {
                mk[x] = -INFINITY;
                lk[x] = 0.f;
#pragma unroll
                for (int c = 0; c < kCols; ++c) ak[x][c] = 0.f;
                if (p0 + x <= w.last) {
                  const float* P =
                      paged_partial(a.ws, p0 + x, w.first, partial_floats(D)) + g * (D + 4);
                  const float2 ml = __ldcg(reinterpret_cast<const float2*>(P + D));
                  mk[x] = ml.x;
                  lk[x] = ml.y;
                  load_columns<kCols>(P + c0, ak[x]);
                }
              }
              float mn = M;
#pragma unroll
              for (int x = 0; x < kParts; ++x) mn = fmaxf(mn, mk[x]);
              const float ref = (mn == -INFINITY) ? 0.f : mn;
              const float s0 = fast_exp2(M - ref);
              L *= s0;
#pragma unroll
              for (int c = 0; c < kCols; ++c) A[c] *= s0;
#pragma unroll
              for (int x = 0; x < kParts; ++x) {
                const float wx = fast_exp2(mk[x] - ref);
                L = fmaf(lk[x], wx, L);
#pragma unroll
                for (int c = 0; c < kCols; ++c) A[c] = fmaf(ak[x][c], wx, A[c]);
              }
              M = mn;
            }
            const int64_t row = out_row(g);
#pragma unroll
            for (int c = 0; c < kCols; ++c) o[row * D + c0 + c] = __float2bfloat16(A[c] / L);
            if (c0 == 0 && a.lse) a.lse[row] = (M + log2f(L)) * kLn2;
          }
        }
      }
      // The segment after the next may stage its queries: the products with this
      // one's have ended.
      if (has_segment(s + 1) && has_segment(s + 2)) stage_q(s + 2);
      mbar_arrive(bar(SM::B_SEGFREE + s % NSEG));
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
  if (tid == 0 && *abort_flag) flag_error(pv.err, kErrWaitTimeout);
}

int grid_of(const PagesView& pv) { return std::min(2 * std::max(pv.sms, 1), kMaxPagedCtas); }

template <int D, int NG>
cudaError_t launch_g(const PagesView& pv, const PagesMaps& maps, const BatchArgs& ba,
                     const AttendArgs& a, cudaStream_t s) {
  Shape sh;
  sh.G = pv.G;
  sh.unit = Divisor(NG);
  sh.box = std::min(pv.P, 32);
  sh.q_stride = a.q_stride;
  auto kern = paged_decode_tc_kernel<D, NG>;
  // Per device (the attribute belongs to the current device's context).
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(grid_of(pv)), dim3(kThreads), Smem<D>::kBytes, s, maps.k32,
                          maps.v32, pv, ba, a, sh, phase_wait_limit_ns());
}

template <int D>
cudaError_t launch_d(const PagesView& pv, const PagesMaps& maps, const BatchArgs& ba,
                     const AttendArgs& a, cudaStream_t s) {
  // The most rows of a unit, where the host knows them; with starts it does not, and takes 8:
  // 64 single tokens of 10 heads over 2048 105.2 us and with starts 108.6, of 32 / 8 heads
  // 87.1 and 89.7, 200 of 10 heads over 600 103.4 and 108.5.
  const int64_t rows = ba.starts ? kRows : (int64_t)ba.each * pv.G;
  if (rows <= 1) return launch_g<D, 1>(pv, maps, ba, a, s);
  if (rows <= 2) return launch_g<D, 2>(pv, maps, ba, a, s);
  if (rows <= 4) return launch_g<D, 4>(pv, maps, ba, a, s);
  return launch_g<D, 8>(pv, maps, ba, a, s);
}

}  // namespace

size_t paged_decode_tc_workspace(const PagesView& pv) {
  return kPagedCounterBytes + (size_t)grid_of(pv) * 2 * partial_floats(pv.d) * sizeof(float);
}

cudaError_t launch_paged_decode_tc(const PagesView& pv, const PagesMaps& maps, const BatchArgs& ba,
                                   const AttendArgs& a, cudaStream_t s) {
  return pv.d == 64 ? launch_d<64>(pv, maps, ba, a, s) : launch_d<128>(pv, maps, ba, a, s);
}

}  // namespace rswa
