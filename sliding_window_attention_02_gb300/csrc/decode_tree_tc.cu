// R-SWA attention of a tree of drafted tokens on the 5th-generation tensor
// cores (tcgen05 + TMEM + TMA), bf16, head_dim 64 and 128.
//
// What it computes is decode_tree.cu's: node i of sequence b is output
// t_b + depth(i); it attends the prefix rows 0..m_b-1, the cached outputs at
// most min(t_b - 1, n - 2 - depth(i)) steps older than the newest, and itself
// and its ancestors fewer than n levels above.
//
// Rows: the G query heads of a KV head see the same keys, so a query tile is
// the rows (node, head of the group) of NPT = 128 / G nodes, fetched as one
// three-dimensional TMA box; a unit is the query tile of one (b, kv head) -
// split: two tensor-core halves share it and take every other key tile - or,
// where the trees have more rows than that, a pair of query tiles, one for
// each half, that read every key tile once between them.
//
// Keys: a unit's prefix rows, its ring slots and its nodes follow each other,
// each from a multiple of 16 on, and are cut into tiles of 128: a tile costs the
// same however many of its keys are real, and only those that lie in the prefix
// whole need no masks (64 sequences 84.2 -> 80.8 us, 64 grouped 123.7 -> 113.8, 51
// sequences of 85 keys 26.5 -> 16.4 when tiles of one source each gave way to
// this).  A tile of several sources is loaded in boxes of 64 and 16 keys.
//
// Work: the key tiles of a unit one after the other, unit after unit, form one
// list, which the CTAs (one per SM) cut into equal ranges.  A CTA streams its
// range through one TMA ring without draining between units; a unit that a range
// covers whole is written out at once, of another the CTA leaves a partial (m, l,
// O) in the workspace.  Each CTA leaves at most two: of the unit that a CTA before
// it began, and of the one that it begins and does not end.  The partials of a cut
// unit are joined
//   pairs, in many units: by the last of the unit's CTAs, from its own
//     accumulators where it is the one that began the unit (64 sequences of
//     32 / 8 heads and 64 nodes: 4 % less time than with the second kernel; a
//     launch without pairs has a quarter to an eighth of the partials and gains
//     nothing)
//   otherwise: by a second, dependent kernel.
// The order of a unit's partials is the same whoever joins it last.
//
// Roles (352 threads): warps 0-3 / 4-7 softmax and epilogue of half 0 / 1
// (thread r owns row r = TMEM lane r), warp 8 TMA producer, warp 9 TMEM
// allocator and MMA issuer, warp 10 planner: it cuts the list, walks the CTA's
// range ahead of the others, hands them, through shared memory, each segment
// (the part of a unit inside the range) and its nodes' depths and ancestors,
// and requests the query tiles.  Steps (a half's turn on a key tile) alternate
// between the halves through the whole range; the MMA order is QK(0) QK(1)
// PV(0) QK(2) PV(1) QK(3) ..., so the tensor core works on one half while the
// other half's softmax runs.  TMEM: S0 | S1 | O0 | O1, P over S.  O is
// rescaled lazily (threshold 2^8, exact because O and l share the reference).
// A key tile's PV takes only the 16-key steps that hold keys; value rows between
// a source's end and the next multiple of 16 are zeroed first (0 x NaN is NaN).
// Every wait is bounded; on a timeout the CTA drains its copies and MMAs, frees
// TMEM and sets the cache's device flag.
//
// What bounds it: for many sequences (64 with prefixes of 256..2048 rows,
// n 128) the issue slots of the softmax, two exchanges of 128 x 128 scores and
// weights with TMEM a tile and half, and one product at a time: 10 heads and 32
// nodes take 80.8 us where the bytes take 57.6 at the copy rate; 32 / 8 heads and
// 64 nodes 111.4, bytes 57.0, products alone 41.  For one long sequence (40 pages)
// latency: 22.8 us, of which 4.6 are state, plan and first keys, and 4.6 the
// second kernel.
#include <cuda.h>

#include <algorithm>

#include "rswa_device.cuh"
#include "tc_pipe.cuh"

namespace rswa {
namespace {

using namespace ptx;

constexpr int BM = 128, BN = 128;
constexpr int kSoftmaxThreads = 256;
constexpr int kThreads = kSoftmaxThreads + 96;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kPlanWarp = 10;
constexpr uint32_t kSub = BM * 64 * 2;         // [128][64] bf16, 128B-swizzled
constexpr int NSEG = 4;                        // segments handed over at a time
constexpr int NTT = 2;                         // tree tiles whose masks are handed over

// Shared memory.  A launch without pairs needs one query tile and so has room
// for a fifth pair of 64-column K/V slots.
template <int D, bool PAIR>
struct Smem {
  static constexpr int NSUB = D / 64;
  static constexpr uint32_t kTile = NSUB * kSub;             // a query, key or value tile
  static constexpr int NQ = PAIR ? 2 : 1;                    // query tiles
  static constexpr int NS = (PAIR ? 8 : 10) / NSUB;          // K/V ring slots
  static constexpr int NODES = PAIR ? 2 * BM : BM;           // most nodes of a unit
  static constexpr uint32_t kNodeWords = NODES * (1 + 4 * NTT);  // depths and masks
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_RING = NQ * kTile;
  static constexpr uint32_t OFF_ML = OFF_RING + NS * kTile;  // [2][2][2][128] floats
  static constexpr uint32_t OFF_BAR = OFF_ML + 2 * 2 * 2 * BM * 4;
  static constexpr uint32_t OFF_SEG = OFF_BAR + 512;
  static constexpr uint32_t OFF_PAR = OFF_SEG + NSEG * 64;   // a sequence's parents
  static constexpr uint32_t OFF_NODE = OFF_PAR + kMaxTreeNodes * 4;
  static constexpr uint32_t kBytes = OFF_NODE + 2 * kNodeWords * 4 + 1024;  // + alignment
  static_assert(kBytes <= 232448, "shared memory of a CTA");
  // barriers
  static constexpr int B_FULL = 0;                 // NS slots landed
  static constexpr int B_EMPTY = B_FULL + NS;      // and free
  static constexpr int B_QF = B_EMPTY + NS;        // NQ query tiles landed
  static constexpr int B_QE = B_QF + NQ;           // and free
  static constexpr int B_S = B_QE + NQ;            // 2 halves: S ready
  static constexpr int B_P = B_S + 2;              // 2 halves: P written
  static constexpr int B_O = B_P + 2;              // 2 halves: the segment's last PV done
  static constexpr int B_F = B_O + 2;              // the segment's O read out
  static constexpr int B_ML = B_F + 1;             // split: both halves' (m, l) in smem
  static constexpr int B_FIN = B_ML + 1;
  static constexpr int B_SEG = B_FIN + 1;          // NSEG segments handed over
  static constexpr int B_NODE = B_SEG + NSEG;      // 2 segments' nodes handed over
  static constexpr int B_NFREE = B_NODE + 2;       // and read by every row
  static constexpr int B_CUT = B_NFREE + 2;        // a cut unit's partial is written
  static constexpr int B_JOIN = B_CUT + 1;         // and who joins it is known
  static constexpr int B_ASK = B_JOIN + 1;         // the same before it is written
  static constexpr int NBAR = B_ASK + 1;
  static_assert(8 * NBAR + 24 <= 512, "barriers");
};

__host__ __device__ constexpr uint32_t tm_s(int half) { return half ? 128u : 0u; }
__host__ __device__ constexpr uint32_t tm_o(int half) { return half ? 384u : 256u; }
constexpr uint32_t TM_COLS = 512;
constexpr int kTurnUnroll = 1;                 // rolled softmax loop
constexpr float kRescaleThreshold = 8.0f;      // log2 units
constexpr uint64_t kWaitLimitNs = 1000000000ull;

// The work list is cut by cost.  Every key tile costs 1, a partial one too: a
// step takes as long as its chain of matrix products and softmax, about the time
// in which an SM's share of HBM brings a whole tile.  A unit's first tile carries
// the unit's start and end as well.  Fitted over the CTAs of a launch (time from
// the dependency wait to the end): 64 sequences of 10 heads and 32 nodes 1.1 us a
// tile and 3.0 us a segment, 64 of 32 / 8 heads and 64 nodes (pairs) 2.05 and 5.2
// us.  A CTA's share is never below kMinCost, so that it holds a tile at least.
constexpr int kUnitCost = 3, kPairUnitCost = 2, kMinCost = 4;
static_assert(kMinCost >= 1 + kUnitCost && kUnitCost >= kPairUnitCost, "a share holds a tile");

// The shape of a launch.
struct Shape {
  int npt;      // nodes of a query tile
  int box;      // nodes of its loads: fewer where no tree has so many
  int pair;     // 1: units of two query tiles
  int G;        // query heads of a KV head
  int evict;    // 1: cache tiles are loaded evict-first
  int flat;     // 1: a CTA for every unit, no unit is cut
  int inl;      // 1: the last CTA of a cut unit joins it, no second kernel
  int joins;    // units of the launch, or its CTAs where those are fewer
};

// What a sequence adds to the work list: `units` units of `tl` key tiles each.
struct Seq {
  int cnt, m_b, ring;
  int64_t t_b;
  int p16, r16, tl, units, extra;
  __device__ __forceinline__ void load(const CacheView& cv, const TreeArgs& a, const Shape& sh,
                                       int b) {
    const int c = a.counts ? a.counts[b] : a.nodes;        // one round trip with m_b and t_b
    m_b = cv.m_dev[b];
    t_b = cv.t_dev[(size_t)b * cv.H];
    cnt = min(max(c, 0), a.nodes);
    if (c != cnt) flag_error(cv.err, kErrBadTree);
    ring = (int)min(min(cv.n, t_b), (int64_t)1 << 30);
    p16 = (m_b + 15) & ~15;
    r16 = (ring + 15) & ~15;
    tl = (p16 + r16 + cnt + BN - 1) / BN;
    extra = sh.pair ? kPairUnitCost : kUnitCost;
    const int per = sh.npt << sh.pair;
    units = (cnt + per - 1) / per * cv.Hkv;
  }
  __device__ int cost(bool flat) const { return flat ? 1 : tl + extra; }   // of a unit
  // Cost of a unit's tiles before tile j, and the first tile that begins at or
  // after cost x (tl: none).  Where no unit is cut, a unit costs 1 as a whole.
  __device__ int before(int j, bool flat) const {
    return j > 0 ? (flat ? 1 : j + extra) : 0;
  }
  __device__ int at(int x, bool flat) const {
    return x <= 0 ? 0 : (flat ? tl : min(max(x - extra, 1), tl));
  }
};

// A segment as the planner hands it over.
struct Segment {
  int b, kvh, node0, cnt;
  int j0, j1;             // key tiles of the unit inside the range; j1 = 0: no more segments
  int p16, t0;            // where the ring's and the tree's keys begin
  int m_b, ring;          // prefix rows, filled ring slots
  int newest, age;        // ring slot of output t_b - 1, and t_b - 1 (clamped)
  uint8_t split, whole, begins, pad;
  int first, last;        // the CTAs that a cut unit begins and ends in
  int tiles;              // the CTA's key tiles before the segment
  // Key x of the unit: prefix row x from 0, ring slot x - p16 from p16, node
  // x - t0 from t0 to the end; p16 and t0 are multiples of 16.
  __device__ int end() const { return t0 + cnt; }
  __device__ int keys(int j) const { return min(BN, end() - j * BN); }   // of tile j
};
static_assert(sizeof(Segment) <= 64, "segment");

// Waits for a segment: its key tiles, and whether it is split in bit 24; 0: no
// more segments, or the wait gave up.
__device__ __noinline__ int enter_segment(uint32_t b, uint32_t phase, const Segment* w,
                                          volatile int* abort_flag, uint64_t ns) {
  if (!mbar_wait(b, phase, abort_flag, ns) || w->j1 == 0) return 0;
  return (w->j1 - w->j0) | w->split << 24;
}

// The join of the cut units is done by the CTAs of a second kernel, one list
// entry for each CTA of the first: the unit that CTA begins and does not end.
struct JoinDesc {
  int b, node0, kvh, last;      // last CTA with a part of the unit; -1: none
  int cnt, pad[3];
};
static_assert(sizeof(JoinDesc) == 32, "join entry");

// A partial: O as [D/4][rows] float4 (a warp's rows are contiguous), then m
// and l [rows].
__host__ __device__ constexpr size_t partial_floats(int D, int pair) {
  return (size_t)(BM << pair) * (D + 2);
}
__device__ __forceinline__ float* partial_at(void* ws, int grid, int slot, int D, int pair) {
  return reinterpret_cast<float*>(static_cast<char*>(ws) +
                                  ((size_t)grid * sizeof(JoinDesc) + 255) / 256 * 256) +
         (size_t)slot * partial_floats(D, pair);
}

// x += wp times the partial's columns 32 c .. 32 c + 31 of the row.
template <int D, bool PAIR>
__device__ __forceinline__ void add_partial(const float* part, int prow, int c, float wp,
                                            float* x) {
  constexpr int prows = BM << (PAIR ? 1 : 0);
  const float4* src = reinterpret_cast<const float4*>(part) + prow;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float4 v = __ldcg(src + (size_t)(c * 8 + e) * prows);
    x[4 * e] = fmaf(v.x, wp, x[4 * e]);
    x[4 * e + 1] = fmaf(v.y, wp, x[4 * e + 1]);
    x[4 * e + 2] = fmaf(v.z, wp, x[4 * e + 2]);
    x[4 * e + 3] = fmaf(v.w, wp, x[4 * e + 3]);
  }
}

// A row's columns from the partials of CTAs first .. last, as the CTA that begins
// a unit joins them to its own O, term by term in the same order.
template <int D, bool PAIR>
__device__ __noinline__ void join_row(void* ws, int grid, int first, int last, int prow, int c_lo,
                                      int c_hi, __nv_bfloat16* orow, float* lse) {
  constexpr int prows = BM << (PAIR ? 1 : 0);
  auto part = [&](int p) { return partial_at(ws, grid, 2 * p + (p == first ? 1 : 0), D, PAIR); };
  auto m_of = [&](int p) { return __ldcg(part(p) + (size_t)prows * D + prow); };
  float top = m_of(first);
  for (int p = first + 1; p <= last; ++p) top = fmaxf(top, m_of(p));
  const float wf = ex2(m_of(first) - top);
  float L = __ldcg(part(first) + (size_t)prows * (D + 1) + prow) * wf;
  for (int p = first + 1; p <= last; ++p)
    L = fmaf(__ldcg(part(p) + (size_t)prows * (D + 1) + prow), ex2(m_of(p) - top), L);
#pragma unroll 1
  for (int c = c_lo; c < c_hi; ++c) {
    float x[32];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(part(first)) + prow +
                              (size_t)(c * 8 + e) * prows);
      x[4 * e] = v.x * wf;
      x[4 * e + 1] = v.y * wf;
      x[4 * e + 2] = v.z * wf;
      x[4 * e + 3] = v.w * wf;
    }
#pragma unroll 1
    for (int p = first + 1; p <= last; ++p)
      add_partial<D, PAIR>(part(p), prow, c, ex2(m_of(p) - top), x);
    store_columns(orow + c * 32, x, 1.f / L);
  }
  if (lse) *lse = (top + log2f(L)) * kLn2;
}

template <int D, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
decode_tree_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmKc,
                      const __grid_constant__ CUtensorMap tmVc,
                      const __grid_constant__ CUtensorMap tmKt,
                      const __grid_constant__ CUtensorMap tmVt,
                      const __grid_constant__ CUtensorMap tmKc16,
                      const __grid_constant__ CUtensorMap tmVc16,
                      const __grid_constant__ CUtensorMap tmKt16,
                      const __grid_constant__ CUtensorMap tmVt16,
                      const __grid_constant__ CUtensorMap tmKc64,
                      const __grid_constant__ CUtensorMap tmVc64, CacheView cv, TreeArgs a,
                      Shape sh, uint64_t wait_ns) {
  using SM = Smem<D, PAIR>;
  constexpr int NSUB = SM::NSUB, NS = SM::NS, NQ = SM::NQ, NODES = SM::NODES;
  constexpr uint32_t kTile = SM::kTile;
  constexpr int NBAR = SM::NBAR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t bar0 = sb + SM::OFF_BAR;
  auto bar = [&](int k) { return bar0 + 8u * (uint32_t)k; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::OFF_BAR + 8 * NBAR);
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(smem + SM::OFF_BAR + 8 * NBAR + 4);
  // Whether this CTA joins a cut unit: two it counted itself in, one it asked for.
  volatile int* joiner = reinterpret_cast<volatile int*>(smem + SM::OFF_BAR + 8 * NBAR + 12);
  volatile int* never = reinterpret_cast<volatile int*>(smem + SM::OFF_BAR + 8 * NBAR + 8);
  const Segment* segs = reinterpret_cast<const Segment*>(smem + SM::OFF_SEG);
  int32_t* nodes_smem = reinterpret_cast<int32_t*>(smem + SM::OFF_NODE);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, grid = gridDim.x;

  if (threadIdx.x == 0) {
    for (int k = 0; k < NBAR; ++k)
      mbar_init(bar(k), k == SM::B_P || k == SM::B_P + 1
                           ? 128u
                           : (k == SM::B_F || k == SM::B_ML || (k >= SM::B_NFREE && k <= SM::B_CUT)
                                  ? 256u
                                  : 1u));
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
  // Segment k, from the planner; false: the wait gave up.
  auto segment = [&](int k, Segment& w) {
    if (!wait_for(bar(SM::B_SEG + k % NSEG), (k / NSEG) & 1, abort_flag, wait_ns)) return false;
    w = segs[k % NSEG];
    return true;
  };

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&tmKc);
      prefetch_tmap(&tmVc);
      prefetch_tmap(&tmKt16);
      prefetch_tmap(&tmVt16);
      prefetch_tmap(&tmKc16);
      prefetch_tmap(&tmVc16);
      prefetch_tmap(&tmKc64);
      prefetch_tmap(&tmVc64);
      const uint64_t normal = evict_normal_policy();
      const uint64_t stream = sh.evict ? evict_first_policy() : normal;
      uint32_t gi = 0;                           // loads issued
      bool ok = true;
      Segment w;
      for (int k = 0; ok && segment(k, w) && w.j1 > 0; ++k) {
        const int64_t slab0 = ((int64_t)w.b * cv.Hkv + w.kvh) * cv.slab_rows;
        for (int j = w.j0; ok && j < w.j1; ++j) {
          const int x0 = j * BN, boxes = (w.keys(j) + 15) / 16;
          // one box of 128 keys where they have one source, or boxes of 64 and 16
          const bool whole = boxes == BN / 16 && (x0 + BN <= w.p16 || x0 >= w.t0 ||
                                                  (x0 >= w.p16 && x0 + BN <= w.t0));
#pragma unroll 1
          for (int isv = 0; isv < 2; ++isv, ++gi) {
            const uint32_t s = gi % NS;
            if (gi >= (uint32_t)NS &&
                !wait_for(bar(SM::B_EMPTY + s), ((gi / NS) - 1) & 1, abort_flag, wait_ns)) {
              ok = false;
              break;
            }
            const uint32_t dst = sb + SM::OFF_RING + s * kTile;
            mbar_arrive_expect_tx(bar(SM::B_FULL + s), (uint32_t)NSUB * boxes * 2048u);
#pragma unroll 1
            for (int r = 0; r < boxes;) {
              const int x = x0 + 16 * r;
              const bool tree = x >= w.t0;
              const int groups =                         // of 16 keys
                  whole ? BN / 16
                        : (!tree && r + 4 <= boxes && x + 64 <= (x < w.p16 ? w.p16 : w.t0)) ? 4 : 1;
              const CUtensorMap* map =
                  whole ? (tree ? (isv ? &tmVt : &tmKt) : (isv ? &tmVc : &tmKc))
                        : tree ? (isv ? &tmVt16 : &tmKt16)
                               : groups == 4 ? (isv ? &tmVc64 : &tmKc64) : (isv ? &tmVc16 : &tmKc16);
              const int col = tree ? w.kvh * D : 0;
              const int row = tree ? w.b * a.nodes + x - w.t0
                                   : (int)(slab0 + (x < w.p16 ? x : cv.m_cap + x - w.p16));
#pragma unroll
              for (int c = 0; c < NSUB; ++c)
                tma_load_2d_pol(dst + c * kSub + r * 2048, map, col + c * 64, row,
                                bar(SM::B_FULL + s), tree ? normal : stream);
              r += groups;
            }
          }
        }
      }
      // Drain: every copy issued has landed before the CTA may exit.
      for (uint32_t k = gi > (uint32_t)NS ? gi - NS : 0; k < gi; ++k)
        wait_for(bar(SM::B_FULL + k % NS), (k / NS) & 1, never, kWaitLimitNs);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // One lane issues.  Step s: PV of step s - 2, then QK of step s, both of half
    // s & 1.  What the lane does between the products holds the tensor core up
    // (2400 cycles a step with 1200 of them in products), so waits are made
    // where their answer can be new only, descriptors advance by constants, and
    // the rare paths are out of line.
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_bf16(BM, BN, false);
      constexpr uint32_t idesc_pv = idesc_bf16(BM, D, true);
      auto wait = [&](int k, uint32_t phase) {
        return wait_for(bar(k), phase & 1, abort_flag, wait_ns);
      };
      // Load 2 t is the key tile of the CTA's tile t, load 2 t + 1 its value
      // tile: `slot` and `phase` of the one a cursor is at.
      struct Cursor {
        int k = 0, left;                 // segment, its tiles left
        bool split, second = false;      // in a pair unit: the second half's turn
        uint32_t slot, phase = 0, q = 0; // q: query tiles before
      };
      auto enter = [&](Cursor& c) {
        const int x = enter_segment(bar(SM::B_SEG + c.k % NSEG), (c.k / NSEG) & 1,
                                    &segs[c.k % NSEG], abort_flag, wait_ns);
        c.left = x & 0xffffff;
        c.split = x >> 24;
        return x != 0;
      };
      auto advance = [&](Cursor& c) {    // false: no more steps
        if (!c.split && !c.second) {
          c.second = true;
          return true;
        }
        c.second = false;
        c.slot += 2;
        if (c.slot >= (uint32_t)NS) {
          c.slot -= NS;
          c.phase ^= 1;
        }
        if (--c.left > 0) return true;
        c.q += c.split ? 1 : 2;
        ++c.k;
        return enter(c);
      };
      Cursor qc, pc;
      qc.slot = 0;
      pc.slot = 1;
      bool qmore = enter(qc), pmore = enter(pc);
      int pfresh = 2, qfresh = 2;        // steps until both halves have had one
      if (pmore && pc.split && pc.left == 1) pfresh = 1;
      if (qmore && qc.split && qc.left == 1) qfresh = 1;
      const uint64_t qdesc = desc_sw128(sb + SM::OFF_Q, 16, 1024);
      const uint64_t kdesc = desc_sw128(sb + SM::OFF_RING, 16, 1024);
      const uint64_t vdesc = desc_sw128(sb + SM::OFF_RING, kSub, 1024);
      // The segment's tiles, and of these, from the first on, those of 128 keys.
      int nf = pmore ? segs[0].end() / BN - segs[0].j0 : 0, tl = pc.left;
#pragma unroll 1
      for (uint32_t s = 0; pmore; ++s) {
        const uint32_t half = s & 1;
        if (s >= 2) {
          const bool first = pfresh > 0, last = pc.left <= (pc.split ? 2 : 1);
          if (first) {
            --pfresh;
            if (pc.k > 0 && !wait(SM::B_F, pc.k - 1)) break;
          }
          if (!wait(SM::B_P + half, (s >> 1) - 1)) break;
          if (!pc.second && !wait(SM::B_FULL + pc.slot, pc.phase)) break;
          tc_fence_after();
          const uint64_t vd = vdesc + (uint64_t)(pc.slot * (kTile >> 4));
          if (tl - pc.left < nf) {
#pragma unroll
            for (int k = 0; k < BN / 16; ++k)
              mma_bf16_ts(tmem + tm_o(half), tmem + tm_s(half) + k * 8, vd + k * 128, idesc_pv,
                          k > 0 ? 1u : (first ? 0u : 1u));
          } else {
            const Segment& w = segs[pc.k % NSEG];
            const int keys = w.keys(w.j1 - pc.left);
#pragma unroll 1
            for (int k = 0; 16 * k < keys; ++k)
              mma_bf16_ts(tmem + tm_o(half), tmem + tm_s(half) + k * 8, vd + k * 128, idesc_pv,
                          (!first || k > 0) ? 1u : 0u);
          }
          if (pc.split || pc.second) mma_commit(bar(SM::B_EMPTY + pc.slot));
          if (last) mma_commit(bar(SM::B_O + half));
          const int at = pc.k;
          pmore = advance(pc);
          if (pc.k != at) {
            pfresh = pc.split && pc.left == 1 ? 1 : 2;
            nf = segs[pc.k % NSEG].end() / BN - segs[pc.k % NSEG].j0;
            tl = pc.left;
          }
        }
        if (qmore) {
          // S = Q K^T
          const uint32_t qt = qc.split ? qc.q : qc.q + half;
          if (qfresh > 0) {
            --qfresh;
            if (!wait(SM::B_QF + qt % NQ, qt / NQ)) break;
          }
          if (!qc.second && !wait(SM::B_FULL + qc.slot, qc.phase)) break;
          tc_fence_after();
          const uint64_t kd = kdesc + (uint64_t)(qc.slot * (kTile >> 4));
          const uint64_t qd = qdesc + (uint64_t)((qt % NQ) * (kTile >> 4));
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * kSub + (k & 3) * 32) >> 4;
            mma_bf16_ss(tmem + tm_s(half), qd + off, kd + off, idesc_qk, k > 0);
          }
          mma_commit(bar(SM::B_S + half));
          if (qc.split || qc.second) {
            mma_commit(bar(SM::B_EMPTY + qc.slot));
            if (qc.left == 1) {
              mma_commit(bar(SM::B_QE + qc.q % NQ));
              if (!qc.split) mma_commit(bar(SM::B_QE + (qc.q + 1) % NQ));
            }
          }
          const int at = qc.k;
          qmore = advance(qc);
          if (qc.k != at) qfresh = qc.split && qc.left == 1 ? 1 : 2;
        }
      }
      // Drain: all MMAs of this CTA have finished before TMEM is freed.
      mma_commit(bar(SM::B_FIN));
      wait_for(bar(SM::B_FIN), 0, never, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == kPlanWarp) {
    // ------------------------------------------------------------ planner
    Segment* out = reinterpret_cast<Segment*>(smem + SM::OFF_SEG);
    int32_t* par = reinterpret_cast<int32_t*>(smem + SM::OFF_PAR);
    if (lane == 0) prefetch_tmap(&tmQ);
    int qi = 0, tiles = 0;                       // query tiles requested, key tiles planned
    // Requests a segment's query tiles once their buffers are free.
    auto queries = [&](const Segment& w) {
      for (int x = 0; x < (w.split ? 1 : 2); ++x, ++qi) {
        const int s = qi % NQ;
        if (qi >= NQ && !__all_sync(0xffffffffu, wait_for(bar(SM::B_QE + s), (qi / NQ - 1) & 1,
                                                           abort_flag, wait_ns)))
          return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(SM::B_QF + s), (uint32_t)NSUB * sh.box * sh.G * 128u);
#pragma unroll
          for (int c = 0; c < NSUB; ++c)
            tma_load_3d(sb + SM::OFF_Q + s * kTile + c * kSub, &tmQ, c * 64, w.kvh * sh.G,
                        w.b * a.nodes + w.node0 + x * sh.npt, bar(SM::B_QF + s));
        }
        __syncwarp();
      }
      return true;
    };
    const bool flat = sh.flat != 0;
    // The list's length, and the sequences of each lane in it.
    const int per = (cv.B + 31) / 32;
    const int b_lo = min(lane * per, cv.B), b_hi = min(b_lo + per, cv.B);
    Seq sq;
    int mine = 0, my_units = 0;
#pragma unroll 2
    for (int b = b_lo; b < b_hi; ++b) {
      sq.load(cv, a, sh, b);
      mine += sq.cost(flat) * sq.units;
      my_units += sq.units;
    }
    int inc = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += x;
    }
    const int total = __shfl_sync(0xffffffffu, inc, 31);
    const int units = __reduce_add_sync(0xffffffffu, my_units);
    // CTA c takes the tiles that begin in [from(c), from(c + 1)).  Few units have
    // the same number of CTAs each, if they are alike: their ends meet CTAs' ends.
    int ctas = min(grid, max(1, flat ? total : total / kMinCost));
    if (units > 0 && units < ctas) ctas -= ctas % units;
    const bool small = total < 1 << 22;          // c * total fits 32 bits
    const int each = total / ctas, rem = total - each * ctas;
    auto from = [&](int c) {
      return small ? (int)((uint32_t)c * (uint32_t)total / (uint32_t)ctas)
                   : c * each + min(c, rem);
    };
    // The last CTA that begins at or before cost x.
    auto owner = [&](int x) {
      if (small) return (int)(((uint32_t)(x + 1) * (uint32_t)ctas - 1) / (uint32_t)total);
      const int cut = rem * (each + 1);
      return min(ctas - 1, x < cut ? x / (each + 1) : rem + (x - cut) / each);
    };
    JoinDesc jd = {0, 0, 0, -1, 0, {0, 0, 0}};
    int k = 0;
    if (cta < ctas && total > 0) {
      const int x0 = from(cta), x1 = from(cta + 1);
      // The sequence that x0 is in, and where it begins.
      int b = 0, base = 0;
      const bool here = inc - mine <= x0 && x0 < inc;
      if (here) {
        base = inc - mine;
        b = b_lo;
        if (per > 1) {
          for (;; ++b) {
            sq.load(cv, a, sh, b);
            if (x0 < base + sq.cost(flat) * sq.units) break;
            base += sq.cost(flat) * sq.units;
          }
        }
      }
      const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
      b = __shfl_sync(0xffffffffu, b, src);
      base = __shfl_sync(0xffffffffu, base, src);
      sq.load(cv, a, sh, b);
      int u = (x0 - base) / sq.cost(flat);
      int ubase = base + u * sq.cost(flat);            // where unit u begins
      int j0 = sq.at(x0 - ubase, flat), par_b = -1;
      const int unit_nodes = sh.npt << sh.pair;
      const int n = (int)min(cv.n, (int64_t)1 << 30);
      for (bool next_unit = j0 == sq.tl;; next_unit = true) {
        if (next_unit) {
          ubase += sq.cost(flat);
          j0 = 0;
          if (++u == sq.units) {
            u = 0;
            sq.units = 0;
            while (sq.units == 0 && b + 1 < cv.B) sq.load(cv, a, sh, ++b);
            if (sq.units == 0) break;            // the list's end
          }
        }
        if (ubase + sq.before(j0, flat) >= x1) break;  // a later CTA's
        Segment w;
        w.b = b;
        w.kvh = u % cv.Hkv;
        w.node0 = u / cv.Hkv * unit_nodes;
        w.cnt = sq.cnt;
        w.j0 = j0;
        w.j1 = sq.at(x1 - ubase, flat);
        w.p16 = sq.p16;
        w.t0 = sq.p16 + sq.r16;
        w.m_b = sq.m_b;
        w.ring = sq.ring;
        w.age = (int)min(sq.t_b - 1, (int64_t)1 << 30);
        w.newest = sq.t_b <= cv.n ? (int)sq.t_b - 1
                   : sq.t_b < (int64_t)1 << 31
                       ? (int)((uint32_t)(sq.t_b - 1) % (uint32_t)cv.n)
                       : (int)((sq.t_b - 1) % cv.n);
        // A unit without rows for a second query tile is split like all
        // others of a launch without pairs.
        w.split = !PAIR || w.node0 + sh.npt >= sq.cnt;
        w.whole = j0 == 0 && w.j1 == sq.tl;
        w.begins = j0 == 0;
        w.first = w.last = cta;
        if (!w.whole) {
          w.first = owner(ubase);
          w.last = owner(ubase + sq.before(sq.tl - 1, flat));
        }
        w.tiles = tiles;
        tiles += w.j1 - j0;
        // Slot k % NSEG was segment k - 4's: all roles had left it when the
        // nodes of segment k - 1 were handed over (which waited until those
        // of segment k - 3 had been read).
        if (lane == 0) {
          out[k % NSEG] = w;
          mbar_arrive(bar(SM::B_SEG + k % NSEG));
        }
        // The first segment's queries come at once, a later one's after its
        // nodes: their buffers are free later than those.
        if (k == 0) queries(w);
        if (j0 == 0 && !w.whole && !sh.inl)  // begun here, ended by the CTA of its last tile
          jd = {b, w.node0, w.kvh, w.last, sq.cnt, {0, 0, 0}};
        // Depths and ancestors of the unit's nodes, where the segment's ring
        // and tree tiles ask for them.
        const bool ask = w.j1 * BN > sq.p16;
        if (ask && par_b != b) {
          __syncwarp();
          for (int i = lane; i < sq.cnt; i += 32) par[i] = a.parents[(size_t)b * a.nodes + i];
          par_b = b;
          __syncwarp();
        }
        if (k >= 2 &&
            !__all_sync(0xffffffffu, wait_for(bar(SM::B_NFREE + (k & 1)), ((k >> 1) - 1) & 1,
                                               abort_flag, wait_ns)))
          break;
        int32_t* nd = nodes_smem + (k & 1) * SM::kNodeWords;
        const int nn = ask ? min(unit_nodes, sq.cnt - w.node0) : 0;
        for (int i = lane; i < nn; i += 32) {
          uint64_t m[2 * NTT];
#pragma unroll
          for (int e = 0; e < 2 * NTT; ++e) m[e] = 0u;
          int up = 0;
          for (int x = w.node0 + i;;) {
            const uint64_t bit = up < n ? (uint64_t)1 << (x & 63) : 0;
#pragma unroll
            for (int e = 0; e < 2 * NTT; ++e) m[e] |= x >> 6 == e ? bit : 0;
            const int p = par[x];
            if (p < -1 || p >= x) flag_error(cv.err, kErrBadTree);
            if (p < 0 || p >= x) break;
            x = p;
            ++up;
          }
          nd[i] = up;
#pragma unroll
          for (int e = 0; e < 4 * NTT; ++e)
            nd[(1 + e) * NODES + i] = (int32_t)(uint32_t)(m[e >> 1] >> (e & 1 ? 32 : 0));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(SM::B_NODE + (k & 1)));
        if (k > 0 && !queries(w)) break;
        ++k;
      }
    }
    if (lane == 0) {
      out[k % NSEG].j1 = 0;              // no more segments
      mbar_arrive(bar(SM::B_SEG + k % NSEG));
      if (!flat && !sh.inl) static_cast<JoinDesc*>(a.ws)[cta] = jd;
      // Drain: every copy issued has landed before the CTA may exit.
      for (int x = max(qi - NQ, 0); x < qi; ++x)
        wait_for(bar(SM::B_QF + x % NQ), (x / NQ) & 1, never, kWaitLimitNs);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------- softmax and epilogue
    const int half = warp >> 2;
    const int r = threadIdx.x & 127;                    // row of the query tile
    const int rg = r / sh.G, hg = r - rg * sh.G;        // its node in the tile, its head
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const float sl2 = rsqrtf((float)D) * kLog2e;
    const uint32_t s_addr = tmem + lane_off + tm_s(half);
    const uint32_t o_addr = tmem + lane_off + tm_o(half);
    const int n = (int)min(cv.n, (int64_t)1 << 30);
    float* ml = reinterpret_cast<float*>(smem + SM::OFF_ML);
    uint32_t step = 0, turns = 0;                       // steps before; this half's among them
    uint32_t o_phase0 = 0, o_phase1 = 0, ml_phase = 0;  // segments with steps of each half; split
    uint32_t cut_phase = 0;                             // cut units left to a join (at most 2)
    bool ok = true;
    Segment w;
    for (int k = 0;; ++k) {
      if (!__all_sync(0xffffffffu, segment(k, w)) || w.j1 == 0) break;
      const bool split = w.split != 0;
      const int nseg = w.j1 - w.j0;
      const int ni = (split ? 0 : half * sh.npt) + rg;  // node of the unit
      const int node = w.node0 + ni;
      const bool live = rg < sh.npt && node < w.cnt;
      const bool any = __any_sync(0xffffffffu, live);
      const int32_t* nd = nodes_smem + (k & 1) * SM::kNodeWords;
      // The planner's depths and masks, first asked for by a ring or tree tile.
      bool have = false;
      auto nodes = [&]() {
        if (!have)
          have = __all_sync(0xffffffffu, wait_for(bar(SM::B_NODE + (k & 1)), (k >> 1) & 1,
                                                   abort_flag, wait_ns));
        return have;
      };
      const int r0 = w.newest;
      float m_run = -INFINITY, l_run = 0.f;
      bool started = false;
      for (int j = w.j0; j < w.j1; ++j) {
        if (split && ((step + (uint32_t)(j - w.j0)) & 1) != (uint32_t)half) continue;
        const int x0 = j * BN;
        const bool full = x0 + BN <= w.m_b;              // every column is a key of every row
        if (x0 + BN > w.p16 && !nodes()) {
          ok = false;
          break;
        }
        // The row's keys among the tile's columns, while S is on its way.
        uint32_t see0 = 0u, see1 = 0u, see2 = 0u, see3 = 0u;
        if (any && !full) {
          // Ring slot s is a key iff its age (r0 - s) mod n is at most lim.
          const int rc = w.p16 - x0, tc = w.t0 - x0;     // columns of slot 0 and node 0
          int a1 = 0, b1 = -1, a2 = 0, b2 = -1;
          if (x0 < w.t0 && x0 + BN > w.p16) {
            const int lim = min(w.age, n - 2 - (live ? nd[ni] : 0));
            if (lim >= 0) {
              a1 = max(r0 - lim, 0) + rc;
              b1 = r0 + rc;
              if (r0 < lim) {
                a2 = r0 - lim + n + rc;
                b2 = n - 1 + rc;
              }
            }
          }
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t see = 0u;
            if (32 * c < w.m_b - x0) see = range_mask(0, w.m_b - 1 - x0, c);
            if (32 * c + 32 > rc && 32 * c < tc)
              see |= range_mask(a1, b1, c) | range_mask(a2, b2, c);
            const int c0 = 32 * c - tc;                  // the chunk's first node
            if (live && c0 > -32 && c0 < w.cnt) {
              if (c0 + 32 <= BN * NTT) {
                const int i = c0 >> 5;                   // -1: nodes from column 16 on
                const uint32_t lo = i < 0 ? 0u : (uint32_t)nd[(1 + i) * NODES + ni];
                const uint32_t hi = c0 & 31 ? (uint32_t)nd[(2 + i) * NODES + ni] : 0u;
                see |= __funnelshift_r(lo, hi, c0 & 31);
              } else {
                // far nodes of a large tree: walk up from the row's
                const int32_t* par = a.parents + (size_t)w.b * a.nodes;
                int up = 0;
                for (int x = node; x >= c0 && up < n; ++up) {
                  if (x < c0 + 32) see |= 1u << (x - c0);
                  const int p = par[x];
                  if (p >= x) break;
                  x = p;
                }
              }
            }
            see0 = see1;
            see1 = see2;
            see2 = see3;
            see3 = see;
          }
        }
        if (!__all_sync(0xffffffffu,
                        wait_for(bar(SM::B_S + half), turns & 1, abort_flag, wait_ns))) {
          ok = false;
          break;
        }
        ++turns;
        tc_fence_after();
        if (any) {
          // Pass 1: the row's maximum; scores of columns that are no keys of it
          // become -inf.  Both passes are short rolled loops: this many warps do
          // not hide the fetch of straight-line code (a turn took 4000-8000
          // cycles unrolled, 2000 rolled).
          float mx[2] = {-INFINITY, -INFINITY};
          uint32_t va[32], vb[32];
          auto maxima = [&](const uint32_t* v) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              mx[0] = fmax3(mx[0], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              mx[1] = fmax3(mx[1], __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
            }
          };
          if (full) {
            tmem_ld32(s_addr, va);
#pragma unroll 1
            for (int c = 0; c < 128; c += 64) {
              tmem_wait_ld32(va);
              tmem_ld32(s_addr + c + 32, vb);
              maxima(va);
              tmem_wait_ld32(vb);
              tmem_ld32(s_addr + ((c + 64) & 127), va);
              maxima(vb);
            }
            tmem_wait_ld32(va);                          // columns 0-31, for pass 2
          } else {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t see = see0;
              see0 = see1;
              see1 = see2;
              see2 = see3;
              tmem_ld32_sync(s_addr + 32 * c, va);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(see >> e & 1u)) va[e] = 0xff800000u;
              tmem_st32(s_addr + 32 * c, va);
              maxima(va);
            }
            tmem_wait_st();
            tmem_ld32_sync(s_addr, va);
          }
          // The reference of a row's exponentials stays until a score exceeds
          // it by more than 2^8 (any reference gives the same o and lse); then O
          // and l are rescaled.  O_h is stable here: S_h of this step completing
          // implies that the half's PV before it has.
          const float tmax = fmaxf(mx[0], mx[1]) * sl2;
          const bool over = tmax > m_run + kRescaleThreshold;      // also where m_run is -inf
          if (__any_sync(0xffffffffu, over)) {
            const float alpha = over ? ex2(m_run - tmax) : 1.f;
            if (over) m_run = tmax;
            l_run *= alpha;
#pragma unroll 1
            for (int c = 0; started && c < D; c += 32) {
              tmem_ld32_sync(o_addr + c, vb);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                vb[e] = __float_as_uint(__uint_as_float(vb[e]) * alpha);
              tmem_st32(o_addr + c, vb);
            }
          }
          // Pass 2: P, over columns of S already read, and its sum.  P is rounded to
          // bf16 for the product with V, whose two operands are of one 16-bit type;
          // l sums it unrounded.  64 sequences of 10 heads and 32 nodes: o is off
          // by 0.0023 relative to 64 bits, 0.0017 of it o's own rounding.
          const float nref = (m_run == -INFINITY) ? 0.f : -m_run;
          const uint64_t sl2x2 = f2_pack(sl2, sl2), nref2 = f2_pack(nref, nref);
          uint64_t ps2 = 0;
          auto exponentials = [&](const uint32_t* v, uint32_t to) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])),
                               sl2x2, nref2),
                        x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              ps2 = f2_add(ps2, f2_pack(p0, p1));
              p[e] = pack_bf16(p0, p1);
            }
            tmem_st16(to, p);
          };
#pragma unroll kTurnUnroll
          for (int c = 0; c < 2; ++c) {
            tmem_ld32(s_addr + 64 * c + 32, vb);
            exponentials(va, s_addr + 32 * c);
            tmem_wait_ld32(vb);
            if (c == 0) tmem_ld32(s_addr + 64, va);
            exponentials(vb, s_addr + 32 * c + 16);
            tmem_wait_ld32(va);
          }
          float s0, s1;
          f2_unpack(ps2, s0, s1);
          l_run += s0 + s1;
          tmem_wait_st();
          tc_fence_before();
        }
        started = true;
        // Value rows from key e, a source's end, to the next multiple of 16 are no
        // keys of any row (of the tree, nodes past the count or the next
        // sequence's) and may hold anything: zero, as 0 x NaN is NaN.
        const int e1 = w.p16 + w.ring, e2 = w.end();
        auto ends = [&](int e) { return (e & 15) != 0 && e >> 7 == j; };
        if ((warp & 3) == 0 && (ends(w.m_b) || ends(e1) || ends(e2))) {
          const uint32_t vi = 2u * (uint32_t)(w.tiles + j - w.j0) + 1u;
          if (__all_sync(0xffffffffu, wait_for(bar(SM::B_FULL + vi % NS), (vi / NS) & 1,
                                                abort_flag, wait_ns))) {
#pragma unroll 1
            for (int i = 0; i < 3; ++i) {
              const int e = i == 0 ? w.m_b : i == 1 ? e1 : e2;
              if (!ends(e)) continue;
              uint8_t* v = smem + SM::OFF_RING + (vi % NS) * kTile + (e & 112) * 128 + lane * 16;
#pragma unroll
              for (int x = 0; x < 16; x += 4)            // a row is 8 lanes
                if (x + (lane >> 3) >= (e & 15)) {
#pragma unroll
                  for (int c = 0; c < NSUB; ++c)
                    *reinterpret_cast<uint4*>(v + x * 128 + c * kSub) = make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();
          }
        }
        mbar_arrive(bar(SM::B_P + half));
      }
      ok = ok && nodes();                                // keeps step with the planner
      mbar_arrive(bar(SM::B_NFREE + (k & 1)));
      // ------------------------------------------------------- epilogue
      // Steps of this half and of the other in this segment.
      const int own = !split ? nseg : ((step & 1) == (uint32_t)half ? (nseg + 1) / 2 : nseg / 2);
      const int other = split ? nseg - own : nseg;
      auto wait_all = [&](int b, uint32_t phase) {
        return __all_sync(0xffffffffu, wait_for(bar(b), phase & 1, abort_flag, wait_ns)) != 0;
      };
      // A cut unit is joined by the last of its CTAs to get here (inl; else by the
      // second kernel): the one that begins it, as a rule, as the others come to
      // it at the start of their ranges.  It then takes their partials from L2 to
      // its own O as it writes the rows, and leaves none itself.  It asks early:
      // the answer comes while the other half's last step runs.
      const bool counted = PAIR && sh.inl && !w.whole;
      int32_t* count = cv.cnt_bh + (size_t)w.b * cv.H + (size_t)w.kvh * sh.G +
                       w.node0 / (sh.npt << sh.pair);
      const bool ask = ok && counted && w.begins;
      if (ask && threadIdx.x == 0) {                    // once a launch: its last unit
        joiner[2] = load_acquire(count) == w.last - w.first;
        mbar_arrive(bar(SM::B_ASK));
      }
      // Weights of the two halves' O, the row's reference and sum.
      float a0 = 1.f, a1 = 0.f, M = m_run, L = l_run;
      if (split) {
        float* own_ml = ml + ((k & 1) * 2 + half) * 2 * BM;
        own_ml[r] = m_run;
        own_ml[BM + r] = l_run;
        mbar_arrive(bar(SM::B_ML));
        if (ok && wait_all(SM::B_ML, ml_phase)) {
          const float* o_ml = ml + ((k & 1) * 2 + 1 - half) * 2 * BM;
          const float m1 = o_ml[r], l1 = o_ml[BM + r];
          M = fmaxf(m_run, m1);
          const float ref = (M == -INFINITY) ? 0.f : M;
          a0 = ex2(m_run - ref);
          a1 = ex2(m1 - ref);
          // The same bits in both halves (no fma): a join from the partials
          // takes half 0's, one from the accumulators each half's own.
          L = __fadd_rn(__fmul_rn(l_run, a0), __fmul_rn(l1, a1));
        } else {
          ok = false;
        }
        ++ml_phase;
      }
      constexpr int prows = BM << (PAIR ? 1 : 0);
      const int prow = (split ? 0 : half * BM) + r;
      auto partial_of = [&](int p) {
        return partial_at(a.ws, grid, 2 * p + (p == w.first ? 1 : 0), D, PAIR);
      };
      bool joins = false;
      float m1 = -INFINITY, l1 = 0.f;          // state of the next CTA's partial
      if (ask) {
        ok = wait_all(SM::B_ASK, 0);
        joins = ok && joiner[2] != 0;
        if (joins && live) {
          m1 = __ldcg(partial_of(cta + 1) + (size_t)prows * D + prow);
          l1 = __ldcg(partial_of(cta + 1) + (size_t)prows * (D + 1) + prow);
        }
      }
      if (ok && own > 0) ok = wait_all(SM::B_O + half, half ? o_phase1 : o_phase0);
      if (ok && split && other > 0) ok = wait_all(SM::B_O + 1 - half, half ? o_phase0 : o_phase1);
      if (!ok) break;
      tc_fence_after();
      const size_t orow = ((size_t)w.b * a.nodes + node) * cv.H + (size_t)w.kvh * sh.G + hg;
      __nv_bfloat16* orow_p = static_cast<__nv_bfloat16*>(a.o) + orow * D;
      // Split: each half writes half of the columns of the joined row.
      const int c_lo = split ? half * (D / 64) : 0, c_hi = split ? c_lo + D / 64 : D / 32;
      const bool final_rows = w.whole || joins;
      if (any) {
        float* part = partial_of(cta);
        float ws = 1.f;
        float top = M;
        if (joins && live) {
          top = fmaxf(M, m1);
          for (int p = cta + 2; p <= w.last; ++p)
            top = fmaxf(top, __ldcg(partial_of(p) + (size_t)prows * D + prow));
          ws = ex2(M - top);
          L = fmaf(l1, ex2(m1 - top), L * ws);
          for (int p = cta + 2; p <= w.last; ++p)
            L = fmaf(__ldcg(partial_of(p) + (size_t)prows * (D + 1) + prow),
                     ex2(__ldcg(partial_of(p) + (size_t)prows * D + prow) - top), L);
          M = top;
        }
        const float inv = 1.f / L;
        const bool use0 = own > 0, use1 = split && other > 0;
#pragma unroll 1
        for (int c = c_lo; c < c_hi; ++c) {
          float x[32];
          uint32_t ov[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 0.f;
          if (use0) {
            tmem_ld32_sync(tmem + lane_off + tm_o(half) + c * 32, ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(ov[e]) * a0;
          }
          if (use1) {
            tmem_ld32_sync(tmem + lane_off + tm_o(1 - half) + c * 32, ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = fmaf(__uint_as_float(ov[e]), a1, x[e]);
          }
          if (live && joins) {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] *= ws;
            add_partial<D, PAIR>(partial_of(cta + 1), prow, c, ex2(m1 - M), x);
            for (int p = cta + 2; p <= w.last; ++p)
              add_partial<D, PAIR>(partial_of(p), prow, c,
                                   ex2(__ldcg(partial_of(p) + (size_t)prows * D + prow) - M), x);
          }
          if (live && final_rows) {
            store_columns(orow_p + c * 32, x, inv);
          } else if (live) {
            float4* dst = reinterpret_cast<float4*>(part) + prow;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[(size_t)(c * 8 + e) * prows] =
                  make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          }
        }
        tc_fence_before();
        mbar_arrive(bar(SM::B_F));
        if (live && (!split || half == 0)) {
          if (!final_rows) {
            part[(size_t)prows * D + prow] = M;
            part[(size_t)prows * (D + 1) + prow] = L;
          } else if (a.lse) {
            a.lse[orow] = (M + log2f(L)) * kLn2;
          }
        }
      } else {
        tc_fence_before();
        mbar_arrive(bar(SM::B_F));
      }
      if (counted && !joins) {
        mbar_arrive(bar(SM::B_CUT));
        if (threadIdx.x == 0 && wait_for(bar(SM::B_CUT), cut_phase & 1, abort_flag, wait_ns)) {
          joiner[cut_phase & 1] = arrive_acq_rel(count) == w.last - w.first;
          mbar_arrive(bar(SM::B_JOIN));
        }
        if (!wait_all(SM::B_JOIN, cut_phase)) break;
        joins = joiner[cut_phase & 1] != 0;
        ++cut_phase;
        if (joins && live) {
          // The last after all, with its O given up.
          join_row<D, PAIR>(a.ws, grid, w.first, w.last, prow, c_lo, c_hi, orow_p,
                            a.lse && (!split || half == 0) ? a.lse + orow : nullptr);
        }
      }
      if (joins && threadIdx.x == 0) *count = 0;        // ready for the next call
      if ((half ? other : own) > 0) ++o_phase0;
      if ((half ? own : other) > 0) ++o_phase1;
      step += split ? nseg : 2 * nseg;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
  if (threadIdx.x == 0 && *abort_flag) flag_error(cv.err, kErrWaitTimeout);
}

// The joins of the units that the CTAs' ranges cut.

// The x-th CTA that begins a unit and does not end it; -1: there are fewer.
// Called by whole warps.
__device__ __forceinline__ int join_owner(const JoinDesc* desc, int ctas, int x) {
  const int lane = threadIdx.x & 31;
  int c = -1;
  for (int c0 = 0; c < 0 && c0 < ctas; c0 += 160) {
    int last[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const int y = c0 + 32 * i + lane;
      last[i] = y < ctas ? desc[y].last : -1;
    }
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const uint32_t on = __ballot_sync(0xffffffffu, last[i] >= 0);
      const int cnt = __popc(on);
      if (c < 0 && x < cnt) c = c0 + 32 * i + (int)__fns(on, 0, x + 1);
      x -= cnt;
    }
  }
  return c;
}

// A row of a cut unit: row y of the workspace's partials.
struct JoinRow {
  int prow, prows;
  bool live;
  size_t orow;                     // of o and lse
  __device__ JoinRow(const CacheView& cv, const TreeArgs& a, const Shape& sh, const JoinDesc& jd,
                     int y) {
    prow = y;
    prows = BM << sh.pair;
    const int r = y & (BM - 1), rg = r / sh.G;
    const int node = jd.node0 + (y >= BM ? sh.npt : 0) + rg;
    live = rg < sh.npt && node < jd.cnt;
    orow = ((size_t)jd.b * a.nodes + node) * cv.H + (size_t)jd.kvh * sh.G + (r - rg * sh.G);
  }
};

// State of a row over the partials seen: reference, sum and NV float4 of o.
template <int NV>
struct JoinState {
  float M = -INFINITY, L = 0.f;
  float4 x[NV];
  __device__ JoinState() {
#pragma unroll
    for (int e = 0; e < NV; ++e) x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ void add(float m, float l, const float4* v) {
    const float mn = fmaxf(M, m), ref = (mn == -INFINITY) ? 0.f : mn;
    const float s0 = fast_exp2(M - ref), s1 = fast_exp2(m - ref);
    M = mn;
    L = L * s0 + l * s1;
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      x[e].x = x[e].x * s0 + v[e].x * s1;
      x[e].y = x[e].y * s0 + v[e].y * s1;
      x[e].z = x[e].z * s0 + v[e].z * s1;
      x[e].w = x[e].w * s0 + v[e].w * s1;
    }
  }
  // float4 col4 .. col4 + NV - 1 of the row, and its lse; self is visible: L > 0.
  template <int D>
  __device__ void store(const TreeArgs& a, size_t orow, int col4) const {
    const float inv = 1.f / L;
    uint2* dst =
        reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + orow * D) + col4;
#pragma unroll
    for (int e = 0; e < NV; ++e)
      dst[e] = make_uint2(pack_bf16(x[e].x * inv, x[e].y * inv),
                          pack_bf16(x[e].z * inv, x[e].w * inv));
    if (col4 == 0 && a.lse) a.lse[orow] = (M + log2f(L)) * kLn2;
  }
};

// Reads partial p's part of a row: m, l and NV float4 from col4 on.
template <int D, int NV>
__device__ __forceinline__ void read_partial(const TreeArgs& a, const Shape& sh, int ctas, int p,
                                             bool first, const JoinRow& w, int col4, float& m,
                                             float& l, float4* v) {
  const float* part = partial_at(a.ws, ctas, 2 * p + (first ? 1 : 0), D, sh.pair);
  m = __ldcg(part + (size_t)w.prows * D + w.prow);
  l = __ldcg(part + (size_t)w.prows * (D + 1) + w.prow);
#pragma unroll
  for (int e = 0; e < NV; ++e)
    v[e] = __ldcg(reinterpret_cast<const float4*>(part) + (size_t)(col4 + e) * w.prows + w.prow);
}

constexpr int kJoinWarps = 4;

// Few units cut into many parts.  Block (x, y, z): unit x, rows 32 y .. 32 y + 31
// (lane = row), float4 z; each of the four warps takes every fourth partial, up
// to four at a time, so that the reads of 16 parts are one round trip.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
join_many_kernel(CacheView cv, TreeArgs a, Shape sh, int ctas) {
  __shared__ float sm[kJoinWarps][6][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const JoinDesc* desc = static_cast<const JoinDesc*>(a.ws);
  const int c = join_owner(desc, ctas, blockIdx.x);
  if (c < 0) return;
  const JoinDesc jd = desc[c];
  const JoinRow w(cv, a, sh, jd, blockIdx.y * 32 + lane);
  if (!__syncthreads_or(w.live)) return;
  constexpr int PB = 4;
  JoinState<1> st;
  for (int p0 = c + warp; p0 <= jd.last; p0 += PB * kJoinWarps) {
    float m[PB], l[PB];
    float4 v[PB];
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      const int p = p0 + i * kJoinWarps;
      m[i] = -INFINITY;
      l[i] = 0.f;
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p <= jd.last && w.live)
        read_partial<D, 1>(a, sh, ctas, p, p == c, w, blockIdx.z, m[i], l[i], &v[i]);
    }
#pragma unroll
    for (int i = 0; i < PB; ++i) st.add(m[i], l[i], &v[i]);
  }
  sm[warp][0][lane] = st.M;
  sm[warp][1][lane] = st.L;
  sm[warp][2][lane] = st.x[0].x;
  sm[warp][3][lane] = st.x[0].y;
  sm[warp][4][lane] = st.x[0].z;
  sm[warp][5][lane] = st.x[0].w;
  __syncthreads();
  if (warp > 0 || !w.live) return;
#pragma unroll
  for (int k = 1; k < kJoinWarps; ++k) {
    const float4 v = make_float4(sm[k][2][lane], sm[k][3][lane], sm[k][4][lane], sm[k][5][lane]);
    st.add(sm[k][0][lane], sm[k][1][lane], &v);
  }
  st.template store<D>(a, w.orow, blockIdx.z);
}

// Many units cut into two or three parts.  Block (x, y, z): unit x, rows 32 y ..
// 32 y + 31 (lane = row), NV float4 a warp, two partials read at a time: all
// columns of the rows where there are many rows (152 units of 256 rows: 1216
// blocks; with NV 1 they were 9728 and took 22 us), a quarter of them otherwise.
// Bound by the partials' traffic through L2.
template <int D, int NV>
__global__ void __launch_bounds__(kJoinWarps * 32)
join_few_kernel(CacheView cv, TreeArgs a, Shape sh, int ctas) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const JoinDesc* desc = static_cast<const JoinDesc*>(a.ws);
  const int c = join_owner(desc, ctas, blockIdx.x);
  if (c < 0) return;
  const JoinDesc jd = desc[c];
  const JoinRow w(cv, a, sh, jd, blockIdx.y * 32 + lane);
  if (!w.live) return;
  const int col4 = ((int)blockIdx.z * kJoinWarps + warp) * NV;
  JoinState<NV> st;
  for (int p = c; p <= jd.last; p += 2) {
    float m0, l0, m1, l1;
    float4 v0[NV], v1[NV];
    read_partial<D, NV>(a, sh, ctas, p, p == c, w, col4, m0, l0, v0);
    if (p < jd.last) read_partial<D, NV>(a, sh, ctas, p + 1, false, w, col4, m1, l1, v1);
    st.add(m0, l0, v0);
    if (p < jd.last) st.add(m1, l1, v1);
  }
  st.template store<D>(a, w.orow, col4);
}

// A cache of more than this is streamed: half of L2.
constexpr uint64_t kEvictBytes = 64u << 20;

Shape shape_of(const CacheView& cv, int nodes) {
  Shape sh;
  sh.G = cv.H / cv.Hkv;
  sh.npt = BM / sh.G;
  sh.pair = nodes > sh.npt ? 1 : 0;
  sh.box = std::min(sh.npt, nodes);
  sh.evict = sh.joins = sh.flat = sh.inl = 0;
  return sh;
}

// Units of the largest work list, and the cost of all of them.
int64_t most_units(const CacheView& cv, int nodes, const Shape& sh) {
  const int per = sh.npt << sh.pair;
  return (int64_t)cv.B * cv.Hkv * ((nodes + per - 1) / per);
}
int64_t most_tiles(const CacheView& cv, int nodes) {
  return ((cv.m_cap + 15) / 16 * 16 + (cv.n + 15) / 16 * 16 + nodes + BN - 1) / BN;
}
int64_t most_cost(const CacheView& cv, int nodes, const Shape& sh) {
  return most_units(cv, nodes, sh) * (most_tiles(cv, nodes) + kUnitCost);
}

// Units, no more of them than SMs, have a CTA each where cutting them would save
// less than the second kernel and the starts of their parts take: at most
// kFlatTiles tiles, of which an even cut would leave a CTA units / SMs.  us for a
// CTA each / cut: 70 units of 9 tiles 15.3 / 21.7, 46 of 7 13.6 / 19.2, 16 pairs
// of 7 24.8 / 28.5, 32 of 10 17.7 / 19.3, but 10 of 10 17.0 / 13.5.
constexpr int kFlatTiles = 10, kFlatSaved = 8;

bool flat_of(const CacheView& cv, int nodes, const Shape& sh) {
  const int64_t units = most_units(cv, nodes, sh), tiles = most_tiles(cv, nodes);
  return units <= cv.sms && tiles <= kFlatTiles && tiles * (cv.sms - units) <= kFlatSaved * cv.sms;
}

// CTAs of the launch: one per SM, no more than the largest list could feed.
int grid_of(const CacheView& cv, int nodes, const Shape& sh) {
  if (sh.flat) return (int)most_units(cv, nodes, sh);
  return (int)std::max<int64_t>(1, std::min<int64_t>(cv.sms, most_cost(cv, nodes, sh) / kMinCost));
}

template <int D, bool PAIR>
cudaError_t launch_d(const CacheView& cv, const TreeArgs& a, const SlabMaps& maps,
                     cudaStream_t s) {
  Shape sh = shape_of(cv, a.nodes);
  sh.flat = flat_of(cv, a.nodes, sh);
  const int grid = grid_of(cv, a.nodes, sh);
  const uint64_t trows = (uint64_t)cv.B * a.nodes;
  const uint64_t crows = (uint64_t)cv.B * cv.Hkv * cv.slab_rows;
  CUtensorMap mq, mkt, mvt, mkt16, mvt16;
  if (!make_tmap_heads_bf16(&mq, a.q, D, cv.H, trows, sh.G, sh.box) ||
      !make_tmap_rows_bf16(&mkt, a.k, (uint64_t)cv.Hkv * D, trows) ||
      !make_tmap_rows_bf16(&mvt, a.v, (uint64_t)cv.Hkv * D, trows) ||
      !make_tmap_rows_bf16(&mkt16, a.k, (uint64_t)cv.Hkv * D, trows, 16) ||
      !make_tmap_rows_bf16(&mvt16, a.v, (uint64_t)cv.Hkv * D, trows, 16))
    return cudaErrorInvalidValue;
  sh.evict = crows * D * 4 > kEvictBytes;
  sh.joins = (int)std::min<int64_t>(most_units(cv, a.nodes, sh), grid);
  // Many units, cut into few parts each, and a counter for each (the cache has
  // one a query head).
  sh.inl = PAIR && !sh.flat && sh.joins == grid &&
           most_units(cv, a.nodes, sh) <= (int64_t)cv.B * cv.Hkv * sh.G;
  // Per device (the attribute belongs to the current device's context).
  cudaError_t e = cudaFuncSetAttribute(decode_tree_tc_kernel<D, PAIR>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, PAIR>::kBytes);
  if (e != cudaSuccess) return e;
  e = launch_dependent(decode_tree_tc_kernel<D, PAIR>, dim3(grid), dim3(kThreads),
                       Smem<D, PAIR>::kBytes, s, mq, maps.k, maps.v, mkt, mvt, maps.k16, maps.v16,
                       mkt16, mvt16, maps.k64, maps.v64, cv, a, sh, phase_wait_limit_ns());
  if (e != cudaSuccess) return e;
  if (sh.flat || sh.inl) return cudaSuccess;
  const int rows = PAIR ? 2 * BM : std::min(a.nodes, sh.npt) * sh.G;
  // More CTAs than units: many parts to a unit.
  if (sh.joins < grid)
    return launch_dependent(join_many_kernel<D>, dim3(sh.joins, (rows + 31) / 32, D / 4),
                            dim3(kJoinWarps * 32), 0, s, cv, a, sh, grid);
  constexpr int NV = D / 4 / kJoinWarps / (PAIR ? 1 : 4);
  return launch_dependent(join_few_kernel<D, NV>,
                          dim3(sh.joins, (rows + 31) / 32, D / 4 / kJoinWarps / NV),
                          dim3(kJoinWarps * 32), 0, s, cv, a, sh, grid);
}

}  // namespace

bool decode_tree_tc_supported(const CacheView& cv, int nodes) {
  // The planner steps over sequences without live nodes one by one (65533 of them
  // in 10.8 ms): so many at most keep that far below the bound of its readers' waits.
  if (cv.dtype != RSWA_BF16 || cv.H / cv.Hkv > BM || cv.B > 65535) return false;
  return most_cost(cv, nodes, shape_of(cv, nodes)) < (int64_t(1) << 31) &&
         (int64_t)cv.B * nodes < (int64_t(1) << 30) &&
         (int64_t)cv.B * cv.Hkv * cv.slab_rows + cv.n < (int64_t(1) << 31);
}

size_t decode_tree_tc_workspace(const CacheView& cv, int nodes) {
  const Shape sh = shape_of(cv, nodes);
  const size_t grid = (size_t)grid_of(cv, nodes, sh);
  return (grid * sizeof(JoinDesc) + 255) / 256 * 256 +
         grid * 2 * partial_floats(cv.d, sh.pair) * sizeof(float);
}

bool make_slab_maps(const CacheView& cv, SlabMaps* maps) {
  const uint64_t rows = (uint64_t)cv.B * cv.Hkv * cv.slab_rows;
  return make_tmap_rows_bf16(&maps->k, cv.K, cv.d, rows) &&
         make_tmap_rows_bf16(&maps->v, cv.V, cv.d, rows) &&
         make_tmap_rows_bf16(&maps->k16, cv.K, cv.d, rows, 16) &&
         make_tmap_rows_bf16(&maps->v16, cv.V, cv.d, rows, 16) &&
         make_tmap_rows_bf16(&maps->k64, cv.K, cv.d, rows, 64) &&
         make_tmap_rows_bf16(&maps->v64, cv.V, cv.d, rows, 64);
}

cudaError_t launch_decode_tree_tc(const CacheView& cv, const TreeArgs& a, const SlabMaps& maps,
                                  cudaStream_t s) {
  if (shape_of(cv, a.nodes).pair)
    return cv.d == 64 ? launch_d<64, true>(cv, a, maps, s) : launch_d<128, true>(cv, a, maps, s);
  return cv.d == 64 ? launch_d<64, false>(cv, a, maps, s) : launch_d<128, false>(cv, a, maps, s);
}

}  // namespace rswa
