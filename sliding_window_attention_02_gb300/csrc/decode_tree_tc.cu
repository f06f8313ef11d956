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
// Work: the key tiles of a unit (prefix, ring, tree; 128 keys each) one after
// the other, unit after unit, form one list, which the CTAs (one per SM) cut
// into equal ranges.  A CTA streams its range through one TMA ring without
// draining between units; a unit that a range covers whole is written out at
// once, of another the CTA leaves a partial (m, l, O) in the workspace, and a
// second, dependent kernel joins the partials of every cut unit.  Each CTA
// leaves at most two: of the unit that a CTA before it began, and of the one
// that it begins and does not end.
//
// Roles (352 threads): warps 0-3 / 4-7 softmax and epilogue of half 0 / 1
// (thread r owns row r = TMEM lane r), warp 8 TMA producer, warp 9 TMEM
// allocator and MMA issuer, warp 10 planner: it cuts the list, walks the CTA's
// range ahead of the others and hands them, through shared memory, each
// segment (the part of a unit inside the range) and its nodes' depths and
// ancestors.  Steps (a half's turn on a key tile) alternate
// between the halves through the whole range; the MMA order is QK(0) QK(1)
// PV(0) QK(2) PV(1) QK(3) ..., so the tensor core works on one half while the
// other half's softmax runs.  TMEM: S0 | S1 | O0 | O1, P over S.  O is
// rescaled lazily (threshold 2^8, exact because O and l share the reference).
// A key tile's PV takes only the 16-key steps that hold keys; keys are loaded
// to the next multiple of 16, and value rows of nodes past the count are
// zeroed first (0 x NaN is NaN).  Every wait is bounded; on a timeout the CTA
// drains its copies and MMAs, frees TMEM and sets the cache's device flag.
#include <cuda.h>

#include <algorithm>

#include "decode_tree.cuh"
#include "rswa_device.cuh"
#include "tc_ptx.cuh"

namespace rswa {
namespace {

using namespace ptx;

constexpr int BM = 128, BN = 128;
constexpr int kSoftmaxThreads = 256;
constexpr int kThreads = kSoftmaxThreads + 96;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kPlanWarp = 10;
constexpr int NS = 4;                          // K/V ring slots
constexpr uint32_t kSub = BM * 64 * 2;         // [128][64] bf16, 128B-swizzled
constexpr uint32_t kTileB = 2 * kSub;          // [128][128] bf16 = 32 KB
constexpr uint32_t OFF_Q = 0;                  // two query tiles
constexpr uint32_t OFF_RING = 2 * kTileB;
constexpr uint32_t OFF_ML = OFF_RING + NS * kTileB;      // [2][2][2][128] floats
constexpr uint32_t OFF_BAR = OFF_ML + 2 * 2 * 2 * BM * 4;
constexpr int NSEG = 4;                        // segments handed over at a time
constexpr uint32_t OFF_SEG = OFF_BAR + 256;
constexpr uint32_t OFF_PAR = OFF_SEG + NSEG * 64;        // a sequence's parents
constexpr int NODES = 2 * BM;                  // most nodes of a unit
constexpr int NTT = 2;                         // tree tiles whose masks are handed over
constexpr uint32_t kNodeWords = NODES * (1 + 4 * NTT);   // depth and masks of a unit's nodes
constexpr uint32_t OFF_NODE = OFF_PAR + kMaxTreeNodes * 4;
constexpr uint32_t kSmemBytes = OFF_NODE + 2 * kNodeWords * 4 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

__host__ __device__ constexpr uint32_t tm_s(int half) { return half ? 128u : 0u; }
__host__ __device__ constexpr uint32_t tm_o(int half) { return half ? 384u : 256u; }
constexpr uint32_t TM_COLS = 512;
constexpr float kRescaleThreshold = 8.0f;      // log2 units
constexpr uint64_t kWaitLimitNs = 1000000000ull;
// A CTA's least share of the list: one key tile for each half.
constexpr int kMinTiles = 2;

constexpr int B_QF = 0;                        // 2 query tiles loaded
constexpr int B_QE = 2;                        // 2 query tiles free
constexpr int B_FULL = 4;                      // NS slots
constexpr int B_EMPTY = B_FULL + NS;           // NS slots
constexpr int B_S = B_EMPTY + NS;              // 2 halves: S ready
constexpr int B_P = B_S + 2;                   // 2 halves: P written
constexpr int B_O = B_P + 2;                   // 2 halves: the segment's last PV done
constexpr int B_F = B_O + 2;                   // the segment's O read out
constexpr int B_ML = B_F + 1;                  // split: both halves' (m, l) in smem
constexpr int B_FIN = B_ML + 1;
constexpr int B_SEG = B_FIN + 1;               // NSEG segments handed over
constexpr int B_NODE = B_SEG + NSEG;           // 2 segments' nodes handed over
constexpr int B_NFREE = B_NODE + 2;            // and read by every row
constexpr int NBAR = B_NFREE + 2;
static_assert(8 * NBAR + 16 <= 256, "barriers");

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x,
                                            int32_t y, int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// The shape of a launch.
struct Shape {
  int npt;      // nodes of a query tile
  int pair;     // 1: units of two query tiles
  int G;        // query heads of a KV head
};

// What a sequence adds to the work list: units of `tl` key tiles each.
struct Seq {
  int cnt, m_b;
  int64_t t_b;
  int np, nr, tl, units;
  __device__ void load(const CacheView& cv, const TreeArgs& a, const Shape& sh, int b) {
    cnt = live_nodes(a.counts, b, a.nodes, cv.err);
    m_b = cv.m_dev[b];
    t_b = cv.t_dev[(size_t)b * cv.H];
    np = (m_b + BN - 1) / BN;
    nr = (int)((min(cv.n, t_b) + BN - 1) / BN);
    tl = np + nr + (cnt + BN - 1) / BN;
    const int per = sh.npt << sh.pair;
    units = (cnt + per - 1) / per * cv.Hkv;
  }
};

enum TileKind { kPrefix = 0, kRing = 1, kTree = 2 };

// A segment as the planner hands it over.
struct Segment {
  int b, kvh, node0, cnt;
  int j0, j1;             // key tiles of the unit inside the range; j1 = 0: no more segments
  int np, nr;             // the unit's prefix and ring tiles, then come the tree's
  int m_b, ring;          // prefix rows, filled ring slots
  int newest, age;        // ring slot of output t_b - 1, and t_b - 1 (clamped)
  int split, whole, begins;
  // Kind of key tile j, its index among its kind, and its keys.
  __device__ void tile(int j, int& kind, int& i, int& keys) const {
    if (j < np) {
      kind = kPrefix;
      i = j;
      keys = m_b;
    } else if (j < np + nr) {
      kind = kRing;
      i = j - np;
      keys = ring;
    } else {
      kind = kTree;
      i = j - np - nr;
      keys = cnt;
    }
    keys = min(BN, keys - i * BN);
  }
};
static_assert(sizeof(Segment) <= 64, "segment");

// Bits e of word c (columns 32 c + e) with lo <= column <= hi.
__device__ __forceinline__ uint32_t range_mask(int lo, int hi, int c) {
  const int a = max(lo - 32 * c, 0), b = min(hi - 32 * c, 31);
  if (a > b) return 0u;
  return (0xffffffffu << a) & (0xffffffffu >> (31 - b));
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
decode_tree_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmKc,
                      const __grid_constant__ CUtensorMap tmVc,
                      const __grid_constant__ CUtensorMap tmKt,
                      const __grid_constant__ CUtensorMap tmVt,
                      const __grid_constant__ CUtensorMap tmKc16,
                      const __grid_constant__ CUtensorMap tmVc16,
                      const __grid_constant__ CUtensorMap tmKt16,
                      const __grid_constant__ CUtensorMap tmVt16, CacheView cv, TreeArgs a,
                      Shape sh, uint64_t wait_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t bar0 = sb + OFF_BAR;
  auto bar = [&](int k) { return bar0 + 8u * (uint32_t)k; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_BAR + 8 * NBAR);
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(smem + OFF_BAR + 8 * NBAR + 4);
  volatile int* never = reinterpret_cast<volatile int*>(smem + OFF_BAR + 8 * NBAR + 8);
  const Segment* segs = reinterpret_cast<const Segment*>(smem + OFF_SEG);
  int32_t* nodes_smem = reinterpret_cast<int32_t*>(smem + OFF_NODE);
  constexpr int NSUB = D / 64;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, grid = gridDim.x;

  if (threadIdx.x == 0) {
    for (int k = 0; k < NBAR; ++k)
      mbar_init(bar(k), k == B_P || k == B_P + 1
                           ? 128u
                           : (k == B_F || k == B_ML || k >= B_NFREE ? 256u : 1u));
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
    if (!mbar_wait(bar(B_SEG + k % NSEG), (k / NSEG) & 1, abort_flag, wait_ns)) return false;
    w = segs[k % NSEG];
    return true;
  };

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmKc);
      prefetch_tmap(&tmVc);
      prefetch_tmap(&tmKt16);
      prefetch_tmap(&tmVt16);
      prefetch_tmap(&tmKc16);
      prefetch_tmap(&tmVc16);
      uint32_t gi = 0, qi = 0;                   // K/V loads and query tiles issued
      bool ok = true;
      const uint32_t qbytes = (uint32_t)NSUB * sh.npt * sh.G * 128u;
      Segment w;
      for (int k = 0; ok && segment(k, w) && w.j1 > 0; ++k) {
        const int nq = w.split ? 1 : 2;
        for (int x = 0; ok && x < nq; ++x, ++qi) {
          const uint32_t s = qi & 1;
          if (qi >= 2 && !mbar_wait(bar(B_QE + s), ((qi >> 1) - 1) & 1, abort_flag, wait_ns)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(B_QF + s), qbytes);
#pragma unroll
          for (int c = 0; c < NSUB; ++c)
            tma_load_3d(sb + OFF_Q + s * kTileB + c * kSub, &tmQ, c * 64, w.kvh * sh.G,
                        w.b * a.nodes + w.node0 + x * sh.npt, bar(B_QF + s));
        }
        const int64_t slab0 = ((int64_t)w.b * cv.Hkv + w.kvh) * cv.slab_rows;
        for (int j = w.j0; ok && j < w.j1; ++j) {
          int kind, i, keys;
          w.tile(j, kind, i, keys);
          const int boxes = (keys + 15) / 16;
          const int x0 = kind == kTree ? w.kvh * D : 0;
          const int y0 = kind == kTree
                             ? w.b * a.nodes + i * BN
                             : (int)(slab0 + (kind == kRing ? cv.m_cap : 0) + (int64_t)i * BN);
          for (int isv = 0; isv < 2; ++isv, ++gi) {
            const uint32_t s = gi % NS;
            if (gi >= (uint32_t)NS &&
                !mbar_wait(bar(B_EMPTY + s), ((gi / NS) - 1) & 1, abort_flag, wait_ns)) {
              ok = false;
              break;
            }
            const uint32_t dst = sb + OFF_RING + s * kTileB;
            mbar_arrive_expect_tx(bar(B_FULL + s), (uint32_t)NSUB * boxes * 2048u);
            if (boxes == BN / 16) {
              const CUtensorMap* map = kind == kTree ? (isv ? &tmVt : &tmKt)
                                                     : (isv ? &tmVc : &tmKc);
#pragma unroll
              for (int c = 0; c < NSUB; ++c)
                tma_load_2d(dst + c * kSub, map, x0 + c * 64, y0, bar(B_FULL + s));
            } else {
              const CUtensorMap* map = kind == kTree ? (isv ? &tmVt16 : &tmKt16)
                                                     : (isv ? &tmVc16 : &tmKc16);
              for (int r = 0; r < boxes; ++r)
#pragma unroll
                for (int c = 0; c < NSUB; ++c)
                  tma_load_2d(dst + c * kSub + r * 2048, map, x0 + c * 64, y0 + 16 * r,
                              bar(B_FULL + s));
            }
          }
        }
      }
      // Drain: every copy issued has landed before the CTA may exit.
      for (uint32_t k = qi > 2 ? qi - 2 : 0; k < qi; ++k)
        mbar_wait(bar(B_QF + (k & 1)), (k >> 1) & 1, never, kWaitLimitNs);
      for (uint32_t k = gi > (uint32_t)NS ? gi - NS : 0; k < gi; ++k)
        mbar_wait(bar(B_FULL + k % NS), (k / NS) & 1, never, kWaitLimitNs);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks; one lane issues.  qc runs two steps ahead of pc.
    constexpr uint32_t idesc_qk = idesc_bf16(BM, BN, false);
    constexpr uint32_t idesc_pv = idesc_bf16(BM, D, true);
    auto wait = [&](int k, uint32_t phase) {
      return __all_sync(0xffffffffu, mbar_wait(bar(k), phase & 1, abort_flag, wait_ns)) != 0;
    };
    struct Cursor {
      Segment w;
      int k;                  // segment
      int j, sub;             // key tile; in a pair unit the first or second half's turn
      uint32_t step, load, q; // steps, key tiles and query tiles before
      bool more;
    };
    auto enter = [&](Cursor& c) {
      const bool got = segment(c.k, c.w);
      c.more = __all_sync(0xffffffffu, got) && c.w.j1 > 0;
      c.j = c.w.j0;
      c.sub = 0;
    };
    auto advance = [&](Cursor& c) {
      ++c.step;
      if (!c.w.split && c.sub == 0) {
        c.sub = 1;
        return;
      }
      c.sub = 0;
      ++c.load;
      if (++c.j == c.w.j1) {
        c.q += c.w.split ? 1 : 2;
        ++c.k;
        enter(c);
      }
    };
    Cursor qc = {}, pc = {};
    enter(qc);
    enter(pc);
    // S = Q K^T of qc's step, then on to the next.
    auto qk = [&]() {
      const uint32_t half = qc.step & 1;
      const uint32_t qt = qc.w.split ? qc.q : qc.q + half;
      const uint32_t ki = 2 * qc.load;
      if (!wait(B_QF + (qt & 1), qt >> 1) || !wait(B_FULL + ki % NS, ki / NS)) return false;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t kb = sb + OFF_RING + (ki % NS) * kTileB;
        const uint32_t qb = sb + OFF_Q + (qt & 1) * kTileB;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * kSub + (k & 3) * 32;
          mma_bf16_ss(tmem + tm_s(half), desc_sw128(qb + off, 16, 1024),
                      desc_sw128(kb + off, 16, 1024), idesc_qk, k > 0);
        }
        mma_commit(bar(B_S + half));
        if (qc.w.split || qc.sub == 1) mma_commit(bar(B_EMPTY + ki % NS));
        if (qc.j + 1 == qc.w.j1 && (qc.w.split || qc.sub == 1)) {
          mma_commit(bar(B_QE + (qc.q & 1)));
          if (!qc.w.split) mma_commit(bar(B_QE + ((qc.q + 1) & 1)));
        }
      }
      __syncwarp();
      advance(qc);
      return true;
    };
    bool ok = true;
    for (int x = 0; x < 2 && ok && qc.more; ++x) ok = qk();
    while (ok && pc.more) {
      const uint32_t half = pc.step & 1;
      const uint32_t vi = 2 * pc.load + 1;
      int kind, i, keys;
      pc.w.tile(pc.j, kind, i, keys);
      // The half's first and last step of the segment.
      const int span = pc.w.split ? 2 : 1;
      const bool first = pc.j - pc.w.j0 < span, last = pc.j + span >= pc.w.j1;
      if (first && pc.k > 0 && !wait(B_F, pc.k - 1)) break;
      if (!wait(B_P + half, pc.step >> 1) || !wait(B_FULL + vi % NS, vi / NS)) break;
      const uint32_t vb = sb + OFF_RING + (vi % NS) * kTileB;
      const int ks = (keys + 15) / 16;
      if (kind == kTree && keys % 16 != 0 && (pc.w.split || pc.sub == 0)) {
        // value rows keys .. 16 ks - 1: nodes past the count
        const int rows = 16 * ks - keys;
        for (int x = lane; x < rows * 8 * NSUB; x += 32) {
          const int c = x / (rows * 8), y = x % (rows * 8);
          *reinterpret_cast<uint4*>(smem + (vb - sb) + c * kSub + keys * 128 + y * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      tc_fence_after();
      if (lane == 0) {
        for (int k = 0; k < ks; ++k)
          mma_bf16_ts(tmem + tm_o(half), tmem + tm_s(half) + k * 8,
                      desc_sw128(vb + k * 2048, kSub, 1024), idesc_pv,
                      (!first || k > 0) ? 1u : 0u);
        if (pc.w.split || pc.sub == 1) mma_commit(bar(B_EMPTY + vi % NS));
        if (last) mma_commit(bar(B_O + half));
      }
      __syncwarp();
      advance(pc);
      if (qc.more) ok = qk();
    }
    // Drain: all MMAs of this CTA have finished before TMEM is freed.
    if (lane == 0) {
      mma_commit(bar(B_FIN));
      mbar_wait(bar(B_FIN), 0, never, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == kPlanWarp) {
    // ------------------------------------------------------------ planner
    Segment* out = reinterpret_cast<Segment*>(smem + OFF_SEG);
    int32_t* par = reinterpret_cast<int32_t*>(smem + OFF_PAR);
    // The list's length, and the sequences of each lane in it.
    const int per = (cv.B + 31) / 32;
    const int b_lo = min(lane * per, cv.B), b_hi = min(b_lo + per, cv.B);
    Seq sq;
    int mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
      sq.load(cv, a, sh, b);
      mine += sq.tl * sq.units;
    }
    int inc = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += x;
    }
    const int total = __shfl_sync(0xffffffffu, inc, 31);
    // Range c: `each` tiles, one more for the first `rem` CTAs.
    const int ctas = min(grid, max(1, total / kMinTiles));
    const int each = total / ctas, rem = total - each * ctas;
    const int g0 = cta * each + min(cta, rem);
    int left = cta < ctas ? each + (cta < rem ? 1 : 0) : 0;
    JoinDesc jd = {0, 0, 0, -1, 0, {0, 0, 0}};
    int k = 0;
    if (left > 0) {
      // The sequence and unit that tile g0 is in.
      int b = 0, off = 0;
      const bool here = inc - mine <= g0 && g0 < inc;
      if (here) {
        int at = inc - mine;
        for (b = b_lo; b < b_hi; ++b) {
          sq.load(cv, a, sh, b);
          if (g0 < at + sq.tl * sq.units) break;
          at += sq.tl * sq.units;
        }
        off = g0 - at;
      }
      const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
      b = __shfl_sync(0xffffffffu, b, src);
      off = __shfl_sync(0xffffffffu, off, src);
      sq.load(cv, a, sh, b);
      int u = off / sq.tl, j0 = off - u * sq.tl, g = g0, par_b = -1;
      const int unit_nodes = sh.npt << sh.pair;
      const int n = (int)min(cv.n, (int64_t)1 << 30);
      for (;;) {
        Segment w;
        w.b = b;
        w.kvh = u % cv.Hkv;
        w.node0 = u / cv.Hkv * unit_nodes;
        w.cnt = sq.cnt;
        w.j0 = j0;
        w.j1 = min(sq.tl, j0 + left);
        w.np = sq.np;
        w.nr = sq.nr;
        w.m_b = sq.m_b;
        w.ring = (int)min(cv.n, sq.t_b);
        w.age = (int)min(sq.t_b - 1, (int64_t)1 << 30);
        w.newest = sq.t_b > cv.n ? (int)((sq.t_b - 1) % cv.n) : (int)sq.t_b - 1;
        // A unit without rows for a second query tile is split like all
        // others of a launch without pairs.
        w.split = !sh.pair || w.node0 + sh.npt >= sq.cnt;
        w.whole = j0 == 0 && w.j1 == sq.tl;
        w.begins = j0 == 0;
        // Slot k % NSEG was segment k - 4's: all roles had left it when the
        // nodes of segment k - 1 were handed over (which waited until those
        // of segment k - 3 had been read).
        if (lane == 0) {
          out[k % NSEG] = w;
          mbar_arrive(bar(B_SEG + k % NSEG));
        }
        if (j0 == 0 && !w.whole) {       // begun here, ended by a later CTA
          const int x = g + sq.tl - 1;   // the unit's last tile
          const int cut = rem * (each + 1);
          jd = {b, w.node0, w.kvh, x < cut ? x / (each + 1) : rem + (x - cut) / each,
                sq.cnt, {0, 0, 0}};
        }
        // Depths and ancestors of the unit's nodes.
        if (par_b != b) {
          __syncwarp();
          for (int i = lane; i < sq.cnt; i += 32) par[i] = a.parents[(size_t)b * a.nodes + i];
          par_b = b;
          __syncwarp();
        }
        if (k >= 2 &&
            !__all_sync(0xffffffffu, mbar_wait(bar(B_NFREE + (k & 1)), ((k >> 1) - 1) & 1,
                                               abort_flag, wait_ns)))
          break;
        int32_t* nd = nodes_smem + (k & 1) * kNodeWords;
        const int nn = min(unit_nodes, sq.cnt - w.node0);
        for (int i = lane; i < nn; i += 32) {
          uint32_t m[4 * NTT];
#pragma unroll
          for (int e = 0; e < 4 * NTT; ++e) m[e] = 0u;
          int up = 0;
          for (int x = w.node0 + i;;) {
            if (up < n) {
#pragma unroll
              for (int e = 0; e < 4 * NTT; ++e)
                if (x >> 5 == e) m[e] |= 1u << (x & 31);
            }
            const int p = par[x];
            if (p < -1 || p >= x) flag_error(cv.err, kErrBadTree);
            if (p < 0 || p >= x) break;
            x = p;
            ++up;
          }
          nd[i] = up;
#pragma unroll
          for (int e = 0; e < 4 * NTT; ++e) nd[(1 + e) * NODES + i] = (int32_t)m[e];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_NODE + (k & 1)));
        ++k;
        g += w.j1 - w.j0;
        left -= w.j1 - w.j0;
        if (left <= 0) break;
        j0 = 0;
        if (++u == sq.units) {
          u = 0;
          sq.units = 0;
          while (sq.units == 0 && b + 1 < cv.B) sq.load(cv, a, sh, ++b);
          if (sq.units == 0) break;      // (the list ends with the last sequence)
        }
      }
    }
    if (lane == 0) {
      out[k % NSEG].j1 = 0;              // no more segments
      mbar_arrive(bar(B_SEG + k % NSEG));
      static_cast<JoinDesc*>(a.ws)[cta] = jd;
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
    float* ml = reinterpret_cast<float*>(smem + OFF_ML);
    uint32_t step = 0, turns = 0;                       // steps before; this half's among them
    uint32_t o_phase0 = 0, o_phase1 = 0, ml_phase = 0;  // segments with steps of each half; split
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
      const int32_t* nd = nodes_smem + (k & 1) * kNodeWords;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(B_NODE + (k & 1)), (k >> 1) & 1, abort_flag,
                                             wait_ns))) {
        ok = false;
        break;
      }
      const int depth = live ? nd[ni] : 0;
      // Ring: slot s is a key iff its age (r0 - s) mod n is at most lim.
      const int lim = min(w.age, n - 2 - depth);
      const int r0 = w.newest;
      float m_run = -INFINITY, l_run = 0.f;
      bool started = false;
      for (int j = w.j0; j < w.j1; ++j) {
        if (split && ((step + (uint32_t)(j - w.j0)) & 1) != (uint32_t)half) continue;
        int kind, i, keys;
        w.tile(j, kind, i, keys);
        const int k0 = i * BN;
        const bool full = kind == kPrefix && keys == BN;
        if (!__all_sync(0xffffffffu,
                        mbar_wait(bar(B_S + half), turns & 1, abort_flag, wait_ns))) {
          ok = false;
          break;
        }
        ++turns;
        tc_fence_after();
        if (any) {
          // This row's keys among the tile's columns.
          uint32_t see[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
          if (!full) {
            if (kind == kTree) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                see[c] = live && i < NTT ? (uint32_t)nd[(1 + 4 * i + c) * NODES + ni] : 0u;
              if (i >= NTT && live) {
                // a further tile of a large tree: walk up from the node
                const int32_t* par = a.parents + (size_t)w.b * a.nodes;
                int up = 0;
                for (int x = node; x >= k0 && up < n; ++up) {
                  if (x < k0 + BN) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      if ((x - k0) >> 5 == e) see[e] |= 1u << (x & 31);
                  }
                  const int p = par[x];
                  if (p >= x) break;
                  x = p;
                }
              }
            } else {
              int a1 = 0, b1 = keys - 1, a2 = 1, b2 = 0;
              if (kind == kRing) {
                if (lim < 0) {
                  b1 = -1;
                } else if (r0 >= lim) {
                  a1 = r0 - lim - k0;
                  b1 = r0 - k0;
                } else {
                  b1 = r0 - k0;
                  a2 = r0 - lim + n - k0;
                  b2 = n - 1 - k0;
                }
              }
#pragma unroll
              for (int c = 0; c < 4; ++c)
                see[c] = range_mask(a1, b1, c) | range_mask(a2, b2, c);
            }
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          uint32_t va[32], vb[32];
          auto max_chunk = [&](uint32_t* v, int c) {
            if (!full) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(see[c] >> e & 1u)) v[e] = 0xff800000u;         // -inf
              tmem_st32(s_addr + 32 * c, v);
            }
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              mx[0] = fmax3(mx[0], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              mx[1] = fmax3(mx[1], __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
              mx[2] = fmax3(mx[2], __uint_as_float(v[e + 4]), __uint_as_float(v[e + 5]));
              mx[3] = fmax3(mx[3], __uint_as_float(v[e + 6]), __uint_as_float(v[e + 7]));
            }
          };
          tmem_ld32(s_addr, va);
          tmem_wait_ld32(va);
          tmem_ld32(s_addr + 32, vb);
          max_chunk(va, 0);
          tmem_wait_ld32(vb);
          tmem_ld32(s_addr + 64, va);
          max_chunk(vb, 1);
          tmem_wait_ld32(va);
          tmem_ld32(s_addr + 96, vb);
          max_chunk(va, 2);
          tmem_wait_ld32(vb);
          max_chunk(vb, 3);
          if (!full) tmem_wait_st();
          const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
          // Lazy rescale.  O_h is stable here: S_h of this step completing
          // implies that the half's PV before it has.
          float alpha = 1.f;
          bool resc = false;
          const float m_new = fmaxf(m_run, tmax);
          if (m_run == -INFINITY) {
            m_run = m_new;
          } else if (m_new > m_run + kRescaleThreshold) {
            alpha = ex2(m_run - m_new);
            m_run = m_new;
            l_run *= alpha;
            resc = true;
          }
          const float nref = (m_run == -INFINITY) ? 0.f : -m_run;
          if (started && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ov[32];
              tmem_ld32_sync(o_addr + c * 32, ov);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              tmem_st32(o_addr + c * 32, ov);
            }
          }
          uint32_t pk[2][32];
          const uint64_t sl2x2 = f2_pack(sl2, sl2), nref2 = f2_pack(nref, nref);
          uint64_t ps2[2] = {0, 0};
          auto exp_chunk = [&](const uint32_t* v, uint32_t* out) {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const int e = 2 * c;
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                               sl2x2, nref2),
                        x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              ps2[c & 1] = f2_add(ps2[c & 1], f2_pack(p0, p1));
              out[c] = pack_bf16(p0, p1);
            }
          };
          tmem_ld32(s_addr, va);
          tmem_wait_ld32(va);
          tmem_ld32(s_addr + 32, vb);
          exp_chunk(va, pk[0]);
          tmem_wait_ld32(vb);
          tmem_ld32(s_addr + 64, va);
          exp_chunk(vb, pk[0] + 16);
          tmem_wait_ld32(va);
          tmem_ld32(s_addr + 96, vb);
          exp_chunk(va, pk[1]);
          tmem_wait_ld32(vb);
          exp_chunk(vb, pk[1] + 16);
          float s0, s1, s2, s3;
          f2_unpack(ps2[0], s0, s1);
          f2_unpack(ps2[1], s2, s3);
          tmem_st32(s_addr, pk[0]);
          tmem_st32(s_addr + 32, pk[1]);
          l_run += (s0 + s1) + (s2 + s3);
          tmem_wait_st();
          tc_fence_before();
        }
        started = true;
        mbar_arrive(bar(B_P + half));
      }
      mbar_arrive(bar(B_NFREE + (k & 1)));
      // ------------------------------------------------------- epilogue
      // Steps of this half and of the other in this segment.
      const int own = !split ? nseg : ((step & 1) == (uint32_t)half ? (nseg + 1) / 2 : nseg / 2);
      const int other = split ? nseg - own : nseg;
      auto wait_all = [&](int b, uint32_t phase) {
        return __all_sync(0xffffffffu, mbar_wait(bar(b), phase & 1, abort_flag, wait_ns)) != 0;
      };
      // Weights of the two halves' O, the row's reference and sum.
      float a0 = 1.f, a1 = 0.f, M = m_run, L = l_run;
      if (split) {
        float* own_ml = ml + ((k & 1) * 2 + half) * 2 * BM;
        own_ml[r] = m_run;
        own_ml[BM + r] = l_run;
        mbar_arrive(bar(B_ML));
        if (ok && wait_all(B_ML, ml_phase)) {
          const float* o_ml = ml + ((k & 1) * 2 + 1 - half) * 2 * BM;
          const float m1 = o_ml[r], l1 = o_ml[BM + r];
          M = fmaxf(m_run, m1);
          const float ref = (M == -INFINITY) ? 0.f : M;
          a0 = ex2(m_run - ref);
          a1 = ex2(m1 - ref);
          L = l_run * a0 + l1 * a1;
        } else {
          ok = false;
        }
        ++ml_phase;
      }
      if (ok && own > 0) ok = wait_all(B_O + half, half ? o_phase1 : o_phase0);
      if (ok && split && other > 0) ok = wait_all(B_O + 1 - half, half ? o_phase0 : o_phase1);
      if (!ok) break;
      tc_fence_after();
      if (any) {
        const int slot = 2 * cta + w.begins;
        float* part = partial_at(a.ws, grid, slot, D, sh.pair);
        const int prow = (split ? 0 : half * BM) + r;
        const int prows = BM << sh.pair;
        const float inv = 1.f / L;
        const bool whole = w.whole != 0;
        const size_t orow = ((size_t)w.b * a.nodes + node) * cv.H + (size_t)w.kvh * sh.G + hg;
        __nv_bfloat16* orow_p = static_cast<__nv_bfloat16*>(a.o) + orow * D;
        // Split: each half writes half of the columns of the joined row.
        const int c_lo = split ? half * (D / 64) : 0, c_hi = split ? c_lo + D / 64 : D / 32;
        const bool use0 = own > 0, use1 = split && other > 0;
#pragma unroll 1
        for (int c = c_lo; c < c_hi; ++c) {
          uint32_t ov[32];
          float x[32];
          if (use0) {
            tmem_ld32_sync(tmem + lane_off + tm_o(half) + c * 32, ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(ov[e]) * a0;
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = 0.f;
          }
          if (use1) {
            tmem_ld32_sync(tmem + lane_off + tm_o(1 - half) + c * 32, ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = fmaf(__uint_as_float(ov[e]), a1, x[e]);
          }
          if (live && whole) {
            uint32_t wv[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) wv[e] = pack_bf16(x[2 * e] * inv, x[2 * e + 1] * inv);
            uint4* dst = reinterpret_cast<uint4*>(orow_p + c * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              dst[e] = make_uint4(wv[4 * e], wv[4 * e + 1], wv[4 * e + 2], wv[4 * e + 3]);
          } else if (live) {
            float4* dst = reinterpret_cast<float4*>(part) + prow;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[(size_t)(c * 8 + e) * prows] =
                  make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          }
        }
        if (live && (!split || half == 0)) {
          if (whole) {
            if (a.lse) a.lse[orow] = (M + log2f(L)) * kLn2;
          } else {
            part[(size_t)prows * D + prow] = M;
            part[(size_t)prows * (D + 1) + prow] = L;
          }
        }
      }
      tc_fence_before();
      mbar_arrive(bar(B_F));
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

// Joins the partials of the units that the CTAs' ranges cut.  Block (c, y):
// rows 32 y .. 32 y + 31 of the unit that CTA c begins and does not end; lane =
// row, each of 16 warps D / 16 columns; 8 partials are read at a time.
constexpr int kJoinWarps = 16;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
join_tree_kernel(CacheView cv, TreeArgs a, Shape sh) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x, grid = gridDim.x;
  const JoinDesc jd = static_cast<const JoinDesc*>(a.ws)[c];
  if (jd.last < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int prow = blockIdx.y * 32 + lane, prows = BM << sh.pair;
  const int r = prow & (BM - 1), rg = r / sh.G;
  const int node = jd.node0 + (prow >= BM ? sh.npt : 0) + rg;
  if (rg >= sh.npt || node >= jd.cnt) return;
  constexpr int NV = D / 4 / kJoinWarps;           // float4 of a thread
  constexpr int PB = 8;                            // partials read at a time
  float M = -INFINITY, L = 0.f;
  float x[4 * NV];
#pragma unroll
  for (int e = 0; e < 4 * NV; ++e) x[e] = 0.f;
  for (int p0 = c; p0 <= jd.last; p0 += PB) {
    float m[PB], l[PB];
    float4 v[PB][NV];
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      const int p = p0 + i;
      if (p <= jd.last) {
        const float* part = partial_at(a.ws, grid, 2 * p + (p == c ? 1 : 0), D, sh.pair);
        m[i] = __ldcg(part + (size_t)prows * D + prow);
        l[i] = __ldcg(part + (size_t)prows * (D + 1) + prow);
#pragma unroll
        for (int e = 0; e < NV; ++e)
          v[i][e] = __ldcg(reinterpret_cast<const float4*>(part) +
                           (size_t)(warp * NV + e) * prows + prow);
      } else {
#pragma unroll
        for (int e = 0; e < NV; ++e) v[i][e] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    float mn = M;
#pragma unroll
    for (int i = 0; i < PB; ++i) mn = fmaxf(mn, m[i]);
    const float ref = (mn == -INFINITY) ? 0.f : mn;
    const float s0 = fast_exp2(M - ref);
    M = mn;
    L *= s0;
#pragma unroll
    for (int e = 0; e < 4 * NV; ++e) x[e] *= s0;
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      const float s = fast_exp2(m[i] - ref);
      L += l[i] * s;
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        x[4 * e] += v[i][e].x * s;
        x[4 * e + 1] += v[i][e].y * s;
        x[4 * e + 2] += v[i][e].z * s;
        x[4 * e + 3] += v[i][e].w * s;
      }
    }
  }
  const float inv = 1.f / L;                       // self is visible: L > 0
  const size_t orow =
      ((size_t)jd.b * a.nodes + node) * cv.H + (size_t)jd.kvh * sh.G + (r - rg * sh.G);
  uint2* dst = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + orow * D) + warp * NV;
#pragma unroll
  for (int e = 0; e < NV; ++e)
    dst[e] = make_uint2(pack_bf16(x[4 * e] * inv, x[4 * e + 1] * inv),
                        pack_bf16(x[4 * e + 2] * inv, x[4 * e + 3] * inv));
  if (warp == 0 && a.lse) a.lse[orow] = (M + log2f(L)) * kLn2;
}

Shape shape_of(const CacheView& cv, int nodes) {
  Shape sh;
  sh.G = cv.H / cv.Hkv;
  sh.npt = BM / sh.G;
  sh.pair = nodes > sh.npt ? 1 : 0;
  return sh;
}

// Key tiles of the largest work list.
int64_t list_bound(const CacheView& cv, int nodes, const Shape& sh) {
  if (sh.npt < 1) return INT64_MAX;
  const int per = sh.npt << sh.pair;
  const int64_t units = (int64_t)cv.B * cv.Hkv * ((nodes + per - 1) / per);
  const int64_t tiles = (cv.m_cap + BN - 1) / BN + (cv.n + BN - 1) / BN + (nodes + BN - 1) / BN;
  return units * tiles;
}

// CTAs of the launch: one per SM, no more than the largest list could feed.
int grid_of(const CacheView& cv, int nodes, const Shape& sh) {
  const int64_t most = list_bound(cv, nodes, sh) / kMinTiles;
  return (int)std::max<int64_t>(1, std::min<int64_t>(cv.sms, most));
}

template <int D>
cudaError_t launch_d(const CacheView& cv, const TreeArgs& a, cudaStream_t s) {
  const Shape sh = shape_of(cv, a.nodes);
  const int grid = grid_of(cv, a.nodes, sh);
  const uint64_t trows = (uint64_t)cv.B * a.nodes;
  const uint64_t crows = (uint64_t)cv.B * cv.Hkv * cv.slab_rows;
  CUtensorMap mq, mkc, mvc, mkt, mvt, mkc16, mvc16, mkt16, mvt16;
  if (!make_tmap_heads_bf16(&mq, a.q, D, cv.H, trows, sh.G, sh.npt) ||
      !make_tmap_rows_bf16(&mkc, cv.K, D, crows) ||
      !make_tmap_rows_bf16(&mvc, cv.V, D, crows) ||
      !make_tmap_rows_bf16(&mkt, a.k, (uint64_t)cv.Hkv * D, trows) ||
      !make_tmap_rows_bf16(&mvt, a.v, (uint64_t)cv.Hkv * D, trows) ||
      !make_tmap_rows_bf16(&mkc16, cv.K, D, crows, 16) ||
      !make_tmap_rows_bf16(&mvc16, cv.V, D, crows, 16) ||
      !make_tmap_rows_bf16(&mkt16, a.k, (uint64_t)cv.Hkv * D, trows, 16) ||
      !make_tmap_rows_bf16(&mvt16, a.v, (uint64_t)cv.Hkv * D, trows, 16))
    return cudaErrorInvalidValue;
  // Per device (the attribute belongs to the current device's context).
  cudaError_t e = cudaFuncSetAttribute(decode_tree_tc_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_dependent(decode_tree_tc_kernel<D>, dim3(grid), dim3(kThreads), kSmemBytes, s, mq,
                       mkc, mvc, mkt, mvt, mkc16, mvc16, mkt16, mvt16, cv, a, sh,
                       phase_wait_limit_ns());
  if (e != cudaSuccess) return e;
  return launch_dependent(join_tree_kernel<D>, dim3(grid, (BM << sh.pair) / 32),
                          dim3(kJoinWarps * 32), 0, s,
                          cv, a, sh);
}

}  // namespace

bool decode_tree_tc_supported(const CacheView& cv, int nodes) {
  const Shape sh = shape_of(cv, nodes);
  return list_bound(cv, nodes, sh) < (int64_t(1) << 31) && cv.dtype == RSWA_BF16 && cv.H / cv.Hkv <= BM &&
         (int64_t)cv.B * nodes < (int64_t(1) << 30) &&
         (int64_t)cv.B * cv.Hkv * cv.slab_rows + cv.n < (int64_t(1) << 31);
}

size_t decode_tree_tc_workspace(const CacheView& cv, int nodes) {
  const Shape sh = shape_of(cv, nodes);
  const size_t grid = (size_t)grid_of(cv, nodes, sh);
  return (grid * sizeof(JoinDesc) + 255) / 256 * 256 +
         grid * 2 * partial_floats(cv.d, sh.pair) * sizeof(float);
}

cudaError_t launch_decode_tree_tc(const CacheView& cv, const TreeArgs& a, cudaStream_t s) {
  return cv.d == 64 ? launch_d<64>(cv, a, s) : launch_d<128>(cv, a, s);
}

}  // namespace rswa
