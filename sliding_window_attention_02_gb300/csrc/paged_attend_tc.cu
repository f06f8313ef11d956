// Attention of a chunk of tokens over a paged cache on the 5th-generation tensor
// cores (tcgen05 + TMEM + TMA), bf16, head_dim 64 and 128.
//
//   o = sum_j exp(s_j - lse) v_j,  s_j = q . k_j / sqrt(d),  lse = log sum_j exp(s_j)
// over the tokens j that the row's token sees (paged.cuh).
//
// Rows: the G query heads of a KV head see the same keys, so a query tile is the
// rows (token, head of the group) of npt = 128 / G tokens, fetched as one
// three-dimensional TMA box.  A unit is a pair of query tiles of one (sequence, KV
// head), one for each half of the softmax warps, that read every key tile once
// between them; one without rows for a second tile is split: both halves share the
// query tile and take every other key tile.
//
// Keys: tiles of 128 tokens, those that hold a token which some row of the unit
// sees.  A tile is fetched page by page (boxes of a page's rows; halves of pages of
// 256), without the pages in which nobody sees a token.  Its product with the
// values takes only the 16-key steps that hold such a token, and in steps that also
// hold others their value rows are zeroed first (they may be any bits, and 0 x NaN
// is NaN).  A half that sees nothing of a tile leaves it out.
//
// Work: PagedPlan cuts the list of all units' tiles evenly over one CTA an SM.  A
// CTA streams its range through one TMA ring without draining between units.  Units
// cut over several CTAs leave partials (m, l, O) in the workspace, which the last
// of a unit's CTAs joins in the order of the CTAs.
//
// Roles (352 threads): warps 0-3 / 4-7 softmax and epilogue of half 0 / 1 (thread r
// owns row r = TMEM lane r), warp 8 TMA producer (a lane for each page of a tile),
// warp 9 TMEM allocator and MMA issuer, warp 10 planner: it walks the CTA's range
// ahead of the others, hands them its segments (the part of a unit inside the
// range) through shared memory and requests the query tiles.  Steps (a half's turn
// on a key tile) alternate between the halves through the whole range; the MMA
// order is QK(0) QK(1) PV(0) QK(2) PV(1) QK(3) ..., so the tensor core works on one
// half while the other half's softmax runs.  TMEM: S0 | S1 | O0 | O1, P over S.  A
// row of S is read twice, 32 columns at a time: for its maximum, then for the
// exponentials.  O is rescaled lazily (threshold 2^8, exact
// because O and l share the reference).  Every wait is bounded; on a timeout the
// CTA drains its copies and MMAs, frees TMEM and sets the pool's device flag.
//
// Bound by the chain of a half's turn: a tile of a pair takes some 2800 cycles, of which
// its products are 2048; beside it the start (plan and first loads, 12 to 15K cycles) and the
// ends of the segments (8 to 12K, a join 13K).  4096 rows of 10 heads behind 6176 tokens:
// 137 us, 172 GFLOP at 0.66 of the measured cuBLAS rate; 24 sequences of 1 to 512 rows of
// 32 / 8 heads, window 1000: 65.6.  What carried it: MMAs issued by an elected lane (20 cycles each; a lane chosen by
// comparison 70), 155 -> 147; P handed over in two parts, 147 -> 144; a cut unit joined from its
// first CTA's accumulators, 144 -> 139.5; costs of pairs and split tiles apart, 78.4 ->
// 74.1 for the ragged chunks; the rolled softmax, 74.1 -> 67.0.
#include <cuda.h>

#include <algorithm>

#include "paged.cuh"
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

// The list's costs, in units of about 1100 cycles: a tile of a pair 3, of a split unit 2,
// a unit's first tile its start and end as well.
constexpr int kTileCost = 3, kSplitCost = 2, kUnitCost = 6, kMinCost = 9;
using Plan = PagedPlan<BN, kTileCost, kSplitCost, kUnitCost, kMinCost>;

template <int D>
struct Smem {
  static constexpr int NSUB = D / 64;
  static constexpr uint32_t kTile = NSUB * kSub;             // a query, key or value tile
  static constexpr int NQ = 2;                               // query tiles
  static constexpr int NS = 8 / NSUB;                        // K/V ring slots
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_RING = NQ * kTile;
  static constexpr uint32_t OFF_ML = OFF_RING + NS * kTile;  // [2][2][2][128] floats
  static constexpr uint32_t OFF_BAR = OFF_ML + 2 * 2 * 2 * BM * 4;
  static constexpr uint32_t OFF_SEG = OFF_BAR + 512;
  static constexpr uint32_t kBytes = OFF_SEG + NSEG * 128 + 1024;   // + alignment
  static_assert(kBytes <= 232448, "shared memory of a CTA");
  // barriers
  static constexpr int B_FULL = 0;                 // NS slots landed
  static constexpr int B_EMPTY = B_FULL + NS;      // and free
  static constexpr int B_QF = B_EMPTY + NS;        // NQ query tiles landed
  static constexpr int B_QE = B_QF + NQ;           // and free
  static constexpr int B_S = B_QE + NQ;            // 2 halves: S ready
  static constexpr int B_P = B_S + 2;              // 2 halves: P of the first 64 keys written
  static constexpr int B_P2 = B_P + 2;             // and of the others
  static constexpr int B_O = B_P2 + 2;             // 2 halves: the segment's last PV done
  static constexpr int B_F = B_O + 2;              // the segment's O read out
  static constexpr int B_ML = B_F + 1;             // split: both halves' (m, l) in smem
  static constexpr int B_FIN = B_ML + 1;
  static constexpr int B_SEG = B_FIN + 1;          // NSEG segments handed over
  static constexpr int B_SFREE = B_SEG + NSEG;     // NSEG segments left by the softmax warps
  static constexpr int B_CUT = B_SFREE + NSEG;     // 2 halves: a cut unit's partial is written
  static constexpr int B_JOIN = B_CUT + 2;         // 2 halves: and who joins it is known
  static constexpr int B_ASK = B_JOIN + 2;         // 2 halves: the same before it is written
  static constexpr int NBAR = B_ASK + 2;
  static_assert(8 * NBAR + 28 + 4 * NS <= 512, "barriers");
};

__host__ __device__ constexpr uint32_t tm_s(int half) { return half ? 128u : 0u; }
__host__ __device__ constexpr uint32_t tm_o(int half) { return half ? 384u : 256u; }
constexpr uint32_t TM_COLS = 512;
constexpr float kRescaleThreshold = 8.0f;      // log2 units
constexpr uint64_t kWaitLimitNs = 1000000000ull;

struct Shape {
  int npt;      // tokens of a query tile
  int G;        // query heads of a KV head
  Divisor unit; // rows of a unit of two query tiles
  int box;      // rows of a K/V box: a page's, at most a tile's
};

// A segment as the planner hands it over.
struct Segment {
  int b, kvh, i0;         // the unit's first chunk row of the sequence
  int row0, T, tok0, m;   // tok0: the token of chunk row 0
  Hull hull;
  int np, kb;             // its tiles, as HullTiles has them
  int j0, j1;             // the tiles inside the range; j1 = 0: no more segments
  int tiles;              // the CTA's key tiles before the segment
  int first, last;        // the CTAs that a cut unit begins and ends in
  int split, whole;
  __device__ __forceinline__ int tile(int j) const { return j < np ? j : kb + (j - np); }
};
static_assert(sizeof(Segment) <= 128, "segment");

// Waits for a segment: its key tiles, and whether it is split in bit 30; 0: no
// more segments, or the wait gave up.
__device__ __noinline__ int enter_segment(uint32_t b, uint32_t phase, const Segment* w,
                                          volatile int* abort_flag, uint64_t ns) {
  if (!mbar_wait(b, phase, abort_flag, ns) || w->j1 == 0) return 0;
  return (w->j1 - w->j0) | w->split << 30;
}

// What a key tile is to the MMA issuer: the 16-key steps that hold a token which
// some row sees, and in bits 8 and 9 whether the halves see one.
__device__ __forceinline__ uint32_t tile_flags(const Hull& h, int x0) {
  uint32_t f = 0;
#pragma unroll
  for (int s = 0; s < BN / 16; ++s)
    if (h.meets(x0 + 16 * s, x0 + 16 * s + 16)) f |= 1u << s;
  return f;
}

// A partial, one of each half: O as [columns/4][128] float4 (a warp's rows are
// contiguous), then m and l.  The halves have their own rows of a pair, and half of the
// columns each of a split unit's; they are published and joined apart, as neither has
// to wait for the other.
__host__ __device__ constexpr size_t partial_floats(int D) { return (size_t)BM * (D + 2); }
__device__ __forceinline__ float* half_partial(void* ws, int p, int first, int half, int D) {
  return paged_partial(ws, p, first, 2 * partial_floats(D)) + half * partial_floats(D);
}

// A row's `chunks` chunks of 32 columns, and its lse, from the partials of CTAs first ..
// last (two at least), in their order; the reads of two are on their way together.
// The same sums in the same order as join_own's: which of them joins a unit depends on
// when its CTAs end, the result does not.
template <int D>
__device__ __noinline__ void join_row(void* ws, int first, int last, int half, int r, int chunks,
                                      __nv_bfloat16* orow, float* lse) {
  auto part = [&](int p) { return half_partial(ws, p, first, half, D); };
  auto stat = [&](int p) { return part(p) + (size_t)BM * D + r; };     // m, and l BM behind
  const float m0 = __ldcg(stat(first)), l0 = __ldcg(stat(first) + BM);
  const float m1 = __ldcg(stat(first + 1)), l1 = __ldcg(stat(first + 1) + BM);
  float M = fmaxf(m0, m1);
  for (int p = first + 2; p <= last; ++p) M = fmaxf(M, __ldcg(stat(p)));
  const float ref = M == -INFINITY ? 0.f : M;
  float L = fmaf(l1, ex2(m1 - ref), __fmul_rn(l0, ex2(m0 - ref)));
  for (int p = first + 2; p <= last; ++p)
    L = fmaf(__ldcg(stat(p) + BM), ex2(__ldcg(stat(p)) - ref), L);
  const float inv = 1.f / L;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    float x[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = 0.f;
#pragma unroll 1
    for (int p = first; p <= last; p += 2) {
      const float* a = part(p);
      const float* b = part(min(p + 1, last));
      const float4* s0 = reinterpret_cast<const float4*>(a) + (size_t)c * 8 * BM + r;
      const float4* s1 = reinterpret_cast<const float4*>(b) + (size_t)c * 8 * BM + r;
      const float w0 = ex2(__ldcg(stat(p)) - ref);
      const float w1 = p < last ? ex2(__ldcg(stat(p + 1)) - ref) : 0.f;
      float4 u[8], v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[e] = __ldcg(s0 + (size_t)e * BM);
        v[e] = __ldcg(s1 + (size_t)e * BM);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[4 * e] = fmaf(v[e].x, w1, fmaf(u[e].x, w0, x[4 * e]));
        x[4 * e + 1] = fmaf(v[e].y, w1, fmaf(u[e].y, w0, x[4 * e + 1]));
        x[4 * e + 2] = fmaf(v[e].z, w1, fmaf(u[e].z, w0, x[4 * e + 2]));
        x[4 * e + 3] = fmaf(v[e].w, w1, fmaf(u[e].w, w0, x[4 * e + 3]));
      }
    }
    store_columns(orow + c * 32, x, inv);
  }
  if (lse) *lse = (M + log2f(L)) * kLn2;
}

// The same in the CTA that begins the unit, from its own O in TMEM (t0 times a0, and t1
// times a1 where the halves share the unit; each where it has had a tile) and the partials of the CTAs behind it.
// Called by whole warps; M, L: of the CTA's own part.
template <int D>
__device__ __noinline__ void join_own(void* ws, int first, int last, int half, int r, bool live,
                                      uint32_t t0, float a0, bool use0, uint32_t t1, float a1,
                                      bool use1, float M, float L, int chunks,
                                      __nv_bfloat16* orow, float* lse) {
  auto part = [&](int p) { return half_partial(ws, p, first, half, D); };
  const float* next = part(first + 1);         // there is one part behind, mostly no more
  auto columns = [&](const float* p, int c) {
    return reinterpret_cast<const float4*>(p) + (size_t)c * 8 * BM + r;
  };
  // its columns of the chunk at hand, asked for a chunk ahead
  float4 u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    u[e] = live ? __ldcg(columns(next, 0) + (size_t)e * BM) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float m1 = live ? __ldcg(next + (size_t)BM * D + r) : -INFINITY;
  const float l1 = live ? __ldcg(next + (size_t)BM * (D + 1) + r) : 0.f;
  const float M0 = M;
  M = fmaxf(M, m1);
  for (int p = first + 2; live && p <= last; ++p)
    M = fmaxf(M, __ldcg(part(p) + (size_t)BM * D + r));
  const float ref = M == -INFINITY ? 0.f : M;
  const float own = ex2(M0 - ref), w1 = ex2(m1 - ref);
  L = fmaf(l1, w1, __fmul_rn(L, own));
  for (int p = first + 2; live && p <= last; ++p) {
    const float* a = part(p) + (size_t)BM * D + r;
    L = fmaf(__ldcg(a + BM), ex2(__ldcg(a) - ref), L);
  }
  const float inv = 1.f / L;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    float x[32];
    uint32_t ov[32];
    float4 v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = u[e];
      if (live && c + 1 < chunks) u[e] = __ldcg(columns(next, c + 1) + (size_t)e * BM);
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = 0.f;
    if (use0) {
      tmem_ld32_sync(t0 + c * 32, ov);
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(ov[e]) * a0;
    }
    if (use1) {
      tmem_ld32_sync(t1 + c * 32, ov);
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = fmaf(__uint_as_float(ov[e]), a1, x[e]);
    }
    if (!live) continue;
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = __fmul_rn(x[e], own);
    auto add = [&](const float4* w, float wp) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[4 * e] = fmaf(w[e].x, wp, x[4 * e]);
        x[4 * e + 1] = fmaf(w[e].y, wp, x[4 * e + 1]);
        x[4 * e + 2] = fmaf(w[e].z, wp, x[4 * e + 2]);
        x[4 * e + 3] = fmaf(w[e].w, wp, x[4 * e + 3]);
      }
    };
    add(v, w1);
#pragma unroll 1
    for (int p = first + 2; p <= last; ++p) {
      const float wp = ex2(__ldcg(part(p) + (size_t)BM * D + r) - ref);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __ldcg(columns(part(p), c) + (size_t)e * BM);
      add(v, wp);
    }
    store_columns(orow + c * 32, x, inv);
  }
  if (lse && live) *lse = (M + log2f(L)) * kLn2;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
paged_attend_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, PagesView pv, BatchArgs ba,
                       AttendArgs a, Shape sh, uint64_t wait_ns) {
  using SM = Smem<D>;
  constexpr int NSUB = SM::NSUB, NS = SM::NS, NQ = SM::NQ;
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
  volatile int* never = reinterpret_cast<volatile int*>(smem + SM::OFF_BAR + 8 * NBAR + 8);
  volatile int* joiner = reinterpret_cast<volatile int*>(smem + SM::OFF_BAR + 8 * NBAR + 12);
  // flags of the tile in each ring slot (tile_flags)
  volatile uint32_t* slot_flags =
      reinterpret_cast<volatile uint32_t*>(smem + SM::OFF_BAR + 8 * NBAR + 28);
  const Segment* segs = reinterpret_cast<const Segment*>(smem + SM::OFF_SEG);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int k = 0; k < NBAR; ++k)
      mbar_init(bar(k), (k >= SM::B_P && k < SM::B_O) || (k >= SM::B_CUT && k < SM::B_JOIN) ? 128u
                        : (k == SM::B_F || k == SM::B_ML ||
                           (k >= SM::B_SFREE && k < SM::B_SFREE + NSEG))
                            ? 256u
                            : 1u);
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
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
    uint32_t gi = 0;                             // loads issued
    bool ok = true;
    Segment w;
    for (int k = 0; ok && __all_sync(0xffffffffu, segment(k, w)) && w.j1 > 0; ++k) {
      // This lane's box of tile j: its page, or -1 where no row sees a token of it.
      auto page_of = [&](int j) {
        const int t0 = w.tile(j) * BN + lane * sh.box;
        if (lane * sh.box >= BN || !w.hull.meets(t0, t0 + sh.box)) return -1;
        return page_at(pv, ba, w.b, t0 >> pv.log2P);
      };
      int page = page_of(w.j0);
      for (int j = w.j0; ok && j < w.j1; ++j) {
        const int next = j + 1 < w.j1 ? page_of(j + 1) : -1;
        const int x0 = w.tile(j) * BN, t0 = x0 + lane * sh.box;
        const int row = (page * pv.Hkv + w.kvh) * pv.P + (t0 & (pv.P - 1));
        const uint32_t bytes =
            __popc(__ballot_sync(0xffffffffu, page >= 0)) * (uint32_t)(sh.box * 128 * NSUB);
        uint32_t flags = tile_flags(w.hull, x0) | 0x300u;
        if (!w.split) {
          // the halves' own tokens: the second has one at least
          const int a0 = w.tok0 + w.i0, a1 = a0 + sh.npt;
          if (!Hull(a0, a1 - 1, w.m, ba.window).meets(x0, x0 + BN)) flags &= ~0x100u;
          if (!Hull(a1, w.hull.end - 1, w.m, ba.window).meets(x0, x0 + BN)) flags &= ~0x200u;
        }
#pragma unroll 1
        for (int isv = 0; isv < 2; ++isv, ++gi) {
          const uint32_t s = gi % NS;
          if (gi >= (uint32_t)NS &&
              !__all_sync(0xffffffffu, wait_for(bar(SM::B_EMPTY + s), ((gi / NS) - 1) & 1,
                                                 abort_flag, wait_ns))) {
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
              tma_load_2d(dst + c * kSub, isv ? &tmV : &tmK, c * 64, row, bar(SM::B_FULL + s));
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
    // One lane issues.  Step s: PV of step s - 2, then QK of step s, both of half
    // s & 1.  What the lane does between the products holds the tensor core up, so
    // descriptors advance by constants and the rare paths are out of line.
    if (elect_one()) {
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
        c.left = x & 0x3fffffff;
        c.split = x >> 30;
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
      uint32_t begun = 0;                // halves whose O holds a product of the segment
      // O_h (+)= P_h V, of the steps that hold keys; S_h = Q_h K^T.
      // pv waits for the two parts of P in turn; false: the wait gave up.
      auto pv = [&](uint32_t half, uint32_t slot, uint32_t flags, uint32_t phase) {
        const uint64_t vd = vdesc + (uint64_t)(slot * (kTile >> 4));
        const bool used = flags >> (8 + half) & 1u;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (!wait((part ? SM::B_P2 : SM::B_P) + half, phase)) return false;
          tc_fence_after();
          if (!used) continue;
          uint32_t acc = begun >> half & 1u;
          if ((flags & 0xffu) == 0xffu) {
            begun |= 1u << half;
#pragma unroll
            for (int k = 4 * part; k < 4 * part + 4; ++k)
              mma_bf16_ts(tmem + tm_o(half), tmem + tm_s(half) + k * 8, vd + k * 128, idesc_pv,
                          k > 0 ? 1u : acc);
          } else {
#pragma unroll 1
            for (int k = 4 * part; k < 4 * part + 4; ++k)
              if (flags >> k & 1u) {
                mma_bf16_ts(tmem + tm_o(half), tmem + tm_s(half) + k * 8, vd + k * 128, idesc_pv,
                            acc);
                acc = 1u;
                begun |= 1u << half;
              }
          }
        }
        return true;
      };
      auto qk = [&](uint32_t half, uint32_t slot, uint32_t qt, uint32_t flags) {
        if (flags >> (8 + half) & 1u) {
          const uint64_t kd = kdesc + (uint64_t)(slot * (kTile >> 4));
          const uint64_t qd = qdesc + (uint64_t)((qt % NQ) * (kTile >> 4));
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * kSub + (k & 3) * 32) >> 4;
            mma_bf16_ss(tmem + tm_s(half), qd + off, kd + off, idesc_qk, k > 0);
          }
        }
        mma_commit(bar(SM::B_S + half));
      };
#pragma unroll 1
      for (uint32_t s = 0; pmore; ++s) {
        const uint32_t half = s & 1;
        // Inside a pair's segment: both halves' turns on a tile in a row, PV of tile
        // t and QK of t + 1, without a question about segments, and with the waits
        // for loads before those for the softmax.
        if (half == 0 && s >= 2 && pfresh == 0 && qfresh == 0 && !pc.split && pc.k == qc.k &&
            !pc.second && !qc.second && qc.left > 1) {
          bool ok = true;
#pragma unroll 1
          for (; qc.left > 1; s += 2) {
            ok = wait(SM::B_FULL + pc.slot, pc.phase) && wait(SM::B_FULL + qc.slot, qc.phase);
            if (!ok) break;
            const uint32_t fv = slot_flags[pc.slot], fk = slot_flags[qc.slot];
            if (!(ok = pv(0, pc.slot, fv, (s >> 1) - 1))) break;
            qk(0, qc.slot, qc.q, fk);
            if (!(ok = pv(1, pc.slot, fv, (s >> 1) - 1))) break;
            mma_commit(bar(SM::B_EMPTY + pc.slot));
            qk(1, qc.slot, qc.q + 1, fk);
            mma_commit(bar(SM::B_EMPTY + qc.slot));
            for (Cursor* c : {&pc, &qc}) {
              c->slot += 2;
              if (c->slot >= (uint32_t)NS) {
                c->slot -= NS;
                c->phase ^= 1;
              }
              --c->left;
            }
          }
          if (!ok) break;
        }
        if (s >= 2) {
          const bool last = pc.left <= (pc.split ? 2 : 1);
          if (pfresh > 0) {
            --pfresh;
            if (pc.k > 0 && !wait(SM::B_F, pc.k - 1)) break;
          }
          if (!pc.second && !wait(SM::B_FULL + pc.slot, pc.phase)) break;
          if (!pv(half, pc.slot, slot_flags[pc.slot], (s >> 1) - 1)) break;
          if (pc.split || pc.second) mma_commit(bar(SM::B_EMPTY + pc.slot));
          if (last) mma_commit(bar(SM::B_O + half));
          const int at = pc.k;
          pmore = advance(pc);
          if (pc.k != at) {
            pfresh = pc.split && pc.left == 1 ? 1 : 2;
            begun = 0;
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
          qk(half, qc.slot, qt, slot_flags[qc.slot]);
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
    if (lane == 0) prefetch_tmap(&tmQ);
    int qi = 0, tiles = 0;                       // query tiles requested, key tiles planned
    int k = 0;
    Plan plan(pv, ba, sh.unit);
    for (bool more = plan.start(cta, gridDim.x); more; more = plan.next()) {
      const PagedUnit& u = plan.u;
      Segment w;
      w.b = u.b;
      w.kvh = u.kvh;
      w.i0 = u.f0 / pv.by_G;
      w.row0 = u.seq.row0;
      w.T = u.seq.T;
      w.tok0 = u.seq.L - u.seq.T;
      w.m = u.seq.m;
      w.hull = u.hull;
      w.np = u.np;
      w.kb = u.kb;
      w.j0 = u.j0;
      w.j1 = u.j1;
      w.tiles = tiles;
      w.first = u.first;
      w.last = u.last;
      // A unit without rows for a second query tile.
      w.split = w.i0 + sh.npt >= w.T;
      w.whole = u.whole();
      tiles += w.j1 - w.j0;
      // The slot's last segment has been left by the softmax warps, the last to
      // leave it (their epilogue follows every step of the others).
      if (k >= NSEG && !__all_sync(0xffffffffu, wait_for(bar(SM::B_SFREE + k % NSEG),
                                                          (k / NSEG - 1) & 1, abort_flag,
                                                          wait_ns)))
        break;
      if (lane == 0) {
        out[k % NSEG] = w;
        mbar_arrive(bar(SM::B_SEG + k % NSEG));
      }
      ++k;
      // its query tiles, once their buffers are free
      bool ok = true;
      for (int x = 0; ok && x < (w.split ? 1 : 2); ++x, ++qi) {
        const int s = qi % NQ;
        ok = qi < NQ || __all_sync(0xffffffffu, wait_for(bar(SM::B_QE + s), (qi / NQ - 1) & 1,
                                                         abort_flag, wait_ns));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(SM::B_QF + s), (uint32_t)NSUB * sh.npt * sh.G * 128u);
#pragma unroll
          for (int c = 0; c < NSUB; ++c)
            tma_load_3d(sb + SM::OFF_Q + s * kTile + c * kSub, &tmQ, c * 64, w.kvh * sh.G,
                        w.row0 + w.i0 + x * sh.npt, bar(SM::B_QF + s));
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    // No more segments: once the slot is free, or at once where all give up.
    if (k >= NSEG)
      __all_sync(0xffffffffu, wait_for(bar(SM::B_SFREE + k % NSEG), (k / NSEG - 1) & 1,
                                       abort_flag, wait_ns));
    if (lane == 0) {
      if (!*abort_flag) out[k % NSEG].j1 = 0;
      if (!*abort_flag) mbar_arrive(bar(SM::B_SEG + k % NSEG));
      // Drain: every copy issued has landed before the CTA may exit.
      for (int x = max(qi - NQ, 0); x < qi; ++x)
        wait_for(bar(SM::B_QF + x % NQ), (x / NQ) & 1, never, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp < kProducerWarp) {
    // -------------------------------------------------- softmax and epilogue
    const int half = warp >> 2;
    const int r = threadIdx.x & 127;                    // row of the query tile
    const int rg = r / pv.by_G, hg = r - rg * sh.G;        // its token in the tile, its head
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const float sl2 = rsqrtf((float)D) * kLog2e;
    const uint32_t s_addr = tmem + lane_off + tm_s(half);
    const uint32_t o_addr = tmem + lane_off + tm_o(half);
    const int n = ba.window;
    float* ml = reinterpret_cast<float*>(smem + SM::OFF_ML);
    uint32_t step = 0, turns = 0;                       // steps before; this half's among them
    uint32_t o_phase0 = 0, o_phase1 = 0, ml_phase = 0;  // segments with steps of each half; split
    uint32_t cut_phase = 0;
    bool ok = true;
    Segment w;
    for (int k = 0;; ++k) {
      if (!__all_sync(0xffffffffu, segment(k, w)) || w.j1 == 0) break;
      const bool split = w.split != 0;
      const int nseg = w.j1 - w.j0;
      const int i = w.i0 + (split ? 0 : half * sh.npt) + rg;       // row of the chunk
      const bool live = rg < sh.npt && i < w.T;
      const bool any = __any_sync(0xffffffffu, live);
      const int tok = w.tok0 + i;
      // the half's first and last token, and what they see
      const int a0 = w.tok0 + w.i0 + (split ? 0 : half * sh.npt);
      const int a1 = min(a0 + sh.npt, w.tok0 + w.T) - 1;
      const Hull own_hull(a0, a1, w.m, n);
      float m_run = -INFINITY, l_run = 0.f;
      bool started = false;
      for (int j = w.j0; j < w.j1; ++j) {
        if (split && ((step + (uint32_t)(j - w.j0)) & 1) != (uint32_t)half) continue;
        const int x0 = w.tile(j) * BN;
        // every column is a token that every row sees
        const bool full = x0 + BN - 1 <= a0 && (x0 + BN <= w.m || x0 > a1 - n);
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
        if (any && !full) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            see[c] = range_mask(0, min(w.m - 1, tok) - x0, c) |
                     range_mask(max(tok - n + 1, 0) - x0, tok - x0, c);
        }
        if (!__all_sync(0xffffffffu,
                        wait_for(bar(SM::B_S + half), turns & 1, abort_flag, wait_ns))) {
          ok = false;
          break;
        }
        ++turns;
        tc_fence_after();
        // Value rows that no row of the unit sees, in steps that hold others that one
        // does (where the prefix ends, the window begins and the chunk ends): zero,
        // as 0 x NaN is NaN.
        const int p = w.hull.p, w0 = w.hull.w0, end = w.hull.end;
        auto edge = [&](int e) { return (e & 15) != 0 && e >> 7 == x0 >> 7; };
        if ((warp & 3) == 0 && ((p < w0 && (edge(p) || edge(w0))) || edge(end))) {
          const uint32_t vi = 2u * (uint32_t)(w.tiles + j - w.j0) + 1u;
          if (__all_sync(0xffffffffu, wait_for(bar(SM::B_FULL + vi % NS), (vi / NS) & 1,
                                                abort_flag, wait_ns))) {
#pragma unroll 1
            for (int z = 0; z < 3; ++z) {
              const int e = z == 0 ? p : z == 1 ? w0 : end;
              if (!edge(e) || (z < 2 && p >= w0)) continue;
              const int t = e & ~15;                     // the step's first token
              uint8_t* v = smem + SM::OFF_RING + (vi % NS) * kTile + (t - x0) * 128 + lane * 16;
#pragma unroll
              for (int y = 0; y < 16; y += 4)            // a row is 8 lanes
                if (!w.hull.has(t + y + (lane >> 3))) {
#pragma unroll
                  for (int c = 0; c < NSUB; ++c)
                    *reinterpret_cast<uint4*>(v + y * 128 + c * kSub) = make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();
          }
        }
        const bool used = own_hull.meets(x0, x0 + BN);
        if (any && used) {
          // In loops of 64 columns: with the row in registers and all 128 columns
          // unrolled the warps waited for instructions (74.1 us for 24 ragged chunks
          // behind their prefixes, 67 in loops; one loop of 32 columns: 67.7, but a
          // chunk behind 20K tokens 146.6 instead of 137).
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
            tmem_wait_ld32(va);
          } else {                                       // masked scores: -inf, back in S
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t m4 = see[0];
              see[0] = see[1];
              see[1] = see[2];
              see[2] = see[3];
              tmem_ld32_sync(s_addr + 32 * c, va);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(m4 >> e & 1u)) va[e] = 0xff800000u;
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
            for (int c = 0; started && c < D; c += 16) {
              uint32_t ov[16];
              tmem_ld16(o_addr + c, ov);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e)
                ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              tmem_st16(o_addr + c, ov);
            }
          }
          // P over S, and its sum.  P is rounded to bf16 (2^-8 of it) for the product with
          // V, whose two operands are of one 16-bit type; l sums it unrounded.  What the
          // rounding takes off as a second operand doubles that product: 4096 rows behind 6176
          // tokens 174.6 us instead of 137.6, 24 ragged chunks 73.1 instead of 65.6, for an
          // error of the output of 0.0017 instead of 0.0023.
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
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            tmem_ld32(s_addr + 64 * c + 32, vb);
            exponentials(va, s_addr + 32 * c);
            tmem_wait_ld32(vb);
            if (c == 0) tmem_ld32(s_addr + 64, va);
            exponentials(vb, s_addr + 32 * c + 16);
            tmem_wait_ld32(va);
            if (c == 0) {
              tmem_wait_st();
              tc_fence_before();
              mbar_arrive(bar(SM::B_P + half));
            }
          }
          float s0, s1;
          f2_unpack(ps2, s0, s1);
          l_run += s0 + s1;
          tmem_wait_st();
          tc_fence_before();
        } else {
          mbar_arrive(bar(SM::B_P + half));
        }
        started = started || used;
        mbar_arrive(bar(SM::B_P2 + half));
      }
      // ------------------------------------------------------- epilogue
      // Steps of this half and of the other in this segment.
      const int own = !split ? nseg : ((step & 1) == (uint32_t)half ? (nseg + 1) / 2 : nseg / 2);
      const int other = split ? nseg - own : nseg;
      auto wait_all = [&](int b, uint32_t phase) {
        return __all_sync(0xffffffffu, wait_for(bar(b), phase & 1, abort_flag, wait_ns)) != 0;
      };
      // The CTA that begins a cut unit comes to it at the end of its range, the others
      // at the start of theirs: as a rule it is the last, and adds their parts to its
      // own O as it writes the rows, without leaving one itself (half of the partials'
      // traffic, which is what cut units cost).  It asks early: the answer comes while
      // the last products run.
      const bool ask = ok && !w.whole && w.j0 == 0;
      if (ask && r == 0) {
        int32_t* count = paged_counter(a.ws, 2 * w.first + half);
        joiner[2 + half] = load_acquire(count) == w.last - w.first;
        if (joiner[2 + half]) *count = 0;               // ready for the next call
        mbar_arrive(bar(SM::B_ASK + half));
      }
      // Weights of the two halves' O, the row's reference and sum.
      float a0w = 1.f, a1w = 0.f, M = m_run, L = l_run;
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
          a0w = ex2(m_run - ref);
          a1w = ex2(m1 - ref);
          // The same bits in both halves (no fma).
          L = __fadd_rn(__fmul_rn(l_run, a0w), __fmul_rn(l1, a1w));
        } else {
          ok = false;
        }
        ++ml_phase;
      }
      if (ok && own > 0) ok = wait_all(SM::B_O + half, half ? o_phase1 : o_phase0);
      if (ok && split && other > 0) ok = wait_all(SM::B_O + 1 - half, half ? o_phase0 : o_phase1);
      bool joins = false;
      if (ok && ask) {                                  // once a launch: its last unit
        ok = wait_all(SM::B_ASK + half, 0);
        joins = ok && joiner[2 + half] != 0;
      }
      if (!ok) break;
      tc_fence_after();
      const size_t orow = ((size_t)w.row0 + i) * pv.H + (size_t)w.kvh * sh.G + hg;
      __nv_bfloat16* orow_p = static_cast<__nv_bfloat16*>(a.o) + orow * D;
      // Split: each half writes half of the columns of the joined row.
      const int c_lo = split ? half * (D / 64) : 0, c_hi = split ? c_lo + D / 64 : D / 32;
      if (joins) {
        if (any)
          join_own<D>(a.ws, w.first, w.last, half, r, live, tmem + lane_off + tm_o(half) + c_lo * 32,
                      a0w, started, tmem + lane_off + tm_o(1 - half) + c_lo * 32, a1w,
                      split && other > 0, M, L, c_hi - c_lo, orow_p + c_lo * 32,
                      a.lse && (!split || half == 0) ? a.lse + orow : nullptr);
        tc_fence_before();
        mbar_arrive(bar(SM::B_F));
      } else if (any) {
        float* part = half_partial(a.ws, cta, w.first, half, D);
        const float inv = 1.f / L;
        const bool use0 = started, use1 = split && other > 0;
#pragma unroll 1
        for (int c = c_lo; c < c_hi; ++c) {
          float x[32];
          uint32_t ov[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 0.f;
          if (use0) {
            tmem_ld32_sync(tmem + lane_off + tm_o(half) + c * 32, ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(ov[e]) * a0w;
          }
          if (use1) {
            tmem_ld32_sync(tmem + lane_off + tm_o(1 - half) + c * 32, ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = fmaf(__uint_as_float(ov[e]), a1w, x[e]);
          }
          if (live && w.whole) {
            store_columns(orow_p + c * 32, x, inv);
          } else if (live) {
            float4* dst = reinterpret_cast<float4*>(part) + (size_t)(c - c_lo) * 8 * BM + r;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[(size_t)e * BM] =
                  make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          }
        }
        tc_fence_before();
        mbar_arrive(bar(SM::B_F));
        if (live) {
          if (!w.whole) {
            part[(size_t)BM * D + r] = M;
            part[(size_t)BM * (D + 1) + r] = L;
          } else if (a.lse && (!split || half == 0)) {
            a.lse[orow] = (M + log2f(L)) * kLn2;
          }
        }
      } else {
        tc_fence_before();
        mbar_arrive(bar(SM::B_F));
      }
      if (!w.whole && !joins) {
        mbar_arrive(bar(SM::B_CUT + half));
        if (r == 0 && wait_for(bar(SM::B_CUT + half), cut_phase & 1, abort_flag, wait_ns)) {
          int32_t* count = paged_counter(a.ws, 2 * w.first + half);
          const bool last = arrive_acq_rel(count) == w.last - w.first;
          if (last) *count = 0;                         // ready for the next call
          joiner[half] = last;
          mbar_arrive(bar(SM::B_JOIN + half));
        }
        if (!wait_all(SM::B_JOIN + half, cut_phase)) break;
        ++cut_phase;
        if (joiner[half] && live)
          join_row<D>(a.ws, w.first, w.last, half, r, c_hi - c_lo, orow_p + c_lo * 32,
                      a.lse && (!split || half == 0) ? a.lse + orow : nullptr);
      }
      mbar_arrive(bar(SM::B_SFREE + k % NSEG));
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
  if (threadIdx.x == 0 && *abort_flag) flag_error(pv.err, kErrWaitTimeout);
}

int grid_of(const PagesView& pv) { return std::min(std::max(pv.sms, 1), kMaxPagedCtas / 2); }

template <int D>
cudaError_t launch_d(const PagesView& pv, const PagesMaps& maps, const BatchArgs& ba,
                     const AttendArgs& a, cudaStream_t s) {
  Shape sh;
  sh.G = pv.G;
  sh.npt = BM / sh.G;
  sh.unit = Divisor(2 * sh.npt * sh.G);
  sh.box = std::min(pv.P, BN);
  CUtensorMap mq;
  const int64_t stride = ba.rows < 2 ? (int64_t)pv.H * D : a.q_stride;
  if (!make_tmap_heads_bf16(&mq, a.q, D, pv.H, ba.rows, sh.G, sh.npt, stride))
    return cudaErrorInvalidValue;
  // Per device (the attribute belongs to the current device's context).
  cudaError_t e = cudaFuncSetAttribute(paged_attend_tc_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_attend_tc_kernel<D>, dim3(grid_of(pv)), dim3(kThreads),
                          Smem<D>::kBytes, s, mq, maps.k, maps.v, pv, ba, a, sh,
                          phase_wait_limit_ns());
}

}  // namespace

bool make_pages_maps(const PagesView& pv, PagesMaps* maps) {
  const uint64_t rows = (uint64_t)pv.pages * pv.Hkv * pv.P;
  const uint32_t box = (uint32_t)std::min(pv.P, BN);
  return make_tmap_rows_bf16(&maps->k, pv.K, pv.d, rows, box) &&
         make_tmap_rows_bf16(&maps->v, pv.V, pv.d, rows, box) &&
         make_tmap_rows_bf16(&maps->k32, pv.K, pv.d, rows, std::min(box, 32u)) &&
         make_tmap_rows_bf16(&maps->v32, pv.V, pv.d, rows, std::min(box, 32u));
}

bool paged_attend_tc_supported(const PagesView& pv) {
  return pv.dtype == RSWA_BF16 && pv.G <= BM;
}

size_t paged_attend_tc_workspace(const PagesView& pv) {
  return kPagedCounterBytes + (size_t)grid_of(pv) * 2 * 2 * partial_floats(pv.d) * sizeof(float);
}

cudaError_t launch_paged_attend_tc(const PagesView& pv, const PagesMaps& maps, const BatchArgs& ba,
                                   const AttendArgs& a, cudaStream_t s) {
  return pv.d == 64 ? launch_d<64>(pv, maps, ba, a, s) : launch_d<128>(pv, maps, ba, a, s);
}

}  // namespace rswa
