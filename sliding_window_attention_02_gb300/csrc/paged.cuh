// Device helpers of the paged-cache kernels: a sequence as the batch describes
// it, the keys that a range of its tokens sees, and the planner that cuts the
// work of a launch into equal ranges.
//
// Token x of sequence b is row x % P of page table[b][x / P].  Row i of the
// chunk's T_b rows is token a = lens[b] - T_b + i, and sees token j <= a when
// j < m_b or j > a - n.
#pragma once

#include "rswa_device.cuh"
#include "rswa_internal.h"

namespace rswa {

__device__ __forceinline__ int operator/(int x, const Divisor& by) {
  return (int)(__umulhi((uint32_t)x << 1, by.m) >> by.s);
}
__device__ __forceinline__ int operator%(int x, const Divisor& by) { return x - x / by * by.d; }
// a / b, a >= 0, b > 0; both mostly fit 32 bits, where a division is far shorter.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// A sequence of the batch.  One that the batch describes wrongly (rows or a
// length outside their range, more rows than tokens) is flagged and taken as empty.
struct PagedSeq {
  int row0, T, L, m;
  __device__ __forceinline__ void load(const PagesView& pv, const BatchArgs& ba, int b) {
    int r1;
    if (ba.starts) {
      row0 = ba.starts[b];
      r1 = ba.starts[b + 1];
    } else {
      row0 = b * ba.each;
      r1 = row0 + ba.each;
    }
    L = ba.lens[b];
    m = ba.prefix ? ba.prefix[b] : 0;
    T = r1 - row0;
    if (row0 < 0 || r1 < row0 || r1 > ba.rows || L < 0 || L > ba.cap || T > L) {
      flag_error(pv.err, kErrBadBatch);
      T = L = 0;
    }
    m = min(max(m, 0), L);
  }
};

// The sequence of chunk row `row`, found by a whole warp; T is 0 where it is nobody's.  Of
// 32 sequences, every lane reads one: where their rows are and what the one that is found
// needs, in one go.  Each range is looked at for itself, so that a wrong one, which need not
// lie between its neighbours, hides no other.
__device__ __forceinline__ int find_row(const PagesView& pv, const BatchArgs& ba, int row,
                                        PagedSeq& s) {
  if (!ba.starts) {
    const int b = row / ba.each;
    s.load(pv, ba, b);
    return b;
  }
  const int lane = (int)(threadIdx.x & 31);
  s.row0 = s.T = s.L = s.m = 0;
  for (int b0 = 0; b0 < ba.B; b0 += 32) {
    PagedSeq mine;
    mine.row0 = mine.T = mine.L = mine.m = 0;
    if (b0 + lane < ba.B) mine.load(pv, ba, b0 + lane);
    const uint32_t on =
        __ballot_sync(0xffffffffu, row >= mine.row0 && row < mine.row0 + mine.T);
    if (!on) continue;
    const int src = __ffs(on) - 1;
    s.row0 = __shfl_sync(0xffffffffu, mine.row0, src);
    s.T = __shfl_sync(0xffffffffu, mine.T, src);
    s.L = __shfl_sync(0xffffffffu, mine.L, src);
    s.m = __shfl_sync(0xffffffffu, mine.m, src);
    return b0 + src;
  }
  return 0;
}

// Page `x` of sequence b; one outside the pool is flagged and read as page 0.  In two
// halves, its read and what waits for it.
__device__ __forceinline__ int page_entry(const BatchArgs& ba, int b, int x) {
  return ba.table[(size_t)b * ba.max_pages + x];
}
__device__ __forceinline__ int page_of_entry(const PagesView& pv, int p) {
  if ((unsigned)p < (unsigned)pv.pages) return p;
  flag_error(pv.err, kErrBadBatch);
  return 0;
}
__device__ __forceinline__ int page_at(const PagesView& pv, const BatchArgs& ba, int b, int x) {
  return page_of_entry(pv, page_entry(ba, b, x));
}

// Tokens that some of the tokens a0 .. a1 see: [0, p) and [w0, end), p <= w0 <= end.
struct Hull {
  int p, w0, end;
  __device__ __forceinline__ Hull() {}
  __device__ __forceinline__ Hull(int a0, int a1, int m, int n) {
    end = a1 + 1;
    p = min(m, end);
    w0 = max(p, a0 - n + 1);
  }
  __device__ __forceinline__ int keys() const { return p + end - w0; }
  __device__ __forceinline__ bool has(int t) const { return t < p || (t >= w0 && t < end); }
  // whether a token of [lo, hi) is one of them
  __device__ __forceinline__ bool meets(int lo, int hi) const {
    return lo < p || (hi > w0 && lo < end);
  }
};

// Tiles of `TILE` tokens (tile x holds tokens x * TILE on) that hold one of a hull's:
// prefix tiles 0 .. np - 1, then band tiles kb on.
template <int TILE>
struct HullTiles {
  int np, kb, nt;
  __device__ __forceinline__ HullTiles() {}
  __device__ __forceinline__ explicit HullTiles(const Hull& h) {
    np = (h.p + TILE - 1) / TILE;
    kb = max(h.w0 / TILE, np);
    nt = np + max(0, (h.end + TILE - 1) / TILE - kb);
  }
};

// Where a CTA's walk over the work list stands: a unit (a number of rows (token,
// head of the group) of one KV head) and its tiles [j0, j1) in the CTA's range.
struct PagedUnit {
  int b, kvh;
  int f0;                 // first of its rows: token f0 / G of the chunk, head f0 % G
  PagedSeq seq;
  Hull hull;
  int np, kb, nt;         // its tiles, as HullTiles has them
  int j0, j1;
  int first, last;        // CTAs that it begins and ends in
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == nt; }
};

// The planner, run by one whole warp with the same state in every lane.  The
// tiles of a unit after each other, unit after unit (sequence by sequence, its rows
// in order, the KV heads of the same rows next to each other), form one list; a tile
// costs COST, or SPLIT in units with half of the rows or fewer, a unit's first one EXTRA
// more.  CTA c of `ctas` takes the tiles that begin in [from(c), from(c + 1)).
//
// A group, the units of the same rows, is one entry of the sums that find a CTA's
// range: 32 groups at a time, a lane each.  What a launch waits for before its first
// loads is this code, run once: it is kept short (40 pages, one sequence of 16 groups:
// 2.7 us; with sums sequence by sequence and 64-bit divisions 4 to 5; with divisions by G
// and by a unit's rows instead of multiplications 24 ragged chunks took 67.8 us for 66.2).
template <int TILE, int COST, int SPLIT, int EXTRA, int MINCOST>
struct PagedPlan {
  static_assert(MINCOST >= COST + EXTRA && COST >= SPLIT, "a range holds a tile at least");
  using Tiles = HullTiles<TILE>;
  const PagesView& pv;
  const BatchArgs& ba;
  const Divisor& unit;                           // rows of a unit
  int lane;
  int64_t total = 0, x1 = 0;
  int ctas = 1;
  PagedUnit u;
  int64_t ubase = 0;
  bool half = false;                             // the unit's tiles cost SPLIT

  __device__ __forceinline__ PagedPlan(const PagesView& pv_, const BatchArgs& ba_, const Divisor& rows)
      : pv(pv_), ba(ba_), unit(rows), lane((int)(threadIdx.x & 31)) {}

  // Finds the start of this CTA's range; false: it has none.
  __device__ bool start(int cta, int grid) {
    PagedSeq s = lane_seq(lane);
    int inc = 0;                                 // groups of the block's sequences up to a lane's
    int64_t groups = 0;
    int64_t c0 = 0, c1 = 0;                      // inclusive costs of the first 64 groups
    for (int b0 = 0; b0 < ba.B; b0 += 32) {
      if (b0 > 0) s = lane_seq(b0 + lane);
      inc = scan(groups_of(s));
      const int count = __shfl_sync(0xffffffffu, inc, 31);
      for (int g0 = 0; g0 < count; g0 += 32) {
        const int64_t c = scan(group_cost(s, inc, count, g0));
        if (b0 == 0 && g0 == 0) c0 = c;
        if (b0 == 0 && g0 == 32) c1 = c;
        total += __shfl_sync(0xffffffffu, c, 31);
      }
      groups += count;
    }
    if (total == 0) return false;
    const int64_t units = groups * pv.Hkv;
    ctas = (int)min((int64_t)grid, max((int64_t)1, total / MINCOST));
    // Few units have the same number of CTAs each, if they are alike: their ends
    // meet CTAs' ends.
    if (units < ctas) ctas -= ctas % (int)units;
    if (cta >= ctas) return false;
    const int64_t x0 = from(cta);
    x1 = from(cta + 1);
    int64_t base = 0;
    for (int b0 = 0;; b0 += 32) {
      if (ba.B > 32) {
        s = lane_seq(b0 + lane);
        inc = scan(groups_of(s));
      }
      const int count = __shfl_sync(0xffffffffu, inc, 31);
      for (int g0 = 0; g0 < count; g0 += 32) {
        const bool known = b0 == 0 && g0 < 64;
        const int64_t c = known ? (g0 == 0 ? c0 : c1) : scan(group_cost(s, inc, count, g0));
        const uint32_t up = __ballot_sync(0xffffffffu, base + c <= x0);   // groups before
        if (up == 0xffffffffu) {
          base += __shfl_sync(0xffffffffu, c, 31);
          continue;
        }
        const int at = __popc(up);
        if (at > 0) base += __shfl_sync(0xffffffffu, c, at - 1);
        // its sequence, and its place there
        const int g = g0 + at;
        const int src = __popc(__ballot_sync(0xffffffffu, inc <= g));
        take(s, b0, src);
        const int before = src > 0 ? __shfl_sync(0xffffffffu, inc, src - 1) : 0;
        enter(g - before);
        u.kvh = (int)quotient(x0 - base, unit_cost());
        ubase = base + (int64_t)u.kvh * unit_cost();
        u.j0 = at_cost(x0 - ubase);
        return u.j0 < u.nt ? clip() : next();
      }
    }
  }

  // The next unit of the range; false: there is none.
  __device__ bool next() {
    ubase += unit_cost();
    if (ubase >= x1) return false;
    u.j0 = 0;
    if (++u.kvh == pv.Hkv) {
      u.kvh = 0;
      int q = u.f0 / unit + 1;
      if (q * unit.d >= u.seq.T * pv.G) {
        q = 0;
        // sequences without rows are passed over; there is one with some, as the
        // list goes on
        for (int b0 = u.b + 1; b0 < ba.B; b0 += 32) {
          const PagedSeq s = lane_seq(b0 + lane);
          const uint32_t live = __ballot_sync(0xffffffffu, s.T > 0);
          if (!live) continue;
          take(s, b0, __ffs(live) - 1);
          break;
        }
      }
      enter(q);
    }
    return clip();
  }

 private:
  // Whether the unit from row f0 on has half of the rows or fewer.
  __device__ __forceinline__ bool is_half(int T, int f0) const {
    return 2 * (T * pv.G - f0) <= unit.d;
  }
  __device__ __forceinline__ int tile_cost() const { return COST != SPLIT && half ? SPLIT : COST; }
  __device__ __forceinline__ int64_t unit_cost() const {
    return (int64_t)u.nt * tile_cost() + EXTRA;
  }
  __device__ __forceinline__ int groups_of(const PagedSeq& s) const {
    return s.T > 0 ? (s.T * pv.G - 1) / unit + 1 : 0;
  }
  __device__ __forceinline__ Hull hull_of(int T, int L, int m, int f0) const {
    const int f1 = min(f0 + unit.d, T * pv.G) - 1;
    return Hull(L - T + f0 / pv.by_G, L - T + f1 / pv.by_G, m, ba.window);
  }
  __device__ __forceinline__ PagedSeq lane_seq(int b) const {
    PagedSeq s;
    if (b < ba.B)
      s.load(pv, ba, b);
    else
      s.row0 = s.T = s.L = s.m = 0;
    return s;
  }
  template <typename X>
  __device__ __forceinline__ X scan(X x) const {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const X y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    return x;
  }
  // Cost of this lane's group g0 + lane of the block's `count`; inc: the groups of
  // the sequences of the lanes up to each.
  __device__ __forceinline__ int64_t group_cost(const PagedSeq& s, int inc, int count,
                                                int g0) const {
    const int g = g0 + lane;
    int src = 0;                                 // sequences that end at or before g
#pragma unroll
    for (int step = 16; step > 0; step >>= 1) {
      const int e = __shfl_sync(0xffffffffu, inc, src + step - 1);
      if (e <= g) src += step;
    }
    src = min(src, 31);
    const int e = __shfl_sync(0xffffffffu, inc, src);
    const int T = __shfl_sync(0xffffffffu, s.T, src);
    const int L = __shfl_sync(0xffffffffu, s.L, src);
    const int m = __shfl_sync(0xffffffffu, s.m, src);
    if (g >= count) return 0;
    const int q = g - (e - (T > 0 ? (T * pv.G - 1) / unit + 1 : 0));
    const int64_t tiles = Tiles(hull_of(T, L, m, q * unit.d)).nt;
    return (tiles * (is_half(T, q * unit.d) ? SPLIT : COST) + EXTRA) * pv.Hkv;
  }
  __device__ __forceinline__ void take(const PagedSeq& s, int b0, int src) {
    u.b = b0 + src;
    u.seq.row0 = __shfl_sync(0xffffffffu, s.row0, src);
    u.seq.T = __shfl_sync(0xffffffffu, s.T, src);
    u.seq.L = __shfl_sync(0xffffffffu, s.L, src);
    u.seq.m = __shfl_sync(0xffffffffu, s.m, src);
  }
  __device__ __forceinline__ void enter(int q) {
    u.f0 = q * unit.d;
    u.hull = hull_of(u.seq.T, u.seq.L, u.seq.m, u.f0);
    const Tiles t(u.hull);
    u.np = t.np;
    u.kb = t.kb;
    u.nt = t.nt;
    half = is_half(u.seq.T, u.f0);
  }
  __device__ __forceinline__ int64_t from(int c) const {
    return quotient(total * c, ctas);
  }
  // The last CTA whose range begins at or before cost x.
  __device__ __forceinline__ int owner(int64_t x) const { return (int)quotient((x + 1) * ctas - 1, total); }
  // The unit's first tile that begins at or after cost x of it.
  __device__ __forceinline__ int at_cost(int64_t x) const {
    return x <= 0 ? 0
           : x <= EXTRA ? 1
                        : min((int)quotient(x - EXTRA + tile_cost() - 1, tile_cost()), u.nt);
  }
  __device__ __forceinline__ bool clip() {
    if (ubase + (u.j0 > 0 ? u.j0 * (int64_t)tile_cost() + EXTRA : 0) >= x1) return false;
    u.j1 = at_cost(x1 - ubase);
    u.first = u.last = 0;
    if (!u.whole()) {
      u.first = owner(ubase);
      u.last = owner(ubase + (u.nt > 1 ? (u.nt - 1) * (int64_t)tile_cost() + EXTRA : 0));
    }
    return true;
  }
};

// Workspace of an attention launch: counters that the CTAs of a cut unit meet
// on, one or two for each CTA that may begin one (zero before the first call, and zero
// again after each), then two partial results for every CTA: of the unit that
// a CTA before it began, and of the one that it begins and does not end.
constexpr int kMaxPagedCtas = 1024;
constexpr size_t kPagedCounterBytes = kMaxPagedCtas * sizeof(int32_t);
__device__ __forceinline__ int32_t* paged_counter(void* ws, int cta) {
  return static_cast<int32_t*>(ws) + cta;
}
// Partial of CTA p of a unit that CTA `first` begins: `floats` floats.
__device__ __forceinline__ float* paged_partial(void* ws, int p, int first, size_t floats) {
  return reinterpret_cast<float*>(static_cast<char*>(ws) + kPagedCounterBytes) +
         (2 * (size_t)p + (p == first ? 1 : 0)) * floats;
}

}  // namespace rswa
