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

// Page `x` of sequence b; one outside the pool is flagged and read as page 0.
__device__ __forceinline__ int page_at(const PagesView& pv, const BatchArgs& ba, int b, int x) {
  const int p = ba.table[(size_t)b * ba.max_pages + x];
  if ((unsigned)p < (unsigned)pv.pages) return p;
  flag_error(pv.err, kErrBadBatch);
  return 0;
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

// Tiles of `TILE` keys that a hull's keys take.  ALIGNED: tiles of the tokens'
// own numbering (tile x holds tokens x * TILE on), those that hold a key of it:
// prefix tiles 0 .. np - 1, then band tiles kb on.  Otherwise its keys packed.
template <int TILE, bool ALIGNED>
struct HullTiles {
  int np, kb, nt;
  __device__ __forceinline__ HullTiles() {}
  __device__ __forceinline__ explicit HullTiles(const Hull& h) {
    if (ALIGNED) {
      np = (h.p + TILE - 1) / TILE;
      kb = max(h.w0 / TILE, np);
      nt = np + max(0, (h.end + TILE - 1) / TILE - kb);
    } else {
      np = kb = 0;
      nt = (h.keys() + TILE - 1) / TILE;
    }
  }
  __device__ __forceinline__ int tile(int j) const { return j < np ? j : kb + (j - np); }
};

// Where a CTA's walk over the work list stands: a unit (unit_rows rows (token,
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
// tiles of a unit after each other, unit after unit (a sequence's units KV head
// by KV head), form one list; every tile costs 1, a unit's first one EXTRA more.
// CTA c of `ctas` takes the tiles that begin in [from(c), from(c + 1)).
template <int TILE, bool ALIGNED, int EXTRA, int MINCOST>
struct PagedPlan {
  static_assert(MINCOST >= 1 + EXTRA, "a range holds a tile at least");
  using Tiles = HullTiles<TILE, ALIGNED>;
  const PagesView& pv;
  const BatchArgs& ba;
  int unit_rows, G, n, lane;
  int64_t total = 0, x1 = 0;
  int ctas = 1;
  PagedUnit u;
  int64_t ubase = 0;
  int nq = 0;

  __device__ __forceinline__ PagedPlan(const PagesView& pv_, const BatchArgs& ba_, int rows)
      : pv(pv_), ba(ba_), unit_rows(rows), G(pv_.G), n(ba_.window),
        lane((int)(threadIdx.x & 31)) {}

  __device__ __forceinline__ Hull hull_of(const PagedSeq& s, int f0) const {
    const int f1 = min(f0 + unit_rows, s.T * G) - 1;
    const int a = s.L - s.T;
    return Hull(a + f0 / G, a + f1 / G, s.m, n);
  }
  __device__ __forceinline__ int units_of(const PagedSeq& s) const {
    return (s.T * G + unit_rows - 1) / unit_rows;
  }
  __device__ __forceinline__ int cost(const PagedSeq& s, int q) const {
    return Tiles(hull_of(s, q * unit_rows)).nt + EXTRA;
  }

  // Cost of the units of one KV head, for the sequences of the warp's lanes:
  // short chunks by their lane, long ones by the warp together.
  __device__ int64_t costs(const PagedSeq& s) const {
    const int mine = units_of(s);
    int64_t c = 0;
    if (mine <= 2)
      for (int q = 0; q < mine; ++q) c += cost(s, q);
    for (uint32_t more = __ballot_sync(0xffffffffu, mine > 2); more; more &= more - 1) {
      const int src = __ffs(more) - 1;
      PagedSeq x;
      x.row0 = 0;
      x.T = __shfl_sync(0xffffffffu, s.T, src);
      x.L = __shfl_sync(0xffffffffu, s.L, src);
      x.m = __shfl_sync(0xffffffffu, s.m, src);
      const int nx = __shfl_sync(0xffffffffu, mine, src);
      int64_t part = 0;
      for (int q = lane; q < nx; q += 32) part += cost(x, q);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
      if (lane == src) c = part;
    }
    return c;
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
  __device__ __forceinline__ int64_t from(int c) const {
    const int64_t p = total * c;
    return p >> 32 ? p / ctas : (int64_t)((uint32_t)p / (uint32_t)ctas);
  }
  // The last CTA whose range begins at or before cost x.
  __device__ __forceinline__ int owner(int64_t x) const {
    const int64_t p = (x + 1) * ctas - 1;
    return (int)((p | total) >> 32 ? p / total : (int64_t)((uint32_t)p / (uint32_t)total));
  }

  // Finds the start of this CTA's range; false: it has none.
  __device__ bool start(int cta, int grid) {
    PagedSeq s0;
    int64_t c0 = 0, inc0 = 0;                    // of the first 32 sequences
    int64_t units = 0;
    for (int b0 = 0; b0 < ba.B; b0 += 32) {
      const PagedSeq s = lane_seq(b0 + lane);
      const int64_t c = costs(s) * pv.Hkv;
      const int64_t inc = scan(c);
      if (b0 == 0) {
        s0 = s;
        c0 = c;
        inc0 = inc;
      }
      total += __shfl_sync(0xffffffffu, inc, 31);
      units += __reduce_add_sync(0xffffffffu, units_of(s)) * (int64_t)pv.Hkv;
    }
    if (total == 0) return false;
    ctas = (int)min((int64_t)grid, max((int64_t)1, total / MINCOST));
    // Few units have the same number of CTAs each, if they are alike: their ends
    // meet CTAs' ends.
    if (units < ctas) ctas -= ctas % (int)units;
    if (cta >= ctas) return false;
    const int64_t x0 = from(cta);
    x1 = from(cta + 1);
    int64_t base = 0;
    int b = 0;
    for (int b0 = 0;; b0 += 32) {
      if (b0 > 0) {
        s0 = lane_seq(b0 + lane);
        c0 = costs(s0) * pv.Hkv;
        inc0 = scan(c0);
      }
      const uint32_t here =
          __ballot_sync(0xffffffffu, base + inc0 - c0 <= x0 && x0 < base + inc0);
      if (here) {
        const int src = __ffs(here) - 1;
        b = b0 + src;
        base += __shfl_sync(0xffffffffu, inc0 - c0, src);
        u.seq.row0 = __shfl_sync(0xffffffffu, s0.row0, src);
        u.seq.T = __shfl_sync(0xffffffffu, s0.T, src);
        u.seq.L = __shfl_sync(0xffffffffu, s0.L, src);
        u.seq.m = __shfl_sync(0xffffffffu, s0.m, src);
        c0 = __shfl_sync(0xffffffffu, c0, src);
        break;
      }
      base += __shfl_sync(0xffffffffu, inc0, 31);
    }
    u.b = b;
    nq = units_of(u.seq);
    const int64_t per = c0 / pv.Hkv;             // of one KV head
    u.kvh = (int)((x0 - base) / per);
    base += u.kvh * per;
    for (int q0 = 0;; q0 += 32) {
      const int64_t c = q0 + lane < nq ? cost(u.seq, q0 + lane) : 0;
      const int64_t inc = scan(c);
      const uint32_t here = __ballot_sync(0xffffffffu, base + inc - c <= x0 && x0 < base + inc);
      if (here) {
        const int src = __ffs(here) - 1;
        base += __shfl_sync(0xffffffffu, inc - c, src);
        enter(q0 + src, base);
        break;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    u.j0 = at(x0 - ubase);
    return u.j0 < u.nt ? clip() : next();
  }

  // The next unit of the range; false: there is none.
  __device__ bool next() {
    const int64_t end = ubase + u.nt + EXTRA;
    int q = u.f0 / unit_rows + 1;
    if (q == nq) {
      q = 0;
      if (++u.kvh == pv.Hkv) {
        u.kvh = 0;
        uint32_t live = 0;
        PagedSeq s;
        int b0 = u.b + 1;
        for (; b0 < ba.B; b0 += 32) {            // sequences without rows are passed over
          s = lane_seq(b0 + lane);
          live = __ballot_sync(0xffffffffu, s.T > 0);
          if (live) break;
        }
        if (!live) return false;
        const int src = __ffs(live) - 1;
        u.b = b0 + src;
        u.seq.row0 = __shfl_sync(0xffffffffu, s.row0, src);
        u.seq.T = __shfl_sync(0xffffffffu, s.T, src);
        u.seq.L = __shfl_sync(0xffffffffu, s.L, src);
        u.seq.m = __shfl_sync(0xffffffffu, s.m, src);
        nq = units_of(u.seq);
      }
    }
    if (end >= x1) return false;
    enter(q, end);
    u.j0 = 0;
    return clip();
  }

 private:
  __device__ __forceinline__ void enter(int q, int64_t base) {
    u.f0 = q * unit_rows;
    u.hull = hull_of(u.seq, u.f0);
    const Tiles t(u.hull);
    u.np = t.np;
    u.kb = t.kb;
    u.nt = t.nt;
    ubase = base;
  }
  // The first tile that begins at or after cost x of the unit.
  __device__ __forceinline__ int at(int64_t x) const {
    return x <= 0 ? 0 : (int)min(max(x - EXTRA, (int64_t)1), (int64_t)u.nt);
  }
  __device__ __forceinline__ bool clip() {
    const int64_t b0 = ubase + (u.j0 > 0 ? u.j0 + EXTRA : 0);
    if (b0 >= x1) return false;
    u.j1 = at(x1 - ubase);
    u.first = u.last = 0;
    if (!u.whole()) {
      u.first = owner(ubase);
      u.last = owner(ubase + (u.nt > 1 ? u.nt - 1 + EXTRA : 0));
    }
    return true;
  }
};

// Workspace of an attention launch: counters that the CTAs of a cut unit meet
// on, one for each CTA that may begin one (zero before the first call, and zero
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
