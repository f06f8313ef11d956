// RMS norm of query and key heads with the position rotation in the same
// pass, for any rows (norm_rope_kernel) and for the next token of every
// sequence on its way into the ring (append_rope_kernel).
//
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w,
//   (a, b) -> (a cos - b sin, b cos + a sin) for each pair of y, angle = pos f_i.
//
// Lanes: a head is 2 L vectors of 16 bytes; L lanes take two each, chosen so
// that both elements of every pair are in one lane's registers (no exchange
// for the rotation; the sum of squares takes log2 L shuffles):
//   half-split pairs    vectors c and c + RC/2 of the RC rotated ones, and
//                       two neighbours of those that are not rotated
//   interleaved pairs   vectors c and c + L
// Each load and store instruction of a warp still covers whole sectors.
//
// Angles: pos f_i / (2 pi) turns, of which only the fraction matters.  f_i /
// (2 pi) is taken as a 64-bit fraction of a turn, by an integer product of f_i's
// mantissa with 2^64 / (2 pi); its product with the position modulo 2^64 is the
// phase, off by at most |pos| max(1, |f_i|) 2^-63 turns (2^64 / (2 pi) is cut to an
// integer, and so is the step) - a 32-bit float angle would be off by 0.006 at
// position 10^5, and 64-bit floats are slow here.  The phase's top 32 bits (2^-32
// turns) are rounded to a float of half turns (2^-26 turns) for sincospi.
//
// Angles and weights depend on the row and the pair, not on the head, so a CTA
// first puts, for each row and for queries and keys,
//   A = wa cos, B = wb sin, C = wb cos, D = wa sin
// of every pair into shared memory, while its warps' first heads are on their
// way, and a head costs a' = r (a A - b B), b' = r (b C + a D), two elements an
// instruction (f32x2): 3.5 instructions an element with the conversions.
#include <atomic>

#include "rswa_device.cuh"

namespace rswa {
namespace {

template <typename T, int D>
struct RopeCfg {
  static constexpr int E = Elt<T>::kPerVec;   // elements of a vector = pairs of a lane
  static constexpr int L = D / E / 2;         // lanes of a head
  static constexpr int HPW = 32 / L;          // heads a warp takes at a time
  static constexpr int P = D / 2;             // pairs of a head = table entries, E * L
};

// Turns per position of frequency f, times 2^64, modulo 2^64.  f = M 2^(x - 63)
// with a 64-bit mantissa M; K = 2^64 / (2 pi); the step is M K 2^(x - 63).
__device__ __forceinline__ uint64_t turn_step(double f) {
  constexpr uint64_t K = 0x28BE60DB9391054Aull;
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int x = (int)(bits >> 52 & 0x7ff) - 1023;
  if (x == -1023) return 0;                    // 0 (and what is too small to turn)
  const uint64_t M = bits << 11 | 1ull << 63;
  const uint64_t hi = __umul64hi(M, K), lo = M * K;
  const int s = 63 - x;                        // shift of the 128-bit product
  uint64_t step = 0;
  if (s >= 64) {
    step = s < 128 ? hi >> (s - 64) : 0;
  } else if (s > 0) {
    step = hi << (64 - s) | lo >> s;
  } else if (s > -64) {
    step = lo << -s;
  }
  return bits >> 63 ? 0 - step : step;
}

// Pair p of a head: lane j's e-th.  Elements a and b, whether it is rotated,
// and its frequency.
template <typename T, int D, bool IL>
struct Pair {
  using C = RopeCfg<T, D>;
  int j, e, a, b, f;
  bool rot;
  __device__ __forceinline__ Pair(int p, int rotary_dim) {
    const int rc = rotary_dim / C::E;          // rotated vectors (even)
    j = p % C::L;
    e = p / C::L;
    if (IL) {
      const int c = e < C::E / 2 ? j : j + C::L, i = e % (C::E / 2);
      a = c * C::E + 2 * i;
      b = a + 1;
      rot = c < rc;
      f = c * (C::E / 2) + i;
    } else {
      rot = j < rc / 2;
      a = (rot ? j : 2 * j) * C::E + e;
      b = (rot ? j + rc / 2 : 2 * j + 1) * C::E + e;
      f = a;
    }
  }
};

// Writes pair p's entry of a table (float4 [E][L]) for phase sine and cosine,
// weights wa and wb: interleaved {A, C, -B, D} in vector p; half-split, for the
// two pairs e, e + 1 of a lane, {A, A', -B, -B'} and {C, C', D, D'}.
template <typename T, int D, bool IL>
__device__ __forceinline__ void put_entry(float4* tab, const Pair<T, D, IL>& pr, float wa,
                                          float wb, float cs, float sn) {
  using C = RopeCfg<T, D>;
  if (IL) {
    tab[pr.e * C::L + pr.j] = make_float4(wa * cs, wb * cs, -wb * sn, wa * sn);
  } else {
    float* t0 = reinterpret_cast<float*>(tab + (pr.e & ~1) * C::L + pr.j) + (pr.e & 1);
    float* t1 = t0 + 4 * C::L;
    t0[0] = wa * cs;
    t0[2] = -wb * sn;
    t1[0] = wb * cs;
    t1[2] = wa * sn;
  }
}

// The entries of one row for this thread's pair, for queries and keys.
template <typename T, int D, bool IL>
struct Coefficients {
  Pair<T, D, IL> pr;
  uint64_t step;
  float w[4];                                  // q's a and b, k's a and b
  __device__ __forceinline__ Coefficients(const rswa_rope& rp, int p) : pr(p, rp.rotary_dim) {
    step = pr.rot ? turn_step(rp.inv_freq[pr.f]) : 0;
    const T* wq = static_cast<const T*>(rp.q_weight);
    const T* wk = static_cast<const T*>(rp.k_weight);
    w[0] = wq ? (float)wq[pr.a] : 1.f;
    w[1] = wq ? (float)wq[pr.b] : 1.f;
    w[2] = wk ? (float)wk[pr.a] : 1.f;
    w[3] = wk ? (float)wk[pr.b] : 1.f;
  }
  __device__ __forceinline__ void put(float4* tab, int64_t pos) const {
    float cs = 1.f, sn = 0.f;
    if (pr.rot) {
      const int64_t phase = (int64_t)((uint64_t)pos * step);
      // half turns in [-1, 1)
      sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &sn, &cs);
    }
    put_entry<T, D, IL>(tab, pr, w[0], w[1], cs, sn);
    put_entry<T, D, IL>(tab + RopeCfg<T, D>::P, pr, w[2], w[3], cs, sn);
  }
};

// This lane's two vectors of a head and whether they are rotated.
template <typename T, int D, bool IL>
struct RopeLane {
  using C = RopeCfg<T, D>;
  int c0, c1;
  bool r0, r1;
  __device__ __forceinline__ RopeLane(int rotary_dim, int lane) {
    const int j = lane % C::L, rc = rotary_dim / C::E;
    if (IL) {
      c0 = j;
      c1 = j + C::L;
      r0 = c0 < rc;
      r1 = c1 < rc;
    } else {
      r0 = r1 = j < rc / 2;
      c0 = r0 ? j : 2 * j;
      c1 = r0 ? j + rc / 2 : 2 * j + 1;
    }
  }
  // The head's vectors, normed (`norm`) and rotated, in place.  Every lane of
  // the warp calls it.  tab: this lane's first table entry; each is used once,
  // straight from shared memory (held in registers for all heads of the row,
  // the entries cost 32 registers and with them a third of the CTAs).
  __device__ __forceinline__ void apply(uint4& v0, uint4& v1, const float4* tab, bool norm,
                                        float eps) const {
    float x0[C::E], x1[C::E];
    Elt<T>::widen(v0, x0);
    Elt<T>::widen(v1, x1);
    uint64_t a[C::E / 2], b[C::E / 2], ss2 = 0;
#pragma unroll
    for (int e = 0; e < C::E / 2; ++e) {
      a[e] = f2_pack(x0[2 * e], x0[2 * e + 1]);
      b[e] = f2_pack(x1[2 * e], x1[2 * e + 1]);
      ss2 = f2_fma(a[e], a[e], f2_fma(b[e], b[e], ss2));
    }
    float s0, s1;
    f2_unpack(ss2, s0, s1);
    float ss = s0 + s1;
#pragma unroll
    for (int off = C::L / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = norm ? rsqrtf(ss * (1.f / D) + eps) : 1.f;
    const uint64_t r2 = f2_pack(r, r);
    if (IL) {
      auto turn = [&](uint64_t x, int e, bool rot) {
        const float4 k = tab[e * C::L];
        uint64_t y = f2_mul(x, f2_pack(k.x, k.y));
        if (rot) {
          float p, q;
          f2_unpack(x, p, q);
          y = f2_fma(f2_pack(q, p), f2_pack(k.z, k.w), y);
        }
        return f2_mul(y, r2);
      };
#pragma unroll
      for (int e = 0; e < C::E / 2; ++e) {
        a[e] = turn(a[e], e, r0);
        b[e] = turn(b[e], e + C::E / 2, r1);
      }
    } else {
#pragma unroll
      for (int e = 0; e < C::E / 2; ++e) {
        const float4 k = tab[2 * e * C::L], l = tab[(2 * e + 1) * C::L];
        uint64_t x = f2_mul(a[e], f2_pack(k.x, k.y)), y = f2_mul(b[e], f2_pack(l.x, l.y));
        if (r0) {
          x = f2_fma(b[e], f2_pack(k.z, k.w), x);
          y = f2_fma(a[e], f2_pack(l.z, l.w), y);
        }
        a[e] = f2_mul(x, r2);
        b[e] = f2_mul(y, r2);
      }
    }
#pragma unroll
    for (int e = 0; e < C::E / 2; ++e) {
      f2_unpack(a[e], x0[2 * e], x0[2 * e + 1]);
      f2_unpack(b[e], x1[2 * e], x1[2 * e + 1]);
    }
    v0 = Elt<T>::narrow(x0);
    v1 = Elt<T>::narrow(x1);
  }
};

constexpr int kRopeThreads = 128, kRopeWarps = kRopeThreads / 32;
constexpr int kRopeBatch = 2;                  // head groups a warp has in flight

// CTAs of 4 warps for R = 1, 2 or 4 rows; the 4 / R warps of a row share its
// head groups (HPW heads, queries then keys).  Bound by HBM: every head is read
// and written once.  Many small CTAs (8 an SM, 64 registers a thread) hide each
// other's start: 32768 rows of 10 + 10 heads, d 128, bf16 take 57.3 us (5.9
// TB/s, 86 % of a plain copy's) so, 63.6 with 4 CTAs of an SM and five groups in
// flight, 72 with CTAs of 8 warps that held the entries in registers.
template <typename T, int D, bool IL>
__global__ void __launch_bounds__(kRopeThreads, 8)
norm_rope_kernel(rswa_rope rp, RopeRows rr, CacheView cv, int R) {
  using C = RopeCfg<T, D>;
  __shared__ float4 tab[kRopeWarps][2][C::P];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpr = kRopeWarps / R;              // warps of a row
  const int64_t row0 = (int64_t)blockIdx.x * R;
  const int lr = warp / wpr;
  const int64_t row = row0 + lr;
  const bool on_row = row < rr.rows;
  const int heads = rr.H + rr.Hkv;
  RopeLane<T, D, IL> rl(rp.rotary_dim, lane);
  griddep_wait();
  griddep_launch_dependents();
  uint4 v0[kRopeBatch], v1[kRopeBatch];
  // Loads batch i: groups warp % wpr + wpr * (kRopeBatch * i + x).
  auto head_of = [&](int i, int x) {
    return (warp % wpr + wpr * (kRopeBatch * i + x)) * C::HPW + lane / C::L;
  };
  auto load = [&](int i) {
#pragma unroll
    for (int x = 0; x < kRopeBatch; ++x) {
      const int h = head_of(i, x);
      v0[x] = v1[x] = make_uint4(0, 0, 0, 0);
      if (on_row && h < heads) {
        const T* in = h >= rr.H
                          ? static_cast<const T*>(rr.k) + row * rr.k_stride + (int64_t)(h - rr.H) * D
                          : static_cast<const T*>(rr.q) + row * rr.q_stride + (int64_t)h * D;
        v0[x] = reinterpret_cast<const uint4*>(in)[rl.c0];
        v1[x] = reinterpret_cast<const uint4*>(in)[rl.c1];
      }
    }
  };
  load(0);
  {
    // kRopeThreads is a multiple of P: a thread has the same pair of every row.
    const Coefficients<T, D, IL> co(rp, threadIdx.x % C::P);
    for (int x = threadIdx.x / C::P; x < R && row0 + x < rr.rows; x += kRopeThreads / C::P) {
      const int64_t y = row0 + x;
      int64_t pos;
      if (rr.pos) {
        pos = rr.pos[y];
      } else {
        const int64_t b = y / rr.tokens;
        pos = cv.m_dev[b] + cv.t_dev[b * cv.H] + (rr.offsets ? rr.offsets[y] : y - b * rr.tokens);
      }
      co.put(&tab[x][0][0], pos);
    }
  }
  __syncthreads();
  const int groups = (heads + C::HPW - 1) / C::HPW;
  for (int i = 0; warp % wpr + wpr * kRopeBatch * i < groups; ++i) {
    if (i > 0) load(i);
#pragma unroll
    for (int x = 0; x < kRopeBatch; ++x) {
      const int h = head_of(i, x);
      const int t = h >= rr.H;
      if (h - lane / C::L >= heads) break;     // the warp's groups end
      rl.apply(v0[x], v1[x], tab[lr][t] + lane % C::L,
               (t ? rp.k_weight : rp.q_weight) != nullptr, rp.eps);
      if (on_row && h < heads) {
        T* out = t ? static_cast<T*>(rr.k_out) + (row * rr.Hkv + h - rr.H) * D
                   : static_cast<T*>(rr.q_out) + (row * rr.H + h) * D;
        reinterpret_cast<uint4*>(out)[rl.c0] = v0[x];
        reinterpret_cast<uint4*>(out)[rl.c1] = v1[x];
      }
    }
  }
}

// One CTA per KV head of a sequence: its query heads and its key, HPW heads a
// warp at a time, and the copy of its value.  The group's copies of t_b
// advance after every thread of the CTA has read t_b.  Bound by latency: the
// heads, t_b, m_b and the frequencies are requested together (one sequence of 10 +
// 10 heads 2.3 us, 64 of 32 + 8 heads 2.5).
constexpr int kAppendThreads = 64;

template <typename T, int D, bool IL>
__global__ void __launch_bounds__(kAppendThreads)
append_rope_kernel(CacheView cv, rswa_rope rp, const T* q, int64_t q_stride, const T* k,
                   int64_t k_stride, const T* v, int64_t v_stride, T* q_out) {
  using C = RopeCfg<T, D>;
  __shared__ float4 tab[2][C::P];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / cv.Hkv, kvh = blockIdx.x % cv.Hkv;
  const int per_kv = cv.H / cv.Hkv;
  int64_t* t_dev = cv.t_dev + (size_t)b * cv.H + (size_t)kvh * per_kv;
  RopeLane<T, D, IL> rl(rp.rotary_dim, lane);
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t_b = t_dev[0];
  const int32_t m_b = cv.m_dev[b];
  uint4 v0, v1, vv = make_uint4(0, 0, 0, 0);
  auto load = [&](int h) {                     // per_kv query heads, then the key
    v0 = v1 = make_uint4(0, 0, 0, 0);
    if (h <= per_kv) {
      const T* in = h == per_kv ? k + b * k_stride + (int64_t)kvh * D
                                : q + b * q_stride + ((int64_t)kvh * per_kv + h) * D;
      v0 = reinterpret_cast<const uint4*>(in)[rl.c0];
      v1 = reinterpret_cast<const uint4*>(in)[rl.c1];
    }
  };
  load(warp * C::HPW + lane / C::L);
  if (threadIdx.x < 2 * C::L)
    vv = reinterpret_cast<const uint4*>(v + b * v_stride + (int64_t)kvh * D)[threadIdx.x];
  if (threadIdx.x < C::P) {
    const Coefficients<T, D, IL> co(rp, threadIdx.x);
    co.put(&tab[0][0], m_b + t_b);
  }
  const size_t slot = ((size_t)b * cv.Hkv + kvh) * cv.slab_rows + cv.m_cap +
                      ((uint64_t)t_b >> 32 ? t_b % cv.n : (int64_t)((uint32_t)t_b % (uint32_t)cv.n));
  if (threadIdx.x < 2 * C::L)
    reinterpret_cast<uint4*>(static_cast<T*>(cv.V) + slot * D)[threadIdx.x] = vv;
  __syncthreads();
  for (int h0 = warp * C::HPW; h0 <= per_kv; h0 += kAppendThreads / 32 * C::HPW) {
    const int h = h0 + lane / C::L;
    const int t = h >= per_kv;
    if (h0 > warp * C::HPW) load(h);
    rl.apply(v0, v1, tab[t] + lane % C::L, (t ? rp.k_weight : rp.q_weight) != nullptr, rp.eps);
    if (h <= per_kv) {
      T* out = t ? static_cast<T*>(cv.K) + slot * D
                 : q_out + ((int64_t)b * cv.H + (int64_t)kvh * per_kv + h) * D;
      reinterpret_cast<uint4*>(out)[rl.c0] = v0;
      reinterpret_cast<uint4*>(out)[rl.c1] = v1;
    }
  }
  for (int h = threadIdx.x; h < per_kv; h += kAppendThreads) t_dev[h] = t_b + 1;
}

template <typename T, int D, bool IL>
cudaError_t norm_rope_t(const rswa_rope& rp, const RopeRows& rr, const CacheView& cv, int sms,
                        cudaStream_t s) {
  // Rows of a CTA: one a warp where that still fills the SMs twice, else fewer,
  // with more warps for each.
  int R = kRopeWarps;
  while (R > 1 && (rr.rows + R - 1) / R < 2 * (int64_t)sms) R >>= 1;
  const int64_t blocks = (rr.rows + R - 1) / R;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return launch_dependent(norm_rope_kernel<T, D, IL>, dim3((unsigned)blocks),
                          dim3(kRopeThreads), 0, s, rp, rr, cv, R);
}

template <typename T, int D>
cudaError_t norm_rope_d(const rswa_rope& rp, const RopeRows& rr, const CacheView& cv, int sms,
                        cudaStream_t s) {
  return rp.interleaved ? norm_rope_t<T, D, true>(rp, rr, cv, sms, s)
                        : norm_rope_t<T, D, false>(rp, rr, cv, sms, s);
}

template <typename T, int D>
cudaError_t append_rope_d(const CacheView& cv, const rswa_rope& rp, const void* q,
                          int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, void* q_out, cudaStream_t s) {
  return launch_dependent(
      rp.interleaved ? append_rope_kernel<T, D, true> : append_rope_kernel<T, D, false>,
      dim3((unsigned)(cv.B * cv.Hkv)), dim3(kAppendThreads), 0, s, cv, rp, (const T*)q, q_stride,
      (const T*)k, k_stride, (const T*)v, v_stride, (T*)q_out);
}

// SMs of the current device.
int current_sms() {
  static std::atomic<int> known[64];           // a device's count does not change
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

}  // namespace

cudaError_t launch_norm_rope(const rswa_rope& rope, const RopeRows& rr, const CacheView* cvp,
                             int d, int dtype, cudaStream_t s) {
  const CacheView cv = cvp ? *cvp : CacheView{};
  const int sms = cvp ? cvp->sms : current_sms();
  if (sms < 1) return cudaErrorInvalidDevice;
  if (dtype == RSWA_F32)
    return d == 64 ? norm_rope_d<float, 64>(rope, rr, cv, sms, s)
                   : norm_rope_d<float, 128>(rope, rr, cv, sms, s);
  return d == 64 ? norm_rope_d<__nv_bfloat16, 64>(rope, rr, cv, sms, s)
                 : norm_rope_d<__nv_bfloat16, 128>(rope, rr, cv, sms, s);
}

cudaError_t launch_append_rope(const CacheView& cv, const rswa_rope& rope, const void* q,
                               int64_t q_stride, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, void* q_out,
                               cudaStream_t s) {
  if ((int64_t)cv.B * cv.Hkv > INT32_MAX) return cudaErrorInvalidValue;
  if (cv.dtype == RSWA_F32)
    return cv.d == 64 ? append_rope_d<float, 64>(cv, rope, q, q_stride, k, k_stride, v,
                                                 v_stride, q_out, s)
                      : append_rope_d<float, 128>(cv, rope, q, q_stride, k, k_stride, v,
                                                  v_stride, q_out, s);
  return cv.d == 64 ? append_rope_d<__nv_bfloat16, 64>(cv, rope, q, q_stride, k, k_stride, v,
                                                       v_stride, q_out, s)
                    : append_rope_d<__nv_bfloat16, 128>(cv, rope, q, q_stride, k, k_stride, v,
                                                        v_stride, q_out, s);
}

}  // namespace rswa
