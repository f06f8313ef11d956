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
// (2 pi) is rounded to a 64-bit fraction of a turn; its product with the
// position modulo 2^64 is the phase, exact but for that rounding (position *
// 2^-52 turns with the 64-bit float it comes from), at the price of one
// integer product - a 32-bit float angle would be off by 0.006 at position
// 10^5.  The phase's top 32 bits go to sincospi.  An angle depends on the row
// and the pair only: a lane computes its sines and cosines once for all heads
// of a row.
#include "rswa_device.cuh"

namespace rswa {
namespace {

template <typename T, int D>
struct RopeCfg {
  static constexpr int E = Elt<T>::kPerVec;   // elements of a vector = angles of a lane
  static constexpr int L = D / E / 2;         // lanes of a head
  static constexpr int HPW = 32 / L;          // heads a warp takes at a time
};

// This lane's two vectors of a head, whether they are rotated, and its pairs'
// turns per position as 64-bit fractions.
template <typename T, int D>
struct RopeLane {
  using C = RopeCfg<T, D>;
  int c0, c1;
  bool r0, r1, il;
  uint64_t step[C::E];

  __device__ __forceinline__ void init(const rswa_rope& rp, int lane) {
    const int j = lane % C::L;
    const int rc = rp.rotary_dim / C::E;       // rotated vectors (even)
    il = rp.interleaved != 0;
    if (il) {
      c0 = j;
      c1 = j + C::L;
      r0 = c0 < rc;
      r1 = c1 < rc;
    } else {
      r0 = r1 = j < rc / 2;
      c0 = r0 ? j : 2 * j;
      c1 = r0 ? j + rc / 2 : 2 * j + 1;
    }
#pragma unroll
    for (int e = 0; e < C::E; ++e) {
      // pair of angle e: half-split, the elements e of both vectors;
      // interleaved, pair e of vector 0, then of vector 1
      const bool second = il && e >= C::E / 2;
      const int i = !il ? c0 * C::E + e
                        : (second ? c1 : c0) * (C::E / 2) + e - (second ? C::E / 2 : 0);
      double turns = 0.0;
      if (second ? r1 : r0) {
        turns = rp.inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
        turns -= floor(turns);
      }
      step[e] = __double2ull_rn(turns * 18446744073709551616.0);
    }
  }

  __device__ __forceinline__ void angles(int64_t pos, float* cs, float* sn) const {
#pragma unroll
    for (int e = 0; e < C::E; ++e) {
      const int64_t phase = (int64_t)((uint64_t)pos * step[e]);
      // half turns in [-1, 1)
      sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &sn[e], &cs[e]);
    }
  }

  // x0, x1 -> their normed and rotated values, in place.  Every lane of the
  // warp calls it (shuffles); w: the head's weight, or NULL for no norm.
  __device__ __forceinline__ void apply(uint4& v0, uint4& v1, const T* w, float eps,
                                        const float* cs, const float* sn) const {
    float x0[C::E], x1[C::E];
    Elt<T>::widen(v0, x0);
    Elt<T>::widen(v1, x1);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < C::E; ++e) ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
#pragma unroll
    for (int off = C::L / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if (w) {
      const float r = rsqrtf(ss * (1.f / D) + eps);
      float w0[C::E], w1[C::E];
      Elt<T>::widen(__ldg(reinterpret_cast<const uint4*>(w) + c0), w0);
      Elt<T>::widen(__ldg(reinterpret_cast<const uint4*>(w) + c1), w1);
#pragma unroll
      for (int e = 0; e < C::E; ++e) {
        x0[e] *= r * w0[e];
        x1[e] *= r * w1[e];
      }
    }
    if (!il) {
      if (r0) {
#pragma unroll
        for (int e = 0; e < C::E; ++e) {
          const float a = x0[e], b = x1[e];
          x0[e] = a * cs[e] - b * sn[e];
          x1[e] = b * cs[e] + a * sn[e];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < C::E / 2; ++e) {
        if (r0) {
          const float a = x0[2 * e], b = x0[2 * e + 1];
          x0[2 * e] = a * cs[e] - b * sn[e];
          x0[2 * e + 1] = b * cs[e] + a * sn[e];
        }
        if (r1) {
          const float a = x1[2 * e], b = x1[2 * e + 1];
          x1[2 * e] = a * cs[C::E / 2 + e] - b * sn[C::E / 2 + e];
          x1[2 * e + 1] = b * cs[C::E / 2 + e] + a * sn[C::E / 2 + e];
        }
      }
    }
    v0 = Elt<T>::narrow(x0);
    v1 = Elt<T>::narrow(x1);
  }
};

// One warp per row: its heads, queries then keys, HPW at a time.
template <typename T, int D>
__global__ void __launch_bounds__(128)
norm_rope_kernel(rswa_rope rp, RopeRows rr, CacheView cv) {
  using C = RopeCfg<T, D>;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (row >= rr.rows) return;
  RopeLane<T, D> rl;
  rl.init(rp, lane);
  int64_t pos;
  if (rr.pos) {
    pos = rr.pos[row];
  } else {
    const int64_t b = row / rr.tokens;
    pos = cv.m_dev[b] + cv.t_dev[b * cv.H] + (rr.offsets ? rr.offsets[row] : row % rr.tokens);
  }
  float cs[C::E], sn[C::E];
  rl.angles(pos, cs, sn);
  const int heads = rr.H + rr.Hkv;
  for (int h0 = 0; h0 < heads; h0 += C::HPW) {
    const int h = h0 + lane / C::L;
    const bool on = h < heads, isk = h >= rr.H;
    const int hh = isk ? h - rr.H : h;
    const uint4* in = reinterpret_cast<const uint4*>(
        isk ? static_cast<const T*>(rr.k) + row * rr.k_stride + (int64_t)hh * D
            : static_cast<const T*>(rr.q) + row * rr.q_stride + (int64_t)hh * D);
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    if (on) {
      v0 = in[rl.c0];
      v1 = in[rl.c1];
    }
    rl.apply(v0, v1, static_cast<const T*>(isk ? rp.k_weight : rp.q_weight), rp.eps, cs, sn);
    if (on) {
      uint4* out = reinterpret_cast<uint4*>(
          isk ? static_cast<T*>(rr.k_out) + (row * rr.Hkv + hh) * D
              : static_cast<T*>(rr.q_out) + (row * rr.H + hh) * D);
      out[rl.c0] = v0;
      out[rl.c1] = v1;
    }
  }
}

// One CTA per KV head of a sequence: its query heads and its key, HPW heads a
// warp at a time, and the copy of its value.  The group's copies of t_b
// advance after every thread of the CTA has read t_b.
template <typename T, int D>
__global__ void __launch_bounds__(128)
append_rope_kernel(CacheView cv, rswa_rope rp, const T* q, int64_t q_stride, const T* k,
                   int64_t k_stride, const T* v, int64_t v_stride, T* q_out) {
  using C = RopeCfg<T, D>;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / cv.Hkv, kvh = blockIdx.x % cv.Hkv;
  const int per_kv = cv.H / cv.Hkv;
  int64_t* t_dev = cv.t_dev + (size_t)b * cv.H + (size_t)kvh * per_kv;
  const int64_t t_b = t_dev[0];
  const size_t slot = ((size_t)b * cv.Hkv + kvh) * cv.slab_rows + cv.m_cap + t_b % cv.n;
  RopeLane<T, D> rl;
  rl.init(rp, lane);
  float cs[C::E], sn[C::E];
  rl.angles(cv.m_dev[b] + t_b, cs, sn);
  for (int h0 = warp * C::HPW; h0 < per_kv + 1; h0 += (blockDim.x >> 5) * C::HPW) {
    const int h = h0 + lane / C::L;            // per_kv query heads, then the key
    const bool on = h <= per_kv, isk = h >= per_kv;
    const int64_t qh = (int64_t)kvh * per_kv + h;
    const uint4* in = reinterpret_cast<const uint4*>(
        isk ? k + b * k_stride + (int64_t)kvh * D : q + b * q_stride + qh * D);
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    if (on) {
      v0 = in[rl.c0];
      v1 = in[rl.c1];
    }
    rl.apply(v0, v1, static_cast<const T*>(isk ? rp.k_weight : rp.q_weight), rp.eps, cs, sn);
    if (on) {
      uint4* out = reinterpret_cast<uint4*>(isk ? static_cast<T*>(cv.K) + slot * D
                                                : q_out + ((int64_t)b * cv.H + qh) * D);
      out[rl.c0] = v0;
      out[rl.c1] = v1;
    }
  }
  if (threadIdx.x < 2 * C::L)
    reinterpret_cast<uint4*>(static_cast<T*>(cv.V) + slot * D)[threadIdx.x] =
        reinterpret_cast<const uint4*>(v + b * v_stride + (int64_t)kvh * D)[threadIdx.x];
  __syncthreads();
  for (int h = threadIdx.x; h < per_kv; h += blockDim.x) t_dev[h] = t_b + 1;
}

template <typename T, int D>
cudaError_t norm_rope_t(const rswa_rope& rp, const RopeRows& rr, const CacheView& cv,
                        cudaStream_t s) {
  const int64_t blocks = (rr.rows + 3) / 4;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return launch_dependent(norm_rope_kernel<T, D>, dim3((unsigned)blocks), dim3(128), 0, s, rp,
                          rr, cv);
}

template <typename T, int D>
cudaError_t append_rope_t(const CacheView& cv, const rswa_rope& rp, const void* q,
                          int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, void* q_out, cudaStream_t s) {
  using C = RopeCfg<T, D>;
  const int warps = min(4, (cv.H / cv.Hkv + C::HPW) / C::HPW);
  return launch_dependent(append_rope_kernel<T, D>, dim3((unsigned)(cv.B * cv.Hkv)),
                          dim3(32 * warps), 0, s, cv, rp, (const T*)q, q_stride,
                          (const T*)k, k_stride, (const T*)v, v_stride, (T*)q_out);
}

}  // namespace

cudaError_t launch_norm_rope(const rswa_rope& rope, const RopeRows& rr, const CacheView* cvp,
                             int d, int dtype, cudaStream_t s) {
  const CacheView cv = cvp ? *cvp : CacheView{};
  if (dtype == RSWA_F32)
    return d == 64 ? norm_rope_t<float, 64>(rope, rr, cv, s)
                   : norm_rope_t<float, 128>(rope, rr, cv, s);
  return d == 64 ? norm_rope_t<__nv_bfloat16, 64>(rope, rr, cv, s)
                 : norm_rope_t<__nv_bfloat16, 128>(rope, rr, cv, s);
}

cudaError_t launch_append_rope(const CacheView& cv, const rswa_rope& rope, const void* q,
                               int64_t q_stride, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, void* q_out,
                               cudaStream_t s) {
  if ((int64_t)cv.B * cv.Hkv > INT32_MAX) return cudaErrorInvalidValue;
  if (cv.dtype == RSWA_F32)
    return cv.d == 64 ? append_rope_t<float, 64>(cv, rope, q, q_stride, k, k_stride, v,
                                                 v_stride, q_out, s)
                      : append_rope_t<float, 128>(cv, rope, q, q_stride, k, k_stride, v,
                                                  v_stride, q_out, s);
  return cv.d == 64 ? append_rope_t<__nv_bfloat16, 64>(cv, rope, q, q_stride, k, k_stride, v,
                                                       v_stride, q_out, s)
                    : append_rope_t<__nv_bfloat16, 128>(cv, rope, q, q_stride, k, k_stride, v,
                                                        v_stride, q_out, s);
}

}  // namespace rswa
