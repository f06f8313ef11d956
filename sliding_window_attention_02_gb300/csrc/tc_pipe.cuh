// Parts of the attention pipelines that several tensor-core kernels share: TMA
// loads with a policy, waits with their polling out of line, masks and stores.
#pragma once

#include "rswa_device.cuh"
#include "tc_ptx.cuh"

namespace rswa {
namespace ptx {

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x,
                                            int32_t y, int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// 2-D load with an L2 policy: evict-first for tiles that are read once a launch, so
// that they do not displace partial results, normal for those that are read again.
__device__ __forceinline__ void tma_load_2d_pol(uint32_t dst, const CUtensorMap* map, int32_t x,
                                                int32_t y, uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(pol)
      : "memory");
}
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t evict_normal_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// One lane of a converged warp.  The compiler knows that a single thread runs what
// depends on it, and keeps descriptors in uniform registers: an MMA takes about 20
// cycles to issue so, 70 where a comparison of lane numbers chooses the thread (40
// pages chunk 155 -> 147 us).
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(on));
  return on != 0;
}

// mbar_wait with its polling loop out of line: the waits are many, and
// instructions that are not there need not be fetched.
static __device__ __noinline__ bool wait_on(uint32_t b, uint32_t phase, volatile int* abort_flag,
                                     uint64_t ns) {
  return mbar_wait(b, phase, abort_flag, ns);
}
__device__ __forceinline__ bool wait_for(uint32_t b, uint32_t phase, volatile int* abort_flag,
                                         uint64_t ns) {
  return mbar_try_wait(b, phase) || wait_on(b, phase, abort_flag, ns);
}

__device__ __forceinline__ int load_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Bits e of word c (columns 32 c + e) with lo <= column <= hi.
__device__ __forceinline__ uint32_t range_mask(int lo, int hi, int c) {
  const int a = max(lo - 32 * c, 0), b = min(hi - 32 * c, 31);
  if (a > b) return 0u;
  return (0xffffffffu << a) & (0xffffffffu >> (31 - b));
}

// 32 columns of a row, times inv, 32 bytes an instruction where o is aligned to
// that: the rows of a warp lie 256 bytes or more apart, and 16 at a time write
// every sector twice (64 grouped sequences 113.8 us for 111.4).
__device__ __forceinline__ void store_columns(__nv_bfloat16* to, const float* x, float inv) {
  uint32_t p[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) p[e] = pack_bf16(x[2 * e] * inv, x[2 * e + 1] * inv);
  if ((reinterpret_cast<uintptr_t>(to) & 31) == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to + 16 * e),
                   "r"(p[8 * e]), "r"(p[8 * e + 1]), "r"(p[8 * e + 2]), "r"(p[8 * e + 3]),
                   "r"(p[8 * e + 4]), "r"(p[8 * e + 5]), "r"(p[8 * e + 6]), "r"(p[8 * e + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      reinterpret_cast<uint4*>(to)[e] =
          make_uint4(p[4 * e], p[4 * e + 1], p[4 * e + 2], p[4 * e + 3]);
  }
}

}  // namespace ptx
}  // namespace rswa
