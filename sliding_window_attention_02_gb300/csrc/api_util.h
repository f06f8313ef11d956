// Host helpers shared by the entry points of the C ABI: argument checks, the
// current device, and the test hook of failing CUDA calls.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rswa_internal.h"

namespace rswa {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// Test hook: simulated CUDA failure before anything is launched (api.cu).
bool injected_failure();

inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

inline int status_of(cudaError_t e) { return e == cudaSuccess ? RSWA_OK : RSWA_ECUDA; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Makes the cache's device current for the duration of a call.
struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) {
      ok = false;
      return;
    }
    if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
  }
  ~DeviceGuard() {
    int cur;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev)
      cudaSetDevice(prev);
  }
};

// `rows` rows of `len` elements, `stride` apart, of 16-byte vectors.
inline bool valid_rows(const void* p, int64_t stride, int64_t len, int64_t rows, int dtype) {
  const int64_t elt = dtype == RSWA_F32 ? 4 : 2;
  if (!p || !aligned16(p) || stride < 0 || stride > (int64_t(1) << 40)) return false;
  return rows < 2 || (stride >= len && stride * elt % 16 == 0);
}

// Bytes that a call reads or writes.
struct Span {
  const void* p;
  int64_t bytes;
  bool meets(const Span& x) const {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(x.p);
    return a < b + x.bytes && b < a + bytes;
  }
};

// Rows of heads as a norm and rotation reads them.
struct InRows {
  const void* p;
  int64_t stride, len;                         // elements
};

// Whether the rows share a byte with the `bytes` bytes at out.
inline bool rows_meet(const InRows& in, int64_t rows, int64_t elt, const void* out, int64_t bytes) {
  const int64_t len = in.len * elt, step = rows < 2 ? len : in.stride * elt;
  const uintptr_t a = reinterpret_cast<uintptr_t>(in.p), o = reinterpret_cast<uintptr_t>(out);
  if (o + bytes <= a || o >= a + (uintptr_t)(rows - 1) * step + len) return false;
  // the first row that ends behind out's first byte
  const int64_t r = o >= a + len ? (int64_t)((o - a - len) / step) + 1 : 0;
  return r < rows && a + r * step < o + bytes;
}

// Whether dense result rows at `out` may be written while `in` is read: apart,
// or row on row of `own` (in place).  Rows are done in any order.
inline bool out_apart(const void* out, int64_t bytes, const InRows& in, int64_t rows, int64_t elt,
               bool own) {
  if (own && out == in.p && (rows < 2 || in.stride == in.len)) return true;
  return !rows_meet(in, rows, elt, out, bytes);
}

}  // namespace rswa
