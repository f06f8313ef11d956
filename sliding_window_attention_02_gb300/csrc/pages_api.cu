// Host side of the paged cache: its handle, the checks of its calls' arguments
// and the launches.  As in api.cu no exception crosses the ABI.
#include <algorithm>
#include <mutex>
#include <new>
#include <unordered_set>

#include "api_util.h"
#include "rswa_internal.h"

using namespace rswa;

struct rswa_pages {
  PagesView pv;
  int device;
  void* buf;
  size_t k_off, v_off;
  PagesMaps maps;                              // of a bf16 pool
};

namespace {

std::mutex g_mu;
std::unordered_set<rswa_pages*> g_live;

bool live(rswa_pages* p) {
  std::lock_guard<std::mutex> lk(g_mu);
  return p != nullptr && g_live.count(p) != 0;
}

int valid_shape(int64_t pages, int page_size, int heads, int kv_heads, int head_dim, int dtype) {
  if (dtype != RSWA_F32 && dtype != RSWA_BF16) return RSWA_EDTYPE;
  if (head_dim != 64 && head_dim != 128) return RSWA_EDTYPE;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0) return RSWA_EINVAL;
  if (heads < 1 || heads > 4096 || kv_heads < 1 || heads % kv_heads != 0) return RSWA_EINVAL;
  if (pages < 1 || pages > (int64_t(1) << 30) / (page_size * kv_heads)) return RSWA_EINVAL;
  return RSWA_OK;
}

struct Layout {
  size_t k_off, v_off, total;
};
Layout make_layout(int64_t pages, int page_size, int kv_heads, int head_dim, int dtype) {
  const size_t elt = dtype == RSWA_F32 ? 4 : 2;
  const size_t pool = elt * (size_t)pages * kv_heads * page_size * head_dim;
  Layout L;
  L.k_off = kAlign;                            // behind the error word
  L.v_off = align_up(L.k_off + pool);
  L.total = align_up(L.v_off + pool);
  return L;
}

// The batch as the kernels take it; RSWA_EINVAL for one that they cannot.
int take_batch(const PagesView& pv, const rswa_batch* bt, int64_t rows, BatchArgs* out) {
  if (!bt || !bt->table || !bt->lens || bt->batch < 1 || bt->batch > (1 << 20) ||
      bt->max_pages < 1 || bt->max_pages > (int64_t(1) << 30) / pv.P || bt->window < 1)
    return RSWA_EINVAL;
  if (!aligned4(bt->table) || !aligned4(bt->lens) || !aligned4(bt->prefix) ||
      !aligned4(bt->starts))
    return RSWA_EINVAL;
  if (rows < 0 || rows > ((int64_t(1) << 31) - 1) / pv.H) return RSWA_EINVAL;
  if (!bt->starts && rows % bt->batch != 0) return RSWA_EINVAL;
  out->table = bt->table;
  out->lens = bt->lens;
  out->prefix = bt->prefix;
  out->starts = bt->starts;
  out->B = bt->batch;
  out->max_pages = (int)bt->max_pages;
  out->rows = (int)rows;
  out->each = (int)(rows / bt->batch);
  out->cap = (int)(bt->max_pages * pv.P);
  out->window = (int)std::min(bt->window, int64_t(1) << 30);
  return RSWA_OK;
}

int64_t pool_bytes(const PagesView& pv) {
  return (int64_t)pv.pages * pv.Hkv * pv.P * pv.d * (pv.dtype == RSWA_F32 ? 4 : 2);
}

// More weights than a 64-bit number of bytes counts.
bool too_many(const PagesView& pv, const BatchArgs& ba) {
  return (int64_t)ba.B * pv.Hkv > (int64_t(1) << 60) / ba.cap;
}

// Whether `out` shares a byte with the pool or with what describes the batch.
bool meets_batch(const PagesView& pv, const BatchArgs& ba, const Span& out) {
  const int64_t B = ba.B;
  const Span in[] = {{pv.K, pool_bytes(pv)},
                     {pv.V, pool_bytes(pv)},
                     {pv.err, 4},
                     {ba.table, B * ba.max_pages * 4},
                     {ba.lens, B * 4},
                     {ba.prefix, ba.prefix ? B * 4 : 0},
                     {ba.starts, ba.starts ? (B + 1) * 4 : 0}};
  if (!out.p || out.bytes == 0) return false;
  for (const Span& x : in)
    if (x.bytes > 0 && out.meets(x)) return true;
  return false;
}

}  // namespace

extern "C" {

int rswa_pages_footprint(int64_t pages, int page_size, int heads, int kv_heads, int head_dim,
                         int dtype, size_t* out_bytes) {
  if (!out_bytes) return RSWA_EINVAL;
  const int st = valid_shape(pages, page_size, heads, kv_heads, head_dim, dtype);
  if (st != RSWA_OK) return st;
  *out_bytes = make_layout(pages, page_size, kv_heads, head_dim, dtype).total;
  return RSWA_OK;
}

int rswa_pages_create(int64_t pages, int page_size, int heads, int kv_heads, int head_dim,
                      int dtype, void* device_buf, size_t buf_bytes, rswa_pages** out) {
  if (!out) return RSWA_EINVAL;
  *out = nullptr;
  const int st = valid_shape(pages, page_size, heads, kv_heads, head_dim, dtype);
  if (st != RSWA_OK) return st;
  if (!device_buf || (reinterpret_cast<uintptr_t>(device_buf) % kAlign) != 0) return RSWA_EINVAL;
  const Layout L = make_layout(pages, page_size, kv_heads, head_dim, dtype);
  if (buf_bytes < L.total) return RSWA_ECAPACITY;
  if (injected_failure()) return RSWA_ECUDA;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return RSWA_ECUDA;
  rswa_pages* p = new (std::nothrow) rswa_pages();
  if (!p) return RSWA_ECUDA;
  char* base = static_cast<char*>(device_buf);
  PagesView& pv = p->pv;
  pv.K = base + L.k_off;
  pv.V = base + L.v_off;
  pv.err = reinterpret_cast<int32_t*>(base);
  pv.pages = (int)pages;
  pv.P = page_size;
  pv.log2P = 0;
  while ((1 << pv.log2P) < page_size) ++pv.log2P;
  pv.H = heads;
  pv.Hkv = kv_heads;
  pv.G = heads / kv_heads;
  pv.by_G = Divisor(pv.G);
  pv.d = head_dim;
  pv.dtype = dtype;
  pv.sms = sms;
  p->device = dev;
  p->buf = device_buf;
  p->k_off = L.k_off;
  p->v_off = L.v_off;
  cudaError_t e = dtype == RSWA_BF16 && !make_pages_maps(pv, &p->maps) ? cudaErrorInvalidValue
                                                                       : cudaSuccess;
  if (e == cudaSuccess) e = cudaMemsetAsync(device_buf, 0, kAlign, 0);
  if (e == cudaSuccess) e = cudaStreamSynchronize(0);
  if (e != cudaSuccess) {
    delete p;
    return RSWA_ECUDA;
  }
  try {
    std::lock_guard<std::mutex> lk(g_mu);
    g_live.insert(p);
  } catch (...) {
    delete p;
    return RSWA_ECUDA;
  }
  *out = p;
  return RSWA_OK;
}

int rswa_pages_destroy(rswa_pages* pages) {
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!pages || g_live.erase(pages) == 0) return RSWA_EHANDLE;
  }
  delete pages;
  return RSWA_OK;
}

int rswa_pages_append(rswa_pages* pages, const rswa_batch* batch, int64_t rows, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride, void* stream) {
  if (!live(pages)) return RSWA_EHANDLE;
  const PagesView& pv = pages->pv;
  BatchArgs ba{};
  const int st = take_batch(pv, batch, rows, &ba);
  if (st != RSWA_OK) return st;
  if (rows == 0) return RSWA_OK;
  const int64_t len = (int64_t)pv.Hkv * pv.d, elt = pv.dtype == RSWA_F32 ? 4 : 2;
  if (!valid_rows(k, k_stride, len, rows, pv.dtype) ||
      !valid_rows(v, v_stride, len, rows, pv.dtype))
    return RSWA_EINVAL;
  for (const InRows& in : {InRows{k, k_stride, len}, InRows{v, v_stride, len}})
    if (rows_meet(in, rows, elt, pv.K, pool_bytes(pv)) ||
        rows_meet(in, rows, elt, pv.V, pool_bytes(pv)))
      return RSWA_EINVAL;
  if (injected_failure()) return RSWA_ECUDA;
  DeviceGuard g(pages->device);
  if (!g.ok) return RSWA_ECUDA;
  return status_of(launch_paged_append(pv, ba, k, k_stride, v, v_stride,
                                       static_cast<cudaStream_t>(stream)));
}

int rswa_pages_attend_workspace(rswa_pages* pages, int64_t rows, size_t* out_bytes) {
  if (!live(pages)) return RSWA_EHANDLE;
  if (!out_bytes || rows < 0 || rows >= (int64_t(1) << 31)) return RSWA_EINVAL;
  *out_bytes = paged_attend_workspace(pages->pv, rows);
  return RSWA_OK;
}

int rswa_pages_attend(rswa_pages* pages, const rswa_batch* batch, int64_t rows, const void* q,
                      int64_t q_stride, void* o, float* lse, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!live(pages)) return RSWA_EHANDLE;
  const PagesView& pv = pages->pv;
  BatchArgs ba{};
  const int st = take_batch(pv, batch, rows, &ba);
  if (st != RSWA_OK) return st;
  if (rows == 0) return RSWA_OK;
  const int64_t len = (int64_t)pv.H * pv.d, elt = pv.dtype == RSWA_F32 ? 4 : 2;
  if (!valid_rows(q, q_stride, len, rows, pv.dtype) || !o || !aligned16(o) || !aligned4(lse) ||
      !workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0)
    return RSWA_EINVAL;
  const size_t need = paged_attend_workspace(pv, rows);
  if (workspace_bytes < need) return RSWA_ECAPACITY;
  const InRows qr{q, q_stride, len};
  const Span out[3] = {{o, rows * len * elt},
                       {lse, lse ? rows * pv.H * 4 : 0},
                       {workspace, (int64_t)need}};
  for (int i = 0; i < 3; ++i) {
    if (!out[i].p) continue;
    if (meets_batch(pv, ba, out[i]) ||
        !out_apart(out[i].p, out[i].bytes, qr, rows, elt, i == 0))
      return RSWA_EINVAL;
    for (int j = 0; j < i; ++j)
      if (out[j].p && out[i].meets(out[j])) return RSWA_EINVAL;
  }
  if (injected_failure()) return RSWA_ECUDA;
  DeviceGuard g(pages->device);
  if (!g.ok) return RSWA_ECUDA;
  AttendArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.o = o;
  a.lse = lse;
  a.ws = workspace;
  return status_of(launch_paged_attend(pv, pages->maps, ba, a, static_cast<cudaStream_t>(stream)));
}

int rswa_pages_weigh(rswa_pages* pages, const rswa_batch* batch, int64_t rows, const void* q,
                     int64_t q_stride, const float* lse, float* weights, float decay,
                     void* stream) {
  if (!live(pages)) return RSWA_EHANDLE;
  const PagesView& pv = pages->pv;
  BatchArgs ba{};
  const int st = take_batch(pv, batch, rows, &ba);
  if (st != RSWA_OK) return st;
  if (!weights || !aligned4(weights) || !(decay >= 0.f) || decay > 1.f || too_many(pv, ba))
    return RSWA_EINVAL;
  const int64_t len = (int64_t)pv.H * pv.d, elt = pv.dtype == RSWA_F32 ? 4 : 2;
  const Span out{weights, (int64_t)ba.B * pv.Hkv * ba.cap * 4};
  if (meets_batch(pv, ba, out)) return RSWA_EINVAL;
  if (rows > 0) {
    if (!valid_rows(q, q_stride, len, rows, pv.dtype) || !lse || !aligned4(lse) ||
        rows_meet(InRows{q, q_stride, len}, rows, elt, weights, out.bytes) ||
        out.meets(Span{lse, rows * pv.H * 4}))
      return RSWA_EINVAL;
  }
  if (injected_failure()) return RSWA_ECUDA;
  DeviceGuard g(pages->device);
  if (!g.ok) return RSWA_ECUDA;
  return status_of(launch_paged_weigh(pv, pages->maps, ba, q, q_stride, lse, weights, decay,
                                      static_cast<cudaStream_t>(stream)));
}

int rswa_pages_evict_workspace(rswa_pages* pages, int batch, int64_t budget, size_t* out_bytes) {
  if (!live(pages)) return RSWA_EHANDLE;
  if (!out_bytes || batch < 1 || batch > (1 << 20) || budget < 1 || budget > (int64_t(1) << 30))
    return RSWA_EINVAL;
  // as many heads as rswa_pages_evict takes of any budget; more of them wrap the bytes
  if ((int64_t)batch * pages->pv.Hkv >= (int64_t(1) << 31)) return RSWA_EINVAL;
  *out_bytes = paged_evict_workspace(pages->pv, batch, budget, false);
  return RSWA_OK;
}

int rswa_pages_evict(rswa_pages* pages, const rswa_batch* batch, const float* weights,
                     int64_t budget, int64_t first, int64_t last, const int32_t* table_out,
                     float* weights_out, int32_t* kept, void* workspace, size_t workspace_bytes,
                     void* stream) {
  if (!live(pages)) return RSWA_EHANDLE;
  const PagesView& pv = pages->pv;
  BatchArgs ba{};
  const int st = take_batch(pv, batch, 0, &ba);
  if (st != RSWA_OK) return st;
  if (budget < 1 || budget > (int64_t(1) << 30) || first < 0 || last < 0 || first > budget ||
      last > budget - first || !weights || !weights_out || !aligned4(weights) ||
      !aligned4(weights_out) || !aligned4(kept) || !aligned4(table_out) || !workspace ||
      (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0)
    return RSWA_EINVAL;
  const int64_t heads = (int64_t)ba.B * pv.Hkv;
  const int64_t rows = std::min<int64_t>(budget, ba.cap);
  if (too_many(pv, ba) || heads * ((rows + 31) / 32) >= (int64_t(1) << 31)) return RSWA_EINVAL;
  const size_t need = paged_evict_workspace(pv, ba.B, budget, kept != nullptr);
  if (workspace_bytes < need) return RSWA_ECAPACITY;
  const int64_t wb = heads * ba.cap * 4;
  const Span in[2] = {{weights, wb}, {table_out, (int64_t)ba.B * ba.max_pages * 4}};
  const Span out[3] = {{weights_out, wb}, {kept, heads * budget * 4}, {workspace, (int64_t)need}};
  for (int i = 0; i < 3; ++i) {
    if (!out[i].p) continue;
    if (meets_batch(pv, ba, out[i])) return RSWA_EINVAL;
    if (out[i].meets(in[0]) && !(i == 0 && weights_out == weights)) return RSWA_EINVAL;
    if (table_out && out[i].meets(in[1])) return RSWA_EINVAL;
    for (int j = 0; j < i; ++j)
      if (out[j].p && out[i].meets(out[j])) return RSWA_EINVAL;
  }
  if (injected_failure()) return RSWA_ECUDA;
  DeviceGuard g(pages->device);
  if (!g.ok) return RSWA_ECUDA;
  EvictArgs a{};
  a.weights = weights;
  a.weights_out = weights_out;
  a.table_out = table_out;
  a.kept = kept;
  a.ws = workspace;
  a.budget = (int)budget;
  a.first = (int)first;
  a.last = (int)last;
  a.in_place = !table_out || table_out == ba.table;
  return status_of(launch_paged_evict(pv, ba, a, static_cast<cudaStream_t>(stream)));
}

int rswa_pages_kv_offsets(rswa_pages* pages, size_t* k_offset, size_t* v_offset) {
  if (!live(pages)) return RSWA_EHANDLE;
  if (!k_offset || !v_offset) return RSWA_EINVAL;
  *k_offset = pages->k_off;
  *v_offset = pages->v_off;
  return RSWA_OK;
}

int rswa_pages_sync_status(rswa_pages* pages) {
  if (!live(pages)) return RSWA_EHANDLE;
  if (injected_failure()) return RSWA_ECUDA;
  DeviceGuard g(pages->device);
  if (!g.ok) return RSWA_ECUDA;
  if (cudaDeviceSynchronize() != cudaSuccess) return RSWA_ECUDA;
  int32_t flag = 0;
  if (cudaMemcpy(&flag, pages->pv.err, sizeof(flag), cudaMemcpyDeviceToHost) != cudaSuccess)
    return RSWA_ECUDA;
  if (flag == 0) return RSWA_OK;
  const int32_t zero = 0;
  if (cudaMemcpy(pages->pv.err, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess)
    return RSWA_ECUDA;
  return RSWA_EDEVICE;
}

}  // extern "C"
