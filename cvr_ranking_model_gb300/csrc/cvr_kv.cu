// Host side of the paged history cache: the cvr_kv_* calls of include/cvr.h. Every size, stride and pointer that the
// host can see is checked here; what only the device sees (lengths, page ids, slots) is checked by the kernels, which
// never leave the pools and report into the handle's error word.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>

#include "../../include/cvr.h"
#include "cvr_kv.cuh"

using namespace cvr;

struct cvr_kv {
  int device = 0;
  int num_sms = 1;
  cudaStream_t stream = nullptr;
  cvr_kv_config cfg{};
  int page_log2 = 0;
  KvAttendKernel attend{};      // (kernel null: no pools)
  CUtensorMap tm_k, tm_v;
  void* ws = nullptr;           // the attention's workspace: parts, then the counters
  float *part_o = nullptr, *part_ml = nullptr;
  unsigned* count = nullptr;
  int n_places = 0;
  size_t count_bytes = 0;
  int* err_host = nullptr;      // pinned, mapped: the error bits since the last sync
  int* err_host_dev = nullptr;  // its device address
  char last_error[256] = "";
};

namespace {

cvr_status kv_fail(cvr_kv* h, cvr_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(h->last_error, sizeof(h->last_error), fmt, ap);
  va_end(ap);
  return s;
}
cvr_status kv_cuda_fail(cvr_kv* h, cudaError_t e, const char* what) {
  cudaGetLastError();
  return kv_fail(h, e == cudaErrorMemoryAllocation ? CVR_E_OOM : CVR_E_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Makes the handle's device current for a call and the caller's current again afterwards.
struct OnDevice {
  int before = -1;
  cudaError_t status;
  explicit OnDevice(int device) {
    status = cudaGetDevice(&before);
    if (status == cudaSuccess && before == device) before = -1;
    else if (status == cudaSuccess) status = cudaSetDevice(device);
  }
  ~OnDevice() {
    if (before >= 0) cudaSetDevice(before);
  }
};

// Lets a call allocate, free and wait while a stream other than its own captures a graph in the calling thread's or the
// global mode, which would end that capture: none of them touches it.
struct BesideCaptures {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  BesideCaptures() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~BesideCaptures() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

// Whether the stream captures, or is the legacy stream while a blocking one does (whose capture any use of it would end).
cudaError_t captures(cudaStream_t s, bool* yes) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing(s, &status);
  *yes = e == cudaErrorStreamCaptureImplicit || (e == cudaSuccess && status != cudaStreamCaptureStatusNone);
  if (e == cudaSuccess) return e;
  cudaGetLastError();
  return *yes ? cudaSuccess : e;
}

bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }

int elt_bytes(int dtype) { return dtype == CVR_DTYPE_I8 ? 1 : 2; }

struct Array {
  const void* p;  // (null: none)
  int64_t bytes;
};
bool overlap(const Array& a, const Array& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && (x < y ? y - x < (uint64_t)a.bytes && b.bytes > 0 : x - y < (uint64_t)b.bytes && a.bytes > 0);
}

// The strides (page, head, token) of a pool, in values: multiples of 16 bytes below 2^40 bytes, and each of them, in
// rising order, steps over everything that the smaller ones span, so that no two rows overlap.
const char* bad_strides(const int64_t* stride, const cvr_kv_config* c) {
  const int64_t size[3] = {c->n_pages, c->kv_heads, c->page_size};
  const int eb = elt_bytes(c->cache_dtype);
  int order[3] = {2, 1, 0};
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) continue;  // (a dimension of one row: its stride is never used)
    if (stride[i] <= 0 || stride[i] >= (int64_t(1) << 40) / eb) return "a pool stride is not in (0, 2^40) bytes";
    if (stride[i] * eb % 16 != 0) return "a pool stride is not a multiple of 16 bytes";
  }
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (stride[order[j]] > stride[order[j + 1]]) {
        const int t = order[j];
        order[j] = order[j + 1];
        order[j + 1] = t;
      }
  int64_t span = c->head_dim;  // values covered by the dimensions so far
  for (int i = 0; i < 3; ++i) {
    const int d = order[i];
    if (size[d] == 1) continue;
    if (stride[d] < span) return "the rows of a pool overlap";
    if (size[d] - 1 > (INT64_MAX / 4 - span) / stride[d]) return "a pool is larger than the address space";
    span += (size[d] - 1) * stride[d];
  }
  return nullptr;
}

const char* bad_config(const cvr_kv_config* c) {
  if (c->kv_heads < 1 || c->kv_heads > 256) return "kv_heads must be in [1, 256]";
  if (c->q_heads < 1 || c->q_heads % c->kv_heads != 0 || c->q_heads / c->kv_heads > 64)
    return "q_heads must be kv_heads times a whole number in [1, 64]";
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return "head_dim must be 32, 64 or 128";
  if (c->page_size < 8 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return "page_size must be a power of two in [8, 256]";
  if (c->max_req < 1 || c->max_req > 65535) return "max_req must be in [1, 65535]";
  if (c->max_pages < 1 || (int64_t)c->max_pages * c->page_size > (int64_t(1) << 30))
    return "max_pages must be >= 1 and max_pages * page_size <= 2^30";
  if (c->n_pages < 1 || c->n_pages > INT32_MAX) return "n_pages must be in [1, 2^31 - 1]";
  if (c->dtype != CVR_DTYPE_BF16 && c->dtype != CVR_DTYPE_F16) return "dtype must be CVR_DTYPE_BF16 or CVR_DTYPE_F16";
  if (c->cache_dtype != c->dtype && c->cache_dtype != CVR_DTYPE_I8) return "cache_dtype must be dtype or CVR_DTYPE_I8";
  if (c->window < 0) return "window must be >= 0";
  if (c->reserved != 0) return "reserved must be 0";
  if (!c->k) return c->v || c->k_scale || c->v_scale ? "v, k_scale and v_scale need k" : nullptr;
  const bool i8 = c->cache_dtype == CVR_DTYPE_I8;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
    return "pools and scales must be 16-byte aligned";
  if (c->k == c->v) return "k and v are the same pool (pass v = NULL for K = V)";
  if (i8 != (c->k_scale != nullptr) || (c->v && i8 != (c->v_scale != nullptr)))
    return "an 8-bit pool needs its scales, a 16-bit pool has none";
  if (i8 && c->v && c->k_scale == c->v_scale) return "k and v need scales of their own";
  if (const char* why = bad_strides(c->k_stride, c)) return why;
  return c->v ? bad_strides(c->v_stride, c) : nullptr;
}

// A pool as [page][head][half][token][line]: a copied box is one page's (or a tile's) rows of one head, in lines of at
// most 128 bytes swizzled as the attention kernel reads them.
bool encode_pool(CUtensorMap* m, void* base, const int64_t* stride, const cvr_kv_config* c, int tile) {
  EncodeTiledFn enc = get_encoder();
  if (!enc) return false;
  const int eb = elt_bytes(c->cache_dtype), row = c->head_dim * eb, line = row < 128 ? row : 128;
  // (the stride of a dimension of one row is never used, but has to be a valid one)
  auto bytes = [&](int d, int64_t size) { return (cuuint64_t)(size == 1 ? 256 : stride[d] * eb); };
  const cuuint64_t dims[5] = {(cuuint64_t)(line / eb), (cuuint64_t)c->page_size, (cuuint64_t)(row / line),
                              (cuuint64_t)c->kv_heads, (cuuint64_t)c->n_pages};
  const cuuint64_t strides[4] = {bytes(2, c->page_size), 128, bytes(1, c->kv_heads), bytes(0, c->n_pages)};
  const cuuint32_t box[5] = {(cuuint32_t)(line / eb), (cuuint32_t)(c->page_size < tile ? c->page_size : tile),
                             (cuuint32_t)(row / line), 1, 1};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  const CUtensorMapSwizzle swizzle = line == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : line == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                  : CU_TENSOR_MAP_SWIZZLE_32B;
  // L2 fetches whole runs of rows where a head's rows are next to each other, else no more than a row
  const bool dense = stride[2] == c->head_dim;
  const CUtensorMapL2promotion l2 = dense || row >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                    : row == 128        ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                    : row == 64         ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                                        : CU_TENSOR_MAP_L2_PROMOTION_NONE;
  return enc(m, eb == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, base, dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, l2, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Everything the attention of a handle with pools needs: the kernel, the pools' tensor maps and the workspace.
cudaError_t prepare_attend(cvr_kv* h) {
  const cvr_kv_config* c = &h->cfg;
  const bool i8 = c->cache_dtype == CVR_DTYPE_I8;
  const int group = c->q_heads / c->kv_heads;
  h->attend = c->head_dim == 32   ? kv_attend_kernel_32(c->dtype, i8, group)
              : c->head_dim == 64 ? kv_attend_kernel_64(c->dtype, i8, group)
                                  : kv_attend_kernel_128(c->dtype, i8, group);
  if (!encode_pool(&h->tm_k, c->k, c->k_stride, c, h->attend.tile)) return cudaErrorInvalidValue;
  h->tm_v = h->tm_k;
  if (c->v && !encode_pool(&h->tm_v, c->v, c->v_stride, c, h->attend.tile)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(h->attend.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, h->attend.smem);
  h->n_places = h->num_sms * h->attend.ctas_per_sm * 2;
  const size_t rows = (size_t)h->n_places * group;
  h->count_bytes = (size_t)h->n_places * 2 * 4;
  if (e == cudaSuccess) e = cudaMalloc(&h->ws, rows * (c->head_dim + 2) * 4 + h->count_bytes);
  if (e != cudaSuccess) {
    h->ws = nullptr;
    return e;
  }
  h->part_o = static_cast<float*>(h->ws);
  h->part_ml = h->part_o + rows * c->head_dim;
  h->count = reinterpret_cast<unsigned*>(h->part_ml + rows * 2);
  // (on the handle's stream, so that it is ordered before the first call whatever stream that is)
  return cudaMemsetAsync(h->count, 0, h->count_bytes, h->stream);
}

}  // namespace

extern "C" {

cvr_status cvr_kv_create(const cvr_kv_config* cfg, void* cuda_stream, cvr_kv** out) {
  if (!out) return CVR_E_ARG;
  *out = nullptr;
  if (!cfg) return CVR_E_ARG;
  if (const char* why = bad_config(cfg)) {
    fprintf(stderr, "cvr_kv_create: %s\n", why);
    return CVR_E_ARG;
  }
  // (a captured clearing of the counters would run with the graph only)
  bool capturing = false;
  cudaError_t e = captures(static_cast<cudaStream_t>(cuda_stream), &capturing);
  if (capturing) fprintf(stderr, "cvr_kv_create: the stream is capturing a graph, or another one that it would wait for\n");
  else if (e != cudaSuccess) fprintf(stderr, "cvr_kv_create: %s\n", cudaGetErrorString(e));
  if (capturing || e != cudaSuccess) return capturing ? CVR_E_ARG : CVR_E_CUDA;
  BesideCaptures beside;
  cvr_kv* h = new (std::nothrow) cvr_kv();
  if (!h) return CVR_E_OOM;
  h->cfg = *cfg;
  h->stream = static_cast<cudaStream_t>(cuda_stream);
  while ((1 << h->page_log2) < cfg->page_size) ++h->page_log2;
  e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e == cudaSuccess) e = cudaHostAlloc(reinterpret_cast<void**>(&h->err_host), 64, cudaHostAllocMapped);
  if (e == cudaSuccess) {
    *h->err_host = 0;
    e = cudaHostGetDevicePointer(reinterpret_cast<void**>(&h->err_host_dev), h->err_host, 0);
  }
  if (e == cudaSuccess && cfg->k) e = prepare_attend(h);
  if (e != cudaSuccess) {
    fprintf(stderr, "cvr_kv_create: %s\n", cudaGetErrorString(e));
    cudaGetLastError();
    cvr_kv_destroy(h);
    return e == cudaErrorMemoryAllocation ? CVR_E_OOM : CVR_E_CUDA;
  }
  *out = h;
  return CVR_OK;
}

cvr_status cvr_kv_tables(cvr_kv* h, int32_t n_req, const int32_t* lens, const int32_t* new_lens, const int32_t* held,
                         const int32_t* free_pages, int32_t n_free, const int32_t* free_head, int32_t* table,
                         int32_t* pages, int32_t* free_head_out, int64_t* slots, int64_t n_slots) {
  if (!h) return CVR_E_ARG;
  if (n_req < 0 || n_req > h->cfg.max_req)
    return kv_fail(h, CVR_E_SHAPE, "need 0 <= n_req <= max_req (%d); got %d", h->cfg.max_req, n_req);
  if (n_free < 0 || n_free == INT32_MAX || n_slots < 0 || n_slots >= INT32_MAX)
    return kv_fail(h, CVR_E_SHAPE, "need 0 <= n_free < 2^31 - 1 and 0 <= n_slots < 2^31 - 1");
  if (n_req > 0 && (!lens || !table)) return kv_fail(h, CVR_E_ARG, "null lens or table");
  if ((n_free > 0 && !free_pages) || (n_slots > 0 && !slots)) return kv_fail(h, CVR_E_ARG, "null free_pages or slots");
  // No CTA waits for another: what one writes, another may still have to read. The written arrays come last.
  const int64_t n = n_req;
  const Array arrays[] = {{lens, n * 4},  {new_lens, n * 4},
                          {held, n * 4},  {free_pages, (int64_t)n_free * 4},
                          {free_head, 4}, {table, n * h->cfg.max_pages * 4},
                          {pages, n * 4}, {free_head_out, 4},
                          {slots, n_slots * 8}};
  constexpr int kArrays = sizeof(arrays) / sizeof(arrays[0]), kRead = 5;
  for (int i = 0; i < kArrays - 1; ++i)
    if (!aligned(arrays[i].p, 4)) return kv_fail(h, CVR_E_ARG, "int32 arrays must be 4-byte aligned");
  if (!aligned(slots, 8)) return kv_fail(h, CVR_E_ARG, "slots must be 8-byte aligned");
  for (int i = kRead; i < kArrays; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(arrays[i], arrays[j])) return kv_fail(h, CVR_E_ARG, "an array that the call writes overlaps another one");
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return kv_cuda_fail(h, on.status, "cudaSetDevice");
  KvTablesArgs a;
  a.lens = lens;
  a.new_lens = new_lens;
  a.held = held;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.table = table;
  a.pages = pages;
  a.free_head_out = free_head_out;
  a.slots = slots;
  a.n_slots = n_slots;
  a.n_pages = h->cfg.n_pages;
  a.n_req = n_req;
  a.n_free = n_free;
  a.max_pages = h->cfg.max_pages;
  a.page_log2 = h->page_log2;
  a.err = h->err_host_dev;
  const cudaError_t e = launch_kv_tables(a, h->num_sms, h->stream);
  return e == cudaSuccess ? CVR_OK : kv_cuda_fail(h, e, "cvr_kv_tables launch");
}

cvr_status cvr_kv_append(cvr_kv* h, int64_t n_tok, const int64_t* slots, const void* k, int64_t k_stride, const void* v,
                         int64_t v_stride) {
  if (!h) return CVR_E_ARG;
  const cvr_kv_config& c = h->cfg;
  if (!c.k) return kv_fail(h, CVR_E_ARG, "the handle was created without pools");
  if (n_tok < 0 || n_tok > INT32_MAX) return kv_fail(h, CVR_E_SHAPE, "need 0 <= n_tok <= 2^31 - 1");
  if (n_tok == 0) return CVR_OK;
  if (!slots || !k || (c.v && !v)) return kv_fail(h, CVR_E_ARG, "null slots or rows");
  if (!c.v && v) return kv_fail(h, CVR_E_ARG, "the cache has K = V: pass v = NULL");
  const int64_t row = (int64_t)c.kv_heads * c.head_dim;
  if (k_stride < row || k_stride % 8 != 0 || (v && (v_stride < row || v_stride % 8 != 0)))
    return kv_fail(h, CVR_E_ARG, "row strides must be multiples of 8 and >= kv_heads * head_dim");
  if (!aligned16(k) || !aligned16(v)) return kv_fail(h, CVR_E_ARG, "rows must be 16-byte aligned");
  if (!aligned(slots, 8)) return kv_fail(h, CVR_E_ARG, "slots must be 8-byte aligned");
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return kv_cuda_fail(h, on.status, "cudaSetDevice");
  KvAppendArgs a;
  a.slots = slots;
  a.src[0] = k;
  a.src[1] = v;
  a.src_stride[0] = k_stride;
  a.src_stride[1] = v_stride;
  a.pool[0] = c.k;
  a.pool[1] = c.v;
  for (int i = 0; i < 3; ++i) {
    a.stride[0][i] = c.k_stride[i];
    a.stride[1][i] = c.v_stride[i];
  }
  a.scale[0] = c.k_scale;
  a.scale[1] = c.v ? c.v_scale : nullptr;
  a.n_tok = n_tok;
  a.n_pages = c.n_pages;
  a.kv_heads = c.kv_heads;
  a.head_dim = c.head_dim;
  a.page_log2 = h->page_log2;
  a.err = h->err_host_dev;
  const cudaError_t e = launch_kv_append(a, c.dtype, c.cache_dtype == CVR_DTYPE_I8, h->num_sms, h->stream);
  return e == cudaSuccess ? CVR_OK : kv_cuda_fail(h, e, "cvr_kv_append launch");
}

cvr_status cvr_kv_attend(cvr_kv* h, int32_t n_req, const void* q, int64_t q_stride, const int32_t* lens,
                         const int32_t* table, float scale, void* out, int64_t out_stride, float* lse) {
  if (!h) return CVR_E_ARG;
  const cvr_kv_config& c = h->cfg;
  if (!c.k) return kv_fail(h, CVR_E_ARG, "the handle was created without pools");
  if (n_req < 0 || n_req > c.max_req)
    return kv_fail(h, CVR_E_SHAPE, "need 0 <= n_req <= max_req (%d); got %d", c.max_req, n_req);
  if (!std::isfinite(scale)) return kv_fail(h, CVR_E_ARG, "scale must be finite");
  if (n_req == 0) return CVR_OK;
  if (!q || !lens || !table || !out) return kv_fail(h, CVR_E_ARG, "null q, lens, table or out");
  const int64_t row = (int64_t)c.q_heads * c.head_dim;
  if (q_stride < row || q_stride % 8 != 0 || out_stride < row || out_stride % 8 != 0)
    return kv_fail(h, CVR_E_ARG, "q and out strides must be multiples of 8 and >= q_heads * head_dim");
  if (!aligned16(q) || !aligned16(out)) return kv_fail(h, CVR_E_ARG, "q and out must be 16-byte aligned");
  if (!aligned(lens, 4) || !aligned(table, 4) || !aligned(lse, 4))
    return kv_fail(h, CVR_E_ARG, "lens, table and lse must be 4-byte aligned");
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return kv_cuda_fail(h, on.status, "cudaSetDevice");
  KvAttendArgs a;
  a.q = q;
  a.v = c.v;
  a.out = out;
  a.lse = lse;
  a.lens = lens;
  a.table = table;
  a.k_scale = c.k_scale;
  a.v_scale = c.v ? c.v_scale : c.k_scale;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.n_pages = c.n_pages;
  a.scale = scale;
  a.n_req = n_req;
  a.q_heads = c.q_heads;
  a.kv_heads = c.kv_heads;
  a.group = c.q_heads / c.kv_heads;
  a.page_log2 = h->page_log2;
  a.max_pages = c.max_pages;
  a.window = c.window;
  a.part_o = h->part_o;
  a.part_ml = h->part_ml;
  a.count = h->count;
  a.n_places = h->n_places;
  a.err = h->err_host_dev;
  // one CTA per tile that there can be at most, at most as many as the SMs hold at once
  const int64_t all = (int64_t)c.max_pages * c.page_size, seen = c.window && c.window < all ? c.window + h->attend.tile : all;
  const int64_t most = n_req * c.kv_heads * ((seen + h->attend.tile - 1) / h->attend.tile);
  const int64_t fit = (int64_t)h->num_sms * h->attend.ctas_per_sm;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(most < fit ? most : fit));
  lc.blockDim = dim3(kKvAttendThreads);
  lc.dynamicSmemBytes = h->attend.smem;
  lc.stream = h->stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  void* args[] = {&a, &h->tm_k, &h->tm_v};
  const cudaError_t e = cudaLaunchKernelExC(&lc, h->attend.kernel, args);
  return e == cudaSuccess ? CVR_OK : kv_cuda_fail(h, e, "cvr_kv_attend launch");
}

cvr_status cvr_kv_sync(cvr_kv* h) {
  if (!h) return CVR_E_ARG;
  OnDevice on(h->device);
  if (on.status != cudaSuccess) return kv_cuda_fail(h, on.status, "cudaSetDevice");
  bool capturing = false;
  cudaError_t e = captures(h->stream, &capturing);
  if (capturing) return kv_fail(h, CVR_E_ARG, "the stream is capturing a graph, or another one that it would wait for");
  BesideCaptures beside;
  if (e == cudaSuccess) e = cudaStreamSynchronize(h->stream);
  if (e != cudaSuccess) return kv_cuda_fail(h, e, "cvr_kv_sync");
  volatile int* word = h->err_host;
  const int ew = *word;
  *word = 0;
  if (ew & kErrTimeout) {
    // a CTA that gave up may have left a counter part-way; the next call starts from zero
    if (h->count) cudaMemsetAsync(h->count, 0, h->count_bytes, h->stream);
    return kv_fail(h, CVR_E_TIMEOUT, "a bounded device-side wait gave up");
  }
  if (ew & kKvErrLens) return kv_fail(h, CVR_E_INPUT, "a length, new length, held count or list head is out of range");
  if (ew & kKvErrPages) return kv_fail(h, CVR_E_PAGES, "the free list ran out of pages");
  if (ew & kKvErrSlots) return kv_fail(h, CVR_E_INPUT, "more new tokens than the slot map holds");
  if (ew & kKvErrSize) return kv_fail(h, CVR_E_SHAPE, "the histories of one call are too long together");
  if (ew & kKvErrPage) return kv_fail(h, CVR_E_ID_RANGE, "a page id is outside the pool");
  if (ew & kKvErrSlot) return kv_fail(h, CVR_E_ID_RANGE, "a slot is outside the pool (its token was skipped)");
  h->last_error[0] = 0;
  return CVR_OK;
}

const char* cvr_kv_last_error(const cvr_kv* h) { return h ? h->last_error : "null handle"; }

void cvr_kv_destroy(cvr_kv* h) {
  if (!h) return;
  {
    OnDevice on(h->device);
    BesideCaptures beside;
    if (h->err_host) {  // (a handle whose creation failed has nothing in flight)
      cudaStreamSynchronize(h->stream);
      cudaFreeHost(h->err_host);
    }
    if (h->ws) cudaFree(h->ws);
  }
  delete h;
}

}  // extern "C"
