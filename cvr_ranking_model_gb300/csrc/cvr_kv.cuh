// Internal definitions of the paged history cache (the cvr_kv_* calls of include/cvr.h): the arguments of its kernels and
// their launchers, and the forms of a pool's rows.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "cvr_internal.cuh"

namespace cvr {

// ---- bits of the handle's error word (pinned host memory; kernels OR into it only when they find an error) ----
constexpr int kKvErrPage = 1;    // a page id outside the pool
constexpr int kKvErrLens = 2;    // a length, new length, held count or list head out of range
constexpr int kKvErrSlot = 4;    // a slot outside the pool
constexpr int kKvErrSlots = 16;  // more new tokens than the slot map holds
constexpr int kKvErrPages = 32;  // the free list ran out
constexpr int kKvErrSize = 64;   // more tiles than one call can take
static_assert(kErrTimeout == 8, "the bounded waits report into the same word");

// How a pool holds its rows: as they are, as 8-bit integers with an fp32 scale per row, or as 4-bit floats (e2m1) with an
// e4m3 scale per 16 values and an fp32 scale per row (a record per page and head: the row scales, then the block scales).
enum KvCode { kKv16 = 0, kKv8 = 1, kKv4 = 2 };
__host__ __device__ constexpr int kv_row_bytes(int code, int dim) { return code == kKv16 ? dim * 2 : code == kKv8 ? dim : dim / 2; }
// bytes of scales per row
__host__ __device__ constexpr int kv_scale_bytes(int code, int dim) { return code == kKv16 ? 0 : code == kKv8 ? 4 : 4 + dim / 16; }

// the record of page * kv_heads + head
template <typename P>
__host__ __device__ inline auto kv4_record(P* records, int64_t page_head, int page_log2, int dim) {
  typedef typename std::conditional<std::is_const<P>::value, const uint8_t, uint8_t>::type Byte;
  return static_cast<Byte*>(records) + page_head * ((int64_t)kv_scale_bytes(kKv4, dim) << page_log2);
}

struct KvTablesArgs {
  const int32_t *lens, *new_lens, *held, *free_pages, *free_head;
  int32_t *table, *pages, *free_head_out;
  int64_t *slots, n_slots;
  int64_t n_pages;
  int n_req, n_free, max_pages, page_log2;
  int* err;
};

struct KvAppendArgs {
  const int64_t* slots;
  const void *src[2];  // keys, values (null: K = V)
  int64_t src_stride[2];
  void* pool[2];
  int64_t stride[2][3];  // page, head, token, in values
  void* scale[2];        // [page][head][token] fp32, or [page][head] records, or null
  int64_t n_tok, n_pages;
  int kv_heads, head_dim, page_log2;
  int* err;
};

struct KvReadArgs {
  const int64_t* slots;
  void* dst[2];  // null: not wanted
  int64_t dst_stride[2];
  const void* pool[2];
  int64_t stride[2][3];
  const void* scale[2];
  int64_t n_tok, n_pages;
  int kv_heads, head_dim, page_log2;
  int* err;
};

struct KvWeighArgs {
  const void *q, *k;
  const int32_t *lens, *new_lens, *table;
  const float* lse;
  const void* k_scale;
  float* weight;  // [page][head][token]
  int64_t q_stride, n_pages, k_stride[3];  // (keys' in bytes: page, head, token)
  float scale, decay;
  int n_req, kv_heads, group, page_log2, max_pages;
  int* err;
};

struct KvEvictArgs {
  const int32_t *lens, *held, *table, *free_head;
  float* weight;
  int32_t *kept, *lens_out, *pages, *free_pages, *free_head_out;
  void* pool[2];  // keys, values (null: K = V)
  int64_t stride[2][3];  // page, head, token, in bytes
  void* scale[2];
  int64_t n_pages;
  int limit, keep, first, last;
  int n_req, n_free, kv_heads, head_dim, page_log2, max_pages;
  int* err;
};

struct KvAttendArgs {
  const void *q, *v;  // v null: K = V
  void* out;
  float* lse;
  const int32_t *lens, *table;
  const void *k_scale, *v_scale;
  int64_t q_stride, out_stride, n_pages;
  float scale;
  int n_req, q_heads, kv_heads, group, page_log2, max_pages, window;
  // workspace: what a CTA leaves of a (request, head) that it shares with others
  float *part_o, *part_ml;  // [n_places][group][head_dim], [n_places][group][m, l]
  unsigned* count;          // [2][n_places] parts of a group, groups of a (request, head) written (zero between calls)
  int n_places;
  int* err;
};

constexpr int kKvAttendThreads = 160;  // four consumer warps and a producer
// An instance of the attention kernel (const KvAttendArgs, K's and V's tensor maps).
struct KvAttendKernel {
  const void* kernel;
  int smem, ctas_per_sm;
  int tile;  // tokens per tile
};
KvAttendKernel kv_attend_kernel_32(int dtype, bool int8, int group);
KvAttendKernel kv_attend_kernel_64(int dtype, bool int8, int group);
KvAttendKernel kv_attend_kernel_128(int dtype, bool int8, int group);
KvAttendKernel kv_attend_kernel_fp4_32(int dtype, int group);
KvAttendKernel kv_attend_kernel_fp4_64(int dtype, int group);
KvAttendKernel kv_attend_kernel_fp4_128(int dtype, int group);

cudaError_t launch_kv_tables(const KvTablesArgs& a, int num_sms, cudaStream_t s);
// dtype: a cvr_dtype of the rows; code: a KvCode
cudaError_t launch_kv_append(const KvAppendArgs& a, int dtype, int code, int num_sms, cudaStream_t s);
cudaError_t launch_kv_read(const KvReadArgs& a, int dtype, int code, int num_sms, cudaStream_t s);
cudaError_t launch_kv_weigh(const KvWeighArgs& a, int dtype, int code, int head_dim, int num_sms, cudaStream_t s);
cudaError_t launch_kv_evict(const KvEvictArgs& a, int code, int num_sms, cudaStream_t s);

}  // namespace cvr
