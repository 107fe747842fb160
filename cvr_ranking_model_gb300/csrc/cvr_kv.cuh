// Internal definitions of the paged history cache (the cvr_kv_* calls of include/cvr.h): the arguments of its three
// kernels and their launchers.
#pragma once

#include <cuda_fp16.h>

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
  float* scale[2];       // [page][head][token] or null
  int64_t n_tok, n_pages;
  int kv_heads, head_dim, page_log2;
  int* err;
};

struct KvAttendArgs {
  const void *q, *v;  // v null: K = V
  void* out;
  float* lse;
  const int32_t *lens, *table;
  const float *k_scale, *v_scale;
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

cudaError_t launch_kv_tables(const KvTablesArgs& a, int num_sms, cudaStream_t s);
// dtype: a cvr_dtype of the rows; int8: the pool holds 8-bit integers
cudaError_t launch_kv_append(const KvAppendArgs& a, int dtype, bool int8, int num_sms, cudaStream_t s);

}  // namespace cvr
