// Pages of the history cache: block tables and slot maps from request lengths, and the new tokens' rows to their
// slots (cvr_kv_tables and cvr_kv_append of include/cvr.h).
#include "../../include/cvr.h"
#include "cvr_kv.cuh"

namespace cvr {

namespace {

// ------------------------------------------------------------------------------------------
// Tables. With n_r = ceil(len_r / P), a request needs f_r = max(0, n_r - held_r) fresh pages, the free list's entries
// from F_r = head + sum_{s<r} f_s on, and its new tokens take the slot map's entries from N_r = sum_{s<r} new_s on.
//
// One launch: every CTA scans all requests, 1024 at a time, and writes its own slice of each batch's table entries and
// slots. A scan reads 12 bytes per request (from L2 in all CTAs but one); no CTA waits for another, and a slot's page
// comes from the free list or the held entries, never from what this call writes.
constexpr int kTabThreads = 512;
constexpr int kTabPer = 2;                           // requests per thread and batch
constexpr int kTabBatch = kTabThreads * kTabPer;     // 1024
constexpr int kTabRun = 256;                         // consecutive items of one warp step, 8 per lane

struct TabReq {
  int len, fresh, fresh_from, new_len, held;
};

// the last index i in [lo, hi] with start[i] <= x (start does not decrease, start[lo] <= x)
__device__ __forceinline__ int last_at_most(const int64_t* start, int lo, int hi, int64_t x) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreads) kv_tables_kernel(const KvTablesArgs a) {
  __shared__ int s_held[kTabBatch], s_len[kTabBatch], s_new[kTabBatch];
  __shared__ int64_t s_fresh_at[kTabBatch], s_new_at[kTabBatch];  // exclusive sums within the batch
  __shared__ int64_t s_warp[2][kTabThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t cta = blockIdx.x, n_cta = gridDim.x;
  const int P = 1 << a.page_log2;
  int bad = 0;
  pdl_trigger();
  pdl_wait();
  int64_t head = a.free_head ? *a.free_head : 0;
  if (head < 0 || head > a.n_free) {
    bad |= kKvErrLens;
    head = head < 0 ? 0 : a.n_free;
  }
  int64_t fresh_base = head, new_base = 0;  // the free list's and slot map's positions at the batch's start
  for (int r0 = 0; r0 < a.n_req; r0 += kTabBatch) {
    const int n = min(kTabBatch, a.n_req - r0);
    int64_t f[kTabPer], w[kTabPer], f_sum = 0, w_sum = 0;
#pragma unroll
    for (int i = 0; i < kTabPer; ++i) {
      const int k = tid * kTabPer + i, r = r0 + k;
      int len = 0, nw = 0, held = 0;
      if (k < n) {
        len = a.lens[r];
        const int64_t most = (int64_t)a.max_pages << a.page_log2;
        if (len < 0 || len > most) {
          bad |= kKvErrLens;
          len = len < 0 ? 0 : (int)most;
        }
        nw = a.new_lens ? a.new_lens[r] : min(len, 1);
        if (nw < 0 || nw > len) {
          bad |= kKvErrLens;
          nw = nw < 0 ? 0 : len;
        }
        held = a.held ? a.held[r] : 0;
        if (held < 0 || held > a.max_pages) {
          bad |= kKvErrLens;
          held = held < 0 ? 0 : a.max_pages;
        }
      }
      s_len[k] = len;
      s_new[k] = nw;
      s_held[k] = held;
      f[i] = max(0, ((len + P - 1) >> a.page_log2) - held);
      w[i] = nw;
      f_sum += f[i];
      w_sum += w[i];
    }
    // exclusive sums over the batch's threads
    int64_t f_in = f_sum, w_in = w_sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, f_in, d), v = __shfl_up_sync(0xffffffffu, w_in, d);
      if (lane >= d) {
        f_in += u;
        w_in += v;
      }
    }
    if (lane == 31) {
      s_warp[0][warp] = f_in;
      s_warp[1][warp] = w_in;
    }
    __syncthreads();
    int64_t f_at = f_in - f_sum, w_at = w_in - w_sum, f_total = 0, w_total = 0;
#pragma unroll
    for (int i = 0; i < kTabThreads / 32; ++i) {
      const int64_t u = s_warp[0][i], v = s_warp[1][i];
      if (i < warp) {
        f_at += u;
        w_at += v;
      }
      f_total += u;
      w_total += v;
    }
#pragma unroll
    for (int i = 0; i < kTabPer; ++i) {
      const int k = tid * kTabPer + i;
      s_fresh_at[k] = f_at;
      s_new_at[k] = w_at;
      f_at += f[i];
      w_at += w[i];
    }
    __syncthreads();
    // the page in entry j of the batch's request k: held already, or taken from the free list; -1: none
    auto page_of = [&](int k, int j) -> int {
      const int held = s_held[k];
      if (j < held) return a.table[(int64_t)(r0 + k) * a.max_pages + j];
      const int64_t at = fresh_base + s_fresh_at[k] + (j - held);
      if (at >= a.n_free) {
        bad |= kKvErrPages;
        return -1;
      }
      return a.free_pages[at];
    };
    // this CTA's slice of the batch's fresh entries, in runs that a warp takes
    const int64_t warps = n_cta * (kTabThreads / 32), my = cta * (kTabThreads / 32) + warp;
    for (int64_t at = my * kTabRun; at < f_total; at += warps * kTabRun) {
      const int64_t end = min(at + kTabRun, f_total);
      const int k0 = last_at_most(s_fresh_at, 0, n - 1, at), k1 = last_at_most(s_fresh_at, k0, n - 1, end - 1);
#pragma unroll
      for (int u = 0; u < kTabRun / 32; ++u) {
        const int64_t x = at + u * 32 + lane;
        if (x >= end) continue;
        const int k = last_at_most(s_fresh_at, k0, k1, x), j = s_held[k] + (int)(x - s_fresh_at[k]);
        int page = page_of(k, j);
        if (page >= a.n_pages || (page < 0 && fresh_base + x < a.n_free)) {
          bad |= kKvErrPage;
          page = -1;
        }
        a.table[(int64_t)(r0 + k) * a.max_pages + j] = page;
      }
    }
    // ... and of its slots
    const int64_t w_end = min(w_total, a.n_slots - new_base);
    if (w_end < w_total && a.slots) bad |= kKvErrSlots;
    for (int64_t at = my * kTabRun; at < w_end; at += warps * kTabRun) {
      const int64_t end = min(at + kTabRun, w_end);
      const int k0 = last_at_most(s_new_at, 0, n - 1, at), k1 = last_at_most(s_new_at, k0, n - 1, end - 1);
#pragma unroll
      for (int u = 0; u < kTabRun / 32; ++u) {
        const int64_t x = at + u * 32 + lane;
        if (x >= end) continue;
        const int k = last_at_most(s_new_at, k0, k1, x);
        const int pos = s_len[k] - s_new[k] + (int)(x - s_new_at[k]);
        const int page = page_of(k, pos >> a.page_log2);
        const bool ok = page >= 0 && page < a.n_pages;
        if (!ok) bad |= kKvErrPage;
        a.slots[new_base + x] = ok ? ((int64_t)page << a.page_log2) + (pos & (P - 1)) : -1;
      }
    }
    if (a.pages)
      for (int64_t k = cta * kTabThreads + tid; k < n; k += n_cta * kTabThreads) {
        const int64_t need = (s_len[k] + P - 1) >> a.page_log2;
        const int64_t left = a.n_free - (fresh_base + s_fresh_at[k]);  // pages of the list from this request on
        const int64_t got = min(max(need - s_held[k], (int64_t)0), max(left, (int64_t)0));
        a.pages[r0 + k] = s_held[k] + (int)got;
      }
    fresh_base += f_total;
    new_base += w_total;
    __syncthreads();  // the batch's arrays have been read
  }
  if (fresh_base > a.n_free) bad |= kKvErrPages;
  for (int64_t x = new_base + cta * kTabThreads + tid; x < a.n_slots; x += n_cta * kTabThreads) a.slots[x] = -1;
  if (cta == 0 && tid == 0 && a.free_head_out) *a.free_head_out = (int)min(fresh_base, (int64_t)a.n_free);
  if (bad) atomicOr(a.err, bad);
}

// ------------------------------------------------------------------------------------------
// Append: 16 bytes (8 values) of a row per thread, keys then values.
template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

constexpr int kAppThreads = 256;

template <typename T, bool I8>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(const KvAppendArgs a) {
  const int vec_row = a.head_dim >> 3;            // vectors of 8 values per row: 4, 8 or 16, within one warp
  const int vec_tok = a.kv_heads * vec_row;
  const int64_t total = a.n_tok * vec_tok;
  const int64_t n_slots = a.n_pages << a.page_log2;
  int bad = 0;
  pdl_trigger();
  pdl_wait();
  // (whole warps stay in the loop together: the 8-bit rows are reduced across lanes)
  for (int64_t base = (int64_t)blockIdx.x * kAppThreads; base < total; base += (int64_t)gridDim.x * kAppThreads) {
    const int64_t i = base + threadIdx.x;
    const bool in = i < total;
    const int64_t tok = in ? i / vec_tok : 0;
    const int c = in ? (int)(i - tok * vec_tok) : 0;
    const int head = c / vec_row, piece = c - head * vec_row;
    const int64_t slot = in ? a.slots[tok] : -1;
    const bool ok = slot >= 0 && slot < n_slots;
    if (slot >= n_slots) bad |= kKvErrSlot;
    const int64_t page = slot >> a.page_log2, pos = slot & ((1 << a.page_log2) - 1);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (!a.src[w]) continue;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (ok) x = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.src[w]) + tok * a.src_stride[w]) + c);
      const int64_t at = page * a.stride[w][0] + head * a.stride[w][1] + pos * a.stride[w][2] + piece * 8;
      if (!I8) {
        if (ok) *reinterpret_cast<uint4*>(static_cast<T*>(a.pool[w]) + at) = x;
        continue;
      }
      // scale = max|x| / 127, q = round-half-even(127 x / max|x|): 127 x is exact in fp32 (at most 11 + 7 bits) and
      // the quotient's one rounding cannot reach or leave a half, so the codes are those of exact arithmetic
      float v[8], big = 0.f;
      bool nan = false;
      const T* e = reinterpret_cast<const T*>(&x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = to_f32(e[j]);
        big = fmaxf(big, fabsf(v[j]));
        nan |= v[j] != v[j];
      }
      for (int d = vec_row >> 1; d > 0; d >>= 1) {
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
        nan |= __shfl_xor_sync(0xffffffffu, (int)nan, d) != 0;
      }
      uint32_t code[2] = {0u, 0u};
      if (big > 0.f && big < INFINITY) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int q = __float2int_rn(__fdiv_rn(v[j] * 127.f, big));
          code[j >> 2] |= (uint32_t)(q & 0xff) << (8 * (j & 3));
        }
      }
      if (ok) {
        *reinterpret_cast<uint2*>(static_cast<int8_t*>(a.pool[w]) + at) = make_uint2(code[0], code[1]);
        if (piece == 0)
          a.scale[w][((page * a.kv_heads + head) << a.page_log2) + pos] =
              nan ? __int_as_float(0x7fc00000) : __fdiv_rn(big, 127.f);
      }
    }
  }
  if (bad) atomicOr(a.err, bad);
}

}  // namespace

cudaError_t launch_kv_tables(const KvTablesArgs& a, int num_sms, cudaStream_t s) {
  // one CTA per 4096 items that the call may write, at most one per SM
  const int64_t entries = (int64_t)a.n_req * a.max_pages;
  const int64_t items = a.n_slots + (entries < a.n_free ? entries : a.n_free);
  const int64_t want = 1 + items / 4096;
  return launch_kernel(kv_tables_kernel, dim3((unsigned)(want < num_sms ? want : num_sms)), dim3(kTabThreads), 0, s, true, a);
}

cudaError_t launch_kv_append(const KvAppendArgs& a, int dtype, bool int8, int num_sms, cudaStream_t s) {
  const int64_t total = a.n_tok * a.kv_heads * (a.head_dim / 8);
  const int64_t want = (total + kAppThreads - 1) / kAppThreads, most = (int64_t)num_sms * 8;
  const dim3 grid((unsigned)(want < most ? want : most));
  auto run = [&](auto kern) { return launch_kernel(kern, grid, dim3(kAppThreads), 0, s, true, a); };
  if (dtype == CVR_DTYPE_BF16) return int8 ? run(kv_append_kernel<__nv_bfloat16, true>) : run(kv_append_kernel<__nv_bfloat16, false>);
  return int8 ? run(kv_append_kernel<__half, true>) : run(kv_append_kernel<__half, false>);
}

}  // namespace cvr
