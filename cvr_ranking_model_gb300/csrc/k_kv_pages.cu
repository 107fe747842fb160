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
// One launch. Every CTA sums all requests (12 bytes each, from L2 in all CTAs but one) and so knows where its own slice
// of the fresh entries and of the slots begins; it scans the slice's requests 512 at a time and writes. No CTA waits for
// another: a slot's page comes from the free list or the held entries, never from what this call writes.
// Bound by latency: 64 requests, a token each, 3.7 us (two dependent loads, a scan); 4095 requests and 5.5 million slots
// 20.1 us, where writing 46 MB takes 7: 5.7 until the slots' requests are known, 3 of them for the table's entries.
constexpr int kTabThreads = 512, kTabWarps = kTabThreads / 32;
// Consecutive items of a warp's step, whose loads are in flight together: a call of one CTA is bound by the latency of its
// few steps (64 requests, a token each: 3.6 us with 128, 4.6 us with 256), a longer one by their number (5.5 million slots:
// 28.5 us with 128, 23.2 us with 256).
constexpr int kTabRunShort = 128, kTabRunLong = 256;

// sums of fresh pages or new tokens; they stop at 2^31 - 1, above any list's or slot map's length
constexpr uint32_t kTabMost = 0x7fffffffu;
__device__ __forceinline__ uint32_t sat_add(uint32_t x, uint32_t y) { return min(x + y, kTabMost); }

struct TabReq {
  int len, fresh, held;
  int n_new;
};

__device__ __forceinline__ TabReq tab_request(const KvTablesArgs& a, int r, int* bad) {
  TabReq q = {0, 0, 0, 0};
  if (r >= a.n_req) return q;
  // (plain loads, here and below: an earlier call of the stream may have written these arrays while this one started)
  const int most = a.max_pages << a.page_log2;  // (at most 2^30)
  const int len = a.lens[r], nw = a.new_lens ? a.new_lens[r] : 1, held = a.held ? a.held[r] : 0;
  q.len = min(max(len, 0), most);
  q.n_new = a.new_lens ? min(max(nw, 0), q.len) : min(q.len, 1);
  q.held = min(max(held, 0), a.max_pages);
  if (q.len != len || (a.new_lens && q.n_new != nw) || q.held != held) *bad |= kKvErrLens;
  q.fresh = max(0, ((q.len + (1 << a.page_log2) - 1) >> a.page_log2) - q.held);
  return q;
}

// Exclusive sums of (f, w) over the block's threads, from (f_base, w_base); the totals behind the last in *_all.
struct TabScan {
  uint32_t f, w, f_all, w_all;
};
__device__ __forceinline__ TabScan tab_scan(uint32_t f, uint32_t w, uint32_t f_base, uint32_t w_base,
                                            uint32_t (*s_warp)[kTabWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t fi = f, wi = w;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, fi, d), v = __shfl_up_sync(0xffffffffu, wi, d);
    if (lane >= d) {
      fi = sat_add(fi, u);
      wi = sat_add(wi, v);
    }
  }
  __syncthreads();  // (the last scan's sums have been read)
  if (lane == 31) {
    s_warp[0][warp] = fi;
    s_warp[1][warp] = wi;
  }
  __syncthreads();
  // lane l < 16 takes warp l's sums; every warp scans them
  uint32_t ft = lane < kTabWarps ? s_warp[0][lane] : 0, wt = lane < kTabWarps ? s_warp[1][lane] : 0;
#pragma unroll
  for (int d = 1; d < kTabWarps; d <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, ft, d), v = __shfl_up_sync(0xffffffffu, wt, d);
    if (lane >= d) {
      ft = sat_add(ft, u);
      wt = sat_add(wt, v);
    }
  }
  const uint32_t fb = __shfl_sync(0xffffffffu, ft, max(warp - 1, 0)), wb = __shfl_sync(0xffffffffu, wt, max(warp - 1, 0));
  TabScan r;
  r.f_all = sat_add(f_base, __shfl_sync(0xffffffffu, ft, kTabWarps - 1));
  r.w_all = sat_add(w_base, __shfl_sync(0xffffffffu, wt, kTabWarps - 1));
  const uint32_t fx = __shfl_up_sync(0xffffffffu, fi, 1), wx = __shfl_up_sync(0xffffffffu, wi, 1);
  r.f = sat_add(sat_add(f_base, warp ? fb : 0), lane ? fx : 0);
  r.w = sat_add(sat_add(w_base, warp ? wb : 0), lane ? wx : 0);
  return r;
}

// the last index i < n (at most kTabThreads) with start[i] <= x, found by a warp; start does not decrease, start[0] <= x
__device__ __forceinline__ int warp_last_at_most(const uint32_t* start, int n, uint32_t x) {
  constexpr int kStep = kTabThreads / 32;
  const int lane = threadIdx.x & 31;
  const int block = __popc(__ballot_sync(0xffffffffu, lane * kStep < n && start[min(lane * kStep, n - 1)] <= x)) - 1;
  const int i = block * kStep + lane % kStep;
  return block * kStep + __popc(__ballot_sync(0xffffffffu, lane < kStep && i < n && start[min(i, n - 1)] <= x)) - 1;
}

// Fresh entries from the kTabMost-th on, of which no sum knows the place: no list reaches them, they are -1. start: a sum per
// thread's run of requests. (Out of line: a table above 8 GB.)
static __device__ __noinline__ void tab_behind(const KvTablesArgs& a, int run, uint32_t before, uint32_t* start) {
  __syncthreads();
  start[threadIdx.x] = before;
  __syncthreads();
  for (int t = blockIdx.x; t < kTabThreads; t += gridDim.x) {
    uint32_t at = start[t];
    for (int r = t * run; r < min((t + 1) * run, a.n_req); ++r) {
      int ignored = 0;
      const TabReq x = tab_request(a, r, &ignored);
      for (uint32_t j = min((uint32_t)x.fresh, kTabMost - at) + threadIdx.x; j < (uint32_t)x.fresh; j += kTabThreads)
        a.table[(int64_t)r * a.max_pages + x.held + j] = -1;
      at = sat_add(at, x.fresh);
    }
  }
}

template <int kTabRun>
__global__ void __launch_bounds__(kTabThreads) kv_tables_kernel(const __grid_constant__ KvTablesArgs a) {
  __shared__ uint32_t s_warp[2][kTabWarps];
  __shared__ uint32_t s_run[2][kTabThreads];  // sums before each thread's run of requests
  // of the requests in hand: the sums before each, its held entries, and with w and f those sums
  __shared__ uint32_t s_f[kTabThreads], s_w[kTabThreads];
  __shared__ int s_held[kTabThreads], s_pos[kTabThreads];  // s_pos: first new token - w, so that item y is token s_pos + y
  __shared__ uint32_t s_at[kTabThreads];                   // head + f - held: entry j's page is s_at + j of the free list
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t cta = blockIdx.x, n_cta = gridDim.x;
  const int P = 1 << a.page_log2;
  int bad = 0;
  pdl_trigger();
  pdl_wait();
  int head = a.free_head ? *a.free_head : 0;
  // ---- sums over every thread's run of requests (one request each for at most 512) ----
  const int run = (a.n_req + kTabThreads - 1) / kTabThreads;
  TabReq q = {0, 0, 0, 0};
  uint32_t f = 0, w = 0;
#pragma unroll 4
  for (int i = 0; i < run; ++i) {
    q = tab_request(a, tid * run + i, &bad);
    f = sat_add(f, q.fresh);
    w = sat_add(w, q.n_new);
  }
  const TabScan all = tab_scan(f, w, 0, 0, s_warp);
  if (head < 0 || head > a.n_free) {
    bad |= kKvErrLens;
    head = head < 0 ? 0 : a.n_free;
  }
  const uint32_t left = a.n_free - head;  // pages in the free list
  if (all.f_all > left) bad |= kKvErrPages;
  const uint32_t n_slots = (uint32_t)min((int64_t)all.w_all, a.n_slots);
  if (a.slots && n_slots < all.w_all) bad |= kKvErrSlots;
  auto in_hand = [&](const TabReq& x, uint32_t f_at, uint32_t w_at) {
    s_f[tid] = f_at;
    s_w[tid] = w_at;
    s_held[tid] = x.held;
    s_pos[tid] = x.len - x.n_new - (int)w_at;
    s_at[tid] = (uint32_t)head + min(f_at, left) - x.held;  // (with j up to 2^27: below 2^32)
  };
  if (run == 1) {
    in_hand(q, all.f, all.w);
  } else {
    s_run[0][tid] = all.f;
    s_run[1][tid] = all.w;
  }
  __syncthreads();

  // a page id as it is written, -1 for none (kNoPage: the list has ended, which is reported above)
  constexpr int kNoPage = INT32_MIN;
  auto checked = [&](int page) {
    if ((unsigned)page < (unsigned)a.n_pages) return page;
    if (page != kNoPage) bad |= kKvErrPage;
    return -1;
  };
  // Kinds of items: 0 fresh table entries, 1 slots. With all requests in hand half of the warps see to each, else all
  // to one after the other.
  const int n_warps = run == 1 ? kTabWarps / 2 : kTabWarps, my_warp = warp % n_warps;
#pragma unroll 1
  for (int kind = warp / n_warps; kind < 2; kind += run == 1 ? 2 : 1) {
    const uint32_t total = kind ? n_slots : all.f_all;
    const uint32_t slice = (total / n_cta + kTabRun) / kTabRun * kTabRun;
    const uint32_t x0 = min((uint64_t)cta * slice, (uint64_t)total), x1 = min((uint64_t)x0 + slice, (uint64_t)total);
    if (x0 >= x1) continue;
    int r0 = 0;  // the first request in hand
    uint32_t f_at = 0, w_at = 0;
    if (run > 1) {
      const int k = warp_last_at_most(s_run[kind], kTabThreads, x0);
      r0 = k * run;
      f_at = s_run[0][k];
      w_at = s_run[1][k];
    }
    uint32_t x = x0;
    while (x < x1 && r0 < a.n_req) {
      uint32_t upto = x1;  // items of the requests in hand
      int n = min(kTabThreads, a.n_req - r0);
      if (run > 1) {
        int ignored = 0;
        const TabReq mine = tab_request(a, r0 + tid, &ignored);
        const TabScan at = tab_scan(mine.fresh, mine.n_new, f_at, w_at, s_warp);
        in_hand(mine, at.f, at.w);
        __syncthreads();
        f_at = at.f_all;
        w_at = at.w_all;
        upto = min(x1, kind ? w_at : f_at);
      }
      const uint32_t* starts = kind ? s_w : s_f;
      // the warp's items: whole steps, the same number for each warp
      const uint32_t step = n_warps * kTabRun, each = (upto - min(x, upto) + step - 1) / step * kTabRun;
      uint32_t b = (uint32_t)min((uint64_t)x + (uint64_t)my_warp * each, (uint64_t)upto);
      const uint32_t mine_end = (uint32_t)min((uint64_t)b + each, (uint64_t)upto);
      while (b < mine_end) {
        constexpr int U = kTabRun / 32;
        const uint32_t e = min(b + kTabRun, mine_end);
        const int k0 = warp_last_at_most(starts, n, b), k1 = warp_last_at_most(starts, n, e - 1);
        // Slots of one request only, as most of a long history's: on to its end or the warp's, 32 pages at a time, their ids one
        // per lane and the next 32 on their way (5.5 million slots: 23.2 -> 20.7 us).
        if (kind == 1 && k0 == k1) {
          const uint32_t stop = min(mine_end, k0 + 1 < n ? s_w[k0 + 1] : upto);
          const int pos0 = s_pos[k0], held = s_held[k0], j_end = (pos0 + (int)stop - 1) >> a.page_log2;
          const uint32_t at0 = s_at[k0];
          const int32_t* const row = a.table + (int64_t)(r0 + k0) * a.max_pages;
          auto id_of = [&](int j) {
            const bool fresh = j >= held;
            if (j > j_end || (fresh && at0 + j >= (uint32_t)a.n_free)) return kNoPage;
            return max(fresh ? a.free_pages[at0 + j] : row[j], -1);
          };
          int j = (pos0 + (int)b) >> a.page_log2, next = id_of(j + lane);
          for (uint32_t y0 = b; y0 < stop; j += 32) {
            const int id = checked(next);
            next = id_of(j + 32 + lane);
            const uint32_t y1 = min(stop, ((uint32_t)(j + 32) << a.page_log2) - (uint32_t)pos0);
#pragma unroll 4
            for (; y0 < y1; y0 += 32) {
              const uint32_t y = y0 + lane;
              const int pos = pos0 + (int)y, p = __shfl_sync(0xffffffffu, id, min((pos >> a.page_log2) - j, 31));
              if (y < y1) a.slots[y] = p < 0 ? -1 : ((int64_t)p << a.page_log2) + (pos & (P - 1));
            }
            y0 = y1;
          }
          b = stop;
          continue;
        }
        // the items' requests, by halving steps that the items of a lane take together
        int of[U], page[U], where[U];
#pragma unroll
        for (int u = 0; u < U; ++u) of[u] = k0;
        for (int step = k1 > k0 ? 1 << (31 - __clz(k1 - k0)) : 0; step > 0; step >>= 1)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int to = min(of[u] + step, k1);  // (past the last: the last itself, which holds if it is reached at all)
            const uint32_t start = starts[to];
            of[u] = start <= b + u * 32 + lane ? to : of[u];
          }
        // where each item goes, and its page's place in the free list
        uint32_t at[U];
        bool held = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t y = min(b + u * 32 + lane, e - 1);
          const int k = of[u];
          if (kind == 0) {
            where[u] = s_held[k] + (int)(y - s_f[k]);
            at[u] = (uint32_t)head + y;
          } else {
            where[u] = s_pos[k] + (int)y;
            const int j = where[u] >> a.page_log2;
            at[u] = s_at[k] + j;
            held |= j < s_held[k];
          }
        }
        if (__any_sync(0xffffffffu, held) || a.n_free == 0) {
          // (some in held entries, or no list: one load each, from either; without branches all are in flight together)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int k = of[u], j = kind ? where[u] >> a.page_log2 : where[u];
            const bool fresh = kind == 0 || j >= s_held[k], none = fresh && at[u] >= (uint32_t)a.n_free;
            const int32_t* from =
                fresh && !none ? a.free_pages + at[u] : a.table + (int64_t)(r0 + k) * a.max_pages + min(j, a.max_pages - 1);
            page[u] = max(*from, -1);
            if (none) page[u] = kNoPage;
          }
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            page[u] = max(a.free_pages[min(at[u], (uint32_t)a.n_free - 1)], -1);
            if (at[u] >= (uint32_t)a.n_free) page[u] = kNoPage;
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t y = b + u * 32 + lane;
          if (y >= e) continue;
          const int p = checked(page[u]);
          if (kind == 0) a.table[(int64_t)(r0 + of[u]) * a.max_pages + where[u]] = p;
          else a.slots[y] = p < 0 ? -1 : ((int64_t)p << a.page_log2) + (where[u] & (P - 1));
        }
        b = e;
      }
      x = upto;
      r0 += kTabThreads;
      if (run > 1) __syncthreads();  // the requests in hand have been read
    }
  }
  // ---- what each request holds now: thread t's run is written by CTA t mod n_cta ----
  if (a.pages && tid % n_cta == cta) {
    uint32_t at = all.f;
    for (int i = 0; i < run; ++i) {
      const int r = tid * run + i;
      if (r >= a.n_req) break;
      int ignored = 0;
      const TabReq x = run == 1 ? q : tab_request(a, r, &ignored);
      a.pages[r] = x.held + (int)min((uint32_t)x.fresh, at < left ? left - at : 0);
      at = sat_add(at, x.fresh);
    }
  }
  if (all.f_all == kTabMost) tab_behind(a, run, all.f, s_run[0]);
  if (a.slots)
    for (int64_t y = (int64_t)n_slots + cta * kTabThreads + tid; y < a.n_slots; y += n_cta * kTabThreads) a.slots[y] = -1;
  if (cta == 0 && tid == 0 && a.free_head_out) *a.free_head_out = head + (int)min(all.f_all, left);
  if (bad) atomicOr(a.err, bad);
}

// ------------------------------------------------------------------------------------------
// Append: 16 bytes (8 values) of a row per thread, the key's and the value's loads in flight together. Bound by HBM:
// 16383 tokens of 8 heads of 128 move 134 MB in 22.9 us (88% of the measured copy rate).
template <typename T>
__device__ __forceinline__ float2 to_f32x2(uint32_t x);
template <>
__device__ __forceinline__ float2 to_f32x2<__nv_bfloat16>(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 to_f32x2<__half>(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// 8-bit codes of 8 values of a row whose largest magnitude is `big`, finite: q = round-half-even(y), y = 127 x / big, as in
// exact arithmetic. r = x (127 / big) is within 2^-23 |y| of y. A y that is no half lies at least 2^-19 |y| from one: 127 x
// and big are whole numbers of at most 18 and 11 bits times powers of two, so y - (k + 1/2) is a multiple of
// |y| / (2 * 127 * 2^11). So an r within 2^-20 |r| of a half stands for that half, any other for a y on its own side of it.
template <typename T>
__device__ __forceinline__ uint2 codes8(const uint4& x, float big) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number, in the low bits
  const float up = big < 0x1p-60f ? 0x1p64f : 1.f;
  const float c2 = big > 0.f ? __fdiv_rn(254.f, big * up) : 0.f;  // 2 * 127 / big (times up, a power of two, for tiny rows)
  uint32_t code[8];
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 v = to_f32x2<T>(w[j >> 1]);
    const float r2 = (j & 1 ? v.y : v.x) * up * c2;
    const float whole = __fadd_rn(__fadd_rn(r2, kMagic), -kMagic);  // 2 y to the nearest half of y
    const float y2 = fabsf(r2 - whole) <= fabsf(r2) * 0x1p-20f ? whole : r2;
    code[j] = __float_as_uint(__fmaf_rn(y2, 0.5f, kMagic));
  }
  auto four = [](const uint32_t* c) {
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  };
  return make_uint2(four(code), four(code + 4));
}

constexpr int kAppThreads = 256;

template <typename T, bool I8>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(const KvAppendArgs a) {
  const unsigned vec_row = a.head_dim >> 3;  // vectors of 8 values per row: 4, 8 or 16, within one warp
  const unsigned vec_tok = a.kv_heads * vec_row;
  const int64_t n_slots = a.n_pages << a.page_log2;
  int bad = 0;
  pdl_trigger();
  pdl_wait();
  // (2^18 tokens at a time, for 32-bit indices; whole warps stay in the loop together: 8-bit rows are reduced across lanes)
  for (int64_t t0 = 0; t0 < a.n_tok; t0 += 1 << 18) {
    const unsigned total = (unsigned)min(a.n_tok - t0, (int64_t)1 << 18) * vec_tok;
    for (unsigned base = blockIdx.x * kAppThreads; base < total; base += gridDim.x * kAppThreads) {
      const unsigned i = base + threadIdx.x;
      const bool in = i < total;
      const unsigned at_tok = in ? i / vec_tok : 0, c = in ? i - at_tok * vec_tok : 0;
      const unsigned head = c / vec_row, piece = c - head * vec_row;
      const int64_t tok = t0 + at_tok, slot = in ? a.slots[tok] : -1;
      const bool ok = slot >= 0 && slot < n_slots;
      if (slot >= n_slots) bad |= kKvErrSlot;
      const int64_t page = slot >> a.page_log2, pos = slot & ((1 << a.page_log2) - 1);
      uint4 row[2];
#pragma unroll
      for (int w = 0; w < 2; ++w)
        row[w] = ok && a.src[w] ? *(reinterpret_cast<const uint4*>(static_cast<const T*>(a.src[w]) + tok * a.src_stride[w]) + c)
                                : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (!a.src[w]) continue;
        const uint4 x = row[w];
        const int64_t at = page * a.stride[w][0] + head * a.stride[w][1] + pos * a.stride[w][2] + piece * 8;
        if (!I8) {
          if (ok) *reinterpret_cast<uint4*>(static_cast<T*>(a.pool[w]) + at) = x;
          continue;
        }
        // the row's largest magnitude on the bits, in pairs: without their sign 16-bit floats order like whole numbers,
        // infinities and NaN last
        uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                              __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
        for (unsigned d = vec_row >> 1; d > 0; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float2 m2 = to_f32x2<T>(max(m & 0xffffu, m >> 16));
        const float big = m2.x;
        const bool finite = big < INFINITY;  // (not for NaN either)
        if (ok) {
          *reinterpret_cast<uint2*>(static_cast<int8_t*>(a.pool[w]) + at) = finite ? codes8<T>(x, big) : make_uint2(0, 0);
          if (piece == 0) a.scale[w][((page * a.kv_heads + head) << a.page_log2) + pos] = __fdiv_rn(big, 127.f);
        }
      }
    }
  }
  if (bad) atomicOr(a.err, bad);
}

}  // namespace

cudaError_t launch_kv_tables(const KvTablesArgs& a, int num_sms, cudaStream_t s) {
  // one CTA per 2048 items, at most one per SM (each sums all requests: two per SM were no faster). How many fresh entries
  // there are only the device knows: with a slot map about one per page of new tokens, else at most what the list holds.
  const int64_t entries = (int64_t)a.n_req * a.max_pages < a.n_free ? (int64_t)a.n_req * a.max_pages : a.n_free;
  const int64_t per_slot = a.n_req + (a.n_slots >> a.page_log2);
  const int64_t want = 1 + (a.n_slots + (a.slots && per_slot < entries ? per_slot : entries)) / 2048;
  return launch_kernel(want == 1 ? kv_tables_kernel<kTabRunShort> : kv_tables_kernel<kTabRunLong>,
                       dim3((unsigned)(want < num_sms ? want : num_sms)), dim3(kTabThreads), 0, s, true, a);
}

cudaError_t launch_kv_append(const KvAppendArgs& a, int dtype, bool int8, int num_sms, cudaStream_t s) {
  const int64_t total = a.n_tok * a.kv_heads * (a.head_dim / 8);
  const int64_t want = (total + kAppThreads - 1) / kAppThreads, most = (int64_t)num_sms * 8;
  const dim3 grid((unsigned)(want < most ? want : most));
  auto run = [&](auto kern) { return launch_kernel(kern, grid, dim3(kAppThreads), 0, s, true, a); };
  if (dtype == CVR_DTYPE_BF16)
    return int8 ? run(kv_append_kernel<__nv_bfloat16, true>) : run(kv_append_kernel<__nv_bfloat16, false>);
  return int8 ? run(kv_append_kernel<__half, true>) : run(kv_append_kernel<__half, false>);
}

}  // namespace cvr
