// Histories over a limit cut to their heaviest tokens, in place (cvr_kv_evict of include/cvr.h). Of a request of n > limit tokens
// every kv head keeps the first `first`, the last `last`, and of the tokens between them the b = keep - first - last of the
// largest weight; what stays moves to places 0 .. keep - 1 in its order. The floor is the bytes of the weights of all tokens and, in and
// out, of the rows that stay.
//
// A (request, kv head) is one cluster's, of 1 to 8 CTAs:
//   1. Selection. Weights become whole numbers that order as they do; the b-th largest is found by its 11, 11 and 10 bits, from the
//      highest: a histogram of the next bits of the numbers that begin like it, summed over the cluster.
//   2. The list `kept`, in order: every warp counts and then writes what stays of its share of the tokens; of the tokens whose
//      weight is the b-th largest the earliest stay.
//   3. Rows. Place i gets the row of token kept[i] >= i. Rounds of places in order: asynchronous copies bring a round's rows to shared
//      memory, two rounds ahead; when the cluster has a round's rows, it meets and writes them to their places. These lie at or before
//      the tokens that this and later rounds read, so nothing is written before it has been read, and reading ahead reads nothing
//      written. A thread writes the pieces that it brought.
// Pages behind the places go back to the free list, in blocks of requests of their own: what they need, the lengths, is known.
//
// Measured (one GB300, copy rate 6.78 TB/s): 64 requests of up to 8191 tokens cut to 1023 each, 8 heads of 128, bf16: 96.8 us. Cut to 8
// tokens each they take 29 us (mostly selection: latency of dependent loads, three passes over shared memory); the other 68 move 410 MB,
// at 89% of the copy rate; on 8 bits 67 us, on 4 bits 56. Rows by bulk copies, two in and two out per token: 181 us, some 20 ns each per SM. Rounds of register-held
// rows whose lookups waited for one another: 187 us. One request of 131071 cut to 32768: 153 us in 8 clusters of 8 CTAs of 1024 threads, 457 us in CTAs of 256.
#include <cstddef>

#include "../../include/cvr.h"
#include "cvr_kv_rows.cuh"

namespace cvr {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kReleased = 256;  // requests whose pages one CTA gives back
constexpr int kBins = 2048;
constexpr int kPieces = 4;      // 16-byte pieces of rows per thread and round

// A CTA's shape: three on an SM, or, where there are too few (request, head)s to fill the GPU, one with rounds of four times the rows.
template <int THREADS>
struct Shape {
  static constexpr int kThreads = THREADS, kWarps = THREADS / 32, kCtasPerSm = THREADS == 256 ? 3 : 1;
  static constexpr int kPerThread = kBins / THREADS;
  static constexpr int kStages = THREADS == 256 ? 3 : 2, kStageBytes = THREADS * kPieces * 16;  // rounds of rows in shared memory, and the most that one takes
  static constexpr int kMaxRows = THREADS == 256 ? 64 : 128;                                  // rows of a round
  static constexpr int kLooked = kStages + 2;  // rounds whose rows' offsets are held: looked up a round before they are read
  // a CTA's share of the weights that shared memory holds; longer shares are read again
  static constexpr int kKeys = kStages * kStageBytes / 4 - kBins;
};

template <int THREADS>
struct __align__(16) Shared : Shape<THREADS> {
  typedef Shape<THREADS> S;
  uint32_t above, ties;   // this CTA's tokens over the b-th largest weight, and of that weight, read by the cluster
  uint32_t w_above[S::kWarps], w_ties[S::kWarps];
  uint32_t found, rest;   // the next bits, and how many are wanted of their bin
  int64_t sum[S::kWarps], sum2[S::kWarps], sum3[S::kWarps];
  int64_t from[S::kLooked][2][S::kMaxRows], to[S::kLooked][2][S::kMaxRows];  // where rows are in the pools, and go (-1: nowhere)
  struct {
    uint2 blocks[2];       // block scales (of rows of 32 values those of two tokens)
    float weight, scale[2];
    int page, pos;         // where the row goes (page -1: nowhere)
  } row[S::kStages][S::kMaxRows];
  union {
    struct {  // while tokens are selected
      uint32_t hist[kBins];  // read by the cluster
      uint32_t keys[S::kKeys];
    };
    uint32_t start[kReleased + 1];
    __align__(16) uint8_t rows[S::kStages * S::kStageBytes];  // while rows move
  };
};
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// all threads of the cluster meet; what they wrote before is seen by all after
__device__ __forceinline__ void meet(uint32_t ctas) {
  if (ctas == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;\n" ::: "memory");
  }
}
__device__ __forceinline__ uint32_t peer_load(const uint32_t* p, uint32_t rank) {
  uint32_t addr, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <int BYTES>
__device__ __forceinline__ void async_in(void* dst, const void* src) {
  if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}

// Numbers that order as weights do, both zeros the same and NaN below all.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t x = __float_as_uint(w + 0.f);  // (-0 becomes 0)
  return w != w ? 0u : x & 0x80000000u ? ~x : x | 0x80000000u;
}

struct Request {
  int len, held;
  bool cut;
};
__device__ __forceinline__ Request request_of(const KvEvictArgs& a, int r, int* bad) {
  Request q;
  const int raw = a.lens[r], most = a.max_pages << a.page_log2;
  q.len = raw < 0 ? 0 : min(raw, most);
  if (q.len != raw) *bad |= kKvErrLens;
  const int need = (q.len + (1 << a.page_log2) - 1) >> a.page_log2;
  q.held = need;
  if (a.held) {
    const int h = a.held[r];
    q.held = min(max(h, 0), a.max_pages);
    if (q.held != h || q.held < need) *bad |= kKvErrLens;
    q.len = min(q.len, q.held << a.page_log2);  // (no entry behind the pages held is used)
  }
  q.cut = q.len > a.limit;
  return q;
}
// entries that a request keeps
__device__ __forceinline__ int stays(const KvEvictArgs& a, const Request& q) {
  return q.cut && a.free_pages ? min(q.held, (a.keep + (1 << a.page_log2) - 1) >> a.page_log2) : q.held;
}

// entries that a request's tokens take
__device__ __forceinline__ int entries_of(const KvEvictArgs& a, const Request& q) { return (q.len + (1 << a.page_log2) - 1) >> a.page_log2; }

// Lengths, page counts and the free list of requests [r0, r0 + kReleased), by one CTA. An id outside the pool among a cut request's tokens'
// is not given back, so where the pages of these requests go depends on the ids of all: every CTA looks at them.
template <int THREADS>
__device__ void release(const KvEvictArgs& a, Shared<THREADS>& s, int r0) {
  constexpr int kThreads = THREADS, kWarps = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int bad = 0, ignored = 0;
  int64_t before = 0, all = 0;  // pages given back by the requests before r0, and by all
  bool gaps = false;            // ids outside the pool among those of these requests
  // (32 requests, one per lane, are one warp's, or where there are few requests several warps')
  const int share = max(kWarps / max((a.n_req + 31) / 32, 1), 1), part = warp % share;
  for (int r = warp / share * 32; r < (a.free_pages ? a.n_req : 0); r += kWarps / share * 32) {
    Request q = {0, 0, false};
    if (r + lane < a.n_req) q = request_of(a, r + lane, &ignored);
    const int left = stays(a, q), n = part == 0 ? q.held - left : 0;
    all += n;
    if (r + lane < r0) before += n;
    // the requests' entries behind those that stay, evenly over the lanes
    const uint32_t look = max(entries_of(a, q) - left, 0);  // (at most 2^27 - 1)
    uint32_t incl = look;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += u;
    }
    const uint32_t start = incl - look, total = __shfl_sync(0xffffffffu, incl, 31);
    constexpr int U = 8;  // (loads in flight together)
    for (int64_t x0 = part * (U * 32); x0 < total; x0 += share * (U * 32)) {
      int of[U], page[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t x = (uint32_t)min(x0 + u * 32 + lane, (int64_t)total - 1);
        int k = 0;
#pragma unroll
        for (int step = 16; step > 0; step >>= 1) {
          const uint32_t to = __shfl_sync(0xffffffffu, start, k + step);
          if (to <= x) k += step;
        }
        of[u] = r + k;
        page[u] = a.table[(int64_t)(r + k) * a.max_pages + (__shfl_sync(0xffffffffu, left, k) + (int)(x - __shfl_sync(0xffffffffu, start, k)))];
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (x0 + u * 32 + lane < total && (unsigned)page[u] >= (unsigned)a.n_pages) {
          --all;
          if (of[u] < r0) --before;
          else if (of[u] < r0 + kReleased) gaps = true;
        }
    }
  }
  if (gaps) bad |= kKvErrPage;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, d);
    all += __shfl_xor_sync(0xffffffffu, all, d);
  }
  const int r = r0 + tid;
  const bool mine = tid < kReleased && r < a.n_req;
  Request q = {0, 0, false};
  if (mine) q = request_of(a, r, &bad);
  const int left = stays(a, q), n = q.held - left;
  if (mine) {
    a.lens_out[r] = q.cut ? a.keep : q.len;
    if (a.pages) a.pages[r] = left;
  }
  int64_t wide = n;  // (kReleased requests of at most 2^27 pages may pass 32 bits)
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, wide, d);
    if (lane >= d) wide += u;
  }
  if (lane == 31) s.sum[warp] = wide;
  if (lane == 0) {
    s.sum2[warp] = before;
    s.sum3[warp] = all;
  }
  gaps = __syncthreads_or(gaps);
  before = all = 0;
  int64_t ahead = wide - n, items = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) ahead += s.sum[w];
    items += s.sum[w];
    before += s.sum2[w];
    all += s.sum3[w];
  }
  if (a.free_pages) {
    int head = *a.free_head;
    if (head < 0 || head > a.n_free) bad |= kKvErrLens;
    head = min(max(head, 0), a.n_free);
    if (r0 == 0 && tid == 0) {
      *a.free_head_out = (int)max((int64_t)head - all, (int64_t)0);
      if (all > head) bad |= kKvErrPages;
    }
    if (tid < kReleased) s.start[tid] = (uint32_t)min(ahead, (int64_t)0xffffffff);
    if (tid == 0) s.start[kReleased] = (uint32_t)min(items, (int64_t)0xffffffff);
    __syncthreads();
    const int64_t at0 = (int64_t)head - all + before;  // where these requests' pages begin (below 0: no room in front of the list)
    const uint32_t end = s.start[kReleased];
    auto page_of = [&](int64_t x, bool* ok) {  // entry x of these requests' pages, and whether it is given back
      int k = 0;
      for (int step = kReleased / 2; step > 0; step >>= 1)
        if (s.start[k + step] <= x) k += step;
      const Request o = request_of(a, r0 + k, &ignored);
      const int entry = stays(a, o) + (int)(x - s.start[k]), page = a.table[(int64_t)(r0 + k) * a.max_pages + entry];
      *ok = (unsigned)page < (unsigned)a.n_pages || entry >= entries_of(a, o);
      return page;
    };
    bool ok = false;
    if (!gaps) {
      for (int64_t x = (at0 < 0 ? -at0 : 0) + tid; x < min((int64_t)end, a.n_free - at0); x += kThreads) a.free_pages[at0 + x] = page_of(x, &ok);
    } else {
      int64_t at = at0;
      for (int64_t x0 = 0; x0 < end; x0 += kThreads) {
        ok = false;
        const int page = x0 + tid < end ? page_of(x0 + tid, &ok) : 0;
        const unsigned there = __ballot_sync(0xffffffffu, ok);
        if (lane == 0) s.w_ties[warp] = __popc(there);
        __syncthreads();
        int64_t to = at + __popc(there & ((1u << lane) - 1));
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) to += s.w_ties[w];
          at += s.w_ties[w];
        }
        if (ok && to >= 0 && to < a.n_free) a.free_pages[to] = page;
        __syncthreads();
      }
    }
  }
  if (bad) atomicOr(a.err, bad);
}

template <int CODE, int THREADS>
__global__ void __launch_bounds__(THREADS, Shape<THREADS>::kCtasPerSm) evict_kernel(const __grid_constant__ KvEvictArgs a, int n_release) {
  typedef Shape<THREADS> S;
  constexpr int kThreads = S::kThreads, kWarps = S::kWarps, kPerThread = S::kPerThread, kStages = S::kStages, kStageBytes = S::kStageBytes;
  constexpr int kMaxRows = S::kMaxRows, kLooked = S::kLooked, kKeys = S::kKeys;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  typedef Shared<THREADS> Mem;
  static_assert(offsetof(Mem, rows) % 16 == 0 && offsetof(Mem, row) % 8 == 0 && sizeof(Mem::row[0][0]) % 8 == 0, "what the copies into shared memory ask for");
  Mem& s = *reinterpret_cast<Mem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t C = cluster_size(), rank = cluster_rank();
  const int64_t n_items = n_release + (int64_t)a.n_req * a.kv_heads;
  const int page_mask = (1 << a.page_log2) - 1;
  // 16-byte pieces of a row in a pool and in both (powers of two), rows of a round
  const int row_vecs = kv_row_bytes(CODE, a.head_dim) / 16, pools = a.pool[1] ? 2 : 1, log2_vecs = 31 - __clz(row_vecs * pools);
  const int rows = min(kMaxRows, kThreads * kPieces >> log2_vecs);
  int bad = 0, ignored = 0;
  pdl_trigger();
  pdl_wait();
  for (int64_t item = blockIdx.x / C; item < n_items; item += gridDim.x / C) {
    if (item < n_release) {
      if (rank == 0) release(a, s, (int)item * kReleased);
      __syncthreads();
      continue;
    }
    const int r = (int)((item - n_release) / a.kv_heads), h = (int)((item - n_release) % a.kv_heads);
    const int n = request_of(a, r, &ignored).len;
    if (n <= a.limit) continue;
    const int32_t* const row = a.table + (int64_t)r * a.max_pages;
    int32_t* const kept = a.kept + ((int64_t)r * a.kv_heads + h) * a.keep;
    auto page_of = [&](int j) {  // of token j, 0 where the entry is none of the pool
      const int p = row[j >> a.page_log2];
      const bool ok = (unsigned)p < (unsigned)a.n_pages;
      bad |= ok ? 0 : kKvErrPage;  // (without a branch: loads of several tokens are in flight together)
      return ok ? p : 0;
    };
    auto weight_of = [&](int j) { return a.weight + ((((int64_t)page_of(j) * a.kv_heads + h) << a.page_log2) + (j & page_mask)); };
    auto key_of = [&](int j) { return order_of(__ldcg(weight_of(j))); };

    // ---- 1. the b-th largest weight of the tokens [first, n - last) ----
    const int m = n - a.first - a.last, b = a.keep - a.first - a.last;  // (b < m)
    const int c0 = a.first + (int)((int64_t)m * rank / C), c1 = a.first + (int)((int64_t)m * (rank + 1) / C);  // this CTA's share
    const bool held = c1 - c0 <= kKeys - 32;  // (a warp's last step may look behind the share)
    // f(token, its number) for tokens from, from + step, .. of this CTA's share, from the share held or from their pages
    auto each = [&](int from, int to, int step, auto f) {
      if (held) {
#pragma unroll 8
        for (int j = from; j < to; j += step) f(j, s.keys[j - c0]);
      } else {
#pragma unroll 8
        for (int j = from; j < to; j += step) f(j, key_of(min(j, n - 1)));
      }
    };
    uint32_t threshold = 0, ties = 0;  // numbers over it stay, and this many of those that are it
    if (b > 0) {
      uint32_t want = b;
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
        __syncthreads();
        if (pass == 0 && held) {
          // (all of a thread's weights are on their way together)
#pragma unroll 16
          for (int j = c0 + tid; j < c1; j += kThreads) async_in<4>(&s.keys[j - c0], weight_of(j));
          asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 8
          for (int j = c0 + tid; j < c1; j += kThreads) {
            const uint32_t k = order_of(__uint_as_float(s.keys[j - c0]));
            s.keys[j - c0] = k;
            atomicAdd(&s.hist[k >> 21], 1u);
          }
        } else {
          each(c0 + tid, c1, kThreads, [&](int, uint32_t k) {
            if (pass == 0 || ((k ^ threshold) >> (shift + (pass == 1 ? 11 : 10))) == 0) atomicAdd(&s.hist[k >> shift & mask], 1u);
          });
        }
        meet(C);
        // The cluster's CTAs have a slice of the bins each, from the top, and a thread some of its CTA's: sums over the CTAs, and
        // from the top down to the bin in which the wanted number lies.
        const int slice = kBins / C, per = slice > kThreads ? slice / kThreads : 1;  // (per: at most kPerThread)
        uint32_t count[kPerThread] = {}, sum = 0;
        const int top = kBins - 1 - (int)rank * slice - tid * per;
        if (tid * per < slice) {
          for (uint32_t c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < kPerThread; ++i)
              if (i < per) count[i] += C == 1 ? s.hist[top - i] : peer_load(&s.hist[top - i], c);
#pragma unroll
          for (int i = 0; i < kPerThread; ++i) sum += count[i];
        }
        uint32_t incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t u = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += u;
        }
        if (lane == 31) s.w_above[warp] = incl;
        __syncthreads();
        uint32_t over = incl - sum, all = 0, owner = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          over += w < warp ? s.w_above[w] : 0;
          all += s.w_above[w];
        }
        if (C > 1) {
          if (tid == 0) s.above = all;
          meet(C);
          uint32_t before = 0;
          for (uint32_t c = 0; c < C; ++c) {  // slices before this one, and the one that has the wanted number
            const uint32_t x = peer_load(&s.above, c);
            if (c < rank) over += x;
            if (before < want && want <= before + x) owner = c;
            before += x;
          }
        }
        if (over < want && want <= over + sum) {
#pragma unroll
          for (int i = 0; i < kPerThread; ++i) {
            if (i < per && over < want && want <= over + count[i]) {
              s.found = top - i;
              s.rest = want - over;
            }
            over += count[i];
          }
        }
        meet(C);  // (also: all have read the histograms)
        if (C > 1) {
          threshold |= peer_load(&s.found, owner) << shift;
          want = peer_load(&s.rest, owner);
          continue;
        }
        threshold |= s.found << shift;
        want = s.rest;
      }
      ties = want;
    }

    // ---- 2. the list: warps take shares of the CTA's share ----
    const int w0 = c0 + (int)((int64_t)(c1 - c0) * warp / kWarps), w1 = c0 + (int)((int64_t)(c1 - c0) * (warp + 1) / kWarps);
    if (b > 0) {
      uint32_t above = 0, equal = 0;
      each(w0 + lane, w1, 32, [&](int, uint32_t k) {
        above += k > threshold;
        equal += k == threshold;
      });
      above = __reduce_add_sync(0xffffffffu, above);
      equal = __reduce_add_sync(0xffffffffu, equal);
      if (lane == 0) {
        s.w_above[warp] = above;
        s.w_ties[warp] = equal;
      }
      __syncthreads();
      uint32_t at = 0, tie = 0, cta_above = 0, cta_ties = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
          at += s.w_above[w];
          tie += s.w_ties[w];
        }
        cta_above += s.w_above[w];
        cta_ties += s.w_ties[w];
      }
      if (C > 1) {
        if (tid == 0) {
          s.above = cta_above;
          s.ties = cta_ties;
        }
        meet(C);
        for (uint32_t c = 0; c < rank; ++c) {
          at += peer_load(&s.above, c);
          tie += peer_load(&s.ties, c);
        }
      }
      // the place of the next that stays: those over the threshold and the ties so far, at most `ties` of them
      at += min(tie, ties);
      const unsigned below = (1u << lane) - 1;
      // (whole warps stay together; places are in bounds whatever the weights do meanwhile, as those of a page that is another
      // request's too)
      each(w0 + lane, w0 + (w1 - w0 + 31) / 32 * 32 + lane, 32, [&](int j, uint32_t k) {
        const bool in = j < w1, is_above = in && k > threshold;
        const unsigned over = __ballot_sync(0xffffffffu, is_above);
        if (__any_sync(0xffffffffu, in && k == threshold) && tie < ties) {
          const unsigned same = __ballot_sync(0xffffffffu, in && k == threshold);
          const uint32_t my_tie = tie + __popc(same & below), before = min(my_tie, ties) - tie;
          const uint32_t place = at + __popc(over & below) + before;
          if ((is_above || (same >> lane & 1 && my_tie < ties)) && place < (uint32_t)b) kept[a.first + place] = j;
          const uint32_t taken = min(tie + __popc(same), ties) - tie;
          tie += taken;
          at += taken;
        } else {
          const uint32_t place = at + __popc(over & below);
          if (is_above && place < (uint32_t)b) kept[a.first + place] = j;
        }
        at += __popc(over);
      });
    }
    for (int i = rank * kThreads + tid; i < a.first; i += C * kThreads) kept[i] = i;
    for (int i = rank * kThreads + tid; i < a.last; i += C * kThreads) kept[a.keep - a.last + i] = n - a.last + i;
    meet(C);  // (the list is written, and every weight has been read)

    // ---- 3. rows, scales and weights, in rounds of `rows` places per CTA ----
    const int n_rounds = (int)(((int64_t)a.keep + (int64_t)C * rows - 1) / ((int64_t)C * rows));
    auto place = [&](int q) { return ((int64_t)q * C + rank) * rows + tid; };  // this thread's of round q
    auto has = [&](int q) { return tid < rows && q < n_rounds && place(q) < a.keep; };
    // Where rows of a round come from and go to. Loads are issued a round before what they bring is used: the list's entry, then the
    // table's entries.
    int listed = has(0) ? __ldcg(kept + place(0)) : 0, token = 0, from_page = 0, to_page = 0;
    auto entries = [&](int q) {  // of round q, whose list entry has come; and the next list entry
      if (has(q)) {
        token = min(max(listed, 0), n - 1);  // (in bounds, as above)
        from_page = row[token >> a.page_log2];
        to_page = row[(int)place(q) >> a.page_log2];
      }
      if (has(q + 1)) listed = __ldcg(kept + place(q + 1));
    };
    auto offset = [&](int w, int page, int pos) { return page * a.stride[w][0] + h * a.stride[w][1] + pos * a.stride[w][2]; };
    auto look_up = [&](int q) {  // round q's offsets, its entries have come
      if (tid < rows && q < n_rounds) {
        const bool there = has(q), ok = there && (unsigned)from_page < (unsigned)a.n_pages, writes = there && (unsigned)to_page < (unsigned)a.n_pages;
        if (there && !(ok && writes)) bad |= kKvErrPage;
        const int from = ok ? from_page : 0, pos = token & page_mask, to_pos = (int)place(q) & page_mask;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (w >= pools) continue;
          s.from[q % kLooked][w][tid] = there ? offset(w, from, pos) : -1;
          s.to[q % kLooked][w][tid] = writes ? offset(w, to_page, to_pos) : -1;
        }
        // this row's scalars (its own thread writes them too)
        auto& x = s.row[q % kStages][tid];
        x.page = writes ? to_page : -1;
        x.pos = to_pos;
        if (there) {
          const int64_t page_head = (int64_t)from * a.kv_heads + h;
          async_in<4>(&x.weight, a.weight + (page_head << a.page_log2) + pos);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (w >= pools) continue;
            if (CODE == kKv8) async_in<4>(&x.scale[w], static_cast<const float*>(a.scale[w]) + (page_head << a.page_log2) + pos);
            if (CODE == kKv4) {
              const uint8_t* const record = kv4_record(a.scale[w], page_head, a.page_log2, a.head_dim);
              const uint8_t* const blocks = record + (4 << a.page_log2) + pos * (a.head_dim >> 4);
              async_in<4>(&x.scale[w], record + pos * 4);
              if (a.head_dim == 128) async_in<8>(&x.blocks[w], blocks);
              else async_in<4>(&x.blocks[w], reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(blocks) & ~(uintptr_t)3));
              if (a.head_dim == 32) x.blocks[w].y = pos & 1;  // (which of the two)
            }
          }
        }
      }
    };
    auto piece_of = [&](int u, int* r, int* w, int* part) {  // a thread's u-th piece of a round: row, pool, bytes into the row
      const int x = tid + u * kThreads, vec = x & ((1 << log2_vecs) - 1);
      *r = x >> log2_vecs;
      *w = vec >= row_vecs;
      *part = (vec & (row_vecs - 1)) * 16;
    };
    auto fetch = [&](int q) {
      if (q < n_rounds) {
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
          int r, w, part;
          piece_of(u, &r, &w, &part);
          if (r >= rows) continue;
          const int64_t from = s.from[q % kLooked][w][r];
          if (from >= 0) async_in<16>(s.rows + q % kStages * kStageBytes + (tid + u * kThreads) * 16, static_cast<const char*>(a.pool[w]) + from + part);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // A round's scalars come with the group of the round before its rows: look_up(q + 1) precedes fetch(q)'s commit.
    entries(0);
    look_up(0);
    entries(1);
    __syncthreads();
    for (int q = 0; q < kStages - 1; ++q) {
      look_up(q + 1);
      entries(q + 2);
      fetch(q);
      __syncthreads();
    }
#pragma unroll 1
    for (int q = 0; q < n_rounds; ++q) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      meet(C);
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        int r, w, part;
        piece_of(u, &r, &w, &part);
        if (r >= rows) continue;
        const int64_t to = s.to[q % kLooked][w][r];
        if (to >= 0) *reinterpret_cast<uint4*>(static_cast<char*>(a.pool[w]) + to + part) = *reinterpret_cast<const uint4*>(s.rows + q % kStages * kStageBytes + (tid + u * kThreads) * 16);
      }
      if (tid < rows) {
        const auto& x = s.row[q % kStages][tid];
        if (x.page >= 0) {
          const int64_t page_head = (int64_t)x.page * a.kv_heads + h;
          a.weight[(page_head << a.page_log2) + x.pos] = x.weight;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (w >= pools) continue;
            if (CODE == kKv8) static_cast<float*>(a.scale[w])[(page_head << a.page_log2) + x.pos] = x.scale[w];
            if (CODE == kKv4) {
              uint8_t* const record = kv4_record(a.scale[w], page_head, a.page_log2, a.head_dim);
              uint8_t* const blocks = record + (4 << a.page_log2) + x.pos * (a.head_dim >> 4);
              reinterpret_cast<float*>(record)[x.pos] = x.scale[w];
              if (a.head_dim == 128) *reinterpret_cast<uint2*>(blocks) = x.blocks[w];
              else if (a.head_dim == 64) *reinterpret_cast<uint32_t*>(blocks) = x.blocks[w].x;
              else *reinterpret_cast<uint16_t*>(blocks) = (uint16_t)(x.blocks[w].x >> (x.blocks[w].y * 16));
            }
          }
        }
      }
      look_up(q + kStages);
      entries(q + kStages + 1);
      fetch(q + kStages - 1);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    meet(C);  // (a CTA's shared memory is read by others until here)
  }
  if (bad) atomicOr(a.err, bad);
}

template <int CODE, int THREADS>
cudaError_t launch(const KvEvictArgs& a, int ctas, cudaStream_t s) {
  const int n_release = a.n_req > 0 ? (a.n_req + kReleased - 1) / kReleased : 1;
  const int64_t items = n_release + (int64_t)a.n_req * a.kv_heads, clusters = items < 65536 ? items : 65536;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(clusters * ctas));
  lc.blockDim = dim3(THREADS);
  lc.dynamicSmemBytes = sizeof(Shared<THREADS>);
  lc.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 2;
  cudaError_t e = cudaFuncSetAttribute(evict_kernel<CODE, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared<THREADS>));
  return e != cudaSuccess ? e : cudaLaunchKernelEx(&lc, evict_kernel<CODE, THREADS>, a, n_release);
}

template <int CODE>
cudaError_t launch(const KvEvictArgs& a, int num_sms, cudaStream_t s) {
  // As many CTAs per (request, head) as the SMs hold, of 1024 tokens at least: a large one per SM for long histories, two small ones for
  // others. A cluster pays for its meetings: 4 requests of 20000 tokens, 8 heads, 51 us in 4 large CTAs each, 67 us in 8 small ones; 512
  // (request, head)s in clusters of two 153 us instead of 104. The lengths are on the device, so it is the table's room that decides: 16
  // histories of up to 2000 events, 4 heads of 32, take 15.6 us in a table of 125 pages of 16 and 22.6 in one of 1024 or more; 8 of up to
  // 2000 tokens, 8 heads of 128, 50 and 33.
  const int64_t pairs = (int64_t)a.n_req * a.kv_heads, most = (int64_t)a.max_pages << a.page_log2;
  const bool large = most >= 16384 && pairs <= num_sms;
  // (clusters of 8 have to find 8 free SMs of one group: 16 of them on 128 SMs run in two waves)
  const auto fit = [&](int n) { return large ? (n == 8 ? num_sms * 2 / 3 : num_sms) : 2 * num_sms; };
  int ctas = 1;
  while (ctas < kMaxCluster && pairs * ctas * 2 <= fit(ctas * 2) && most / (ctas * 2) >= 1024) ctas *= 2;
  return large ? launch<CODE, 1024>(a, ctas, s) : launch<CODE, 256>(a, ctas, s);
}

}  // namespace

cudaError_t launch_kv_evict(const KvEvictArgs& a, int code, int num_sms, cudaStream_t s) {
  return code == kKv16 ? launch<kKv16>(a, num_sms, s) : code == kKv8 ? launch<kKv8>(a, num_sms, s) : launch<kKv4>(a, num_sms, s);
}

}  // namespace cvr
