// Histories over a limit cut to their heaviest tokens, in place (cvr_kv_evict of include/cvr.h). Of a request of n > limit tokens
// every kv head keeps the first `first`, the last `last`, and of the tokens between them the b = keep - first - last of the
// largest weight; what stays moves to places 0 .. keep - 1 in its order. The floor is the bytes of the weights of all tokens and, in and
// out, of the rows that stay.
//
// A (request, kv head) is one cluster's, of 1 to 8 CTAs:
//   1. Selection. Weights become whole numbers that order as they do; the b-th largest is found by its four bytes, from the
//      highest: a histogram of the next byte of the numbers that begin like it, summed over the cluster.
//   2. The list `kept`, in order: every warp counts and then writes what stays of its share of the tokens; of the tokens whose
//      weight is the b-th largest the earliest stay.
//   3. Rows. Place i gets the row of token kept[i] >= i. In rounds, places in order: the cluster reads a round's rows into
//      registers, meets, and writes them. A round's places lie at or before the tokens that it and later rounds read, and behind none of
//      them is written before all have been read: so nothing is lost, and rows that do not move are the same again.
// Pages behind the places go back to the free list, in blocks of requests of their own: what they need, the lengths, is known.
#include "../../include/cvr.h"
#include "cvr_kv_rows.cuh"

namespace cvr {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 256, kCopies = 8;  // a histogram's copies: lanes that meet in one bin mostly count in different ones
constexpr int kKeys = 8192;              // a CTA's share of the weights that shared memory holds; longer shares are read again
constexpr int kInFlight = 8;             // 16-byte pieces of rows in flight per thread

struct __align__(16) Shared {
  uint32_t hist[kBins * kCopies];
  uint32_t mine[kBins];   // this CTA's histogram, read by the cluster
  uint32_t total[kBins];  // the cluster's
  uint32_t above, ties;   // this CTA's tokens over the b-th largest weight, and of that weight, read by the cluster
  uint32_t w_above[kWarps], w_ties[kWarps];
  uint32_t found, rest;   // the byte, and how many are wanted of its bin
  int64_t sum[kWarps], sum2[kWarps];
  uint32_t start[kThreads + 1];
  uint32_t keys[kKeys];
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
  }
  q.cut = q.len > a.limit;
  return q;
}
// entries that a request keeps
__device__ __forceinline__ int stays(const KvEvictArgs& a, const Request& q) {
  return q.cut && a.free_pages ? min(q.held, (a.keep + (1 << a.page_log2) - 1) >> a.page_log2) : q.held;
}

// Lengths, page counts and the free list of requests [r0, r0 + kThreads), by one CTA.
__device__ void release(const KvEvictArgs& a, Shared& s, int r0) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int bad = 0, ignored = 0;
  int64_t before = 0, all = 0;  // pages given back by the requests before r0, and by all
  if (a.free_pages)
    for (int r = tid; r < a.n_req; r += kThreads) {
      const Request q = request_of(a, r, &ignored);
      const int n = q.held - stays(a, q);
      all += n;
      if (r < r0) before += n;
    }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, d);
    all += __shfl_xor_sync(0xffffffffu, all, d);
  }
  const int r = r0 + tid;
  Request q = {0, 0, false};
  if (r < a.n_req) q = request_of(a, r, &bad);
  const int left = stays(a, q), n = q.held - left;
  if (r < a.n_req) {
    a.lens_out[r] = q.cut ? a.keep : q.len;
    if (a.pages) a.pages[r] = left;
  }
  int64_t wide = n;  // (512 requests of at most 2^27 pages may pass 32 bits)
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, wide, d);
    if (lane >= d) wide += u;
  }
  if (lane == 31) s.sum[warp] = wide;
  if (lane == 0) {
    s.sum2[warp] = before;
    reinterpret_cast<int64_t*>(s.hist)[warp] = all;
  }
  __syncthreads();
  before = all = 0;
  int64_t ahead = wide - n, items = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) ahead += s.sum[w];
    items += s.sum[w];
    before += s.sum2[w];
    all += reinterpret_cast<int64_t*>(s.hist)[w];
  }
  if (a.free_pages) {
    int head = *a.free_head;
    if (head < 0 || head > a.n_free) bad |= kKvErrLens;
    head = min(max(head, 0), a.n_free);
    if (r0 == 0 && tid == 0) {
      *a.free_head_out = (int)max((int64_t)head - all, (int64_t)0);
      if (all > head) bad |= kKvErrPages;
    }
    // entry x of these requests' pages goes to position head - all + before + x
    s.start[tid] = (uint32_t)min(ahead, (int64_t)0xffffffff);
    if (tid == 0) s.start[kThreads] = (uint32_t)min(items, (int64_t)0xffffffff);
    __syncthreads();
    const int64_t at0 = (int64_t)head - all + before;
    const int64_t skip = at0 < 0 ? -at0 : 0;  // (no room in front of the list)
    const uint32_t end = s.start[kThreads];
    for (int64_t x = skip + tid; x < end; x += kThreads) {
      int k = 0;
      for (int step = kThreads / 2; step > 0; step >>= 1)
        if (s.start[k + step] <= x) k += step;
      const Request o = request_of(a, r0 + k, &ignored);
      a.free_pages[at0 + x] = a.table[(int64_t)(r0 + k) * a.max_pages + stays(a, o) + (int)(x - s.start[k])];
    }
  }
  if (bad) atomicOr(a.err, bad);
}

template <int CODE>
__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const __grid_constant__ KvEvictArgs a, int n_release) {
  extern __shared__ uint8_t smem_raw[];
  Shared& s = *reinterpret_cast<Shared*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t C = cluster_size(), rank = cluster_rank();
  const int64_t n_items = n_release + (int64_t)a.n_req * a.kv_heads;
  const int page_mask = (1 << a.page_log2) - 1;
  int bad = 0, ignored = 0;
  pdl_trigger();
  pdl_wait();
  for (int64_t item = blockIdx.x / C; item < n_items; item += gridDim.x / C) {
    if (item < n_release) {
      if (rank == 0) release(a, s, (int)item * kThreads);
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
      if ((unsigned)p < (unsigned)a.n_pages) return p;
      bad |= kKvErrPage;
      return 0;
    };
    auto key_of = [&](int j) { return order_of(__ldcg(a.weight + ((((int64_t)page_of(j) * a.kv_heads + h) << a.page_log2) + (j & page_mask)))); };

    // ---- 1. the b-th largest weight of the tokens [first, n - last) ----
    const int m = n - a.first - a.last, b = a.keep - a.first - a.last;  // (b < m)
    const int c0 = a.first + (int)((int64_t)m * rank / C), c1 = a.first + (int)((int64_t)m * (rank + 1) / C);  // this CTA's share
    const bool held = c1 - c0 <= kKeys;
    auto key = [&](int j) { return held ? s.keys[j - c0] : key_of(j); };
    uint32_t threshold = 0, ties = 0;  // weights over it stay, and this many of those that are it
    if (b > 0) {
      if (held) {
#pragma unroll 4
        for (int j = c0 + tid; j < c1; j += kThreads) s.keys[j - c0] = key_of(j);
      }
      uint32_t want = b;
#pragma unroll 1
      for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < kBins * kCopies; i += kThreads) s.hist[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int j = c0 + tid; j < c1; j += kThreads) {
          const uint32_t k = key(j);
          if (shift == 24 || (k ^ threshold) >> (shift + 8) == 0) atomicAdd(&s.hist[(k >> shift & 255u) * kCopies + (lane & (kCopies - 1))], 1u);
        }
        __syncthreads();
        if (tid < kBins) {
          uint32_t sum = 0;
#pragma unroll
          for (int i = 0; i < kCopies; ++i) sum += s.hist[tid * kCopies + i];
          s.mine[tid] = sum;
        }
        meet(C);
        if (tid < kBins) {
          uint32_t sum = 0;
          if (C == 1) sum = s.mine[tid];
          else
            for (uint32_t c = 0; c < C; ++c) sum += peer_load(&s.mine[tid], c);
          s.total[tid] = sum;
        }
        __syncthreads();
        if (warp == 0) {
          // lane l has bins 255 - 8 l .. 248 - 8 l: sums from the top
          uint32_t sum = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) sum += s.total[255 - lane * 8 - i];
          uint32_t incl = sum;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += u;
          }
          const unsigned reach = __ballot_sync(0xffffffffu, incl >= want);
          if (lane == __ffs(reach) - 1) {
            uint32_t over = incl - sum;
            int bin = 255 - lane * 8;
            while (over + s.total[bin] < want) over += s.total[bin--];
            s.found = bin;
            s.rest = want - over;
          }
        }
        meet(C);  // (also: all have read the histograms)
        threshold |= s.found << shift;
        want = s.rest;
      }
      ties = want;
    }

    // ---- 2. the list: warps take shares of the CTA's share ----
    const int w0 = c0 + (int)((int64_t)(c1 - c0) * warp / kWarps), w1 = c0 + (int)((int64_t)(c1 - c0) * (warp + 1) / kWarps);
    if (b > 0) {
      uint32_t above = 0, equal = 0;
      for (int j = w0 + lane; j < w1; j += 32) {
        const uint32_t k = key(j);
        above += k > threshold;
        equal += k == threshold;
      }
      above = __reduce_add_sync(0xffffffffu, above);
      equal = __reduce_add_sync(0xffffffffu, equal);
      if (lane == 0) {
        s.w_above[warp] = above;
        s.w_ties[warp] = equal;
      }
      __syncthreads();
      uint32_t at = 0, tie = 0, cta_above = 0, cta_ties = 0;
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
      for (int j0 = w0; j0 < w1; j0 += 32) {
        const int j = j0 + lane;
        const uint32_t k = j < w1 ? key(j) : 0u;
        const bool is_above = j < w1 && k > threshold, is_tie = j < w1 && k == threshold;
        const unsigned over = __ballot_sync(0xffffffffu, is_above), same = __ballot_sync(0xffffffffu, is_tie), below = (1u << lane) - 1;
        const uint32_t my_tie = tie + __popc(same & below);
        const uint32_t place = at + __popc(over & below) + min(my_tie, ties);
        // (in bounds whatever the weights do meanwhile, as those of a page that is another request's too)
        if ((is_above || (is_tie && my_tie < ties)) && place < (uint32_t)b) kept[a.first + place] = j;
        at += __popc(over);
        tie += __popc(same);
      }
    }
    for (int i = rank * kThreads + tid; i < a.first; i += C * kThreads) kept[i] = i;
    for (int i = rank * kThreads + tid; i < a.last; i += C * kThreads) kept[a.keep - a.last + i] = n - a.last + i;
    meet(C);  // (the list is written, and every weight has been read)

    // ---- 3. rows, scales and weights, in rounds of `rows` places per CTA ----
    const int row_vecs = kv_row_bytes(CODE, a.head_dim) / 16, pools = a.pool[1] ? 2 : 1, vecs = row_vecs * pools;  // (powers of two)
    const int at_once = kThreads / vecs, rows = min(kThreads, at_once * kInFlight);
    const int vec = tid % vecs, w = vec / row_vecs, part = vec % row_vecs;
    auto where = [&](int p, int j) {
      return static_cast<char*>(a.pool[w]) + p * a.stride[w][0] + h * a.stride[w][1] + (j & page_mask) * a.stride[w][2] + part * 16;
    };
    // (a row of a page that is none of the pool's is not written)
    auto token = [&](int64_t i) { return min(max(__ldcg(kept + i), 0), n - 1); };  // (in bounds, as above)
    auto writable = [&](int j) { return (unsigned)row[j >> a.page_log2] < (unsigned)a.n_pages; };
#pragma unroll 1
    for (int64_t i0 = (int64_t)rank * rows; i0 - (int64_t)rank * rows < a.keep; i0 += (int64_t)C * rows) {
      const int n_rows = (int)max((int64_t)0, min((int64_t)rows, a.keep - i0));
      uint4 x[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int i = tid / vecs + u * at_once;
        if (i < n_rows) {
          const int j = token(i0 + i);
          x[u] = __ldcg(reinterpret_cast<const uint4*>(where(page_of(j), j)));
        }
      }
      float weight = 0.f, scale[2] = {0.f, 0.f};
      uint2 blocks[2] = {};
      if (tid < n_rows) {
        const int j = token(i0 + tid);
        const int64_t page_head = (int64_t)page_of(j) * a.kv_heads + h;
        const int pos = j & page_mask;
        weight = __ldcg(a.weight + (page_head << a.page_log2) + pos);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          if (CODE == kKv16 || v >= pools) continue;
          if (CODE == kKv8) scale[v] = __ldcg(static_cast<const float*>(a.scale[v]) + (page_head << a.page_log2) + pos);
          if (CODE == kKv4) {
            const uint8_t* const record = kv4_record(a.scale[v], page_head, a.page_log2, a.head_dim);
            scale[v] = __ldcg(reinterpret_cast<const float*>(record) + pos);
            const uint8_t* const from = record + (4 << a.page_log2) + pos * (a.head_dim >> 4);
            if (a.head_dim == 128) blocks[v] = __ldcg(reinterpret_cast<const uint2*>(from));
            else if (a.head_dim == 64) blocks[v].x = __ldcg(reinterpret_cast<const uint32_t*>(from));
            else blocks[v].x = __ldcg(reinterpret_cast<const uint16_t*>(from));
          }
        }
      }
      meet(C);
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int i = tid / vecs + u * at_once;
        if (i < n_rows) {
          const int to = (int)i0 + i;
          if (writable(to)) *reinterpret_cast<uint4*>(where(page_of(to), to)) = x[u];
        }
      }
      if (tid < n_rows && writable((int)i0 + tid)) {
        const int to = (int)i0 + tid;
        const int64_t page_head = (int64_t)page_of(to) * a.kv_heads + h;
        const int pos = to & page_mask;
        a.weight[(page_head << a.page_log2) + pos] = weight;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          if (CODE == kKv16 || v >= pools) continue;
          if (CODE == kKv8) static_cast<float*>(a.scale[v])[(page_head << a.page_log2) + pos] = scale[v];
          if (CODE == kKv4) {
            uint8_t* const record = kv4_record(a.scale[v], page_head, a.page_log2, a.head_dim);
            reinterpret_cast<float*>(record)[pos] = scale[v];
            uint8_t* const to_blocks = record + (4 << a.page_log2) + pos * (a.head_dim >> 4);
            if (a.head_dim == 128) *reinterpret_cast<uint2*>(to_blocks) = blocks[v];
            else if (a.head_dim == 64) *reinterpret_cast<uint32_t*>(to_blocks) = blocks[v].x;
            else *reinterpret_cast<uint16_t*>(to_blocks) = (uint16_t)blocks[v].x;
          }
        }
      }
    }
    meet(C);  // (a CTA's shared memory is read by others until here)
  }
  if (bad) atomicOr(a.err, bad);
}

template <int CODE>
cudaError_t launch(const KvEvictArgs& a, int num_sms, cudaStream_t s) {
  const int n_release = a.n_req > 0 ? (a.n_req + kThreads - 1) / kThreads : 1;
  const int64_t pairs = (int64_t)a.n_req * a.kv_heads, most = (int64_t)a.max_pages << a.page_log2;
  // as many CTAs per (request, head) as the SMs hold, of 1024 tokens at least
  int ctas = 1;
  while (ctas < kMaxCluster && pairs * ctas * 2 <= num_sms * 2 && most / (ctas * 2) >= 1024) ctas *= 2;
  const int64_t items = n_release + pairs, clusters = items < 65536 ? items : 65536;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(clusters * ctas));
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = sizeof(Shared);
  lc.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 2;
  cudaError_t e = cudaFuncSetAttribute(evict_kernel<CODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
  return e != cudaSuccess ? e : cudaLaunchKernelEx(&lc, evict_kernel<CODE>, a, n_release);
}

}  // namespace

cudaError_t launch_kv_evict(const KvEvictArgs& a, int code, int num_sms, cudaStream_t s) {
  return code == kKv16 ? launch<kKv16>(a, num_sms, s) : code == kKv8 ? launch<kKv8>(a, num_sms, s) : launch<kKv4>(a, num_sms, s);
}

}  // namespace cvr
