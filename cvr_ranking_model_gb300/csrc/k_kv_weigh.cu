// Attention weights of one query token per request, added up per cached token and kv head (cvr_kv_weigh of include/cvr.h):
//   weight[j] = decay weight[j] + sum_i exp(scale q_i . k_j - lse_i)  over the query heads i of the kv head.
// The softmax's denominators are known (lse), so no token depends on another: every K row is read once, nothing is joined, and each
// weight has one writer. The floor is the bytes of the K rows and of the weights, in and out.
//
// Work: blocks of 16 tokens of a (request, kv head). The blocks of all requests form one line (request, then head, then
// position), which the warps of a persistent grid cut into equal runs, so ragged lengths load the SMs alike. A warp computes S =
// K Q^T on mma.sync m16n8k16 with the tokens on M and 8 query heads on N: a row's sum over the heads is then a sum of two
// accumulators and two shuffles, and up to 8 heads nothing is padded but the heads themselves. The products' k index is permuted so
// that a thread's values of a row are 16 consecutive bytes: every thread copies what it will use to shared memory, asynchronously and
// some blocks ahead, and reads it back itself, so no warp waits for another and no registers hold what is in flight.
//
// Measured (one GB300, copy rate 6.78 TB/s): 64 requests of up to 8191 tokens, 32 / 8 heads of 128, bf16: 65.4 us, 85% of the copy rate;
// straight into registers 77.6 us (two CTAs per SM, the next block's loads in flight). 32 requests of up to 16383 on 4 bits, 64 / 8 heads:
// 42.8 us, 43%: 328 warp instructions per block of 16 tokens, issued 68% of the time; 64 of them convert and scale codes, the others are
// the copies' addresses and predicates, logits, exponents and sums. The first requests on 8 bits 44.8 us, 66%. 16 query heads per kv head
// 74 us on bf16. More are far from their bytes (24: 110 us on bf16; 64: 220, and 206 on 4 bits where 8 take 42.8): their query fragments
// leave an SM one CTA, two warps per scheduler, which cannot cover a head tile's one chain of products (issue 44%), and the grid, of
// two CTAs per SM, runs in two waves.
#include "../../include/cvr.h"
#include "cvr_kv_rows.cuh"

namespace cvr {
namespace {

using namespace kv;

constexpr int kWarps = 8, kThreads = kWarps * 32;

template <int CODE, int D>
struct Rows {
  static constexpr int kWords = kv_row_bytes(CODE, D) / 16;             // 32-bit words of a row per thread (4 threads a row)
  static constexpr int kLoad = kWords < 4 ? kWords : 4;                 // words of one load
  static constexpr int kRun = kLoad * 4 * D / kv_row_bytes(CODE, D);    // values of one load
  // a warp's ring of blocks in shared memory: per block and thread its words of rows gid and gid + 8, the rows' scales and block
  // scales, the old weight and where the new one goes
  static constexpr int kStages = kWords >= 16 ? 2 : kWords == 8 ? 3 : 4, kScaled = CODE == kKv16 ? 0 : CODE == kKv8 ? 2 : 4;
  static constexpr int oScale = kWords * 2 * 128, oOld = oScale + kScaled * 128, oWeight = oOld + 128, kStage = oWeight + 256;
  static constexpr int kWarpBytes = kStages * kStage;
  // the first of this thread's 4 values of k-step ks
  static __device__ __forceinline__ int dim(int ks, int tig) { return ks * 4 / kRun * 4 * kRun + tig * kRun + ks * 4 % kRun; }
};

// BYTES copied to shared memory asynchronously
template <int BYTES>
__device__ __forceinline__ void copy(void* dst, const void* src) {
  if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}

// the smaller, NaN if either is
__device__ __forceinline__ float min_or_nan(float x, float y) {
  float z;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}

__device__ __forceinline__ int64_t scan_before(int64_t x, int64_t* sums, int64_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += u;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int64_t before = incl - x, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  *all = total;
  return before;
}

// CTAs that share an SM by their registers (two head tiles of rows of 128, or many, need more); with many, shared memory may hold fewer
constexpr int ctas_per_sm(int dim, int tiles) { return tiles == 1 || dim < 128 ? 3 : 2; }

// TILES: head tiles held in registers (1 or 2), or 0: any number, in shared memory
template <typename T, int CODE, int D, int TILES>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, TILES)) weigh_kernel(const __grid_constant__ KvWeighArgs a) {
  typedef Rows<CODE, D> R;
  constexpr bool SCALED = CODE != kKv16;
  typedef typename std::conditional<SCALED, __half, T>::type M;  // operand type of the products
  constexpr int KS = D / 16, kHeld = TILES ? TILES : 1;
  // the warps' rings, then (TILES = 0) per warp [tile][ks][lane][2] fragments, [tile * 8] factors and lse
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_before[kThreads + 1], s_sums[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int H = a.kv_heads, G = a.group, page_mask = (1 << a.page_log2) - 1;
  const int n_tiles = TILES ? TILES : (G + 7) / 8;
  uint8_t* const my_ring = smem + warp * R::kWarpBytes;
  uint32_t* const my_q = reinterpret_cast<uint32_t*>(smem + kWarps * R::kWarpBytes) + warp * n_tiles * (KS * 64 + 16);
  float* const my_c = reinterpret_cast<float*>(my_q + n_tiles * KS * 64);
  float* const my_l = my_c + n_tiles * 8;
  pdl_trigger();
  pdl_wait();  // (what an earlier call of the stream wrote is read with plain loads)

  // ---- the line of blocks: every thread sums a few requests ----
  auto length = [&](int r) {
    const int len = a.lens[r];
    return len < 0 ? 0 : min(len, a.max_pages << a.page_log2);  // (at most 2^30)
  };
  auto blocks_of = [](int len) { return (len + 15) >> 4; };
  const int few = (a.n_req + kThreads - 1) / kThreads;
  int64_t mine = 0, all = 0;
  int bad = 0;
  for (int r = min(tid * few, a.n_req); r < min((tid + 1) * few, a.n_req); ++r) {
    const int len = length(r);
    if (len != a.lens[r]) bad = kKvErrLens;
    if (a.new_lens && (a.new_lens[r] < 0 || a.new_lens[r] > len)) bad = kKvErrLens;
    mine += blocks_of(len);
  }
  s_before[tid] = scan_before(mine, s_sums, &all);
  if (tid == 0) s_before[kThreads] = all;
  __syncthreads();
  if (blockIdx.x != 0) bad = 0;
  const int64_t total = all * H, warps = (int64_t)gridDim.x * kWarps, per = (total + warps - 1) / warps;
  // (a CTA's warps take neighbouring runs)
  const int64_t begin = min(((int64_t)blockIdx.x * kWarps + warp) * per, total), end = min(begin + per, total);
  if (begin < end) {
    // the requests of the thread whose share holds `begin`, 32 at a time, one per lane
    int t = 0;
    for (int step = kThreads / 2; step > 0; step >>= 1)
      if (s_before[t + step] * H <= begin) t += step;
    int wb = t * few, wl = 0;
    uint32_t w_incl = 0;                   // the window's first request; its lane's length and sum of blocks up to it
    int64_t base = s_before[t];            // blocks per head before the window
    auto window = [&]() {
      wl = wb + lane < a.n_req ? length(wb + lane) : 0;
      w_incl = blocks_of(wl);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, w_incl, d);
        if (lane >= d) w_incl += u;  // (at most 32 requests of 2^26 blocks)
      }
    };
    int64_t at = begin;
    window();
    while (at < end) {
      // ---- a segment: the blocks of one (request, head) in this run ----
      unsigned has;
      while (true) {
        has = __ballot_sync(0xffffffffu, at < (base + w_incl) * H);
        if (has) break;
        base += __shfl_sync(0xffffffffu, w_incl, 31);
        wb += 32;
        window();
      }
      const int f = __ffs(has) - 1, r = wb + f, len = __shfl_sync(0xffffffffu, wl, f), n = blocks_of(len);
      const int64_t in = at - (base + __shfl_sync(0xffffffffu, w_incl, f) - n) * H;  // (below 2^34)
      const int h = (int)(in / n), t0 = (int)(in - (int64_t)h * n), count = (int)min((int64_t)(n - t0), end - at);
      at += count;
      const int n_new = a.new_lens ? min(max(a.new_lens[r], 0), len) : 1, old_end = a.decay == 0.f ? 0 : len - n_new;

      // page ids of the request's table row, 32 entries at a time, the next 32 ahead of use
      const int32_t* const row = a.table + (int64_t)r * a.max_pages;
      int e0 = (t0 * 16) >> a.page_log2;
      auto entries = [&](int e) { return e + lane < a.max_pages ? row[e + lane] : 0; };
      int ids = entries(e0), more_ids = entries(e0 + 32);

      // what does not depend on the page: this head's, this thread's
      const char* const k_head = static_cast<const char*>(a.k) + h * a.k_stride[1] + gid * a.k_stride[2] + tig * (R::kLoad * 4);
      const uint32_t page_places = (uint32_t)H << a.page_log2;  // rows of a page
      float* const weight_head = a.weight + ((uint32_t)h << a.page_log2) + gid;
      const uint32_t record_bytes = (uint32_t)kv_scale_bytes(CODE, D) << a.page_log2;
      const uint8_t* const scale_head = static_cast<const uint8_t*>(a.k_scale) + (SCALED ? h * record_bytes + gid * 4 : 0);
      // (4 bytes of the row's block scales, this thread's among them)
      const int blocks_at = (4 << a.page_log2) + gid * (D / 16 - 4) + (D == 128 ? tig & 2 ? 4 : 0 : 0);
      auto fetch = [&](int b) {
        if (b < count) {
          const int j0 = (t0 + b) * 16;
          if ((j0 + 15) >> a.page_log2 >= e0 + 32) {  // (a block of two pages never straddles: 32 entries begin at an even one)
            ids = more_ids;
            e0 += 32;
            more_ids = entries(e0 + 32);
          }
          uint8_t* const slot = my_ring + (b % R::kStages) * R::kStage;
          const int e = (j0 >> a.page_log2) - e0, pos = j0 & page_mask;
          const uint32_t p0 = __shfl_sync(0xffffffffu, ids, e);
          const bool small = a.page_log2 == 3;  // (8 tokens a page: the block has two)
          const uint32_t p1 = small ? __shfl_sync(0xffffffffu, ids, e + 1) : p0;
          const bool ok0 = p0 < (uint32_t)a.n_pages, ok1 = p1 < (uint32_t)a.n_pages;
          const uint32_t from0 = ok0 ? p0 : 0, from1 = ok1 ? p1 : 0;
          const char* const row0 = k_head + from0 * a.k_stride[0] + pos * a.k_stride[2];
          const char* const row1 = small ? k_head + from1 * a.k_stride[0] : row0 + 8 * a.k_stride[2];
          const uint8_t* const record0 = scale_head + (SCALED ? (uint64_t)from0 * (H * record_bytes) + pos * 4 : 0);
          const uint8_t* const record1 = small ? scale_head + (SCALED ? (uint64_t)from1 * (H * record_bytes) : 0) : record0 + 32;
          const uint8_t* const blocks0 = record0 + blocks_at + pos * (D / 16 - 4);
          const uint8_t* const blocks1 = small ? record1 + blocks_at : blocks0 + D / 2;
          // threads 0 and 1 of a row's four keep the weights of tokens gid and gid + 8
          float* const at = weight_head + (uint64_t)(tig ? from1 : from0) * page_places + (small ? 0 : pos + 8 * (tig & 1));
          auto bring = [&](auto all) {
            // (of tokens behind the history, and of a page that is none of the pool's, nothing is read: the products' rows do not mix, and
            // theirs go nowhere)
            constexpr bool ALL = decltype(all)::value;
            const bool there0 = ALL || (j0 + gid < len && ok0), there1 = ALL || (j0 + gid + 8 < len && ok1);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              if (!(u ? there1 : there0)) continue;
#pragma unroll
              for (int c = 0; c < R::kWords / R::kLoad; ++c)
                copy<R::kLoad * 4>(slot + (u * R::kWords / R::kLoad + c) * (R::kLoad * 128) + lane * (R::kLoad * 4), (u ? row1 : row0) + c * 64);
              if (SCALED) copy<4>(slot + R::oScale + u * 128 + lane * 4, u ? record1 : record0);
              if (CODE == kKv4) {
                const uint8_t* const blocks = u ? blocks1 : blocks0;
                copy<4>(slot + R::oScale + (2 + u) * 128 + lane * 4, D == 32 ? (const uint8_t*)((uintptr_t)blocks & ~(uintptr_t)3) : blocks);
              }
            }
            const bool there = tig == 0 ? there0 : tig == 1 && there1;
            *reinterpret_cast<float**>(slot + R::oWeight + lane * 8) = there ? at : nullptr;
            if (there && j0 + gid + 8 * (tig & 1) < old_end) copy<4>(slot + R::oOld + lane * 4, at);
          };
          if (j0 + 16 <= len && ok0 && ok1) {
            bring(std::true_type());
          } else {
            bad |= (j0 < len && !ok0) || (j0 + 8 < len && !ok1) ? kKvErrPage : 0;
            bring(std::false_type());
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
      for (int b = 0; b < R::kStages - 1; ++b) fetch(b);

      // ---- the query rows: fragments, and per head the logits' factor and lse ----
      // As in the attention: q times the scale's sign, -1, 0 or 1; bf16 rows times a power of two, which goes into the factor (on 16-bit
      // pools those whose largest value is 2^16 or more, on others all: fp16 operands are relative to the row's largest value).
      const float sign = a.scale > 0.f ? 1.f : a.scale < 0.f ? -1.f : 0.f;
      uint32_t qf[kHeld][KS][2];
      float c0[kHeld], c1[kHeld], l0[kHeld], l1[kHeld];
      auto query = [&](int tile, uint32_t (*f)[2], float& factor, float& lse) {  // of head tile * 8 + gid
        const int head = tile * 8 + gid;
        const bool in = head < G;
        const T* q = static_cast<const T*>(a.q) + r * a.q_stride + ((int64_t)h * G + (in ? head : 0)) * D;
        uint2 x[KS];
        float big = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          x[ks] = in ? *reinterpret_cast<const uint2*>(q + R::dim(ks, tig)) : make_uint2(0, 0);
          const float2 u = unpack2<T>(x[ks].x), v = unpack2<T>(x[ks].y);
          big = fmaxf(fmaxf(big, fmaxf(fabsf(u.x), fabsf(u.y))), fmaxf(fabsf(v.x), fabsf(v.y)));
        }
        lse = in ? a.lse[((int64_t)r * H + h) * G + head] : 0.f;
        float up = sign;
        factor = fabsf(a.scale);
        if (std::is_same<T, __nv_bfloat16>::value) {
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          const uint32_t e = __float_as_uint(big) >> 23;
          const uint32_t to = SCALED ? min(max(e, 1u), 253u) : min(max(e, 142u), 254u) - 15;
          up *= __uint_as_float((254u - to) << 23);
          factor *= __uint_as_float(to << 23);
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const float2 u = unpack2<T>(x[ks].x), v = unpack2<T>(x[ks].y);
          f[ks][0] = pack2<M>(u.x * up, u.y * up);
          f[ks][1] = pack2<M>(v.x * up, v.y * up);
        }
      };
      if (TILES == 0) {
        __syncwarp();  // (the segment before has been computed)
        for (int tile = 0; tile < n_tiles; ++tile) {
          float factor, lse;
          query(tile, qf[0], factor, lse);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
            reinterpret_cast<uint2*>(my_q)[(tile * KS + ks) * 32 + lane] = make_uint2(qf[0][ks][0], qf[0][ks][1]);
          if (tig == 0) {
            my_c[tile * 8 + gid] = factor;
            my_l[tile * 8 + gid] = lse;
          }
        }
        __syncwarp();
      } else {
#pragma unroll
        for (int tile = 0; tile < kHeld; ++tile) {
          float factor, lse;
          query(tile, qf[tile], factor, lse);
          // (the accumulators' columns are heads 2 tig and 2 tig + 1)
          c0[tile] = __shfl_sync(0xffffffffu, factor, tig * 8);
          c1[tile] = __shfl_sync(0xffffffffu, factor, tig * 8 + 4);
          l0[tile] = __shfl_sync(0xffffffffu, lse, tig * 8);
          l1[tile] = __shfl_sync(0xffffffffu, lse, tig * 8 + 4);
        }
      }

      auto compute = [&](int b) {
        const uint8_t* const slot = my_ring + (b % R::kStages) * R::kStage;
        const int row0 = (t0 + b) * 16 + gid;
        uint32_t sc[2][2] = {};  // 4 bits: the block scales of the thread's words, of tokens gid and gid + 8, as pairs
        if (CODE == kKv4)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x = *reinterpret_cast<const uint32_t*>(slot + R::oScale + (2 + u) * 128 + lane * 4);
            // rows of 128: bytes 2 (tig mod 2) and the next; of 64: tig; of 32: the row's two of the four, tig / 2
            const uint32_t first = D == 128 ? (tig & 1) * 2 : D == 64 ? tig : (row0 & 1) * 2 + (tig >> 1);
            sc[u][0] = e4m3_f16x2(__byte_perm(x, 0, first * 0x11));
            sc[u][1] = D == 128 ? e4m3_f16x2(__byte_perm(x, 0, first * 0x11 + 0x11)) : sc[u][0];
          }
        uint32_t words[2][R::kLoad];
        auto bring = [&](int c) {  // the thread's words of load c of both rows
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint8_t* from = slot + (u * R::kWords / R::kLoad + c) * (R::kLoad * 128) + lane * (R::kLoad * 4);
            if (R::kLoad == 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(from);
              words[u][0] = v.x;
              words[u][1 % R::kLoad] = v.y;
              words[u][2 % R::kLoad] = v.z;
              words[u][3 % R::kLoad] = v.w;
            } else if (R::kLoad == 2) {
              const uint2 v = *reinterpret_cast<const uint2*>(from);
              words[u][0] = v.x;
              words[u][1 % R::kLoad] = v.y;
            } else {
              words[u][0] = *reinterpret_cast<const uint32_t*>(from);
            }
          }
        };
        // k-steps of a word: half a one on 16-bit pools, one on 8-bit pools, two on 4-bit pools
        auto fragment = [&](int ks, uint32_t* k) {
          const int word = CODE == kKv16 ? 2 * ks : CODE == kKv8 ? ks : ks / 2;
          if (word % R::kLoad == 0 && (CODE != kKv4 || ks % 2 == 0)) bring(word / R::kLoad);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x = words[u][word % R::kLoad];
            if (CODE == kKv16) {
              k[u] = x;
              k[2 + u] = words[u][(word + 1) % R::kLoad];
            } else if (CODE == kKv8) {
              const uint32_t v = x ^ 0x80808080u;
              k[u] = i8_pair<0x4140>(v);
              k[2 + u] = i8_pair<0x4342>(v);
            } else {
              const uint32_t scale = sc[u][word * 2 / R::kWords % 2];
              k[u] = mul2<M>(ks & 1 ? e2m1_f16x2<2>(x) : e2m1_f16x2<0>(x), scale);
              k[2 + u] = mul2<M>(ks & 1 ? e2m1_f16x2<3>(x) : e2m1_f16x2<1>(x), scale);
            }
          }
        };
        const float sA = SCALED ? *reinterpret_cast<const float*>(slot + R::oScale + lane * 4) : 1.f;
        const float sB = SCALED ? *reinterpret_cast<const float*>(slot + R::oScale + 128 + lane * 4) : 1.f;
        // A finite logit above lse is so by the rounding of both and counts as lse: of logits about 2^24 that rounding is a factor of e, and a
        // weight that it made infinite would never fade. (A row of an infinity gives no head a finite product, so one head's shows it.)
        float sumA = 0.f, sumB = 0.f, mostA = 0.f, mostB = 0.f;
        auto add = [&](const float* s, int tile, float c0, float c1, float l0, float l1) {
          // (a head that there is none of weighs nothing, also where its 0 times an infinity of a row is no number)
          const bool in0 = tile * 8 + 2 * tig < G, in1 = tile * 8 + 2 * tig + 1 < G;
          const float x[4] = {SCALED ? s[0] * sA : s[0], SCALED ? s[1] * sA : s[1], SCALED ? s[2] * sB : s[2], SCALED ? s[3] * sB : s[3]};
          if (tile == 0) {
            mostA = fabsf(x[0]) < INFINITY ? 0.f : INFINITY;
            mostB = fabsf(x[2]) < INFINITY ? 0.f : INFINITY;
          }
          auto weight = [&](float x, float most, float c, float l, bool in) {
            const float p = ex2(min_or_nan(fmaf(x, c, -l) * kLog2e, most));
            return in ? p : 0.f;
          };
          sumA += weight(x[0], mostA, c0, l0, in0) + weight(x[1], mostA, c1, l1, in1);
          sumB += weight(x[2], mostB, c0, l0, in0) + weight(x[3], mostB, c1, l1, in1);
        };
        if (TILES == 0) {
          uint32_t k[KS][4];
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) fragment(ks, k[ks]);
#pragma unroll 1
          for (int tile = 0; tile < n_tiles; ++tile) {
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              const uint2 q = reinterpret_cast<const uint2*>(my_q)[(tile * KS + ks) * 32 + lane];
              mma16816<M>(s, k[ks], q.x, q.y);
            }
            const float2 c = *reinterpret_cast<const float2*>(my_c + tile * 8 + 2 * tig), l = *reinterpret_cast<const float2*>(my_l + tile * 8 + 2 * tig);
            add(s, tile, c.x, c.y, l.x, l.y);
          }
        } else {
          float s[kHeld][4];
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t k[4];
            fragment(ks, k);
#pragma unroll
            for (int tile = 0; tile < kHeld; ++tile) {
              if (ks == 0) mma16816<M, true>(s[tile], k, qf[tile][ks][0], qf[tile][ks][1]);
              else mma16816<M>(s[tile], k, qf[tile][ks][0], qf[tile][ks][1]);
            }
          }
#pragma unroll
          for (int tile = 0; tile < kHeld; ++tile) add(s[tile], tile, c0[tile], c1[tile], l0[tile], l1[tile]);
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          sumA += __shfl_xor_sync(0xffffffffu, sumA, d);
          sumB += __shfl_xor_sync(0xffffffffu, sumB, d);
        }
        float* const weight = *reinterpret_cast<float* const*>(slot + R::oWeight + lane * 8);
        if (weight) {
          // (the old weight of a token that has none, or of no decay, was not read)
          const float sum = tig & 1 ? sumB : sumA, old = *reinterpret_cast<const float*>(slot + R::oOld + lane * 4);
          *weight = row0 + 8 * (tig & 1) < old_end ? fmaf(a.decay, old, sum) : sum;
        }
      };
#pragma unroll 1
      for (int b = 0; b < count; ++b) {
        fetch(b + R::kStages - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(R::kStages - 1) : "memory");
        compute(b);
      }
    }
  }
  if (bad) atomicOr(a.err, bad);
}

template <typename T, int CODE, int D>
cudaError_t launch(const KvWeighArgs& a, int num_sms, cudaStream_t s) {
  const int tiles = (a.group + 7) / 8;
  const int64_t blocks = (((int64_t)a.max_pages << a.page_log2) + 15) / 16 * a.n_req * a.kv_heads;  // at most
  const int64_t want = (blocks + kWarps - 1) / kWarps, fit = (int64_t)num_sms * ctas_per_sm(D, tiles > 2 ? 0 : tiles);
  const dim3 grid((unsigned)(want < fit ? want : fit)), block(kThreads);
  // (a kernel's limit of shared memory is the process's: always what its largest launch asks for, or a handle of fewer heads would lower
  // it between another thread's setting and launch)
  const auto smem_of = [](int tiles) { return kWarps * (Rows<CODE, D>::kWarpBytes + (tiles > 2 ? tiles * (D / 16 * 64 + 16) * 4 : 0)); };
  const int smem = smem_of(tiles), most = smem_of(tiles > 2 ? 64 / 8 : tiles);
  auto run = [&](auto kern) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return e != cudaSuccess ? e : launch_kernel(kern, grid, block, smem, s, true, a);
  };
  return tiles == 1 ? run(weigh_kernel<T, CODE, D, 1>) : tiles == 2 ? run(weigh_kernel<T, CODE, D, 2>) : run(weigh_kernel<T, CODE, D, 0>);
}

}  // namespace

cudaError_t launch_kv_weigh(const KvWeighArgs& a, int dtype, int code, int head_dim, int num_sms, cudaStream_t s) {
  auto of = [&](auto t, auto c) {
    typedef decltype(t) T;
    constexpr int CODE = decltype(c)::value;
    return head_dim == 32   ? launch<T, CODE, 32>(a, num_sms, s)
           : head_dim == 64 ? launch<T, CODE, 64>(a, num_sms, s)
                            : launch<T, CODE, 128>(a, num_sms, s);
  };
  auto by_code = [&](auto t) {
    return code == kKv16  ? of(t, std::integral_constant<int, kKv16>())
           : code == kKv8 ? of(t, std::integral_constant<int, kKv8>())
                          : of(t, std::integral_constant<int, kKv4>());
  };
  return dtype == CVR_DTYPE_BF16 ? by_code(__nv_bfloat16()) : by_code(__half());
}

}  // namespace cvr
