// Attention weights of one query token per request, added up per cached token and kv head (cvr_kv_weigh of include/cvr.h):
//   weight[j] = decay weight[j] + sum_i exp(scale q_i . k_j - lse_i)  over the query heads i of the kv head.
// The softmax's denominators are known (lse), so no token depends on another: every K row is read once, nothing is joined, and each
// weight has one writer. The floor is the bytes of the K rows and of the weights, in and out.
//
// Work: blocks of 16 tokens of a (request, kv head). The blocks of all requests form one line (request, then head, then
// position), which the warps of a persistent grid cut into equal runs, so ragged lengths load the SMs alike. A warp computes S =
// K Q^T on mma.sync m16n8k16 with the tokens on M and 8 query heads on N: a row's sum over the heads is then a sum of two
// accumulators and two shuffles, and up to 8 heads nothing is padded but the heads themselves. K goes from global memory straight
// into the fragments: the products' k index is permuted so that a thread's values of a row are 16 consecutive bytes, and the next
// block's loads are in flight while this one is computed.
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
  // the first of this thread's 4 values of k-step ks
  static __device__ __forceinline__ int dim(int ks, int tig) { return ks * 4 / kRun * 4 * kRun + tig * kRun + ks * 4 % kRun; }
};

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

// TILES: head tiles held in registers (1 or 2), or 0: any number, in shared memory
template <typename T, int CODE, int D, int TILES>
__global__ void __launch_bounds__(kThreads, 2) weigh_kernel(const __grid_constant__ KvWeighArgs a) {
  typedef Rows<CODE, D> R;
  constexpr bool SCALED = CODE != kKv16;
  typedef typename std::conditional<SCALED, __half, T>::type M;  // operand type of the products
  constexpr int KS = D / 16, kHeld = TILES ? TILES : 1;
  extern __shared__ uint32_t s_q[];  // TILES = 0: per warp [tile][ks][2][lane] fragments, then [tile * 8] factors and lse
  __shared__ int64_t s_before[kThreads + 1], s_sums[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int H = a.kv_heads, G = a.group, page_mask = (1 << a.page_log2) - 1;
  const int n_tiles = TILES ? TILES : (G + 7) / 8;
  uint32_t* const my_q = s_q + warp * n_tiles * (KS * 64 + 16);
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

      // a block's rows as loaded: tokens gid and gid + 8
      struct Block {
        uint32_t w[2][R::kWords];
        float scale[2], old;
        uint32_t block_scale[2];
        int page[2];
      };
      auto load = [&](Block& x, int b) {
        const int j0 = (t0 + b) * 16;
        if ((j0 + 15) >> a.page_log2 >= e0 + 32) {  // (a block of two pages never straddles: 32 entries begin at an even one)
          ids = more_ids;
          e0 += 32;
          more_ids = entries(e0 + 32);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j = j0 + gid + 8 * u;
          int page = __shfl_sync(0xffffffffu, ids, ((j >> a.page_log2) - e0) & 31);
          if (j >= len) page = -1;
          else if ((unsigned)page >= (unsigned)a.n_pages) {
            bad |= kKvErrPage;
            page = -1;
          }
          x.page[u] = page;
          const int pos = j & page_mask;
          const int64_t from = page * a.k_stride[0] + h * a.k_stride[1] + pos * a.k_stride[2];
          const char* p = static_cast<const char*>(a.k) + (CODE == kKv16 ? from * 2 : CODE == kKv8 ? from : from >> 1) + tig * (R::kLoad * 4);
#pragma unroll
          for (int c = 0; c < R::kWords / R::kLoad; ++c) {
            uint32_t* d = x.w[u] + c * R::kLoad;
            if (R::kLoad == 4) {
              uint4 v = make_uint4(0, 0, 0, 0);
              if (page >= 0) v = *reinterpret_cast<const uint4*>(p + c * 64);
              d[0] = v.x;
              d[1 % R::kLoad] = v.y;
              d[2 % R::kLoad] = v.z;
              d[3 % R::kLoad] = v.w;
            } else if (R::kLoad == 2) {
              uint2 v = make_uint2(0, 0);
              if (page >= 0) v = *reinterpret_cast<const uint2*>(p);
              d[0] = v.x;
              d[1 % R::kLoad] = v.y;
            } else {
              d[0] = page >= 0 ? *reinterpret_cast<const uint32_t*>(p) : 0u;
            }
          }
          const int64_t page_head = (int64_t)page * H + h;
          if (CODE == kKv8) x.scale[u] = page >= 0 ? static_cast<const float*>(a.k_scale)[(page_head << a.page_log2) + pos] : 0.f;
          if (CODE == kKv4) {
            const uint8_t* record = kv4_record(a.k_scale, page_head, a.page_log2, D);
            const uint8_t* blocks = record + (4 << a.page_log2) + pos * (D / 16);
            x.scale[u] = page >= 0 ? reinterpret_cast<const float*>(record)[pos] : 0.f;
            x.block_scale[u] = page < 0 ? 0u : D == 128 ? reinterpret_cast<const uint16_t*>(blocks)[tig] : D == 64 ? blocks[tig] : blocks[tig >> 1];
          }
        }
        // threads 0 and 1 of a row's four keep the weights of tokens gid and gid + 8
        const int j = j0 + gid + 8 * (tig & 1), page = tig & 1 ? x.page[1] : x.page[0];
        x.old = tig < 2 && page >= 0 && j < old_end ? a.weight[(((int64_t)page * H + h) << a.page_log2) + (j & page_mask)] : 0.f;
      };
      Block now, next;
      load(now, 0);

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

      auto compute = [&](const Block& x, int b) {
        uint32_t sc[2][2] = {};  // 4 bits: the block scales of the thread's words, of tokens gid and gid + 8, as pairs
        if (CODE == kKv4)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            sc[u][0] = e4m3_f16x2(__byte_perm(x.block_scale[u], 0, 0x00));
            sc[u][1] = D == 128 ? e4m3_f16x2(__byte_perm(x.block_scale[u], 0, 0x11)) : sc[u][0];
          }
        auto fragment = [&](int ks, uint32_t* k) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (CODE == kKv16) {
              k[u] = x.w[u][(2 * ks) % R::kWords];
              k[2 + u] = x.w[u][(2 * ks + 1) % R::kWords];
            } else if (CODE == kKv8) {
              const uint32_t v = x.w[u][ks % R::kWords] ^ 0x80808080u;
              k[u] = i8_pair<0x4140>(v);
              k[2 + u] = i8_pair<0x4342>(v);
            } else {
              const uint32_t v = x.w[u][ks / 2 % R::kWords], s = sc[u][ks / 2 * 2 / R::kWords % 2];
              k[u] = mul2<M>(ks & 1 ? e2m1_f16x2<2>(v) : e2m1_f16x2<0>(v), s);
              k[2 + u] = mul2<M>(ks & 1 ? e2m1_f16x2<3>(v) : e2m1_f16x2<1>(v), s);
            }
          }
        };
        const float sA = SCALED ? x.scale[0] : 1.f, sB = SCALED ? x.scale[1] : 1.f;
        float sumA = 0.f, sumB = 0.f;
        auto add = [&](const float* s, int tile, float c0, float c1, float l0, float l1) {
          auto weight = [&](float s, float scale, float c, float l, int head) {
            const float p = ex2(fmaf(SCALED ? s * scale : s, c, -l) * kLog2e);
            return head < G ? p : 0.f;
          };
          const int head = tile * 8 + 2 * tig;
          sumA += weight(s[0], sA, c0, l0, head) + weight(s[1], sA, c1, l1, head + 1);
          sumB += weight(s[2], sB, c0, l0, head) + weight(s[3], sB, c1, l1, head + 1);
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
        const int j = (t0 + b) * 16 + gid + 8 * (tig & 1), page = tig & 1 ? x.page[1] : x.page[0];
        if (tig < 2 && page >= 0) {
          // (the old weight of a token that has none, or of no decay, was not read)
          const float sum = tig & 1 ? sumB : sumA;
          a.weight[(((int64_t)page * H + h) << a.page_log2) + (j & page_mask)] = j < old_end ? fmaf(a.decay, x.old, sum) : sum;
        }
      };
#pragma unroll 1
      for (int b = 0; b < count; b += 2) {
        if (b + 1 < count) load(next, b + 1);
        compute(now, b);
        if (b + 1 == count) break;
        if (b + 2 < count) load(now, b + 2);
        compute(next, b + 1);
      }
    }
  }
  if (bad) atomicOr(a.err, bad);
}

template <typename T, int CODE, int D>
cudaError_t launch(const KvWeighArgs& a, int num_sms, cudaStream_t s) {
  const int tiles = (a.group + 7) / 8;
  const int64_t blocks = (((int64_t)a.max_pages << a.page_log2) + 15) / 16 * a.n_req * a.kv_heads;  // at most
  const int64_t want = (blocks + kWarps - 1) / kWarps, fit = (int64_t)num_sms * 2;
  const dim3 grid((unsigned)(want < fit ? want : fit)), block(kThreads);
  if (tiles == 1) return launch_kernel(weigh_kernel<T, CODE, D, 1>, grid, block, 0, s, true, a);
  if (tiles == 2) return launch_kernel(weigh_kernel<T, CODE, D, 2>, grid, block, 0, s, true, a);
  const int smem = kWarps * tiles * (D / 16 * 64 + 16) * 4;
  const cudaError_t e = cudaFuncSetAttribute(weigh_kernel<T, CODE, D, 0>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return e != cudaSuccess ? e : launch_kernel(weigh_kernel<T, CODE, D, 0>, grid, block, smem, s, true, a);
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
