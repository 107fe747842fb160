// The consumer warps' part of the paged history attention on pools of 4 bits (k_kv_attn.cuh): logits, softmax and sums of a block of
// 16 tokens at a time, for 8 NT query heads.
//
// Here the tokens and the values lie on M and the heads on N of mma.sync m16n8k16: S^T = K Q^T (16 tokens x 8 heads) and O^T = V^T P^T (16
// values x 8 heads), so that up to 8 heads nothing is computed for padding rows, O takes half the registers that it takes with the heads
// on M, and three CTAs of rows of 128 share an SM: codes and their scales have to become fp16 first, which is what the instructions of
// a token are spent on, and more warps hide its latency. A word of 8 codes costs 4 conversions (cvt e2m1x2) and 4 products with the
// block's scale, exact in fp16 (2 and 4 bits); V's words a regrouping of nibbles besides, after which a byte holds one value of two
// neighbouring tokens, the pair that a fragment wants.
//   - S^T leaves the tensor cores with a token's heads side by side; as P^T it has to enter with a head's tokens side by side: movmatrix
//     transposes the packed weights.
//   - Weights, times V's row scale and a power of two, enter as two fp16 halves, as on 8-bit pools (there: the rule for that power).
//
// Measured (one GB300, copy rate 6.78 TB/s): 64 requests of up to 8191 tokens, 32 / 8 heads of 128: 70.8 us, 45% of the copy rate (pages
// of 16; 65.7 us with pages of 32 and more, whose rows take fewer copies), against 112.6 us on bf16 rows; one request of 131071: 48.5 us,
// 48%. 26 to 28 warp instructions per token and kv head, about 10 of them conversions, scaling and regrouping; no pipe is full: the
// schedulers issue half of the time, the ALU pipe is 48% busy, the tensor pipe 22 to 24%. 3.4 warps per scheduler do not cover what they
// wait for: of 6.7 warp cycles per instruction issued 2.0 are loads and barriers of tiles (1.3 of 6.3 on the long request), 1.2 the last
// instruction's own latency, 0.5 a busy pipe. With the heads on M (112.3 and 61.4 us) the sums
// took twice the registers and two CTAs shared an SM. 512 histories of up to 2000 events, 4 heads of 32, K = V: 46.4 us, 35.1 us on bf16
// rows: rows of 32 are mostly softmax, and 4 bits add conversions. One request of 200: 6.0 us, latency.
#pragma once

#include "cvr_kv_rows.cuh"

namespace cvr {
namespace kv {

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
// c (+)= a b like mma16816, free to move among the conversions
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x times the low or high half of y, on both halves
template <bool HIGH>
__device__ __forceinline__ uint32_t mul_half(uint32_t x, uint32_t y) {
  const __half2 s = *reinterpret_cast<const __half2*>(&y);
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), HIGH ? __high2half2(s) : __low2half2(s));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// What a consumer warp holds of 8 NT heads. Lane (gid, tig): of K^T's and V^T's fragments tokens or values gid and gid + 8, of results
// heads 2 tig and 2 tig + 1 of each 8. PER_LANE = 1: of at most 4 heads, which take every other column: softmax is per column and lane,
// used or not, and half of the columns are then left out.
template <typename T, int D, int NT, int PER_LANE>
struct Heads4 {
  static constexpr int kPieces = D / 32;  // 32 values: 16 bytes of a row
  static constexpr float kGrow = 6.f;     // weights are at most 2^kGrow
  static constexpr int kQBytes = NT * D / 16 * 256;  // a warp's query fragments in shared memory: [k-step][tile][lane], 8 bytes each
  uint2* qf;                                          // this lane's
  float o[NT][kPieces][2][4];  // values 32 g + 4 gid + (0, 1 | 2, 3) of columns (2 tig, 2 tig + 1)
  static constexpr int N = PER_LANE;
  float m[NT][N], l[NT][N], c[NT][N], mul[NT][N];
  uint32_t range;  // a V scale's bits plus this are at most 11 << 23 where it lies in [hi / 2^11, hi]

  // Query rows `q` (row_bytes apart, `rows` of them there) of up to 16 heads; scale: of the logits.
  __device__ __forceinline__ void begin(uint8_t* fragments, const uint8_t* q, int row_bytes, int rows, float scale) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    qf = reinterpret_cast<uint2*>(fragments) + lane;
    const float sign = scale > 0.f ? 1.f : scale < 0.f ? -1.f : 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int head = N == 2 ? t * 8 + gid : gid & 1 ? rows : gid >> 1;  // (of column gid)
      uint4 x[kPieces];
      uint32_t big = 0;
#pragma unroll
      for (int g = 0; g < kPieces; ++g) {
        x[g] = head < rows ? *reinterpret_cast<const uint4*>(q + head * row_bytes + g * 64 + tig * 16) : make_uint4(0, 0, 0, 0);
        big = __vmaxu2(big, __vmaxu2(__vmaxu2(x[g].x & 0x7fff7fffu, x[g].y & 0x7fff7fffu), __vmaxu2(x[g].z & 0x7fff7fffu, x[g].w & 0x7fff7fffu)));
      }
      float up = sign;
      uint32_t e = 127;
      if (std::is_same<T, __nv_bfloat16>::value) {
        // in fp16, the largest value brought to [1, 2): exact down to 2^-14 of it, 2^-25 of it below (both factors are normal)
        big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, 2));
        e = min(max(max(big >> 16, big & 0xffffu) >> 7, 1u), 253u);
        up *= __uint_as_float((254u - e) << 23);
      }
#pragma unroll
      for (int g = 0; g < kPieces; ++g) {
        auto pair = [&](uint32_t y) {
          const float2 f = unpack2<T>(y);
          return pack2<__half>(f.x * up, f.y * up);
        };
        qf[((2 * g) * NT + t) * 32] = make_uint2(pair(x[g].x), pair(x[g].y));
        qf[((2 * g + 1) * NT + t) * 32] = make_uint2(pair(x[g].z), pair(x[g].w));
      }
      const float f = scale == 0.f ? 1.f : fmaxf(fabsf(scale) * __uint_as_float(e << 23) * kLog2e, 1.4e-45f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        c[t][i] = __shfl_sync(0xffffffffu, f, tig * 8 + i * 4);
        m[t][i] = -INFINITY;
        l[t][i] = mul[t][i] = 0.f;
      }
#pragma unroll
      for (int g = 0; g < kPieces; ++g)
#pragma unroll
        for (int e2 = 0; e2 < 8; ++e2) o[t][g][e2 >> 2][e2 & 3] = 0.f;
    }
    range = 0x80000000u;  // (none yet: every scale is outside)
  }

  // NBS blocks of 16 tokens of a tile: block b is its tokens key(b) .. key(b) + 15, of which those in [j0, j1) are seen (MASK: not all
  // need be). load_k(b, piece, f), load_v(b, piece, f): fragments of two pieces' words (rows of 32 values: of one), tokens 0-7 and 8-15
  // of each. wait_v: before V is touched.
  // The scales of a tile are a record per box of 2^log2_box tokens: the rows' fp32 scales, then their block scales.
  template <bool MASK, int NBS, typename Key, typename LoadK, typename LoadV, typename Wait>
  __device__ __forceinline__ bool step(const uint8_t* k_rec, const uint8_t* v_rec, int log2_box, int j0, int j1, Key key, LoadK load_k, LoadV load_v,
                                       Wait wait_v) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    constexpr int kRec = kv_scale_bytes(kKv4, D);
    if (D == 128) asm volatile("" : "+r"(log2_box));  // (offsets are computed where they are used: held over the loop of tiles they would spill)
    // offsets of token j's row scale and block scales, and from token gid's to token gid + 8's
    auto row_at = [&](int j) { return (j >> log2_box) * (kRec << log2_box) + (j & ((1 << log2_box) - 1)) * 4; };
    auto blocks_at = [&](int j) { return (j >> log2_box) * (kRec << log2_box) + (4 << log2_box) + (j & ((1 << log2_box) - 1)) * (D / 16); };
    const int row_8 = log2_box == 3 ? 8 * kRec : 32, blocks_8 = log2_box == 3 ? 8 * kRec : D / 2;
    constexpr int kTwo = D == 32 ? 1 : 2;  // pieces of a load
    // ---- S^T = K Q^T ----
    float s[NBS][NT][4];
    uint32_t bs[NBS][2][2];  // block scales of tokens gid and gid + 8
    bool any[NBS];
#pragma unroll
    for (int b = 0; b < NBS; ++b) {
      any[b] = !MASK || (key(b) + 16 > j0 && key(b) < j1);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[b][t][e] = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t* at = k_rec + blocks_at(key(b)) + gid * (D / 16) + u * blocks_8;
        if (D == 128) {
          const uint2 x = *reinterpret_cast<const uint2*>(at);
          bs[b][u][0] = x.x;
          bs[b][u][1] = x.y;
        } else {
          bs[b][u][0] = bs[b][u][1] = D == 64 ? *reinterpret_cast<const uint32_t*>(at) : *reinterpret_cast<const uint16_t*>(at);
        }
      }
    }
#pragma unroll
    for (int p = 0; p < kPieces; p += kTwo) {
      uint2 q[kTwo][2][NT];
#pragma unroll
      for (int i = 0; i < kTwo; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int t = 0; t < NT; ++t) q[i][e][t] = qf[((2 * (p + i) + e) * NT + t) * 32];
#pragma unroll
      for (int b = 0; b < NBS; ++b) {
        if (MASK && !any[b]) continue;
        uint32_t f[4], sc[2];
        load_k(b, p, f);
        // (this thread's words are of the first or second block of each piece)
#pragma unroll
        for (int u = 0; u < 2; ++u) sc[u] = e4m3_f16x2(__byte_perm(bs[b][u][p >> 1], 0, 0x20 + (tig >> 1) * 0x11));
#pragma unroll
        for (int i = 0; i < kTwo; ++i) {
          const uint32_t x = f[2 * i], y = f[2 * i + 1];
          uint32_t k[2][4];
          auto scaled = [&](uint32_t v, int u) { return i ? mul_half<true>(v, sc[u]) : mul_half<false>(v, sc[u]); };
          k[0][0] = scaled(e2m1_f16x2<0>(x), 0);
          k[0][1] = scaled(e2m1_f16x2<0>(y), 1);
          k[0][2] = scaled(e2m1_f16x2<1>(x), 0);
          k[0][3] = scaled(e2m1_f16x2<1>(y), 1);
          k[1][0] = scaled(e2m1_f16x2<2>(x), 0);
          k[1][1] = scaled(e2m1_f16x2<2>(y), 1);
          k[1][2] = scaled(e2m1_f16x2<3>(x), 0);
          k[1][3] = scaled(e2m1_f16x2<3>(y), 1);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) mma_f16(s[b][t], k[e], q[i][e][t].x, q[i][e][t].y);
        }
      }
    }
    if (!wait_v()) return false;
    // ---- row scales, tokens that are not seen, the heads' largest logits ----
    float sv[NBS][2], top[NT][N];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < N; ++i) top[t][i] = -INFINITY;
#pragma unroll
    for (int b = 0; b < NBS; ++b)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j = key(b) + u * 8 + gid;
        const int at = row_at(key(b)) + gid * 4 + u * row_8;
        const float sk = *reinterpret_cast<const float*>(k_rec + at);
        sv[b][u] = *reinterpret_cast<const float*>(v_rec + at);
        const bool seen = !MASK || (j >= j0 && j < j1);
        if (MASK && !seen) sv[b][u] = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            float& x = s[b][t][2 * u + i];
            x = seen ? x * sk : -INFINITY;
            top[t][i] = fmaxf(top[t][i], x);
          }
      }
    // (rounded before the base is taken off, as the base was: a rest of the product's bits would be far above 0 in a large one)
    auto logit = [](float x, float f) { return __fmul_rn(x, f); };
    bool grows = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        top[t][i] = logit(top[t][i], c[t][i]);
        grows = grows || top[t][i] > m[t][i] + kGrow;
      }
    // the magnitude of one token's V scale in each lane, as bits (not seen, or nothing to weigh: 0)
    auto size = [&]() -> uint32_t {
      const int j = key(NBS == 2 ? lane >> 4 : 0) + (lane & 15);
      return !MASK || (j >= j0 && j < j1) ? *reinterpret_cast<const uint32_t*>(v_rec + row_at(j)) & 0x7fffffffu : 0u;
    };
    auto is_outside = [&](uint32_t x) { return x + range > 11u << 23 && x != 0u; };
    if (__any_sync(0xffffffffu, grows || is_outside(size()))) rescale<NBS>(s, sv, top, size, is_outside);
    // ---- O^T += V^T P^T ----
    float base[NT][N];  // (a base of -infinity is left out of the exponent: nothing was seen yet, or every logit is -infinity)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < N; ++i) base[t][i] = m[t][i] == -INFINITY ? 0.f : m[t][i];
#pragma unroll
    for (int b = 0; b < NBS; ++b) {
      if (MASK && !any[b]) continue;
      uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float w[2] = {0.f, 0.f};
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float p = ex2(logit(s[b][t][2 * u + i], c[t][i]) - base[t][i]);
            l[t][i] += p;
            w[i] = p * (sv[b][u] * mul[t][i]);
          }
          const uint32_t h = pack2<__half>(w[0], w[1]);
          const float2 f = unpack2<__half>(h);
          hi[t][u] = transposed(h);
          lo[t][u] = transposed(pack2<__half>(w[0] - f.x, N == 2 ? w[1] - f.y : 0.f));
        }
      // block scales of tokens 2 tig, 2 tig + 1 and of those 8 further; unseen tokens' cleared (they may be no numbers)
      uint32_t vs[2][4], keep[2] = {0xffffffffu, 0xffffffffu};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j = key(b) + u * 8 + 2 * tig;
        const uint8_t* at = v_rec + blocks_at(key(b)) + 2 * tig * (D / 16) + u * blocks_8;
        if (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(at);
          vs[u][0] = x.x;
          vs[u][1] = x.y;
          vs[u][2] = x.z;
          vs[u][3] = x.w;
        } else if (D == 64) {
          const uint2 x = *reinterpret_cast<const uint2*>(at);
          vs[u][0] = vs[u][1] = x.x;
          vs[u][2] = vs[u][3] = x.y;
        } else {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(at);
          vs[u][0] = vs[u][1] = x;
          vs[u][2] = vs[u][3] = x >> 16;
        }
        if (MASK) keep[u] = (j >= j0 && j < j1 ? 0xffu : 0u) | (j + 1 >= j0 && j + 1 < j1 ? 0xff00u : 0u);
      }
      const uint32_t pick = (gid >> 2) * 0x11 + 0x40;  // block gid / 4 of a piece's two, of either token
#pragma unroll
      for (int p = 0; p < kPieces; p += kTwo) {
        uint32_t f[4];
        load_v(b, p, f);
#pragma unroll
        for (int i = 0; i < kTwo; ++i) {
          const int g = p + i;
          uint32_t sc[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t both = __byte_perm(vs[u][g >> 1], vs[u][2 + (g >> 1)], pick + (g & 1) * 0x22);
            if (MASK) both &= keep[u];
            sc[u] = e4m3_f16x2(both);
          }
          // 4 values of two tokens each: bytes of a value's two tokens, values 0 and 2 in `even`, 1 and 3 in `odd`
          const uint32_t first = __byte_perm(f[2 * i], f[2 * i + 1], 0x5410), second = __byte_perm(f[2 * i], f[2 * i + 1], 0x7632);
          const uint32_t even = (first & 0x0f0f0f0fu) | (second << 4 & 0xf0f0f0f0u), odd = (first >> 4 & 0x0f0f0f0fu) | (second & 0xf0f0f0f0u);
          uint32_t v[2][4];
          v[0][0] = mul2<__half>(e2m1_f16x2<0>(even), sc[0]);
          v[0][1] = mul2<__half>(e2m1_f16x2<0>(odd), sc[0]);
          v[0][2] = mul2<__half>(e2m1_f16x2<2>(even), sc[1]);
          v[0][3] = mul2<__half>(e2m1_f16x2<2>(odd), sc[1]);
          v[1][0] = mul2<__half>(e2m1_f16x2<1>(even), sc[0]);
          v[1][1] = mul2<__half>(e2m1_f16x2<1>(odd), sc[0]);
          v[1][2] = mul2<__half>(e2m1_f16x2<3>(even), sc[1]);
          v[1][3] = mul2<__half>(e2m1_f16x2<3>(odd), sc[1]);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mma_f16(o[t][g][e], v[e], hi[t][0], hi[t][1]);
              mma_f16(o[t][g][e], v[e], lo[t][0], lo[t][1]);
            }
        }
      }
    }
    return true;
  }

  // A logit passed its base by more than kGrow, or a V scale lies outside: bases and powers of two follow.
  template <int NBS, typename Size, typename Outside>
  __device__ __forceinline__ void rescale(const float (&s)[NBS][NT][4], const float (&sv)[NBS][2], float (&top)[NT][N], Size size, Outside is_outside) {
    auto exponent = [](float x) { return (int)(__float_as_uint(x) >> 23 & 255u); };
    auto power = [](int e) { return __uint_as_float((uint32_t)e << 23); };
    const uint32_t my_size = size(), most = __reduce_max_sync(0xffffffffu, my_size);
    const int largest = (int)(most >> 23);
    if (mul[0][0] == 0.f && most != 0u) {  // (scales of zero set none: their tokens add nothing)
      const float first = power(262 - min(max(largest + 4, 12), 254));
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < N; ++i) mul[t][i] = first;
      range = __float_as_uint(first) - (251u << 23);
    }
    const bool far = __any_sync(0xffffffffu, is_outside(my_size));
    if (far) range = 0x80000000u;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float n = top[t][i];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, d));
        n = fmaxf(n, m[t][i]);
        const float f = n == m[t][i] ? 1.f : ex2(m[t][i] - n), up = m[t][i] - n;
        m[t][i] = n;
        l[t][i] *= f;
        float g = f;
        if (far) {
          // the head's largest weight times V scale becomes 2^7 to 2^8, unless what was summed so far holds a larger one, and a scale
          // times mul stays finite (its weight may be zero)
          const float sub = n == -INFINITY ? 0.f : n;
          float x = 0.f;
#pragma unroll
          for (int b = 0; b < NBS; ++b)
#pragma unroll
            for (int u = 0; u < 2; ++u) x = fmaxf(x, fabsf(ex2(__fmul_rn(s[b][t][2 * u + i], c[t][i]) - sub) * sv[b][u]));
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          const int was = exponent(mul[t][i]), held = f == 1.f ? was : exponent(mul[t][i] * ex2(-up));
          const int e = min(max(min(min(held, 261 - exponent(x)), 379 - largest), 8), 250);
          mul[t][i] = power(e);
          g = f == 1.f ? power(127 + max(e - was, -127)) : ex2(up + (float)(e - was));
        }
#pragma unroll
        for (int q = 0; q < kPieces; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            o[t][q][e][i] *= g;
            o[t][q][e][2 + i] *= g;
          }
      }
  }

  // The sums to shared memory: rows of the heads (those below `rows`), `stride` floats apart, and their m and l.
  __device__ __forceinline__ void store(float* dst, float* dst_m, float* dst_l, int stride, int rows) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float sum = l[t][i];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const int head = N == 2 ? t * 8 + 2 * tig + i : tig;
        if (head >= rows) continue;
        const float back = __uint_as_float(254u - (__float_as_uint(mul[t][i]) >> 23) << 23);  // 1 / mul
#pragma unroll
        for (int g = 0; g < kPieces; ++g)
          *reinterpret_cast<float4*>(dst + head * stride + g * 32 + 4 * gid) =
              make_float4(o[t][g][0][i] * back, o[t][g][0][2 + i] * back, o[t][g][1][i] * back, o[t][g][1][2 + i] * back);
        if (gid == 0) {
          dst_m[head] = m[t][i];
          dst_l[head] = sum;
        }
      }
  }
};

}  // namespace kv
}  // namespace cvr
