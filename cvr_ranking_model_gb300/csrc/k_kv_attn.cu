// Attention of one query token per request over a paged history (cvr_kv_attend of include/cvr.h): for query head i of
// request r, with s_j = scale q . k_j over the tokens j that it sees,
//   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  m = max_j s_j,  lse = m + ln sum_j exp(s_j - m).
//
// One CTA per request and query head: its warps take every fourth token, a lane holds head_dim / 32 values of a row, and
// the four running (m, l, o) are joined in shared memory.
#include "../../include/cvr.h"
#include "cvr_kv.cuh"

namespace cvr {

namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32(int8_t x) { return (float)x; }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }

template <typename T, typename C, int D>
__global__ void __launch_bounds__(128) kv_attend_kernel(const KvAttendArgs a) {
  constexpr int E = D / 32;
  __shared__ float s_o[4][D], s_m[4], s_l[4];
  const int r = blockIdx.x, head = blockIdx.y, kv = head / a.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  int len = a.lens[r];
  const int64_t most = (int64_t)a.max_pages << a.page_log2;
  if (len < 0 || len > most) {
    if (threadIdx.x == 0) atomicOr(a.err, kKvErrLens);
    len = len < 0 ? 0 : (int)most;
  }
  const int lo = a.window ? max(0, len - a.window) : 0;
  const T* q = static_cast<const T*>(a.q) + r * a.q_stride + head * D;
  float qf[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qf[e] = to_f32(q[lane * E + e]);
    o[e] = 0.f;
  }
  for (int j = lo + warp; j < len; j += 4) {
    int page = a.table[(int64_t)r * a.max_pages + (j >> a.page_log2)];
    if (page < 0 || page >= a.n_pages) {
      if (lane == 0) atomicOr(a.err, kKvErrPage);
      page = 0;
    }
    const int pos = j & ((1 << a.page_log2) - 1);
    const C* kr = static_cast<const C*>(a.k) + page * a.k_stride[0] + kv * a.k_stride[1] + pos * a.k_stride[2] + lane * E;
    const C* vr = a.v ? static_cast<const C*>(a.v) + page * a.v_stride[0] + kv * a.v_stride[1] + pos * a.v_stride[2] + lane * E : kr;
    const int64_t sc = (((int64_t)page * a.kv_heads + kv) << a.page_log2) + pos;
    const float ks = a.k_scale ? a.k_scale[sc] : 1.f, vs = a.v_scale && a.v ? a.v_scale[sc] : ks;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(qf[e], to_f32(kr[e]), s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= ks * a.scale;
    const float n = fmaxf(m, s), base = n == -INFINITY ? 0.f : n;
    const float f = expf(m - base), p = expf(s - base);
    m = n;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * (to_f32(vr[e]) * vs);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  if (warp != 0) return;
  float top = -INFINITY;
  for (int w = 0; w < 4; ++w) top = fmaxf(top, s_m[w]);
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int w = 0; w < 4; ++w) {
    const float f = expf(s_m[w] - base);
    sum += s_l[w] * f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += s_o[w][lane * E + e] * f;
  }
  T* out = static_cast<T*>(a.out) + r * a.out_stride + head * D;
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane * E + e] = from_f32<T>(len > 0 ? acc[e] / sum : 0.f);
  if (lane == 0 && a.lse) a.lse[(int64_t)r * a.q_heads + head] = len > 0 ? base + logf(sum) : -INFINITY;
}

}  // namespace

cudaError_t launch_kv_attend(const KvAttendArgs& a, int dtype, bool int8, int head_dim, int num_sms, cudaStream_t s) {
  (void)num_sms;
  auto run = [&](auto kern) { return launch_kernel(kern, dim3(a.n_req, a.q_heads), dim3(128), 0, s, true, a); };
  auto by_dim = [&](auto t, auto c) {
    typedef decltype(t) T;
    typedef decltype(c) C;
    if (head_dim == 32) return run(kv_attend_kernel<T, C, 32>);
    if (head_dim == 64) return run(kv_attend_kernel<T, C, 64>);
    return run(kv_attend_kernel<T, C, 128>);
  };
  if (dtype == CVR_DTYPE_BF16) return int8 ? by_dim(__nv_bfloat16(), int8_t()) : by_dim(__nv_bfloat16(), __nv_bfloat16());
  return int8 ? by_dim(__half(), int8_t()) : by_dim(__half(), __half());
}

}  // namespace cvr
