// Attention of one query token per request over a paged history (cvr_kv_attend of include/cvr.h): for query head i of
// request r, with s_j = scale q . k_j over the tokens j that it sees,
//   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  m = max_j s_j,  lse = m + ln sum_j exp(s_j - m).
// Every K and V row is read once for all the query heads that share it, so the floor is the bytes of the seen rows.
//
// Work: a tile is 8 or 16 KB of one kv head's K rows (at most 256) and the V rows beside them. The tiles of all requests
// and heads form one line (request, then head, then position; in long runs with a place or two in front of each head's tiles for
// what its start and end cost); a persistent grid cuts it into equal runs, so ragged lengths, few long histories and many
// short ones load the SMs alike. A CTA finds its run by scanning the lengths itself. What
// a CTA leaves of a (request, head) that it shares with others goes to the workspace as (m, l, o); the last of them to
// arrive joins the parts in order, so results do not depend on which it is.
//
// A CTA is one producer warp and four consumer warps. The producer turns page ids into TMA copies (a box per page)
// into a ring of units, K and V in turn, swizzled so that ldmatrix reads without bank conflicts, and runs ahead across
// requests. A consumer warp takes every fourth block of 16 tokens of a tile (or, for more than 16 query heads per kv head,
// 16 of the heads): S = Q K^T and O += P V on mma.sync m16n8k16 with the running maximum, sum and O in registers.
//   - mma.sync, not tcgen05: a tile has 1 (one head, 16 bits) to 256 (64 heads, int8, K = V) operations per byte read, and P
//     stays in registers between the two products. For up to 8 heads the tensor pipe is active less than 30% of the time. With the
//     heads on M an M = 128 MMA would be mostly padding; with the tokens on M it would not, which is not built: the forms for 32
//     and 64 heads, whose warps load and convert the same rows for 16 heads each, stand far from their bytes.
//   - P enters the second product as two 16-bit halves (p = hi + lo), so that its rounding (2^-8 in bf16) does not add to
//     the output's. With at most 8 query rows the halves sit in the two halves of the 16-row tile, at no extra cost.
//   - 8-bit rows become fp16 exactly (1024 + q by a byte permute, minus 1152); K's scale multiplies the logit, V's scale
//     the weight, whose products enter as fp16 times a power of two that the first scales choose. Where scales lie farther apart
//     than the halves' bits allow, each query row has its own, which follows the row's largest product, so that a large scale
//     without weight leaves the other tokens their bits.
//
// Measured (one GB300, copy rate 6.67 TB/s): 64 requests of up to 8191 tokens, 32 / 8 heads of 128, bf16: 113 us, 6.5 TB/s;
// one request of 131071: 85 us, 6.3 TB/s; both bound by HBM. 32 requests on int8 rows, 64 / 8 heads of 128: 74 us, 5.2 TB/s: 2.4
// warps per scheduler, which issue 49% of the time, and no registers for more. 512 histories of up to 2000 events, 4 heads of 32,
// K = V: 35 us, 3.7 TB/s: softmax, masks and copies of 1 KB once per head, issued 53% of the time. One request of 200: 4.6 us, latency.
#pragma once

#include <type_traits>

#include "../../include/cvr.h"
#include "cvr_kv.cuh"

namespace cvr {
namespace kv {

constexpr int kConsumers = 4;                       // consumer warps
constexpr int kThreads = (kConsumers + 1) * 32;     // and the producer
static_assert(kThreads == kKvAttendThreads, "the launch's block");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A part: the tiles of one (request, kv head) in a CTA's run.
struct __align__(16) Part {
  int r, h, k0, n_tiles;     // request, kv head, first token of the first tile; n_tiles negated: the run's last part
  int lo, len, i0, n_parts;  // tokens seen: [lo, len); the (request, head) has n_parts parts, of CTAs i0, i0 + 1, ..
};
constexpr int kGroup = 16;  // parts that are joined at once

// MODE: query rows per kv head 0: at most 8, 1: 16, 2: 32, 3: 64
template <bool I8, int D, int MODE>
struct Shape {
  static constexpr int MT = MODE == 3 ? 4 : MODE == 2 ? 2 : 1;  // 16-row tiles of query heads
  static constexpr int KP = kConsumers / MT;                    // consumer warps that share a row tile's tokens
  static constexpr int kRow = D * (I8 ? 1 : 2);                 // bytes of a row
  static constexpr int kLine = kRow < 128 ? kRow : 128;         // bytes of a swizzled line
  static constexpr int kHalves = kRow / kLine;
  static constexpr int kCtasPerSm = D == 32 ? (MT == 1 ? 4 : 3) : D == 64 ? (MT == 1 && I8 ? 3 : 2) : 2;
  static constexpr int kUnitMost = kCtasPerSm == 2 && (MT == 1 || D < 128) ? 16384 : 8192;
  static constexpr int TK = kUnitMost / kRow < 256 ? kUnitMost / kRow : 256;  // tokens per tile
  static constexpr int kUnit = TK * kRow;
  static constexpr int kQRow = D * 2 + 16;                      // padded: conflict-free fragment loads
  static constexpr int kQBytes = (MODE == 0 ? 8 : MT * 16) * kQRow;
  static constexpr int kORow = D + (I8 ? 16 : 8);               // padded fp32 rows of the joining area
  static constexpr int kORows = MODE == 0 ? 8 : 16;             // a warp's rows in the joining area
  static constexpr int kOBytes = kConsumers * kORows * (kORow + 2) * 4;  // with the rows' m and l
  static constexpr int kOAreas = D == 32 && MODE == 0 ? 2 : 1;           // (two spare a barrier per use, where they fit)
  static constexpr int kScaleBytes = I8 ? TK * 4 : 0;
  static constexpr int kPartCost = MT == 1 ? 1 : 2;  // what a part costs beside its tiles, in tiles (see attend_kernel's runs)
  // blocks of 16 tokens that a warp takes per tile, and per softmax step
  static constexpr int NB = TK / 16 / KP, NBS = NB < 2 ? NB : 2;
  // ring units: what is left of this CTA's share of the SM's 228 KB (1 KB of it reserved, 1 KB for the ring's alignment)
  static constexpr int kShare = kCtasPerSm == 1 ? 232448 : 233472 / kCtasPerSm - 1024;
  static constexpr int kFixed = 2 * kQBytes + kOAreas * kOBytes + 3 * (int)sizeof(Part) + 5 * 8 + 64 + 1024;
  static constexpr int kRing = (kShare - kFixed) / (kUnit + kScaleBytes + 16);
  // shared memory
  static constexpr int oScale = kRing * kUnit;
  static constexpr int oQ = oScale + kRing * kScaleBytes;
  static constexpr int oO = oQ + 2 * kQBytes;
  static constexpr int oPart = oO + kOAreas * kOBytes;
  static constexpr int oBar = oPart + 3 * (int)sizeof(Part);
  static constexpr int kSmem = oBar + (2 * kRing + 5) * 8 + 64 + 1024;
  static_assert(kSmem <= kShare && kRing >= 4, "K and V units of two tiles at least");
};


template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) { return pack_bf16(a, b); }
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t x);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// the product of two pairs
template <typename T>
__device__ __forceinline__ uint32_t mul2(uint32_t x, uint32_t y);
template <>
__device__ __forceinline__ uint32_t mul2<__nv_bfloat16>(uint32_t x, uint32_t y) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t mul2<__half>(uint32_t x, uint32_t y) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// c (+)= a b; FIRST: the accumulator starts from zero
template <typename T, bool FIRST = false>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (FIRST) {
    if (std::is_same<T, __half>::value)
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
          : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
          : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
          : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
          : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  } else {
    if (std::is_same<T, __half>::value)
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
          : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
          : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
          : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
          : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two of the four bytes of x, biased signed values (q ^ 0x80 = q + 128), as an fp16 pair: SEL picks the bytes (0x4140: 0 and
// 1, 0x4342: 2 and 3, 0x4240: 0 and 2, 0x4341: 1 and 3); the bits 0x64.. are 1024 + (q + 128).
template <int SEL>
__device__ __forceinline__ uint32_t i8_pair(uint32_t x) {
  const uint32_t u = __byte_perm(x, 0x64646464u, SEL);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// A wait of a whole warp, bounded like mbar_wait: the hardware may hold a polling warp for up to 1 ms at a time, so that
// waiting warps do not take the others' issue slots.
__device__ __forceinline__ bool try_wait_1ms(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (__all_sync(0xffffffffu, try_wait_1ms(bar, parity))) return true;
    const bool late = global_timer_ns() - t0 > 1000000000ull;
    if (__any_sync(0xffffffffu, *abort_flag != 0 || late)) {
      if (late) {
        *abort_flag = 1;
        atomicOr(err, kErrTimeout);
      }
      __syncwarp();
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_on(bar, parity, abort_flag, err);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// the tokens that a request of length `len` sees begin at the result
__device__ __forceinline__ int seen_from(const KvAttendArgs& a, int len) { return a.window ? max(0, len - a.window) : 0; }
__device__ __forceinline__ int clamped_len(const KvAttendArgs& a, int len) {
  const int most = a.max_pages << a.page_log2;  // (at most 2^30)
  return len < 0 ? 0 : min(len, most);
}
template <int TK>
__device__ __forceinline__ int tiles_of(const KvAttendArgs& a, int len) {
  return (len + TK - 1) / TK - seen_from(a, len) / TK;
}

// Exclusive sums of x over the block's threads, saturating at 2^31 - 1, and the sum of all; sums: a word per warp.
struct Scanned {
  uint32_t before, all;
};
__device__ __forceinline__ Scanned scan_block(uint32_t x, uint32_t* sums) {
  auto add = [](uint32_t x, uint32_t y) { return min(x + y, 0x7fffffffu); };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl = add(incl, u);
  }
  if (lane == 31) sums[warp] = incl;
  cta_sync();
  Scanned s = {incl - x, 0};
#pragma unroll
  for (int w = 0; w <= kConsumers; ++w) {
    if (w < warp) s.before = add(s.before, sums[w]);
    s.all = add(s.all, sums[w]);
  }
  return s;
}
// (the same out of line, for calls whose line is scanned twice: in line it costs every small call 0.2 us of instruction fetches)
static __device__ __noinline__ Scanned scan_block_again(uint32_t x, uint32_t* sums) { return scan_block(x, sums); }
// n > 0 tiles filled up to whole runs (out of line for the same reason)
static __device__ __noinline__ int whole_runs(int n, int per) { return (n + per - 1) / per * per; }

// where part p of a (request, head) that begins in CTA i0's run lies in the workspace: a CTA has two places, [1] for what
// begins in its run and goes on, [0] for what began before
__device__ __forceinline__ int part_place(int i0, int p) { return (i0 + p) * 2 + (p == 0); }

__device__ __forceinline__ unsigned add_acq_rel(unsigned* p) {
  unsigned v;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
  return v;
}

template <typename T, bool I8, int D, int MODE>
__global__ void __launch_bounds__(kThreads, Shape<I8, D, MODE>::kCtasPerSm)
    attend_kernel(const __grid_constant__ KvAttendArgs a, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v) {
  typedef Shape<I8, D, MODE> S;
  constexpr int MT = S::MT, KP = S::KP, TK = S::TK, NB = S::NB, NBS = S::NBS, RING = S::kRing;
  constexpr bool R8 = MODE == 0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* const full = reinterpret_cast<uint64_t*>(sm + S::oBar);
  uint64_t* const empty = full + RING;
  uint64_t* const q_full = empty + RING;   // [2]
  uint64_t* const q_empty = q_full + 2;    // [2]
  uint64_t* const meet = q_empty + 2;      // the consumer warps' barrier
  volatile int* const abort_flag = reinterpret_cast<int*>(meet + 1);
  int* const s_last = const_cast<int*>(abort_flag) + 1;
  uint32_t* const s_sum = reinterpret_cast<uint32_t*>(sm + S::oPart);  // scan scratch, before the first part
  int* const s_start = s_last + 1;  // request of the CTA's first tile, the places per head before it, and its own
  Part* const s_part = reinterpret_cast<Part*>(sm + S::oPart);  // [2] with the query rows, [1] the early part
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.kv_heads, G = a.group;
  const bool two = a.v != nullptr;  // V is a pool of its own

  if (tid == 0) {
    for (int i = 0; i < RING; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, kConsumers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, kConsumers);
    }
    mbar_init(meet, kConsumers);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    if (two) tma_prefetch_desc(&tm_v);
  }
  pdl_trigger();
  pdl_wait();  // (lengths and page ids are read with plain loads: an earlier call may have written them while this one started)

  // ---- this CTA's run of the line of tiles: every thread sums a few requests' tiles, saturating ----
  const int few = (a.n_req + kThreads - 1) / kThreads;
  const int r0 = min(tid * few, a.n_req), r1 = min(r0 + few, a.n_req);
  auto add = [](uint32_t x, uint32_t y) { return min(x + y, 0x7fffffffu); };
  uint32_t mine = 0;
  int nonempty = 0;
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    const int raw = a.lens[r], len = clamped_len(a, raw);
    bad |= raw != len;
    mine = add(mine, tiles_of<TK>(a, len));
    nonempty += len > 0;
  }
  if (bad && blockIdx.x == 0) atomicOr(a.err, kKvErrLens);
  // In runs of 8 tiles or more a (request, head) has kPartCost empty places in front of its tiles, or a run of many short
  // requests would end last: 32 requests of 1 to 16383 tokens in 8 bits 80.5 -> 74.3 us, 48 of up to 6001 tokens, 8 x 32 heads
  // over rows of 64, 56.9 -> 47.9 us.
  // In shorter ones of two tiles or more a (request, head) is filled up to whole runs behind its tiles, if the grid has room for
  // that: no CTA then has one's end and another's beginning, two joins one after the other. 48 requests with a window of 1000:
  // 10.6 -> 9.6 us; 4 requests of up to 3000 tokens, 8 / 4 heads of 128, 13.6 -> 11.2 us.
  int lead = 0, pad = 1;
  const int grid = gridDim.x;
  Scanned line = scan_block(mine, s_sum);  // places per head before this thread's requests, and of all
  const uint64_t tiles = (uint64_t)line.all * H;
  const bool fits = tiles <= 0x7fff0000u;  // (sums with a grid's size stay below 2^31)
  int total = fits ? (int)tiles : 0;
  // A run's places: an even share of the line; at least two tiles where requests have two or more on average: a split costs a
  // join (about 2 us at a call's end), a second tile about 0.5 us. One request of 200 tokens of 4 x 32: 4.7 us in 4 runs, 5.8 us
  // in 8.
  auto share = [&](int n) { return (int)(((unsigned)n + grid - 1) / (unsigned)grid); };
  int per = max(share(total), (int)line.all >= 2 * a.n_req ? 2 : 1);
  if (__builtin_expect(per >= 8 && fits && tiles <= 0x7fff0000u / (1 + S::kPartCost), 0)) {
    lead = S::kPartCost;
    mine += nonempty * lead;
    line = scan_block_again(mine, s_sum + 8);
    total = (int)line.all * H;
    per = share(total);
  } else if (__builtin_expect(per > 1 && per < 8 && a.n_req * H <= grid && (a.n_req > 1 || (int)line.all > per), 0)) {
    uint32_t filled_up = 0;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) filled_up += whole_runs(tiles_of<TK>(a, clamped_len(a, a.lens[r])), per);
    const Scanned l = scan_block_again(filled_up, s_sum + 8);
    if ((uint64_t)l.all * H <= (uint64_t)grid * per) {
      pad = per;
      line = l;
      mine = filled_up;
      total = (int)l.all * H;
    }
  }
  uint32_t before = line.before;
  if (!fits && tid == 0 && blockIdx.x == 0) atomicOr(a.err, kKvErrSize);
  auto extent = [&](int n) { return n <= 0 ? 0 : pad > 1 ? whole_runs(n, pad) : n + lead; };  // places of a request of n tiles, per head
  const int begin = min((int64_t)blockIdx.x * per, (int64_t)total), end = min((int64_t)begin + per, (int64_t)total);
  const bool some = end > begin;  // (a run without tiles is none: the line ends with a tile, other runs are longer than kPartCost)
  if (some && begin >= (int)before * H && begin < (int)(before + mine) * H) {
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
      const int n = r1 - r0 == 1 ? (int)mine : extent(tiles_of<TK>(a, clamped_len(a, a.lens[r])));
      if (begin < ((int)before + n) * H) {
        s_start[0] = r;
        s_start[1] = (int)before;
        s_start[2] = n;
        break;
      }
      before += n;
    }
  }
  cta_sync();

  if (warp == kConsumers) {
    // ================= producer =================
    const int log2_br = min(a.page_log2, 31 - __clz(TK));  // rows of a box: a page, or a tile of a longer page
    const int br = 1 << log2_br, n_box_max = TK >> log2_br;
    int slot = 0, filled = 0;  // the ring's next unit, and the units filled so far (at most RING)
    uint32_t phase = 0;        // parity of the ring's round
    int parts = 0;             // parts begun
    if (some) {
      // Page ids come 32 entries of a table row at a time, one per lane, and ahead of their use: the row's next 32, and the
      // first 32 of the next request. A tile's entries never straddle two batches (both begin at a multiple of its count).
      auto entries = [&](int row, int e) {
        return e + lane < a.max_pages ? a.table[(int64_t)row * a.max_pages + e + lane] : 0;
      };
      int wb = s_start[0], wl = 0;  // lengths of the 32 requests from wb on, one per lane
      auto window = [&](int from) {
        wb = from;
        wl = wb + lane < a.n_req ? clamped_len(a, a.lens[wb + lane]) : 0;
      };
      auto first_entry = [&](int length) { return (seen_from(a, length) / TK * TK) >> a.page_log2; };
      // the next request with a tile from `from` on (n_req: none), its length and first page ids
      int n_r = 0, n_len = 0, n_ids = 0;
      auto look_ahead = [&](int from) {
        unsigned some;
        while (true) {
          if (from >= wb + 32) window(from);
          some = __ballot_sync(0xffffffffu, wl > 0 && wb + lane >= from);
          if (some || wb + 32 >= a.n_req) break;
          from = wb + 32;
        }
        n_r = some ? wb + __ffs(some) - 1 : a.n_req;
        n_len = some ? __shfl_sync(0xffffffffu, wl, __ffs(some) - 1) : 0;
        n_ids = some ? entries(n_r, first_entry(n_len)) : 0;
      };
      int P = s_start[1], r = 0, h = 0, t = 0, n_t = 1, t0 = 0, len = 0, lo = 0;  // P: places per head before request r
      int w_t = 1;  // the request's places per head
      int e0 = 0, ids = 0, more_ids = 0;  // entries e0 + lane and e0 + 32 + lane of the request's table row
      int ids0 = 0, more0 = 0;            // the same from the request's first entry on, for its next head
      auto enter = [&]() {  // the request that was looked ahead to
        r = n_r;
        len = n_len;
        lo = seen_from(a, len);
        t0 = lo / TK;
        n_t = max(1, tiles_of<TK>(a, len));
        w_t = n_t + lead;
      };
      window(wb);
      look_ahead(wb);
      enter();
      w_t = s_start[2];  // (filled up, it is the run's only part)
      h = (begin - P * H) / w_t;
      t = max((begin - P * H) - h * w_t - lead, 0);
      e0 = ((t0 + t) * TK) >> a.page_log2;  // (the run may begin anywhere in its request)
      ids = entries(r, e0);
      more_ids = entries(r, e0 + 32);
      ids0 = n_ids;
      more0 = entries(r, first_entry(len) + 32);
      bool ok = true;
      const uint32_t box_bytes = br * (S::kRow + (I8 ? 4 : 0)), tile_bytes = TK * (S::kRow + (I8 ? 4 : 0));
      const bool long_pages = a.page_log2 > log2_br;  // several tiles per page, one box per tile
      while (ok) {
        // ---- a part: its query rows and description, and its tiles ----
        const int first = P * H + h * w_t + lead;  // the (request, head)'s first tile's place
        const int n = min(n_t - t, end - first - t), b = parts & 1;
        const bool more = n == n_t - t && first + w_t < end;  // the run goes on
        ok = wait_warp(q_empty + b, ((parts >> 1) & 1) ^ 1, abort_flag, a.err);
        if (!ok) break;
        if (lane == 0) {
          const int last = first + n_t - 1;
          Part pt;
          pt.r = r;
          pt.h = h;
          pt.k0 = (t0 + t) * TK;
          pt.n_tiles = more ? n : -n;
          pt.lo = lo;
          pt.len = len;
          pt.i0 = first >= begin ? blockIdx.x : (unsigned)first / (unsigned)per;
          pt.n_parts = (last < end ? blockIdx.x : (unsigned)last / (unsigned)per) - pt.i0 + 1;
          s_part[b] = pt;
          mbar_expect_tx(q_full + b, (uint32_t)G * D * 2);
        }
        __syncwarp();
        const T* q = static_cast<const T*>(a.q) + r * a.q_stride + (int64_t)h * G * D;
        for (int g = lane; g < G; g += 32)
          bulk_load(smem_u32(sm + S::oQ + b * S::kQBytes + g * S::kQRow), q + g * D, D * 2, q_full + b);
        ++parts;
        if (more && h + 1 == H) look_ahead(r + 1);  // (its lengths and page ids arrive meanwhile)
        for (int i = 0; i < n && ok; ++i) {
          const int k0 = (t0 + t + i) * TK;
          if ((k0 >> a.page_log2) >= e0 + 32) {
            ids = more_ids;
            e0 += 32;
            more_ids = entries(r, e0 + 32);
          }
          // in lane b: box b of the tile, wanted if any of its tokens is seen
          const int row = long_pages ? k0 & ((1 << a.page_log2) - 1) : 0;
          int page = __shfl_sync(0xffffffffu, ids, ((k0 >> a.page_log2) - e0 + (long_pages ? 0 : lane)) & 31);
          unsigned want = n_box_max == 32 ? 0xffffffffu : (1u << n_box_max) - 1;
          uint32_t bytes = tile_bytes;
          if (k0 < lo || k0 + TK > len) {
            const int from = k0 + (lane << log2_br);
            want &= __ballot_sync(0xffffffffu, from < len && from + br > lo);
            bytes = __popc(want) * box_bytes;
          }
          if ((want >> lane & 1) && (unsigned)page >= (unsigned)a.n_pages) {
            atomicOr(a.err, kKvErrPage);
            page = 0;
          }
#pragma unroll 1
          for (int w = 0; w < (two ? 2 : 1); ++w) {
            ok = wait_warp(empty + slot, phase ^ 1, abort_flag, a.err);
            if (!ok) break;
            if (lane == 0) mbar_expect_tx(full + slot, bytes);
            __syncwarp();
            if (want >> lane & 1) {
              tma_load_5d(sm + slot * S::kUnit + (lane << log2_br) * S::kRow, w ? &tm_v : &tm_k, full + slot, 0, row, 0, h,
                          page);
              if (I8)
                bulk_load(smem_u32(sm + S::oScale + slot * S::kScaleBytes + (lane << log2_br) * 4),
                          (w ? a.v_scale : a.k_scale) + ((((int64_t)page * H + h) << a.page_log2) + row), 4 << log2_br,
                          full + slot);
            }
            filled = min(filled + 1, RING);
            if (++slot == RING) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
        // on to the next head, or the next request
        if (!more) break;
        t = 0;
        if (++h == H) {
          h = 0;
          P += w_t;
          enter();
          ids0 = n_ids;
          more0 = entries(r, first_entry(len) + 32);
        }
        e0 = first_entry(len);
        ids = ids0;
        more_ids = more0;
      }
    }
    // requests that see nothing, shared out over the grid: this CTA's are blockIdx, blockIdx + grid, ..
    for (int64_t r0 = blockIdx.x; r0 < a.n_req; r0 += 32 * (int64_t)gridDim.x) {
      const int64_t mine = r0 + (int64_t)lane * gridDim.x;
      unsigned none = __ballot_sync(0xffffffffu, mine < a.n_req && clamped_len(a, a.lens[min(mine, (int64_t)a.n_req - 1)]) == 0);
      for (; none; none &= none - 1) {
        const int64_t r = r0 + (int64_t)(__ffs(none) - 1) * gridDim.x;
        uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + r * a.out_stride);
        for (int i = lane; i < a.q_heads * (D / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
          for (int i = lane; i < a.q_heads; i += 32) a.lse[r * a.q_heads + i] = -INFINITY;
      }
    }
    // the copies in flight land before the CTA's shared memory can go, also when a consumer's wait gave up
    for (int u = 0; u < filled; ++u) {
      if (--slot < 0) {
        slot = RING - 1;
        phase ^= 1;
      }
      mbar_drain(full + slot, phase);
    }
    for (int p = max(0, parts - 2); p < parts; ++p) mbar_drain(q_full + (p & 1), (p >> 1) & 1);
    return;
  }

  // ================= consumers =================
  const int gid = lane >> 2, tig = lane & 3;
  const int mt = warp % MT, kp = warp / MT;  // row tile, share of the tokens
  const int log2_br = min(a.page_log2, 31 - __clz(TK));
  // Logits in units of ln 2 are c q . k with c > 0 (a token that is not seen has q . k = -infinity, whose product must stay
  // that), q times the scale's sign: -1, 0 or 1. bf16 rows may enter times a power of two, which goes back into c: q . k alone may
  // leave fp32's range where scale times q does not. On 16-bit pools rows whose largest value is 2^16 or more are brought to
  // [2^15, 2^16) (128 products with keys up to 2^104 then stay below 2^127), others stay as they are.
  const float sign = a.scale > 0.f ? 1.f : a.scale < 0.f ? -1.f : 0.f;
  auto factor = [&](uint32_t e) {  // c of rows over 2^(e - 127), at least the least number above 0
    return a.scale == 0.f ? 1.f : fmaxf(fabsf(a.scale) * __uint_as_float(e << 23) * kLog2e, 1.4e-45f);
  };
  // In fp16 weights are kept times a power of two (p is at most 2^kGrow), so that small ones keep their bits: times 2^8, with
  // 8-bit rows and their V scales over a power of two (below). The two halves hold a weight to 2^-22 of it, or to 2^-25, 2^-33
  // of a weight of 1.
  constexpr float kGrow = 6.f;
  constexpr bool kF16 = !I8 && std::is_same<T, __half>::value;
  constexpr float kShift = kF16 ? 8.f : 0.f;
  typedef typename std::conditional<I8, __half, T>::type M;  // operand type of the products
  // fp16 weights are summed by a product of their halves, 2^-22 of each, with ones; others as they are (bf16's halves hold 2^-16)
  constexpr bool kOnesSum = kF16;
  constexpr uint32_t kOnes = 0x3c003c00u;  // 1, 1
  uint32_t meets = 0;
  bool ok = true;
  auto consumer_sync = [&]() {  // a bounded barrier of the four warps
    __syncwarp();
    if (lane == 0) mbar_arrive(meet);
    ok = wait_warp(meet, meets & 1, abort_flag, a.err) && ok;
    ++meets;
  };
  // Addresses of ldmatrix rows in a unit. A unit is boxes of [half][row][line]; block_at is the offset of a 16-token
  // block's first row, a lane adds its row and its 16-byte piece, swizzled by the row (row_off, piece below): matrices
  // 0 .. 3 are (rows 0-7, 8-15) x (two pieces), in the order that the K or the V fragments want. 32 bytes further along the
  // rows is an exclusive or (lines are 128-byte aligned, or the bits above the swizzle's belong to the row).
  const uint32_t half_step = (uint32_t)S::kLine << log2_br;
  const int l7 = lane & 7, up8 = (lane >> 3) & 1, up16 = lane >> 4;
  const uint32_t swz = (S::kLine == 128 ? l7 : S::kLine == 64 ? (l7 >> 1) & 3 : (l7 >> 2) & 1) << 4;
  auto row_off = [&](int upper) -> uint32_t {
    return l7 * S::kLine + upper * (log2_br >= 4 ? 8 * S::kLine : S::kHalves * 8 * S::kLine);
  };
  const uint32_t ring = smem_u32(sm);
  const uint32_t lane_k = ring + row_off(up16) + ((up8 << 4) ^ swz), lane_v = ring + row_off(up8) + ((up16 << 4) ^ swz);
  auto block_at = [&](int key) -> uint32_t {
    return (uint32_t)(((key >> log2_br) * S::kHalves << log2_br) + (key & ((1 << log2_br) - 1))) * S::kLine;
  };
  auto piece = [&](uint32_t addr, int k) -> uint32_t {
    return (addr ^ (uint32_t)(k * 32 % S::kLine)) + (k * 32 / S::kLine) * half_step;
  };

  int ks = 0, parts = 0, areas = 0;  // the ring's next unit, parts begun, joining areas used
  uint32_t phase = 0;
  // A part that the CTA before began and that ends within this run: counted when it is done, looked at when the run is
  // through (in s_part[2]).
  bool early = false;
  unsigned early_count = 0;  // (thread 0: the parts counted before it)

  for (bool last = !some; !last;) {
    // ---- a part: the tiles of one (request, head) in this CTA's run ----
    uint32_t qf[D / 16][4];
    float o[D / 8][4], ls[4] = {0.f, 0.f, 0.f, 0.f};  // ls: sums of the weights by products
    float mA = -INFINITY, mB = -INFINITY, lA = 0.f, lB = 0.f;
    float cA = factor(127), cB = cA;  // logit factors of rows A (gid) and B (gid + 8)
    // 8 bits: weight times V scale times |mul| enters the second product. Rows A and B have the same 2^8 / hi (none yet: 0), hi
    // a power of two, as long as the scales lie in [hi / 2^11, hi]: a row's largest weight is 1 or more, so that the halves'
    // 2^-33 hi per token is within 2^-22 of the row's sum. The first scales set hi to 8 to 16 times their largest; one outside
    // makes the rows `far` below: powers of two of their own, that of A negative, which puts every scale outside. 32 requests of 1
    // to 16383 tokens: 73.3 us with scales within 4 of each other, 80.6 us with scales within 2^16.
    float mulA = 0.f, mulB = 0.f;
    auto exponent = [](float x) { return (int)(__float_as_uint(x) >> 23 & 255u); };
    auto power = [](int e) { return __uint_as_float((uint32_t)e << 23); };
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    const int qb = parts & 1;
    ok = wait_warp(q_full + qb, (parts >> 1) & 1, abort_flag, a.err);
    if (!ok) return;
    const Part pt = s_part[qb];
    const int n_tiles = abs(pt.n_tiles);
    last = pt.n_tiles < 0;
    {
      const uint8_t* qs = sm + S::oQ + qb * S::kQBytes + mt * 16 * S::kQRow;
      const bool inA = mt * 16 + gid < G, inB = !R8 && mt * 16 + gid + 8 < G;
      if (!I8) {
        uint32_t bigA = 0, bigB = 0;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint8_t* pa = qs + gid * S::kQRow + k * 32 + tig * 4;
          qf[k][0] = inA ? *reinterpret_cast<const uint32_t*>(pa) : 0u;
          qf[k][2] = inA ? *reinterpret_cast<const uint32_t*>(pa + 16) : 0u;
          qf[k][1] = inB ? *reinterpret_cast<const uint32_t*>(pa + 8 * S::kQRow) : 0u;
          qf[k][3] = inB ? *reinterpret_cast<const uint32_t*>(pa + 8 * S::kQRow + 16) : 0u;
          bigA = __vmaxu2(bigA, __vmaxu2(qf[k][0] & 0x7fff7fffu, qf[k][2] & 0x7fff7fffu));  // (magnitudes order as their bits)
          bigB = __vmaxu2(bigB, __vmaxu2(qf[k][1] & 0x7fff7fffu, qf[k][3] & 0x7fff7fffu));
        }
        float upA = sign, upB = sign;
        if (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
          for (int d = 1; d < 4; d <<= 1) {
            bigA = __vmaxu2(bigA, __shfl_xor_sync(0xffffffffu, bigA, d));
            if (!R8) bigB = __vmaxu2(bigB, __shfl_xor_sync(0xffffffffu, bigB, d));
          }
          auto row_exponent = [](uint32_t big) { return min(max(max(big >> 16, big & 0xffffu) >> 7, 142u), 254u) - 15; };
          const uint32_t eA = row_exponent(bigA), eB = row_exponent(bigB);
          upA *= __uint_as_float((254u - eA) << 23);
          upB *= __uint_as_float((254u - eB) << 23);
          cA = factor(eA);
          cB = factor(eB);
        }
        const uint32_t upA2 = pack2<T>(upA, upA), upB2 = pack2<T>(upB, upB);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[k][0] = mul2<T>(qf[k][0], upA2);
          qf[k][2] = mul2<T>(qf[k][2], upA2);
          if (!R8) {
            qf[k][1] = mul2<T>(qf[k][1], upB2);
            qf[k][3] = mul2<T>(qf[k][3], upB2);
          }
        }
      } else {
        // a K row's bytes 4 tig .. 4 tig + 3 of each 16 are this thread's: the products' k index is permuted to match
        float upA = sign, upB = sign;
        uint2 xa[D / 16], xb[D / 16];
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint8_t* pa = qs + gid * S::kQRow + k * 32 + tig * 8;
          xa[k] = inA ? *reinterpret_cast<const uint2*>(pa) : make_uint2(0, 0);
          xb[k] = inB ? *reinterpret_cast<const uint2*>(pa + 8 * S::kQRow) : make_uint2(0, 0);
        }
        if (std::is_same<T, __nv_bfloat16>::value) {
          // in fp16, the largest value brought to [1, 2): exact down to 2^-14 of it, 2^-25 of it below
          float bigA = 0.f, bigB = 0.f;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const float2 u = unpack2<T>(xa[k].x), v = unpack2<T>(xa[k].y), w = unpack2<T>(xb[k].x), z = unpack2<T>(xb[k].y);
            bigA = fmaxf(fmaxf(bigA, fmaxf(fabsf(u.x), fabsf(u.y))), fmaxf(fabsf(v.x), fabsf(v.y)));
            bigB = fmaxf(fmaxf(bigB, fmaxf(fabsf(w.x), fabsf(w.y))), fmaxf(fabsf(z.x), fabsf(z.y)));
          }
#pragma unroll
          for (int d = 1; d < 4; d <<= 1) {
            bigA = fmaxf(bigA, __shfl_xor_sync(0xffffffffu, bigA, d));
            bigB = fmaxf(bigB, __shfl_xor_sync(0xffffffffu, bigB, d));
          }
          // (the exponents at the type's ends, subnormals' and the highest, take the power beside theirs: both factors are normal)
          auto row_exponent = [](float big) { return min(max(__float_as_uint(big) >> 23, 1u), 253u); };
          const uint32_t eA = row_exponent(bigA), eB = row_exponent(bigB);
          upA *= __uint_as_float((254u - eA) << 23);
          upB *= __uint_as_float((254u - eB) << 23);
          cA = factor(eA);
          cB = factor(eB);
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const float2 u = unpack2<T>(xa[k].x), v = unpack2<T>(xa[k].y), w = unpack2<T>(xb[k].x), z = unpack2<T>(xb[k].y);
          qf[k][0] = pack2<__half>(u.x * upA, u.y * upA);
          qf[k][2] = pack2<__half>(v.x * upA, v.y * upA);
          qf[k][1] = pack2<__half>(w.x * upB, w.y * upB);
          qf[k][3] = pack2<__half>(z.x * upB, z.y * upB);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(q_empty + qb);
    ++parts;

    // One tile: its K and V units, and its tokens [j0, j1) that are seen. Whole tiles take the instance without masks.
    auto step = [&](auto masked, int k_slot, int v_slot, uint32_t v_phase, int j0, int j1) {
      constexpr bool MASK = decltype(masked)::value;
      const float* k_sc = reinterpret_cast<const float*>(sm + S::oScale + k_slot * S::kScaleBytes);
      const float* v_sc = reinterpret_cast<const float*>(sm + S::oScale + v_slot * S::kScaleBytes);
#pragma unroll 1
      for (int sub = 0; sub < NB / NBS; ++sub) {
        // S = Q K^T
        float s[NBS][2][4];
#pragma unroll
        for (int b = 0; b < NBS; ++b) {
          const int key = ((sub * NBS + b) * KP + kp) * 16;
          if (MASK && !(key + 16 > j0 && key < j1)) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[b][n][e] = 0.f;
            continue;
          }
          const uint32_t base = lane_k + k_slot * S::kUnit + block_at(key);
          if (!I8) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              uint32_t f[4];
              ldsm4(f, piece(base, k));
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                if (k == 0) mma16816<M, true>(s[b][n], qf[k], f[2 * n], f[2 * n + 1]);
                else mma16816<M>(s[b][n], qf[k], f[2 * n], f[2 * n + 1]);
              }
            }
          } else {
#pragma unroll
            for (int k = 0; k < D / 16; k += 2) {
              uint32_t f[4];
              ldsm4(f, piece(base, k / 2));
#pragma unroll
              for (int e = 0; e < 4; ++e) f[e] ^= 0x80808080u;
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const uint32_t e0 = i8_pair<0x4140>(f[2 * n]), e1 = i8_pair<0x4342>(f[2 * n]);
                const uint32_t d0 = i8_pair<0x4140>(f[2 * n + 1]), d1 = i8_pair<0x4342>(f[2 * n + 1]);
                if (k == 0) mma16816<M, true>(s[b][n], qf[k], e0, e1);
                else mma16816<M>(s[b][n], qf[k], e0, e1);
                mma16816<M>(s[b][n], qf[k + 1], d0, d1);
              }
            }
          }
        }
        if (sub == 0 && two) {
          ok = wait_warp(full + v_slot, v_phase, abort_flag, a.err);
          if (!ok) return;
        }
        float nA = -INFINITY, nB = -INFINITY;
        float2 sv[NBS][2];  // 8 bits: V's row scales
#pragma unroll
        for (int b = 0; b < NBS; ++b)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int key = ((sub * NBS + b) * KP + kp) * 16 + n * 8 + 2 * tig;
            if (I8) {
              const float2 sk = *reinterpret_cast<const float2*>(k_sc + key);
              sv[b][n] = *reinterpret_cast<const float2*>(v_sc + key);
              s[b][n][0] *= sk.x;
              s[b][n][1] *= sk.y;
              if (!R8) {
                s[b][n][2] *= sk.x;
                s[b][n][3] *= sk.y;
              }
            }
            if (MASK) {  // tokens that are not seen are out
              if (key < j0 || key >= j1) {
                s[b][n][0] = s[b][n][2] = -INFINITY;
                if (I8) sv[b][n].x = 0.f;
              }
              if (key + 1 < j0 || key + 1 >= j1) {
                s[b][n][1] = s[b][n][3] = -INFINITY;
                if (I8) sv[b][n].y = 0.f;
              }
            }
            nA = fmaxf(nA, fmaxf(s[b][n][0], s[b][n][1]));
            if (!R8) nB = fmaxf(nB, fmaxf(s[b][n][2], s[b][n][3]));
          }
        // (rounded before the base is taken off, as the base was: a rest of the product's bits would be far above 0 in a large one)
        auto logit = [](float s, float c) { return __fmul_rn(s, c); };
        nA = logit(nA, cA);
        if (!R8) nB = logit(nB, cB);
        // 8 bits: the magnitude of one token's V scale in each lane, as bits plus x (not seen: 0), and whether it is outside
        auto size_and = [&](uint32_t x) -> uint32_t {
          const int key = ((sub * NBS + (NBS == 2 ? lane >> 4 : 0)) * KP + kp) * 16 + (lane & 15);
          return !MASK || (key >= j0 && key < j1) ? (__float_as_uint(v_sc[key]) & 0x7fffffffu) + x : 0u;
        };
        auto is_outside = [&]() { return size_and(__float_as_uint(mulA) - (251u << 23)) > 11u << 23; };  // (less the bits of hi / 2^11)
        const bool outside = I8 && is_outside();
        // The exponents' base follows the running maximum only when a logit passes it by more than kGrow: most steps then need
        // neither shuffles nor a rescaling.
        if (__any_sync(0xffffffffu, nA > mA + kGrow || (!R8 && nB > mB + kGrow) || outside)) {
#pragma unroll
          for (int d = 1; d < 4; d <<= 1) {
            nA = fmaxf(nA, __shfl_xor_sync(0xffffffffu, nA, d));
            if (!R8) nB = fmaxf(nB, __shfl_xor_sync(0xffffffffu, nB, d));
          }
          nA = fmaxf(nA, mA);
          nB = fmaxf(nB, mB);
          const float fA = nA == mA ? 1.f : ex2(mA - nA), fB = R8 ? fA : nB == mB ? 1.f : ex2(mB - nB);
          const float upA = mA - nA, upB = mB - nB;
          mA = nA;
          mB = nB;
          float gA = fA, gB = fB;
          if (kOnesSum) {
            ls[0] *= fA;
            ls[2] *= fB;
          } else {
            lA *= fA;
            if (!R8) lB *= fB;
          }
          if (I8) {
            const int top = (int)(__reduce_max_sync(0xffffffffu, size_and(0u)) >> 23);
            if (mulA == 0.f) mulA = mulB = power(262 - min(max(top + 4, 12), 254));
            if (__any_sync(0xffffffffu, is_outside())) {
              // far: the row's largest weight times V scale becomes 2^7 to 2^8, unless what was summed so far holds a larger one, and
              // a scale times mul stays finite (its weight may be zero)
              const float subA = mA == -INFINITY ? 0.f : mA, subB = mB == -INFINITY ? 0.f : mB;
              float xA = 0.f, xB = 0.f;
#pragma unroll
              for (int b = 0; b < NBS; ++b)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    const float v = i ? sv[b][n].y : sv[b][n].x;
                    xA = fmaxf(xA, fabsf(ex2(logit(s[b][n][i], cA) - subA) * v));
                    if (!R8) xB = fmaxf(xB, fabsf(ex2(logit(s[b][n][2 + i], cB) - subB) * v));
                  }
              auto follow = [&](float x, float f, float up, float& mul) {
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                const int was = exponent(mul), held = f == 1.f ? was : exponent(fabsf(mul) * ex2(-up));
                const int e = min(max(min(min(held, 261 - exponent(x)), 379 - top), 8), 250);
                mul = power(e);
                return f == 1.f ? power(127 + max(e - was, -127)) : ex2(up + (float)(e - was));
              };
              gA = follow(xA, fA, upA, mulA);
              mulA = -mulA;
              if (!R8) gB = follow(xB, fB, upB, mulB);
            }
          }
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            o[j][0] *= gA;
            o[j][1] *= gA;
            o[j][2] *= gB;
            o[j][3] *= gB;
          }
        }
        // (a base of -infinity is left out of the exponent: nothing was seen yet, or every logit is -infinity)
        const float subA = kShift - (mA == -INFINITY ? 0.f : mA), subB = kShift - (mB == -INFINITY ? 0.f : mB);
#pragma unroll
        for (int b = 0; b < NBS; ++b) {
          const int key0 = ((sub * NBS + b) * KP + kp) * 16;
          if (MASK && !(key0 + 16 > j0 && key0 < j1)) continue;
          uint32_t hi[4], lw[4];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float pA0 = ex2(logit(s[b][n][0], cA) + subA), pA1 = ex2(logit(s[b][n][1], cA) + subA), pB0 = 0.f, pB1 = 0.f;
            if (!R8) {
              pB0 = ex2(logit(s[b][n][2], cB) + subB);
              pB1 = ex2(logit(s[b][n][3], cB) + subB);
            }
            if (!kOnesSum) {
              lA += pA0 + pA1;
              if (!R8) lB += pB0 + pB1;
            }
            if (I8) {
              pA0 *= sv[b][n].x * fabsf(mulA);
              pA1 *= sv[b][n].y * fabsf(mulA);
              if (!R8) {
                pB0 *= sv[b][n].x * mulB;
                pB1 *= sv[b][n].y * mulB;
              }
            }
            const uint32_t hA = pack2<M>(pA0, pA1);
            const float2 fA = unpack2<M>(hA);
            const uint32_t dA = pack2<M>(pA0 - fA.x, pA1 - fA.y);
            hi[2 * n] = hA;
            if (R8) {
              hi[2 * n + 1] = dA;
            } else {
              const uint32_t hB = pack2<M>(pB0, pB1);
              const float2 fB = unpack2<M>(hB);
              hi[2 * n + 1] = hB;
              lw[2 * n] = dA;
              lw[2 * n + 1] = pack2<M>(pB0 - fB.x, pB1 - fB.y);
            }
          }
          if (kOnesSum) {
            mma16816<M>(ls, hi, kOnes, kOnes);
            if (!R8) mma16816<M>(ls, lw, kOnes, kOnes);
          }
          // rows of V that are not seen may hold anything: their bits are cleared (0 times an infinity is no number)
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
          if (!I8 && MASK) {
            const int key = key0 + 2 * tig;
            keep0 = (key >= j0 && key < j1 ? 0xffffu : 0u) | (key + 1 >= j0 && key + 1 < j1 ? 0xffff0000u : 0u);
            keep1 = (key + 8 >= j0 && key + 8 < j1 ? 0xffffu : 0u) | (key + 9 >= j0 && key + 9 < j1 ? 0xffff0000u : 0u);
          }
          const uint32_t base = lane_v + v_slot * S::kUnit + block_at(key0);
          if (!I8) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t f[4];
              ldsm4_trans(f, piece(base, c));
              if (MASK) {
                f[0] &= keep0;
                f[1] &= keep1;
                f[2] &= keep0;
                f[3] &= keep1;
              }
              mma16816<M>(o[2 * c], hi, f[0], f[1]);
              mma16816<M>(o[2 * c + 1], hi, f[2], f[3]);
              if (!R8) {
                mma16816<M>(o[2 * c], lw, f[0], f[1]);
                mma16816<M>(o[2 * c + 1], lw, f[2], f[3]);
              }
            }
          } else {
            // a loaded pair of bytes is two dims of one token: the even and the odd dims of 16 form one n-tile each
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t f[4];
              ldsm4_trans(f, piece(base, c));
#pragma unroll
              for (int e = 0; e < 4; ++e) f[e] ^= 0x80808080u;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t e0 = i8_pair<0x4240>(f[2 * e]), e1 = i8_pair<0x4240>(f[2 * e + 1]);
                const uint32_t d0 = i8_pair<0x4341>(f[2 * e]), d1 = i8_pair<0x4341>(f[2 * e + 1]);
                mma16816<M>(o[4 * c + 2 * e], hi, e0, e1);
                mma16816<M>(o[4 * c + 2 * e + 1], hi, d0, d1);
                if (!R8) {
                  mma16816<M>(o[4 * c + 2 * e], lw, e0, e1);
                  mma16816<M>(o[4 * c + 2 * e + 1], lw, d0, d1);
                }
              }
            }
          }
        }
      }
    };
    for (int i = 0; i < n_tiles; ++i) {
      ok = wait_warp(full + ks, phase, abort_flag, a.err);
      if (!ok) return;
      const int v_slot = two ? (ks + 1 == RING ? 0 : ks + 1) : ks;
      const uint32_t v_phase = v_slot < ks ? phase ^ 1 : phase;
      const int k0 = pt.k0 + i * TK;
      if (D < 128 && k0 >= pt.lo && k0 + TK <= pt.len) step(std::false_type(), ks, v_slot, v_phase, 0, TK);
      else step(std::true_type(), ks, v_slot, v_phase, max(pt.lo - k0, 0), min(pt.len - k0, TK));
      if (!ok) return;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(empty + ks);
        if (two) mbar_arrive(empty + v_slot);
      }
      phase = v_slot + 1 == RING ? v_phase ^ 1 : v_phase;
      ks = v_slot + 1 == RING ? 0 : v_slot + 1;
    }

    // ---- the part's end: the warps' (m, l, o) to shared memory, and summed ----
    if (!kOnesSum) {
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        lA += __shfl_xor_sync(0xffffffffu, lA, d);
        if (!R8) lB += __shfl_xor_sync(0xffffffffu, lB, d);
      }
    } else {
      lA = R8 ? ls[0] + ls[2] : ls[0];
      lB = ls[2];
    }
    const float o_mulA = I8 ? power(254 - exponent(mulA)) : 1.f, o_mulB = I8 ? power(254 - exponent(mulB)) : 1.f;  // (1 / mul)
    // values c .. c + 3 of query row g of a (request, head), all tokens joined: the output; or so far: to a place of the
    // workspace
    auto finish = [&](const Part& of, int g, int c, float m, float l, const float* acc) {
      const int qh = of.h * G + g;
      T* dst = static_cast<T*>(a.out) + (int64_t)of.r * a.out_stride + (int64_t)qh * D + c;
      const float inv = 1.f / l;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(acc[0] * inv, acc[1] * inv), pack2<T>(acc[2] * inv, acc[3] * inv));
      if (c == 0 && a.lse) a.lse[(int64_t)of.r * a.q_heads + qh] = (m == -INFINITY ? 0.f : m) * kLn2 + logf(l * (kF16 ? 0x1p-8f : 1.f));
    };
    auto keep = [&](int to, int g, int c, float m, float l, const float* acc) {
      __stcg(reinterpret_cast<float4*>(a.part_o + ((int64_t)to * G + g) * D + c), make_float4(acc[0], acc[1], acc[2], acc[3]));
      if (c == 0) __stcg(reinterpret_cast<float2*>(a.part_ml) + (int64_t)to * G + g, make_float2(m, l));
    };
    const int part = (int)blockIdx.x - pt.i0, place = part_place(pt.i0, part);
    constexpr int kPerRow = D / 4;  // 4 values per thread
    {
      if (S::kOAreas == 1) {
        consumer_sync();  // (the previous part has been read; with two areas the part between has said so)
        if (!ok) return;
      }
      float* const s_o = reinterpret_cast<float*>(sm + S::oO + (S::kOAreas == 1 ? 0 : (areas & 1)) * S::kOBytes);
      float* const s_m = s_o + kConsumers * S::kORows * S::kORow;
      float* const s_l = s_m + kConsumers * S::kORows;
      ++areas;
#pragma unroll
      for (int half = 0; half < S::kORows / 8; ++half) {
        const bool upper = half != 0;
        if (mt * 16 + upper * 8 + gid >= G) continue;
        const int row = warp * S::kORows + half * 8 + gid;
        const float o_mul = upper ? o_mulB : o_mulA;
        float* dst = s_o + row * S::kORow;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const float x = (R8 ? o[j][0] + o[j][2] : upper ? o[j][2] : o[j][0]) * o_mul;
          const float y = (R8 ? o[j][1] + o[j][3] : upper ? o[j][3] : o[j][1]) * o_mul;
          if (!I8) {
            *reinterpret_cast<float2*>(dst + j * 8 + 2 * tig) = make_float2(x, y);
          } else if (j & 1) {
            // (even dims from the tile before: dims 4 tig .. 4 tig + 3 of the 16)
            const float u = (R8 ? o[j - 1][0] + o[j - 1][2] : upper ? o[j - 1][2] : o[j - 1][0]) * o_mul;
            const float v = (R8 ? o[j - 1][1] + o[j - 1][3] : upper ? o[j - 1][3] : o[j - 1][1]) * o_mul;
            *reinterpret_cast<float4*>(dst + (j >> 1) * 16 + 4 * tig) = make_float4(u, x, v, y);
          }
        }
        if (tig == 0) {
          s_m[row] = upper ? mB : mA;
          s_l[row] = upper ? lB : lA;
        }
      }
      consumer_sync();
      if (!ok) return;
      // (rows behind the last head are summed too, so that the loop's rounds run together, and left out)
      constexpr int kItems = S::kORows * MT * kPerRow, kRounds = (kItems + kConsumers * 32 - 1) / (kConsumers * 32);
#pragma unroll (kRounds < 4 ? kRounds : 4)
      for (int i = 0; i < kRounds; ++i) {
        const int x = tid + i * kConsumers * 32;
        if (kItems % (kConsumers * 32) != 0 && x >= kItems) break;
        const int rx = x / kPerRow, c = (x - rx * kPerRow) * 4;
        const int rt = rx / S::kORows, rr = rx % S::kORows, g = rt * 16 + rr;
        float top = -INFINITY;
#pragma unroll
        for (int p = 0; p < KP; ++p) top = fmaxf(top, s_m[(p * MT + rt) * S::kORows + rr]);
        const float base = top == -INFINITY ? 0.f : top;
        float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < KP; ++p) {
          const int w = (p * MT + rt) * S::kORows + rr;
          const float f = ex2(s_m[w] - base);
          l += f * s_l[w];
          const float4 v = *reinterpret_cast<const float4*>(s_o + w * S::kORow + c);
          acc[0] += f * v.x;
          acc[1] += f * v.y;
          acc[2] += f * v.z;
          acc[3] += f * v.w;
        }
        if (g >= G) continue;
        if (pt.n_parts == 1) finish(pt, g, c, top, l, acc);
        else keep(place, g, c, top, l, acc);
      }
    }

    // ---- joining: the last of a group of 16 parts to get here joins the group, the last group's joiner the groups ----
    // A release by one thread after the warps' meeting covers what all of them wrote.
    if (pt.n_parts > 1 && !last) {
      // (not the run's last part: counted now, looked at when the run is through)
      consumer_sync();
      if (!ok) return;
      early = true;
      if (tid == 0) s_part[2] = pt;
      if (tid == 0) early_count = add_acq_rel(a.count + part_place(pt.i0, part / kGroup * kGroup));
    }
    if (!last) continue;
    // This part and the early one; of each its group of parts, then the groups. A count is of what precedes the own.
#pragma unroll 1
    for (int k = early ? 3 : 1; k >= 0; --k) {
      const bool groups = !(k & 1);
      const Part of = k >> 1 ? s_part[2] : pt;
      const int g0 = groups ? 0 : ((int)blockIdx.x - of.i0) / kGroup * kGroup;
      const int n_groups = (of.n_parts + kGroup - 1) / kGroup;
      const int n = groups ? n_groups : min(kGroup, of.n_parts - g0), every = groups ? kGroup : 1;
      if (of.n_parts == 1 || (groups && n_groups == 1)) continue;
      unsigned* const count = a.count + (groups ? a.n_places : 0) + part_place(of.i0, g0);
      consumer_sync();
      if (ok && tid == 0) {
        const bool is_last = (k == 3 ? early_count : add_acq_rel(count)) == (unsigned)(n - 1);
        if (is_last) *count = 0u;  // ready for the next call
        *s_last = is_last;
      }
      consumer_sync();
      if (!ok) return;
      if (!*s_last) {
        if (!groups) --k;  // (another CTA joins this group, and sees to the groups)
        continue;
      }
      // parts g0, g0 + every, .. (n of them): a thread joins 4 values of a row at a time, kInFlight loads in flight: of that
      // many parts, or of 4 parts for several rows where there are no more
      constexpr int kInFlight = D == 128 ? 16 : 8;
      auto join = [&](auto parts_at_once) {
        constexpr int NP = decltype(parts_at_once)::value, NX = kInFlight / NP;
        for (int x0 = warp * 32; x0 < G * kPerRow; x0 += NX * kConsumers * 32) {
          float m[NX], l[NX], acc[NX][4];
#pragma unroll
          for (int i = 0; i < NX; ++i) {
            m[i] = -INFINITY;
            l[i] = acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
          }
          for (int b = 0; b < n; b += NP) {
            float2 ml[NX][NP];
            float4 v[NX][NP];
#pragma unroll
            for (int i = 0; i < NX; ++i)
#pragma unroll
              for (int u = 0; u < NP; ++u) {
                const int x = min(x0 + i * kConsumers * 32 + lane, G * kPerRow - 1), g = x / kPerRow;
                const int64_t from = (int64_t)part_place(of.i0, g0 + min(b + u, n - 1) * every) * G + g;
                ml[i][u] = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + from);
                v[i][u] = __ldcg(reinterpret_cast<const float4*>(a.part_o + from * D + (x - g * kPerRow) * 4));
              }
#pragma unroll
            for (int i = 0; i < NX; ++i) {
              float top = m[i];
#pragma unroll
              for (int u = 0; u < NP; ++u) top = fmaxf(top, ml[i][u].x);
              const float base = top == -INFINITY ? 0.f : top, f = ex2(m[i] - base);
              l[i] *= f;
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][e] *= f;
#pragma unroll
              for (int u = 0; u < NP; ++u)
                if (b + u < n) {
                  const float w = ex2(ml[i][u].x - base);
                  l[i] += w * ml[i][u].y;
                  acc[i][0] += w * v[i][u].x;
                  acc[i][1] += w * v[i][u].y;
                  acc[i][2] += w * v[i][u].z;
                  acc[i][3] += w * v[i][u].w;
                }
              m[i] = top;
            }
          }
          __syncwarp();  // (a row's lanes, one warp, have read the first part, whose place the group's sum takes)
#pragma unroll
          for (int i = 0; i < NX; ++i) {
            const int x = x0 + i * kConsumers * 32 + lane, g = x / kPerRow, c = (x - g * kPerRow) * 4;
            if (x >= G * kPerRow) continue;
            if (groups || n_groups == 1) finish(of, g, c, m[i], l[i], acc[i]);
            else keep(part_place(of.i0, g0), g, c, m[i], l[i], acc[i]);
          }
        }
      };
      if (n <= 4) join(std::integral_constant<int, 4>());
      else join(std::integral_constant<int, kInFlight>());
    }
  }
}

// The instance for a configuration: its kernel, shared memory, CTAs per SM and tile.
template <int D>
KvAttendKernel instance(int dtype, bool int8, int group) {
  const int mode = group <= 8 ? 0 : group <= 16 ? 1 : group <= 32 ? 2 : 3;
  auto of = [&](auto t, auto i8, auto m) {
    typedef decltype(t) T;
    typedef Shape<decltype(i8)::value, D, decltype(m)::value> S;
    return KvAttendKernel{reinterpret_cast<const void*>(&attend_kernel<T, decltype(i8)::value, D, decltype(m)::value>), S::kSmem,
                          S::kCtasPerSm, S::TK};
  };
  auto by_mode = [&](auto t, auto i8) {
    if (mode == 0) return of(t, i8, std::integral_constant<int, 0>());
    if (mode == 1) return of(t, i8, std::integral_constant<int, 1>());
    if (mode == 2) return of(t, i8, std::integral_constant<int, 2>());
    return of(t, i8, std::integral_constant<int, 3>());
  };
  if (dtype == CVR_DTYPE_BF16) return int8 ? by_mode(__nv_bfloat16(), std::true_type()) : by_mode(__nv_bfloat16(), std::false_type());
  return int8 ? by_mode(__half(), std::true_type()) : by_mode(__half(), std::false_type());
}

}  // namespace kv
}  // namespace cvr
