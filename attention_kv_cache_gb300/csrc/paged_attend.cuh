// Attention of one new query row per head over a request's rows in the paged pool.
//
// z_t = scale <q, k_t> (capped, biased), o = sum_t softmax(z)_t v_t over the visible rows t of a request;
// the G query heads of a KV head share its rows, so K and V are read once for all of them.
//
// Bound: the bytes of K and V (4 to 16 flop per byte).  The work is cut into steps of 32 consecutive rows
// of one request; the steps of all requests, laid end to end, are dealt evenly to `lanes`, and a lane is
// one warp per (KV head, tile of query heads), so every warp of one resident wave has the same number of
// steps whatever the lengths are.  A warp walks its steps with three of them in shared memory or in flight;
// lane r of the warp owns row r of a step: it finds the row's page and its visibility.
//
// Arithmetic: the step's rows are the M side of mma.sync m16n8k16 and 8 query heads the N side, so
// S^T = K Q^T needs no padding at G = 8; P^T moves from the accumulator to the B operand by movmatrix, and
// O^T += V^T P^T with V transposed by ldmatrix.  P is taken as a high and a low 16-bit part.  The softmax
// keeps an exponent offset that moves only when a score passes it by 2^lag, so the common step forms no
// maximum, and the sums stay in the lanes until a row ends.
// The parts are of weights times a power of two, which O is divided by at the end.  An fp16 part is a multiple of 2^-24, so of
// weights near 1 those below 2^-25 would be left out of O while their sum counts them: a long tail behind one high score
// would be lost.  Over fp16 products the factor is 2^13 and the lag 2: weights end at 2^15, inside fp16, and what is lost of
// one is below 2^-38 of the largest.  bf16 parts have fp32's exponents, and values up to fp32's largest: a lag of 8 and a
// factor of 2^-8, so that none is above one.  (The factor taken by the offset instead would round every distance at 13 or 8.)
//
// A request cut between lanes leaves one partial (O, offset, sum) per piece, which paged_join merges; a request within
// one lane is written at once.
//
// A call whose tables hold few rows is a CTA per (request, unit) instead: its warps share the request's steps and merge
// their parts in shared memory, one launch and no partials.  (A CTA holds an SM whatever its request's length, so the
// tables' size and not the lengths decide: see geometry().)
//
// Stages: 192 KB of an SM's shared memory, four warps of three 16 KB steps (16-bit pools, d = 128) or eight of 8 KB.  At
// 128 KB in flight a read of the whole cache runs at the copy rate; three or six warps lose 5-15 %, twelve warps of two
// stages 8 %.  cp.async by all lanes, rows without a source zero-filled, rather than boxes of a tensor map: the boxes
// took 2-4 % longer, and left V rows that are not seen to be cleared by hand.
//
// Measured (GB300, device time, join included): 32 requests of 2048-65536 rows, 8 KV heads of 128, bf16, 642 us (4430 MB,
// 6.9 TB/s); 1 x 131072 rows 86 us (537 MB, 6.3 TB/s); 256 requests of 1-4095 rows, e4m3, capped, window 2048, 137 us
// (813 MB, 5.9 TB/s; 566 instructions per step of 8 KB against 523 of 16 KB); 1 x 517 rows 5.5 us (by lanes
// 7.2), 16 x 800 rows 13.3 us (17.3).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "paged.cuh"
#include "sm100.cuh"

namespace kvsel {

constexpr int kKeys = 32;             // rows per step: one per lane
constexpr int kSoloSteps = 8;         // steps per warp of a short call at most
constexpr float kLog2e = 1.4426950408889634f;
enum Kind { kBf16 = 0, kF16 = 1, kE4m3 = 2 };

struct PagedArgs {
  const void *q, *k, *v;
  const int32_t* tables;
  const int64_t* lens;
  const float *slopes, *k_scale, *v_scale;
  void* o;
  float* lse;
  float* part;          // [2 * lanes][h_kv * tiles * 8 * NT][d]: partial O
  float2* part_ml;      // [2 * lanes][h_kv * tiles * 8 * NT]: its offset (base 2) and sum
  // What paged_join merges: of every request its first and last lane, or (more requests than lanes, by_lane) of every
  // lane the request that begins in it and goes on, and that request's last lane.  First >= last: nothing.
  int2* span;
  DeviceError* err;
  int64_t page_stride, head_stride, row_stride, q_stride;
  float scale, softcap;
  float unit;           // weight_unit() of the kernel (for paged_join)
  int32_t h_q, h_kv, G, P, batch, max_blocks, n_pages, window, out_f16;
  uint32_t p_mul, p_shift;   // division of a row below 2^31 by P: (mulhi(p_mul, t) + t) >> p_shift
  int32_t tiles;        // tiles of query heads per KV head
  int32_t lanes;        // lanes the grid can hold
  int32_t by_lane;
  int32_t solo;         // a CTA per request and unit (no lanes, no join)
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tanh from its definition, 1 - 2 / (1 + e^2x), off by at most 2^-21 (absolute: 2^-22 relative of ex2, an ulp of rcp and
// the roundings, each weighted by its share), and where that cancels (|x| < 1/4) from its odd series to x^7, within 2^-20 of
// the value.
__device__ __forceinline__ float tanh_fast(float x) {
  const float x2 = x * x;
  const float small = x * fmaf(x2, fmaf(x2, fmaf(x2, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(x * 2.885390081777927f)));
  return x2 < 0.0625f ? small : fmaf(-2.f, r, 1.f);
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const uint32_t n = valid ? 16u : 0u;          // 0 source bytes: the destination is zero-filled
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int KIND>
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (KIND == kBf16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (a, b) as two 16-bit values of the products' type, and what they leave of a and b
template <int KIND>
__device__ __forceinline__ uint32_t pack_hi(float a, float b, float& ra, float& rb) {
  if constexpr (KIND == kBf16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    ra = a - __low2float(p);
    rb = b - __high2float(p);
    return *reinterpret_cast<const uint32_t*>(&p);
  } else {
    const __half2 p = __floats2half2_rn(a, b);
    ra = a - __low2float(p);
    rb = b - __high2float(p);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
}
// four e4m3 values as fp16, exactly: the low two and the high two
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(x));
}

// Binary orders that a score may pass the offset by before it moves, and the factor on the weights that are split.
template <int KIND>
__host__ __device__ constexpr float weight_lag() { return KIND == kBf16 ? 8.f : 2.f; }
template <int KIND>
__host__ __device__ constexpr float weight_unit() { return KIND == kBf16 ? 0x1p-8f : 0x1p13f; }

template <int KIND>
__host__ __device__ constexpr int elem_bytes() { return KIND == kE4m3 ? 1 : 2; }
template <int D, int KIND>
__host__ __device__ constexpr int row_bytes() { return D * elem_bytes<KIND>(); }
template <int D, int KIND>
__host__ __device__ constexpr int stage_bytes() { return 2 * kKeys * row_bytes<D, KIND>(); }   // K, then V
// Warps per CTA and stages per warp: one CTA per SM, 190 KB of stages.
template <int D, int KIND>
__host__ __device__ constexpr int n_warps() { return stage_bytes<D, KIND>() >= 16384 ? 4 : 8; }
template <int D, int KIND>
__host__ __device__ constexpr int n_stages() { return 196608 / (n_warps<D, KIND>() * stage_bytes<D, KIND>()); }
template <int D, int KIND>
__host__ __device__ constexpr int smem_bytes(int batch) {
  return 1024 + n_warps<D, KIND>() * n_stages<D, KIND>() * stage_bytes<D, KIND>() + 8 * (batch + 1);
}

// Byte offset of 16-byte chunk c of row x: halves of 128-byte rows one after another, chunks of eight rows
// spread over the banks.
template <int RB>
__device__ __forceinline__ uint32_t chunk_at(int x, int c) {
  if constexpr (RB >= 128) return (uint32_t)((c >> 3) * (kKeys * 128) + x * 128 + (((c & 7) ^ (x & 7)) << 4));
  else return (uint32_t)(x * 64 + ((c ^ ((x >> 1) & 3)) << 4));
}
// From the address `at` of chunk c0 of a row (c0 below 2), the address of its chunk c0 + c of the row 16 mt rows on, for even c.
template <int RB>
__device__ __forceinline__ uint32_t chunk_from(uint32_t at, int mt, int c) {
  if constexpr (RB >= 128) return (at ^ (uint32_t)((c & 7) << 4)) + (c >> 3) * (kKeys * 128) + mt * 16 * 128;
  else return (at ^ (uint32_t)(c << 4)) + mt * 16 * 64;
}

// two output values in the output's type
__device__ __forceinline__ uint32_t pack_out(const PagedArgs& a, float u, float v) {
  if (a.out_f16) {
    const __half2 y = __floats2half2_rn(u, v);
    return *reinterpret_cast<const uint32_t*>(&y);
  }
  const __nv_bfloat162 y = __floats2bfloat162_rn(u, v);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// First visible row of a request of n rows.
__device__ __forceinline__ int first_row(int n, int window) { return window > 0 && n > window ? n - window : 0; }
// Steps of a request of n rows (n may be 2^31 - 2: what is added to it is not 32-bit signed).
__device__ __forceinline__ int steps_of(int n, int window) {
  return (int)(((uint32_t)n + kKeys - 1) / kKeys) - first_row(n, window) / kKeys;
}
// First step of lane i of N over T steps.
__device__ __forceinline__ int quotient(uint64_t x, int y) { return (x >> 32) == 0 ? (int)((uint32_t)x / (uint32_t)y) : (int)(x / y); }
__device__ __forceinline__ int lane_begin(int i, int T, int N) { return quotient((uint64_t)i * T, N); }
// The lane that holds step x.
__device__ __forceinline__ int lane_of(int x, int T, int N) { return quotient((uint64_t)(x + 1) * N + T - 1, T) - 1; }

// cum[b] = (steps of the requests before b, rows of b), in shared memory; returns all steps.  Every CTA forms it.
template <int THREADS>
__device__ int step_sums(const PagedArgs& a, int2* cum) {
  __shared__ int32_t warp_sum[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.batch + THREADS - 1) / THREADS;
  const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
  const int64_t cap = (int64_t)a.max_blocks * a.P;
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    int64_t L = a.lens[b];
    if (L < 0 || L > cap) {
      if (blockIdx.x == 0) set_device_error(a.err, KVSEL_ERR_INVALID_ARG, (uint32_t)b);
      L = 0;
    }
    const int n = (int)L;
    const int steps = steps_of(n, a.window);
    cum[b] = make_int2(steps, n);
    sum += steps;
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int base = 0, total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) base = total;
    total += warp_sum[w];
  }
  int at = base + inc - sum;
  for (int b = b0; b < b1; ++b) {
    const int s = cum[b].x;
    cum[b].x = at;
    at += s;
  }
  if (tid == 0) cum[a.batch] = make_int2(total, 0);
  __syncthreads();
  return total;
}

// The same for request b alone.
template <int THREADS>
__device__ int one_request(const PagedArgs& a, int b, int2* cum) {
  int64_t L = a.lens[b];
  if (L < 0 || L > (int64_t)a.max_blocks * a.P) {
    if (threadIdx.x == 0) set_device_error(a.err, KVSEL_ERR_INVALID_ARG, (uint32_t)b);
    L = 0;
  }
  const int n = (int)L;
  const int steps = steps_of(n, a.window);
  if (threadIdx.x == 0) {
    cum[0] = make_int2(0, n);
    cum[1] = make_int2(steps, 0);
  }
  __syncthreads();
  return steps;
}

__device__ __forceinline__ int find_request(const int2* cum, int batch, int x) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid].x <= x) lo = mid; else hi = mid;
  }
  return lo;
}

template <int D, int KIND, int NT>
__global__ void __launch_bounds__(32 * n_warps<D, KIND>(), 1) paged_attend(const __grid_constant__ PagedArgs a) {
  constexpr int W = n_warps<D, KIND>(), NS = n_stages<D, KIND>(), RB = row_bytes<D, KIND>();
  constexpr int KV = kKeys * RB;                    // bytes of a step's K (or V)
  constexpr int CPR = RB / 16;                      // 16-byte chunks per row
  constexpr int KS = D / 16;                        // 16-wide slices of the head dim
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int2* cum = reinterpret_cast<int2*>(sbase + W * NS * stage_bytes<D, KIND>());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;
  const uint32_t st0 = sm100::smem_addr(sbase) + warp * NS * stage_bytes<D, KIND>();
  // the rows and chunks that this lane addresses for ldmatrix
  const uint32_t k_lane = chunk_at<RB>(lane & 15, lane >> 4);
  const uint32_t v_lane = KIND == kE4m3 ? k_lane : chunk_at<RB>(((lane >> 4) << 3) + (lane & 7), (lane >> 3) & 1);

  wait_for_earlier_kernels();
  const int units = a.h_kv * a.tiles;
  // A short call is a CTA per (request, unit), which knows its one request alone; requests are counted from b0.
  const bool solo = a.solo != 0;
  const int b0 = solo ? blockIdx.x / units : 0;
  const int batch = solo ? 1 : a.batch;
  int T, N = 1;
  if (solo) {
    T = one_request<32 * W>(a, b0, cum);
  } else {
    let_later_kernels_start();                      // (paged_join: it waits for this grid's end)
    T = step_sums<32 * W>(a, cum);
    N = max(1, min(a.lanes, T));
  }
  if (a.by_lane && blockIdx.x == 0)                 // lanes without a step
    for (int i = threadIdx.x; i < a.lanes; i += 32 * W)
      if (i >= N || lane_begin(i, T, N) == lane_begin(i + 1, T, N)) a.span[i] = make_int2(0, -1);
  // requests without a row: o = 0, lse = -inf
  for (int b = blockIdx.x; b < a.batch && !solo; b += gridDim.x) {
    if (cum[b].x != cum[b + 1].x) continue;
    uint32_t* ob = reinterpret_cast<uint32_t*>(a.o) + (int64_t)b * a.h_q * (D / 2);
    for (int x = threadIdx.x; x < a.h_q * (D / 2); x += 32 * W) ob[x] = 0u;
    if (a.lse != nullptr)
      for (int x = threadIdx.x; x < a.h_q; x += 32 * W) a.lse[(int64_t)b * a.h_q + x] = -INFINITY;
    if (!a.by_lane && threadIdx.x == 0) a.span[b] = make_int2(0, -1);
  }
  const int heads_pad = units * 8 * NT;
  // a warp's part of a short call: O of its steps by head, offset and sum
  constexpr int kSoloPitch = D + 4, kSoloHeads = 8 * NT;
  float* solo_o = reinterpret_cast<float*>(sbase + warp * NS * stage_bytes<D, KIND>());
  float2* solo_ml = reinterpret_cast<float2*>(solo_o + kSoloHeads * kSoloPitch);
  static_assert(kSoloHeads * (kSoloPitch * 4 + 8) <= NS * stage_bytes<D, KIND>(), "a warp's part fits its stages");
  const int first_w = solo ? 0 : (int)blockIdx.x * W + warp, n_w = solo ? 1 : N * units, step_w = solo ? 1 : (int)gridDim.x * W;
  for (int w = first_w; w < n_w; w += step_w) {
    const int li = solo ? 0 : w / units, unit = solo ? (int)blockIdx.x - b0 * units : w - li * units;
    const int g = unit / a.tiles, tile = unit - g * a.tiles;
    const int x0 = solo ? T * warp / W : lane_begin(li, T, N), x1 = solo ? T * (warp + 1) / W : lane_begin(li + 1, T, N);
    if (x0 >= x1 && !solo) continue;
    const uint8_t* kbase = static_cast<const uint8_t*>(a.k) + (int64_t)g * a.head_stride * elem_bytes<KIND>();
    const uint8_t* vbase = static_cast<const uint8_t*>(a.v) + (int64_t)g * a.head_stride * elem_bytes<KIND>();

    // ---- what all requests share: scales and slopes of the unit's heads (2 tq, 2 tq + 1 of each tile); in base 2, but for
    // capped scores, which get it with the cap
    const float ksc = a.scale * (a.k_scale != nullptr ? a.k_scale[g] : 1.f) * (a.softcap != 0.f ? 1.f : kLog2e);
    const float vsc = (a.v_scale != nullptr ? a.v_scale[g] : 1.f) / weight_unit<KIND>();
    const float cap2 = a.softcap * kLog2e, icap = a.softcap != 0.f ? 1.f / a.softcap : 0.f;
    const bool plain = a.softcap == 0.f && a.slopes == nullptr;
    float sl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hl = (tile * NT + nt) * 8 + 2 * tq + e;
        sl[nt][e] = a.slopes != nullptr && hl < a.G ? a.slopes[g * a.G + hl] * kLog2e : 0.f;
      }
    // Query rows of a request (heads 8 nt + gq of the tile) as they are: elements 2 tq, +1 and 8 + 2 tq, +1 of every 16,
    // or 4 tq .. 4 tq + 3 where the K fragments come from bytes.  With one tile per warp they are fetched a request
    // ahead (two tiles leave no registers for that).
    uint32_t qn[NT][KS][2];
    auto load_q = [&](int request, uint32_t (*to)[KS][2]) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int hl = (tile * NT + nt) * 8 + gq;
        const bool live = hl < a.G;
        const uint32_t* qrow = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) +
                                                                 (int64_t)(b0 + request) * a.q_stride +
                                                                 (int64_t)(live ? g * a.G + hl : 0) * D);
#pragma unroll
        for (int c = 0; c < KS; ++c) {
          const int e0 = KIND == kE4m3 ? 2 * tq : tq, e1 = KIND == kE4m3 ? 2 * tq + 1 : 4 + tq;
          to[nt][c][0] = live ? qrow[8 * c + e0] : 0u;
          to[nt][c][1] = live ? qrow[8 * c + e1] : 0u;
        }
      }
    };
    int b = find_request(cum, batch, x0);           // request of the next piece
    if (NT == 1) load_q(b, qn);

    // ---- the steps' rows, ahead of the arithmetic -----------------------------------------------
    int pb = b;                                     // request of the next step to look up
    int px = x0;
    // This lane's row of a step: its page's entry in the table (read ahead: nothing waits for it here) and its row there.
    struct Row {
      int32_t id, within, b;
      bool seen;
    };
    auto look = [&]() -> Row {
      Row r{0, 0, 0, false};
      if (px < x1) {
        while (px >= cum[pb + 1].x) ++pb;
        const int2 at = cum[pb];
        const int pn = at.y, f = first_row(pn, a.window);
        const int t = (f / kKeys + (px - at.x)) * kKeys + lane;
        r.b = pb;
        r.seen = t >= f && t < pn;
        if (r.seen) {
          const int blk = (int)((__umulhi(a.p_mul, (uint32_t)t) + (uint32_t)t) >> a.p_shift);   // t / P
          r.within = t - blk * a.P;
          r.id = a.tables[(int64_t)(b0 + pb) * a.max_blocks + blk];
        }
        ++px;
      }
      return r;
    };
    // Copies a step into stage `buf`, 16-byte chunks by all lanes, whole rows at a time, and returns the rows it has;
    // rows without a source are zeros.
    auto issue = [&](const Row& r, int buf) -> uint32_t {
      const bool ok = r.seen && r.id >= 0 && r.id < a.n_pages;
      if (r.seen && !ok) set_device_error(a.err, KVSEL_ERR_DEVICE, (uint32_t)(b0 + r.b));
      const int64_t off = (ok ? (int64_t)r.id * a.page_stride + (int64_t)r.within * a.row_stride : 0) * elem_bytes<KIND>();
      const uint32_t seen = __ballot_sync(0xffffffffu, ok);
      constexpr int KPI = 32 / CPR;                 // rows per copy instruction
      const uint32_t ks = st0 + buf * stage_bytes<D, KIND>();
      const int c = lane % CPR;
#pragma unroll
      for (int i = 0; i < kKeys / KPI; ++i) {
        const int x = i * KPI + lane / CPR;
        const int64_t ox = __shfl_sync(0xffffffffu, off, x) + c * 16;
        const bool has = (seen >> x) & 1u;
        const uint32_t dst = ks + chunk_at<RB>(x, c);
        cp_async16(dst, kbase + ox, has);
        cp_async16(dst + KV, vbase + ox, has);
      }
      return seen;
    };
    uint32_t seen[NS];                              // rows of the stages, by age: seen[0] is the step computed
#pragma unroll
    for (int i = 0; i < NS; ++i) seen[i] = 0;
    Row next;                                       // of the step to copy next
    {
      Row ahead[NS];
#pragma unroll
      for (int i = 0; i < NS; ++i) ahead[i] = look();
#pragma unroll
      for (int i = 0; i < NS - 1; ++i) {
        if (x0 + i < x1) seen[i] = issue(ahead[i], i);
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      next = ahead[NS - 1];
    }

    // ---- the row pieces of this lane --------------------------------------------------------------
    int buf = 0, x = x0;
    while (x < x1) {
      const int first = cum[b].x, last = cum[b + 1].x;         // the request's steps
      const int n = cum[b].y;
      const int f = first_row(n, a.window);
      const int row_end = min(x1, last);
      const bool starts = x == first, ends = row_end == last;
      if (unit == 0 && lane == 0 && !solo) {        // (one warp of the lane speaks for all)
        if (!a.by_lane && starts) a.span[b] = make_int2(li, ends ? li : lane_of(last - 1, T, N));
        if (a.by_lane && row_end == x1) a.span[li] = make_int2(b, starts && !ends ? lane_of(last - 1, T, N) : -1);
      }
      // the query rows as B fragments, fp16 where the pool is e4m3
      uint32_t qb[NT][KS][2];
      float sc[NT][2];                              // score factors of heads 2 tq, 2 tq + 1 of each tile
      if (NT > 1) load_q(b, qn);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < KS; ++c) qb[nt][c][0] = qn[nt][c][0], qb[nt][c][1] = qn[nt][c][1];
        sc[nt][0] = sc[nt][1] = ksc;
        if constexpr (KIND == kE4m3) {
          // bf16 queries: the row divided by the power of two at its largest value
          if (!a.out_f16) {
            float mx = 0.f;
#pragma unroll
            for (int c = 0; c < KS; ++c)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(qb[nt][c][e] << 16)), fabsf(__uint_as_float(qb[nt][c][e] & 0xffff0000u))));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // powers 2^-100 .. 2^100 keep both the factor and its inverse normal
            const int ex = min(100, max(-100, (int)((__float_as_uint(mx) >> 23) & 0xff) - 127));
            const float by = __uint_as_float((uint32_t)(ex + 127) << 23), inv = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
            for (int e = 0; e < 2; ++e) sc[nt][e] *= __shfl_sync(0xffffffffu, by, (2 * tq + e) * 4);
#pragma unroll
            for (int c = 0; c < KS; ++c)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const __half2 h = __floats2half2_rn(__uint_as_float(qb[nt][c][e] << 16) * inv,
                                                    __uint_as_float(qb[nt][c][e] & 0xffff0000u) * inv);
                qb[nt][c][e] = *reinterpret_cast<const uint32_t*>(&h);
              }
          }
        }
      }
      const int now = b;
      if (ends) {                                   // on to the next request with a row; its queries are fetched by then
        do ++b; while (b < batch && cum[b + 1].x == last);
        if (NT == 1 && row_end < x1) load_q(b, qn);
      }
      bool fresh = true;                            // one of this lane's heads has no offset yet
      float o[KS][NT][4], l[NT][2], m[NT][2], mo[NT][2];   // mo: the offset taken off, 0 while there is none
#pragma unroll
      for (int c = 0; c < KS; ++c)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) o[c][nt][0] = o[c][nt][1] = o[c][nt][2] = o[c][nt][3] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        mo[nt][0] = mo[nt][1] = 0.f;
        l[nt][0] = l[nt][1] = 0.f;
      }
      for (; x < row_end; ++x) {
        // the step NS - 1 ahead into the stage read last
        uint32_t ahead = 0;
        if (x + NS - 1 < x1) {
          ahead = issue(next, buf == 0 ? NS - 1 : buf - 1);
          next = look();
        }
        seen[NS - 1] = ahead;
        const uint32_t ks = st0 + buf * stage_bytes<D, KIND>(), vs = ks + KV;
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
        __syncwarp();
        // S^T: element e of tile mt is row 16 mt + gq + 8 (e / 2), head 2 tq + e % 2
        float s[2][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
        if constexpr (KIND == kE4m3) {
#pragma unroll
          for (int c = 0; c < KS; c += 2)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              uint32_t r[4];
              ldsm4(r, chunk_from<RB>(ks + k_lane, mt, c));
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t kf[4];
                e4m3x4_to_f16(r[2 * h], kf[0], kf[2]);
                e4m3x4_to_f16(r[2 * h + 1], kf[1], kf[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma<KIND>(s[mt][nt], kf, qb[nt][c + h][0], qb[nt][c + h][1]);
              }
            }
        } else {
#pragma unroll
          for (int c = 0; c < KS; ++c)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              uint32_t kf[4];
              ldsm4(kf, chunk_from<RB>(ks + k_lane, mt, 2 * c));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma<KIND>(s[mt][nt], kf, qb[nt][c][0], qb[nt][c][1]);
            }
        }
        if (!plain) {                               // capped and biased scores, in base 2
          const int t0 = (f / kKeys + (x - first)) * kKeys + gq - (n - 1);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float z = s[mt][nt][e] * sc[nt][e & 1];
                if (a.softcap != 0.f) z = cap2 * tanh_fast(z * icap);
                s[mt][nt][e] = fmaf(sl[nt][e & 1], (float)(t0 + 16 * mt + 8 * (e >> 1)), z);
              }
        }
        // plain scores are multiplied by their factor when their distance is taken, or here
        const bool whole = seen[0] == 0xffffffffu;
        float mul[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) mul[nt][e] = plain && whole ? sc[nt][e] : 1.f;
        if (!whole) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool ok = (seen[0] >> (16 * mt + gq + 8 * (e >> 1))) & 1u;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                s[mt][nt][e] = ok ? s[mt][nt][e] * (plain ? sc[nt][e & 1] : 1.f) : -INFINITY;
            }
        }
        // distances to the offset; where one passes the lag the offset moves to the step's largest score
        constexpr float kLag = weight_lag<KIND>(), kUnit = weight_unit<KIND>();
        float z[2][NT][4], top = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              z[mt][nt][e] = fmaf(s[mt][nt][e], mul[nt][e & 1], -mo[nt][e & 1]);
              top = fmaxf(top, z[mt][nt][e]);
            }
        if (__any_sync(0xffffffffu, top > (fresh ? -INFINITY : kLag))) {
          fresh = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float mm = mul[nt][e];
              float mx = fmaxf(fmaxf(s[0][nt][e] * mm, s[0][nt][e + 2] * mm), fmaxf(s[1][nt][e] * mm, s[1][nt][e + 2] * mm));
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
              if (mx > m[nt][e] + kLag) {
                const float alpha = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - mx);
                m[nt][e] = mo[nt][e] = mx;
                l[nt][e] *= alpha;
#pragma unroll
                for (int c = 0; c < KS; ++c) {
                  o[c][nt][e] *= alpha;
                  o[c][nt][e + 2] *= alpha;
                }
              }
#pragma unroll
              for (int mt = 0; mt < 2; ++mt) {
                z[mt][nt][e] = fmaf(s[mt][nt][e], mm, -mo[nt][e]);
                z[mt][nt][e + 2] = fmaf(s[mt][nt][e + 2], mm, -mo[nt][e]);
              }
              fresh |= m[nt][e] == -INFINITY;
            }
        }
        // P^T as B fragments (rows 16 mt + 2 tq, +1 and 8 + ..., head gq)
        uint32_t ph[2][NT][2], pl[2][NT][2];          // high and low parts
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              p[e] = ex2(z[mt][nt][e]);
              l[nt][e & 1] += p[e];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float r0, r1, d0, d1;
              ph[mt][nt][h] = transpose8x8(pack_hi<KIND>(p[2 * h] * kUnit, p[2 * h + 1] * kUnit, r0, r1));
              pl[mt][nt][h] = transpose8x8(pack_hi<KIND>(r0, r1, d0, d1));
            }
          }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          if constexpr (KIND == kE4m3) {
#pragma unroll
            for (int c = 0; c < KS; c += 2) {
              uint32_t r[4];
              ldsm4_t(r, chunk_from<RB>(vs + v_lane, mt, c));
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                // bytes (row 2 tq: d 2 gq, 2 gq + 1; row 2 tq + 1: the same) to row pairs of one d each
                uint32_t vf[4];
                e4m3x4_to_f16(__byte_perm(r[2 * h], 0, 0x3120), vf[0], vf[1]);
                e4m3x4_to_f16(__byte_perm(r[2 * h + 1], 0, 0x3120), vf[2], vf[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma<KIND>(o[c + h][nt], vf, ph[mt][nt][0], ph[mt][nt][1]);
                  mma<KIND>(o[c + h][nt], vf, pl[mt][nt][0], pl[mt][nt][1]);
                }
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < KS; ++c) {
              uint32_t vf[4];
              ldsm4_t(vf, chunk_from<RB>(vs + v_lane, mt, 2 * c));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma<KIND>(o[c][nt], vf, ph[mt][nt][0], ph[mt][nt][1]);
                mma<KIND>(o[c][nt], vf, pl[mt][nt][0], pl[mt][nt][1]);
              }
            }
          }
        }
        __syncwarp();                               // the stage is read before it is refilled
        buf = buf == NS - 1 ? 0 : buf + 1;
#pragma unroll
        for (int i = 0; i < NS - 1; ++i) seen[i] = seen[i + 1];
      }
      // the piece's sums over the rows a lane did not hold
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
      // d of accumulator element e of slice c: rows gq and gq + 8 of the slice, or 2 gq and 2 gq + 1 from bytes
      const int d0 = KIND == kE4m3 ? 2 * gq : gq, d1 = KIND == kE4m3 ? 2 * gq + 1 : gq + 8;
      if (solo) {                                   // to the warp's own stages, all read by now
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* to = solo_o + (nt * 8 + 2 * tq + e) * kSoloPitch;
#pragma unroll
            for (int c = 0; c < KS; ++c) {
              to[16 * c + d0] = o[c][nt][e];
              to[16 * c + d1] = o[c][nt][e + 2];
            }
            if (gq == 0) solo_ml[nt * 8 + 2 * tq + e] = make_float2(m[nt][e], l[nt][e]);
          }
      } else if (starts && ends) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float inv[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            inv[e] = l[nt][e] == 0.f ? 0.f : vsc / l[nt][e];
            const int hl = (tile * NT + nt) * 8 + 2 * tq + e;
            if (a.lse != nullptr && gq == 0 && hl < a.G)
              a.lse[(int64_t)now * a.h_q + g * a.G + hl] = (m[nt][e] + log2f(l[nt][e])) * 0.6931471805599453f;
          }
          // transposed back, a lane holds consecutive d of one head: 2 tq, +1 of both halves of a slice, or 4 tq .. + 3
          const int hl = (tile * NT + nt) * 8 + gq;
          uint32_t* orow = static_cast<uint32_t*>(a.o) + ((int64_t)now * a.h_q + g * a.G + hl) * (D / 2);
#pragma unroll
          for (int c = 0; c < KS; ++c) {
            const uint32_t y0 = transpose8x8(pack_out(a, o[c][nt][0] * inv[0], o[c][nt][1] * inv[1]));
            const uint32_t y1 = transpose8x8(pack_out(a, o[c][nt][2] * inv[0], o[c][nt][3] * inv[1]));
            if (hl >= a.G) continue;
            if constexpr (KIND == kE4m3) {
              *reinterpret_cast<uint2*>(orow + 8 * c + 2 * tq) = make_uint2(__byte_perm(y0, y1, 0x5410), __byte_perm(y0, y1, 0x7632));
            } else {
              orow[8 * c + tq] = y0;
              orow[8 * c + 4 + tq] = y1;
            }
          }
        }
      } else {
        const int64_t row = (int64_t)(2 * li + (starts ? 1 : 0)) * heads_pad + unit * 8 * NT;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float* pr = a.part + (row + nt * 8 + 2 * tq + e) * D;
#pragma unroll
            for (int c = 0; c < KS; ++c) {
              pr[16 * c + d0] = o[c][nt][e];
              pr[16 * c + d1] = o[c][nt][e + 2];
            }
            if (gq == 0) a.part_ml[row + nt * 8 + 2 * tq + e] = make_float2(m[nt][e], l[nt][e]);
          }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    if (!solo) continue;
    // the warps' parts merged as paged_join does, here
    if (x0 >= x1 && lane < kSoloHeads) solo_ml[lane] = make_float2(-INFINITY, 0.f);
    __syncthreads();
    constexpr int part = NS * stage_bytes<D, KIND>() / 4;         // floats from one warp's part to the next
    const float* o0 = reinterpret_cast<const float*>(sbase);
    for (int y = threadIdx.x; y < kSoloHeads * (D / 2); y += 32 * W) {
      const int h = y / (D / 2), d = 2 * (y - h * (D / 2)), hl = tile * kSoloHeads + h;
      if (hl >= a.G) continue;
      float2 ml[W];
      float M = -INFINITY, num0 = 0.f, num1 = 0.f, den = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        ml[i] = reinterpret_cast<const float2*>(o0 + i * part + kSoloHeads * kSoloPitch)[h];
        M = fmaxf(M, ml[i].x);
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (ml[i].x == -INFINITY && ml[i].y == 0.f) continue;     // no step, or no score
        const float wt = ml[i].x == M ? 1.f : exp2f(ml[i].x - M);
        const float2 v = *reinterpret_cast<const float2*>(o0 + i * part + h * kSoloPitch + d);
        num0 = fmaf(wt, v.x, num0);
        num1 = fmaf(wt, v.y, num1);
        den = fmaf(wt, ml[i].y, den);
      }
      const float inv = den == 0.f ? 0.f : vsc / den;
      const int64_t oh = (int64_t)b0 * a.h_q + g * a.G + hl;
      static_cast<uint32_t*>(a.o)[(oh * D + d) / 2] = pack_out(a, num0 * inv, num1 * inv);
      if (a.lse != nullptr && d == 0) a.lse[oh] = (M + log2f(den)) * 0.6931471805599453f;
    }
  }
}

using PagedKernel = void (*)(const PagedArgs);
struct PagedVariant {
  PagedKernel kern;
  int warps, smem;       // warps per CTA; shared memory without the batch's sums
};
template <int D, int KIND>
PagedVariant paged_variant(int nt) {
  return {nt == 1 ? paged_attend<D, KIND, 1> : paged_attend<D, KIND, 2>, n_warps<D, KIND>(), smem_bytes<D, KIND>(0)};
}
// The kernels of a pool type, each in a file of its own (paged_attend_*.cu): head dim, tiles of 8 query heads per warp.
PagedVariant paged_variant_bf16(int d, int nt);
PagedVariant paged_variant_f16(int d, int nt);
PagedVariant paged_variant_e4m3(int d, int nt);

}  // namespace kvsel
