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
// keeps an exponent offset that moves only when a score passes it by 2^8, so the common step forms no
// maximum, and the sums stay in the lanes until a row ends.
//
// A request cut between lanes leaves one partial (O, offset, sum) per piece, which paged_join merges in
// lane order; a request within one lane is written at once.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <mutex>

#include "paged.cuh"
#include "sm100.cuh"

namespace kvsel {
namespace {

constexpr int kKeys = 32;             // rows per step: one per lane
constexpr int kMinSteps = 2;          // a lane is not given fewer steps than this
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
  int32_t* cum;         // [batch + 1] first step of each request, then the lanes in use
  DeviceError* err;
  int64_t page_stride, head_stride, row_stride, q_stride;
  float scale, softcap;
  int32_t h_q, h_kv, G, P, batch, max_blocks, n_pages, window, out_f16;
  int32_t tiles;        // tiles of query heads per KV head
  int32_t lanes;        // lanes the grid can hold
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
// two e4m3 values (the low 16 bits) as fp16, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xffffu), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

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
  return 1024 + n_warps<D, KIND>() * n_stages<D, KIND>() * stage_bytes<D, KIND>() + 4 * (batch + 1);
}

// Byte offset of 16-byte chunk c of row x: halves of 128-byte rows one after another, chunks of eight rows
// spread over the banks.
template <int RB>
__device__ __forceinline__ uint32_t chunk_at(int x, int c) {
  if constexpr (RB >= 128) return (uint32_t)((c >> 3) * (kKeys * 128) + x * 128 + (((c & 7) ^ (x & 7)) << 4));
  else return (uint32_t)(x * 64 + ((c ^ ((x >> 1) & 3)) << 4));
}

// First and last visible step of a request of n rows.
__device__ __forceinline__ int first_row(int n, int window) { return window > 0 && n > window ? n - window : 0; }
// First step of lane i of N over T steps.
__device__ __forceinline__ int lane_begin(int i, int T, int N) { return (int)((int64_t)i * T / N); }
// The lane that holds step x.
__device__ __forceinline__ int lane_of(int x, int T, int N) { return (int)(((int64_t)(x + 1) * N + T - 1) / T) - 1; }

// cum[b] = steps of the requests before b, in shared memory; returns all steps.  Every CTA forms it.
template <int THREADS>
__device__ int step_sums(const PagedArgs& a, int32_t* cum) {
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
    const int steps = (n + kKeys - 1) / kKeys - first_row(n, a.window) / kKeys;
    cum[b] = steps;
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
    const int s = cum[b];
    cum[b] = at;
    at += s;
  }
  if (tid == 0) cum[a.batch] = total;
  __syncthreads();
  return total;
}

__device__ __forceinline__ int find_request(const int32_t* cum, int batch, int x) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= x) lo = mid; else hi = mid;
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
  int32_t* cum = reinterpret_cast<int32_t*>(sbase + W * NS * stage_bytes<D, KIND>());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;
  const uint32_t st0 = sm100::smem_addr(sbase) + warp * NS * stage_bytes<D, KIND>();

  const int T = step_sums<32 * W>(a, cum);
  const int N = max(1, min(a.lanes, T / kMinSteps));
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b <= a.batch; b += 32 * W) a.cum[b] = cum[b];
    if (threadIdx.x == 0) a.cum[a.batch + 1] = N;
  }
  // requests without a row: o = 0, lse = -inf
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    if (cum[b] != cum[b + 1]) continue;
    uint32_t* ob = reinterpret_cast<uint32_t*>(a.o) + (int64_t)b * a.h_q * (D / 2);
    for (int x = threadIdx.x; x < a.h_q * (D / 2); x += 32 * W) ob[x] = 0u;
    if (a.lse != nullptr)
      for (int x = threadIdx.x; x < a.h_q; x += 32 * W) a.lse[(int64_t)b * a.h_q + x] = -INFINITY;
  }
  const int units = a.h_kv * a.tiles;
  const int heads_pad = units * 8 * NT;
  for (int64_t w = (int64_t)blockIdx.x * W + warp; w < (int64_t)N * units; w += (int64_t)gridDim.x * W) {
    const int li = (int)(w / units), unit = (int)(w - (int64_t)li * units);
    const int g = unit / a.tiles, tile = unit - g * a.tiles;
    const int x0 = lane_begin(li, T, N), x1 = lane_begin(li + 1, T, N);
    if (x0 >= x1) continue;
    const uint8_t* kbase = static_cast<const uint8_t*>(a.k) + (int64_t)g * a.head_stride * elem_bytes<KIND>();
    const uint8_t* vbase = static_cast<const uint8_t*>(a.v) + (int64_t)g * a.head_stride * elem_bytes<KIND>();

    // ---- the steps' rows, ahead of the arithmetic -----------------------------------------------
    int pb = find_request(cum, a.batch, x0);        // request of the next step to look up
    int pn = (int)a.lens[pb];
    int px = x0;
    // This lane's row of step px: page id (or -1 when the row is not seen), fetched a step before its copy.
    int32_t id = -1, within = 0;
    auto look = [&]() {
      id = -1;
      if (px < x1) {
        while (px >= cum[pb + 1]) {
          ++pb;
          pn = (int)a.lens[pb];
        }
        const int f = first_row(pn, a.window);
        const int t = (f / kKeys + (px - cum[pb])) * kKeys + lane;
        if (t >= f && t < pn) {
          const int blk = t / a.P;
          within = t - blk * a.P;
          id = __ldg(a.tables + (int64_t)pb * a.max_blocks + blk);
          if (id < 0 || id >= a.n_pages) {
            set_device_error(a.err, KVSEL_ERR_DEVICE, (uint32_t)pb);
            id = -1;
          }
        }
        ++px;
      }
    };
    // Copies the looked-up step into stage `buf` and returns the rows it has; rows without a source are zeros.
    auto issue = [&](int buf) -> uint32_t {
      const int64_t off = (id < 0 ? 0 : (int64_t)id * a.page_stride + (int64_t)within * a.row_stride) * elem_bytes<KIND>();
      const uint32_t seen = __ballot_sync(0xffffffffu, id >= 0);
      constexpr int KPI = 32 / CPR;                 // rows per copy instruction
      const uint32_t ks = st0 + buf * stage_bytes<D, KIND>();
      const int c = lane % CPR;
#pragma unroll
      for (int i = 0; i < kKeys / KPI; ++i) {
        const int x = i * KPI + lane / CPR;
        const int64_t ox = __shfl_sync(0xffffffffu, off, x) + c * 16;
        const bool ok = (seen >> x) & 1u;
        const uint32_t dst = ks + chunk_at<RB>(x, c);
        cp_async16(dst, kbase + ox, ok);
        cp_async16(dst + KV, vbase + ox, ok);
      }
      return seen;
    };
    uint32_t seen[NS];                              // rows of the stages, by age: seen[0] is the step computed
#pragma unroll
    for (int i = 0; i < NS; ++i) seen[i] = 0;
    look();
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) {
      if (x0 + i < x1) {
        seen[i] = issue(i);
        look();
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }

    // ---- the row pieces of this lane --------------------------------------------------------------
    int buf = 0, x = x0;
    int b = find_request(cum, a.batch, x0);
    while (x < x1) {
      while (x >= cum[b + 1]) ++b;
      const int n = (int)a.lens[b];
      const int f = first_row(n, a.window);
      const int row_end = min(x1, cum[b + 1]);
      const bool starts = x == cum[b], ends = row_end == cum[b + 1];
      // B fragments of the query rows (head 8 nt + gq of the tile): elements 2 tq, +1 and 8 + 2 tq, +1 of
      // every 16, or 4 tq .. 4 tq + 3 where the K fragments come from bytes
      uint32_t qb[NT][KS][2];
      float qs[NT];                                 // what the row of head 8 nt + gq was divided by
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int hl = (tile * NT + nt) * 8 + gq;
        const bool live = hl < a.G;
        const uint32_t* qrow = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) +
                                                                 (int64_t)b * a.q_stride +
                                                                 (int64_t)(live ? g * a.G + hl : 0) * D);
        qs[nt] = 1.f;
#pragma unroll
        for (int c = 0; c < KS; ++c) {
          const int e0 = KIND == kE4m3 ? 2 * tq : tq, e1 = KIND == kE4m3 ? 2 * tq + 1 : 4 + tq;
          qb[nt][c][0] = live ? __ldg(qrow + 8 * c + e0) : 0u;
          qb[nt][c][1] = live ? __ldg(qrow + 8 * c + e1) : 0u;
        }
        if constexpr (KIND == kE4m3) {
          // bf16 queries to fp16: the row divided by the power of two at its largest value
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
            qs[nt] = __uint_as_float((uint32_t)(ex + 127) << 23);
            const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
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
      // per accumulator column (heads 2 tq, 2 tq + 1 of each tile): score factor and bias slope
      const float ksc = a.scale * (a.k_scale != nullptr ? a.k_scale[g] : 1.f);
      float sc[NT][2], sl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int hl = (tile * NT + nt) * 8 + 2 * tq + e;
          sc[nt][e] = ksc * (KIND == kE4m3 ? __shfl_sync(0xffffffffu, qs[nt], (2 * tq + e) * 4) : 1.f);
          sl[nt][e] = a.slopes != nullptr && hl < a.G ? a.slopes[g * a.G + hl] * 1.4426950408889634f : 0.f;
        }
      const bool plain = a.softcap == 0.f && a.slopes == nullptr;
      float o[KS][NT][4], m[NT][2], l[NT][2];
#pragma unroll
      for (int c = 0; c < KS; ++c)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) o[c][nt][0] = o[c][nt][1] = o[c][nt][2] = o[c][nt][3] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
      }
      for (; x < row_end; ++x) {
        // the step NS - 1 ahead into the stage read last
        uint32_t ahead = 0;
        if (x + NS - 1 < x1) {
          ahead = issue(buf == 0 ? NS - 1 : buf - 1);
          look();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        seen[NS - 1] = ahead;
        asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
        __syncwarp();
        const uint32_t ks = st0 + buf * stage_bytes<D, KIND>(), vs = ks + KV;
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
              ldsm4(r, ks + chunk_at<RB>(mt * 16 + (lane & 15), c + (lane >> 4)));
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t kf[4] = {e4m3x2_to_f16x2(r[2 * h]), e4m3x2_to_f16x2(r[2 * h + 1]),
                                        e4m3x2_to_f16x2(r[2 * h] >> 16), e4m3x2_to_f16x2(r[2 * h + 1] >> 16)};
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
              ldsm4(kf, ks + chunk_at<RB>(mt * 16 + (lane & 15), 2 * c + (lane >> 4)));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma<KIND>(s[mt][nt], kf, qb[nt][c][0], qb[nt][c][1]);
            }
        }
        // scores in base 2: element e of tile mt is row 16 mt + gq + 8 (e / 2), head 2 tq + e % 2
        if (plain) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[mt][nt][e] *= sc[nt][e & 1] * 1.4426950408889634f;
        } else {
          const int t0 = (f / kKeys + (x - cum[b])) * kKeys + gq - (n - 1);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float z = s[mt][nt][e] * sc[nt][e & 1];
                if (a.softcap != 0.f) z = a.softcap * tanhf(z / a.softcap);
                s[mt][nt][e] = fmaf(sl[nt][e & 1], (float)(t0 + 16 * mt + 8 * (e >> 1)), z * 1.4426950408889634f);
              }
        }
        if (seen[0] != 0xffffffffu) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((seen[0] >> (16 * mt + gq + 8 * (e >> 1))) & 1u))
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[mt][nt][e] = -INFINITY;
        }
        bool up = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            up |= fmaxf(s[0][nt][e], s[1][nt][e]) > m[nt][e & 1] + 8.f;
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(fmaxf(s[0][nt][e], s[0][nt][e + 2]), fmaxf(s[1][nt][e], s[1][nt][e + 2]));
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
              if (mx > m[nt][e] + 8.f) {
                const float alpha = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - mx);
                m[nt][e] = mx;
                l[nt][e] *= alpha;
#pragma unroll
                for (int c = 0; c < KS; ++c) {
                  o[c][nt][e] *= alpha;
                  o[c][nt][e + 2] *= alpha;
                }
              }
            }
        }
        // P^T as B fragments (rows 16 mt + 2 tq, +1 and 8 + ..., head gq), high and low parts
        uint32_t ph[2][NT][2], pl[2][NT][2];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              p[e] = s[mt][nt][e] == -INFINITY ? 0.f : ex2(s[mt][nt][e] - m[nt][e & 1]);
              l[nt][e & 1] += p[e];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float r0, r1, d0, d1;
              ph[mt][nt][h] = transpose8x8(pack_hi<KIND>(p[2 * h], p[2 * h + 1], r0, r1));
              pl[mt][nt][h] = transpose8x8(pack_hi<KIND>(r0, r1, d0, d1));
            }
          }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          if constexpr (KIND == kE4m3) {
#pragma unroll
            for (int c = 0; c < KS; c += 2) {
              uint32_t r[4];
              ldsm4_t(r, vs + chunk_at<RB>(mt * 16 + (lane & 15), c + (lane >> 4)));
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                // bytes (row 2 tq: d 2 gq, 2 gq + 1; row 2 tq + 1: the same) to row pairs of one d each
                const uint32_t u0 = __byte_perm(r[2 * h], 0, 0x3120), u1 = __byte_perm(r[2 * h + 1], 0, 0x3120);
                const uint32_t vf[4] = {e4m3x2_to_f16x2(u0), e4m3x2_to_f16x2(u0 >> 16), e4m3x2_to_f16x2(u1),
                                        e4m3x2_to_f16x2(u1 >> 16)};
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
              ldsm4_t(vf, vs + chunk_at<RB>(mt * 16 + ((lane >> 4) << 3) + (lane & 7), 2 * c + ((lane >> 3) & 1)));
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
      if (starts && ends) {
        const float vsc = a.v_scale != nullptr ? a.v_scale[g] : 1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int hl = (tile * NT + nt) * 8 + 2 * tq + e;
            if (hl >= a.G) continue;
            const int64_t oh = (int64_t)b * a.h_q + g * a.G + hl;
            const float inv = l[nt][e] == 0.f ? 0.f : vsc / l[nt][e];
#pragma unroll
            for (int c = 0; c < KS; ++c) {
              const float y0 = o[c][nt][e] * inv, y1 = o[c][nt][e + 2] * inv;
              if (a.out_f16) {
                __half* orow = static_cast<__half*>(a.o) + oh * D + 16 * c;
                orow[d0] = __float2half_rn(y0);
                orow[d1] = __float2half_rn(y1);
              } else {
                __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.o) + oh * D + 16 * c;
                orow[d0] = __float2bfloat16_rn(y0);
                orow[d1] = __float2bfloat16_rn(y1);
              }
            }
            if (a.lse != nullptr && gq == 0) a.lse[oh] = (m[nt][e] + log2f(l[nt][e])) * 0.6931471805599453f;
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
  }
}

// o of a request that several lanes hold: sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over its pieces in lane
// order.  blockIdx.y is the request, or (more requests than lanes) the lane in which one begins that goes on.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join(const __grid_constant__ PagedArgs a, int NT8, int by_lane) {
  constexpr int GR = kJoinThreads / D;
  __shared__ float red[kJoinThreads];
  __shared__ float redl[GR];
  const int h = blockIdx.x, T = a.cum[a.batch], N = a.cum[a.batch + 1];
  int b = blockIdx.y;
  if (by_lane) {
    const int li = blockIdx.y;
    if (li >= N) return;
    const int end = lane_begin(li + 1, T, N);
    if (end <= lane_begin(li, T, N) || end >= T) return;
    b = find_request(a.cum, a.batch, end - 1);     // the request of the lane's last step
    if (a.cum[b] < lane_begin(li, T, N)) return;   // it began in an earlier lane
  }
  const int c0 = a.cum[b], c1 = a.cum[b + 1];
  if (c0 == c1) return;
  const int i0 = lane_of(c0, T, N), i1 = lane_of(c1 - 1, T, N);
  if (i0 == i1) return;
  const int g = h / a.G, hl = h - g * a.G;
  const int units8 = a.h_kv * a.tiles * NT8;
  const int at = g * a.tiles * NT8 + hl;            // the head among the padded heads
  const int d = threadIdx.x % D, gr = threadIdx.x / D;
  auto row_of = [&](int i) -> int64_t { return (int64_t)(2 * i + (i == i0 ? 1 : 0)) * units8 + at; };
  float M = -INFINITY;
  for (int i = i0 + (threadIdx.x & 31); i <= i1; i += 32) M = fmaxf(M, a.part_ml[row_of(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float num = 0.f, den = 0.f;
#pragma unroll 8
  for (int i = i0 + gr; i <= i1; i += GR) {
    const int64_t r = row_of(i);
    const float2 ml = a.part_ml[r];
    const float w = ml.x == M ? 1.f : exp2f(ml.x - M);   // (both -inf: scores that are all NaN, or no score)
    num = fmaf(w, a.part[r * D + d], num);
    den = fmaf(w, ml.y, den);
  }
  red[threadIdx.x] = num;
  if (d == 0) redl[gr] = den;
  __syncthreads();
  if (gr != 0) return;
  den = 0.f;
  num = 0.f;
#pragma unroll
  for (int i = 0; i < GR; ++i) {
    num += red[i * D + d];
    den += redl[i];
  }
  const float vsc = a.v_scale != nullptr ? a.v_scale[g] : 1.f;
  const float y = den == 0.f ? 0.f : num * (vsc / den);
  const int64_t oh = (int64_t)b * a.h_q + h;
  if (a.out_f16) static_cast<__half*>(a.o)[oh * D + d] = __float2half_rn(y);
  else static_cast<__nv_bfloat16*>(a.o)[oh * D + d] = __float2bfloat16_rn(y);
  if (a.lse != nullptr && d == 0) a.lse[oh] = (M + log2f(den)) * 0.6931471805599453f;
}

using PagedKernel = void (*)(const PagedArgs);
struct Variant {
  PagedKernel kern;
  int warps, smem;       // warps per CTA; shared memory without the batch's sums
};
template <int D, int KIND>
Variant variant_of(int nt) {
  return {nt == 1 ? paged_attend<D, KIND, 1> : paged_attend<D, KIND, 2>, n_warps<D, KIND>(), smem_bytes<D, KIND>(0)};
}
Variant variant(const PagedShape& p, int nt) {
  const int kind = p.cache_dtype == KVSEL_DTYPE_E4M3 ? kE4m3 : p.dtype == KVSEL_DTYPE_F16 ? kF16 : kBf16;
  if (p.d == 64) return kind == kBf16 ? variant_of<64, kBf16>(nt) : kind == kF16 ? variant_of<64, kF16>(nt) : variant_of<64, kE4m3>(nt);
  return kind == kBf16 ? variant_of<128, kBf16>(nt) : kind == kF16 ? variant_of<128, kF16>(nt) : variant_of<128, kE4m3>(nt);
}

// SMs of the current device (0: it cannot be queried), asked once per device.
int sm_count() {
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static int cache[kMaxDev] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < kMaxDev && cache[dev] > 0) return cache[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  if (dev >= 0 && dev < kMaxDev) cache[dev] = n;
  return n;
}

struct Geometry {
  int nt, tiles, lanes, grid;
  size_t cum_off, ml_off, part_off, total;
};
// One CTA per SM, fewer when the bound on the steps needs fewer warps.
bool geometry(const PagedShape& p, Geometry* out) {
  const int sms = sm_count();
  if (sms <= 0) return false;
  const int G = p.h_q / p.h_kv;
  Geometry& o = *out;
  o.nt = G <= 8 ? 1 : 2;
  o.tiles = (int)ceil_div(G, 8 * o.nt);
  const Variant v = variant(p, o.nt);
  const int64_t units = (int64_t)p.h_kv * o.tiles;
  const int64_t most = ceil_div((int64_t)p.max_blocks * p.P, kKeys) + 1;     // steps of one request, bounded
  const int64_t lanes = std::min<int64_t>(std::max<int64_t>(1, (int64_t)sms * v.warps / units),
                                          std::max<int64_t>(1, most * p.batch / kMinSteps));
  o.lanes = (int)lanes;
  o.grid = (int)std::min<int64_t>(sms, ceil_div(lanes * units, v.warps));
  const int64_t heads = units * 8 * o.nt;
  auto up = [](size_t x) { return (x + KVSEL_WS_ALIGN - 1) / KVSEL_WS_ALIGN * KVSEL_WS_ALIGN; };
  o.cum_off = sizeof(DeviceError);
  o.ml_off = up(o.cum_off + sizeof(int32_t) * ((size_t)p.batch + 2));
  o.part_off = up(o.ml_off + sizeof(float2) * 2 * (size_t)(lanes * heads));
  o.total = up(o.part_off + sizeof(float) * 2 * (size_t)(lanes * heads) * p.d);
  return true;
}

}  // namespace

size_t paged_attend_ws(const PagedShape& p) {
  Geometry geo;
  return geometry(p, &geo) ? geo.total : 0;
}

kvsel_status launch_paged_attend(const PagedShape& p, const void* q, const void* k, const void* v,
                                 const int32_t* tables, const int64_t* lens, const float* slopes,
                                 const float* k_scale, const float* v_scale, void* o, float* lse, void* ws,
                                 cudaStream_t s) {
  Geometry geo;
  if (!geometry(p, &geo)) return KVSEL_ERR_CUDA;
  const Variant var = variant(p, geo.nt);
  char* base = static_cast<char*>(ws);
  PagedArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.tables = tables;
  a.lens = lens;
  a.slopes = slopes;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.o = o;
  a.lse = lse;
  a.cum = reinterpret_cast<int32_t*>(base + geo.cum_off);
  a.part_ml = reinterpret_cast<float2*>(base + geo.ml_off);
  a.part = reinterpret_cast<float*>(base + geo.part_off);
  a.err = reinterpret_cast<DeviceError*>(ws);
  a.page_stride = p.page_stride;
  a.head_stride = p.head_stride;
  a.row_stride = p.row_stride;
  a.q_stride = p.q_stride;
  a.scale = p.scale;
  a.softcap = p.softcap;
  a.h_q = p.h_q;
  a.h_kv = p.h_kv;
  a.G = p.h_q / p.h_kv;
  a.P = p.P;
  a.batch = p.batch;
  a.max_blocks = p.max_blocks;
  a.n_pages = p.n_pages;
  a.window = p.window;
  a.out_f16 = p.dtype == KVSEL_DTYPE_F16;
  a.tiles = geo.tiles;
  a.lanes = geo.lanes;
  const size_t smem = var.smem + sizeof(int32_t) * (size_t)p.batch;
  if (set_smem((const void*)var.kern, smem) != cudaSuccess) return KVSEL_ERR_CUDA;
  {
    TraceScope ts("paged_attend", s);
    var.kern<<<geo.grid, 32 * var.warps, smem, s>>>(a);
    const kvsel_status st = launch_status();
    if (st != KVSEL_OK) return st;
  }
  TraceScope ts("paged_join", s);
  const int by_lane = p.batch > geo.lanes;
  const dim3 grid((unsigned)p.h_q, (unsigned)(by_lane ? geo.lanes : p.batch));
  if (p.d == 64) paged_join<64><<<grid, kJoinThreads, 0, s>>>(a, 8 * geo.nt, by_lane);
  else paged_join<128><<<grid, kJoinThreads, 0, s>>>(a, 8 * geo.nt, by_lane);
  return launch_status();
}

}  // namespace kvsel
