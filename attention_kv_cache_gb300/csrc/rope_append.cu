// RMS norm of every query and key head, rotary positions, and the new K / V rows into the paged pool.
//
// y = x rsqrt(mean(x^2) + eps) (w + bias), then the pairs (a, b) of the first `rot` elements become
// factor (a cos - b sin, b cos + a sin) of the angle position * inv_freq.
//
// The angle is formed in turns as a 64-bit fraction: inv_freq / (2 pi) as a multiple of 2^-64 (off by less than one of
// them) times the position, modulo 2^64.  So it is off by less than position * 2^-64 and the rounding to its top 32
// bits: 2^-32 of a turn at any position below 2^31.
//
// One pass over the data, by single warps: a unit is up to kUnitBytes of a token's rows, queries,
// keys and values end to end.  Every
// warp has an equal share of all units; its units come by bulk copies into a ring of stages (one copy where the rows are contiguous), are
// normed and turned where they lie, and go out by bulk copies from there; 16-bit value rows go through untouched.
// A row is d / 16 lanes of 16 elements, chosen so that both elements of a pair lie in one lane (elements 8 j .. and
// rot / 2 + 8 j .. of a half layout, 16 j .. of an interleaved one), and the lanes of a row sum its squares by shuffles.
//
// Bound: the bytes of the rows, if enough of them are in flight (which is why the stages are shared memory and not
// registers) and the arithmetic stays below the issue rate:
//   - weight, cosine and sine are one 2x2 matrix per pair, formed once per token (two pairs per lane) and read by
//     every row: (a, b) -> r (A a - B b, C b + D a) with A = w_a cos, B = w_b sin, C = w_b cos, D = w_a sin and r
//     the row's norm;
//   - two pairs share an instruction (packed fp32);
//   - units of queries alone share the matrices' reads between rows (32768 tokens 227 -> 219 us);
//   - frequencies in turns are formed once per CTA, a token's slot and
//     position are read a token ahead.
//
// Measured (GB300, device time): 8200 tokens of 32 + 8 + 8 heads of 128, bf16, 37 us (202 MB, 5.5 TB/s; the copies
// without the arithmetic 35 us); 32768 tokens of 64 + 8 + 8 heads into e4m3, 208 us (1276 MB, 6.1 TB/s; copies alone
// 205 us); one token 4.8 us.  With rows in registers instead (steps of 4 rows, 16 warps per SM): 52 and 288 us.  Few
// heads leave little to a unit: 8200 tokens of 8 + 1 + 1 heads take 19 us (42 MB, 2.2 TB/s; with a unit for each kind of
// row 21 us).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "sm100.cuh"

namespace kvsel {
namespace {

constexpr int kWarps = 5;              // per CTA
constexpr int kRopeThreads = 32 * kWarps;
constexpr int kUnitBytes = 4096;       // of a unit at most
constexpr int kRingBytes = 3 * kUnitBytes;   // of a warp's stages: three of that, or up to kMaxStages of smaller ones
constexpr int kMaxStages = 12;

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 get(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t put(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
};
template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 get(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
  static __device__ __forceinline__ uint32_t put(float a, float b) {
    const __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
};

// two fp32 values in one register pair
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 get(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Two quotients x / s, correctly rounded, of the negated x: q = x (1 / s) and its residual s q - x, which one fused
// multiply-add forms exactly, correct one another (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990, whose condition is a correctly rounded reciprocal).  A product with 1 / s alone can miss a quotient
// that lies between two e4m3 numbers, and then goes to the wrong one; plain divisions take 10 to 23 % of an append into an
// 8-bit pool, this 1 to 5 %.  A q that is infinite (of a finite x too) has an infinite residual or none: its magnitude is
// limited, and q stays.  Scales below 2^-60 (inv_res zero) leave q as it is.  The signs keep a negative zero.
struct Divisor {
  F2 s, inv, inv_res;        // s, -1 / s, and -1 / s on the residual
};
// x with its magnitude at most 2^60; NaN is 2^60
__device__ __forceinline__ float limited(float x) {
  float r;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(0x1p60f));
  return r;
}
__device__ __forceinline__ F2 divide_neg(F2 neg_x, const Divisor& d) {
  const F2 q = mul(neg_x, d.inv);
  const float2 r = get(fma(q, d.s, neg_x));
  return fma(f2(limited(r.x), limited(r.y)), d.inv_res, q);
}

// A lane's 16 elements as four packed pairs of first elements and four of second ones.
template <typename T, bool HALF>
__device__ __forceinline__ void unpack16(const uint4* r, F2* a, F2* b) {
  const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const float2 x = Pair<T>::get(w[HALF ? m : 2 * m]), y = Pair<T>::get(w[HALF ? m + 4 : 2 * m + 1]);
    a[m] = HALF ? f2(x.x, x.y) : f2(x.x, y.x);
    b[m] = HALF ? f2(y.x, y.y) : f2(x.y, y.y);
  }
}
// the packed pairs back in the order of the elements
template <bool HALF>
__device__ __forceinline__ void order16(const F2* a, const F2* b, float* x) {
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const float2 u = get(a[m]), v = get(b[m]);
    x[HALF ? 2 * m : 4 * m] = u.x;
    x[HALF ? 2 * m + 1 : 4 * m + 2] = u.y;
    x[HALF ? 8 + 2 * m : 4 * m + 1] = v.x;
    x[HALF ? 9 + 2 * m : 4 * m + 3] = v.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(Pair<T>::put(f[0], f[1]), Pair<T>::put(f[2], f[3]), Pair<T>::put(f[4], f[5]), Pair<T>::put(f[6], f[7]));
}
// 8 values as e4m3, nearest, clamped to +-448 (NaN stays NaN)
__device__ __forceinline__ uint2 pack8_e4m3(const float* f) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Turns per position, inv_freq / (2 pi), as a multiple of 2^-64 modulo 2^64 (whole turns drop out; below 0: its complement):
// the frequency's mantissa times 130 bits of 1 / (2 pi), shifted by its exponent, off by less than one multiple for
// frequencies below 2^54 (0 above).  In whole numbers, because a double product is off by 2^-25 of a turn at 2^31
// positions and its correction in doubles takes 0.2 us of a small call.
__device__ __forceinline__ uint64_t turns_of(double inv_freq) {
  constexpr uint64_t kHi = 0xa2f9836e4e441529ull, kLo = 0xfc2757d1f534ddc0ull;      // 2^130 / (2 pi)
  const uint64_t bits = (uint64_t)__double_as_longlong(inv_freq);
  const uint64_t m = (bits & ((uint64_t(1) << 52) - 1)) | (uint64_t(1) << 52);
  const uint64_t part = m * kHi, lo = part + __umul64hi(m, kLo), hi = __umul64hi(m, kHi) + (lo < part ? 1 : 0);
  const int shift = 1077 - (int)((bits >> 52) & 0x7ff);                  // (hi, lo) 2^-shift
  uint64_t t = 0;
  if (shift >= 64 && shift < 128) t = hi >> (shift - 64);
  else if (shift > 0 && shift < 64) t = (lo >> shift) | (hi << (64 - shift));
  return (bits >> 63) != 0 ? 0 - t : t;
}

// Sines and cosines of two turns given in multiples of 2^-32: the nearest quarter taken off, and of what is left (u quarters,
// |u| <= 1/2) the Taylor polynomials to u^9 and u^8, whose next terms are below 2^-29 and 2^-25.  With the conversion of u and
// the roundings, all are within 2^-22.  (The fast functions' 2^-21 of an angle rounded to fp32 are 2^-20, and fp16 rows show
// them where a pair nearly cancels; they take 3 % less of an append of ten rows per token, and no less of one of 48.)
__device__ __forceinline__ void turn_sincos(uint32_t turn0, uint32_t turn1, float* sine, float* cosine) {
  const uint32_t quarter[2] = {(turn0 + 0x20000000u) >> 30, (turn1 + 0x20000000u) >> 30};
  auto both = [](float x) { return f2(x, x); };
  const F2 left = f2((float)(int32_t)(turn0 - (quarter[0] << 30)), (float)(int32_t)(turn1 - (quarter[1] << 30)));
  const F2 u = mul(left, both(0x1p-30f)), v = mul(u, u);
  // (pi / 2)^k / k!, their signs in turn
  F2 odd = fma(v, both(1.6044118479e-04f), both(-4.6817541353e-03f)), even = fma(v, both(9.1926027484e-04f), both(-2.0863480763e-02f));
  odd = fma(v, fma(v, fma(v, odd, both(7.9692626246e-02f)), both(-6.4596409751e-01f)), both(1.5707963268e+00f));
  even = fma(v, fma(v, fma(v, even, both(2.5366950790e-01f)), both(-1.2337005501e+00f)), both(1.f));
  const float2 sn = get(mul(u, odd)), cs = get(even);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float sv = e == 0 ? sn.x : sn.y, cv = e == 0 ? cs.x : cs.y;
    const float s = (quarter[e] & 1) != 0 ? cv : sv, c = (quarter[e] & 1) != 0 ? sv : cv;
    sine[e] = __uint_as_float(__float_as_uint(s) ^ (quarter[e] & 2) << 30);
    cosine[e] = __uint_as_float(__float_as_uint(c) ^ ((quarter[e] + 1) & 2) << 30);
  }
}

// Shared memory, in this order: the warps' stages, the warps' matrices of a token's pairs ([2 kinds][8][chunks + 1] float4:
// entry 2 m of chunk j holds (A, -B) of its pairs 2 m and 2 m + 1, entry 2 m + 1 holds (C, D)), weights [2][d], turns
// [rot / 2], the stages' barriers.
__host__ __device__ inline size_t rope_smem(int d, int rot) {
  return (size_t)kWarps * (kRingBytes + 2 * 8 * (d / 16 + 1) * 16) + (size_t)2 * d * 4 + (size_t)rot / 2 * 8 +
         (size_t)kWarps * kMaxStages * 8;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// GROUP: lanes of a head row (the power of two >= d / 16), or 0: found at run time.
template <typename T, bool HALF, int GROUP>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_append(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int chunks = a.d / 16, pitch = chunks + 1, pairs = a.rot / 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* stages = smem + (size_t)warp * kRingBytes;
  uint8_t* after = smem + (size_t)kWarps * kRingBytes;
  float4* mats = reinterpret_cast<float4*>(after) + warp * 2 * 8 * pitch;
  float* wts = reinterpret_cast<float*>(after + (size_t)kWarps * 2 * 8 * pitch * 16);
  uint64_t* turns = reinterpret_cast<uint64_t*>(wts + 2 * a.d);
  const uint32_t bar0 = sm100::smem_addr(turns + pairs) + warp * kMaxStages * 8;
  const uint32_t st0 = sm100::smem_addr(stages);
  int group = GROUP;
  if (GROUP == 0)
    for (group = 1; group < chunks;) group <<= 1;
  const int rows = 32 / group, sub = lane / group, j = lane % group;   // this lane: chunk j of row `sub` of `rows`
  const bool live = j < chunks, rotate = j < a.rot / 16;
  const int o0 = HALF && rotate ? 8 * j : 16 * j, o1 = HALF && rotate ? pairs + 8 * j : 16 * j + 8;

  if (lane == 0) {
    for (int i = 0; i < a.stages; ++i) sm100::mbar_init(bar0 + 8 * i, 1);
    sm100::fence_barrier_init();
  }
  __syncwarp();
  wait_for_earlier_kernels();
  const float inv_d = 1.f / (float)a.d;
  const int row_bytes = a.d * 2;
  // a token's rows, end to end: queries from 0, keys from bk, values from bv, `all` in all; a unit is unit_rows of them
  const int bk = a.q != nullptr ? a.h_q : 0, bv = bk + (a.k != nullptr ? a.h_kv : 0), all = bv + (a.k != nullptr ? a.h_kv : 0);
  const int total = (all + a.unit_rows - 1) / a.unit_rows;
  // This warp's units: a.rounds whole tokens, one in every n_w (so that all warps read and write near each other), then an
  // equal share of the units of the tokens that remain, `left` in all.  (i, u) is a unit, r the tokens before it.
  const int n_w = gridDim.x * kWarps, w = blockIdx.x * kWarps + warp;
  const int64_t first = a.share * w + min((int64_t)w, a.extra);
  const int rest_i = (first >> 31) == 0 ? (int)first / total : (int)(first / total);   // (a 32-bit division where it will do)
  const int rest_u = (int)(first - (int64_t)rest_i * total);
  int64_t left = (int64_t)a.rounds * total + a.share + (w < a.extra ? 1 : 0);
  auto next_token = [&](int i, int r) { return r < a.rounds ? i + n_w : r == a.rounds ? a.rounds * n_w + rest_i : i + 1; };
  int i = a.rounds > 0 ? w : rest_i, u = a.rounds > 0 ? 0 : rest_u, r = 0;

  // ---- the units' loads, a.stages - 2 ahead: the stage between them is the one whose rows are leaving
  int64_t lleft = left;
  int li = i, lu = u, lr = 0, lst = 0;                        // next unit to load, its stage
  auto load = [&]() {
    if (lleft == 0) return;
    --lleft;
    const int r0 = lu * a.unit_rows, r1 = min(r0 + a.unit_rows, all);
    const uint32_t dst = st0 + lst * a.stage_bytes, bar = bar0 + 8 * lst;
    if (lane == 0) sm100::mbar_expect_tx(bar, (r1 - r0) * row_bytes);
    __syncwarp();
    // rows lo .. hi - 1 of the unit, heads lo - base and on: one copy where they are contiguous
    auto part = [&](const void* p, int64_t ts, int64_t hs, int base, int end) {
      const int lo = max(r0, base), hi = min(r1, end);
      if (lo >= hi) return;
      const T* src = static_cast<const T*>(p) + li * ts + (lo - base) * hs;
      const uint32_t to = dst + (lo - r0) * row_bytes;
      if (hs == a.d) {
        if (lane == 0) bulk_load(to, src, (hi - lo) * row_bytes, bar);
      } else {
        for (int h = lane; h < hi - lo; h += 32) bulk_load(to + h * row_bytes, src + h * hs, row_bytes, bar);
      }
    };
    part(a.q, a.q_stride, a.q_head, 0, bk);
    part(a.k, a.k_stride, a.k_head, bk, bv);
    part(a.v, a.v_stride, a.v_head, bv, all);
    lst = lst == a.stages - 1 ? 0 : lst + 1;
    if (++lu == total) {
      ++lr;
      li = next_token(li, lr);
      lu = lr == a.rounds ? rest_u : 0;
    }
  };
  for (int e = 0; e < a.stages - 2; ++e) load();

  // ---- what all tokens share, while those land
  for (int x = threadIdx.x; x < 2 * a.d; x += kRopeThreads) {
    const T* w = static_cast<const T*>(x < a.d ? a.q_weight : a.k_weight);
    wts[x] = w != nullptr ? (float)w[x < a.d ? x : x - a.d] + a.bias : 1.f;
  }
  for (int x = threadIdx.x; x < pairs; x += kRopeThreads) turns[x] = turns_of(a.inv_freq[x]);
  __syncthreads();
  // the matrices of the elements that pass: their weights alone
  for (int x = lane; x < 2 * 8 * (chunks - a.rot / 16); x += 32) {
    const int kind = x / (8 * (chunks - a.rot / 16)), y = x % (8 * (chunks - a.rot / 16));
    const int c = a.rot / 16 + y / 8, p = y % 8;
    float* ab = reinterpret_cast<float*>(mats + (kind * 8 + p / 2 * 2) * pitch + c) + (p & 1);
    float* cd = reinterpret_cast<float*>(mats + (kind * 8 + p / 2 * 2 + 1) * pitch + c) + (p & 1);
    ab[0] = wts[kind * a.d + 16 * c + (HALF ? p : 2 * p)];
    cd[0] = wts[kind * a.d + 16 * c + (HALF ? 8 + p : 2 * p + 1)];
    ab[2] = cd[2] = 0.f;
  }


  int st = 0, phase = 0;
  int64_t next_slot = 0, next_pos = 0;                          // of the next token, read while this one is worked on
  auto look = [&](int token) {
    next_slot = a.slots != nullptr ? a.slots[token] : 0;
    next_pos = pairs > 0 ? a.positions[token] : 0;
  };
  if (left > 0) look(i);
  while (left > 0) {
    const int64_t slot = next_slot, pos = next_pos;
    if (left > total - u) look(next_token(i, r + 1));
    const bool cached = slot >= 0 && slot < a.n_slots;
    if (a.k != nullptr && !cached && slot != -1 && lane == 0 && u == 0) set_device_error(a.err, KVSEL_ERR_DEVICE, (uint32_t)i);
    int64_t at = 0;                                             // of the slot in the pool
    if (cached) {
      const int64_t page = (slot >> 31) == 0 ? (int)slot / a.P : slot / a.P;
      at = page * a.page_stride + (slot - page * a.P) * a.row_stride;
    }
    if (pairs > 0 && u * a.unit_rows < bv && slot != -1) {
      __syncwarp();                                             // the last token's matrices are read
      for (int c = lane; c < pairs / 2; c += 32) {              // pairs 2 c and 2 c + 1
        float sn[2], cs[2];
        auto turn_of = [&](int x) { return (uint32_t)((turns[x] * (uint64_t)pos + 0x80000000u) >> 32); };
        turn_sincos(turn_of(2 * c), turn_of(2 * c + 1), sn, cs);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sn[e] *= a.factor;
          cs[e] *= a.factor;
        }
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
          const float* wk = wts + kind * a.d;
          float2 wa, wb;
          if (HALF) {
            wa = *reinterpret_cast<const float2*>(wk + 2 * c);
            wb = *reinterpret_cast<const float2*>(wk + pairs + 2 * c);
          } else {
            const float4 v = *reinterpret_cast<const float4*>(wk + 4 * c);
            wa = make_float2(v.x, v.z);
            wb = make_float2(v.y, v.w);
          }
          float4* to = mats + (kind * 8 + c % 4 * 2) * pitch + c / 4;
          to[0] = make_float4(wa.x * cs[0], wa.y * cs[1], -(wb.x * sn[0]), -(wb.y * sn[1]));
          to[pitch] = make_float4(wb.x * cs[0], wb.y * cs[1], wa.x * sn[0], wa.y * sn[1]);
        }
      }
      __syncwarp();
    }
    for (; u < total && left > 0; ++u, --left) {
      const int r0 = u * a.unit_rows, r1 = min(r0 + a.unit_rows, all);
      // the next load goes into the stage stored before the last one: its bytes have left
      asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      __syncwarp();
      load();
      if (!__all_sync(0xffffffffu, sm100::mbar_wait(bar0 + 8 * st, phase))) {
        // the copies in flight land (or their own wait runs out) before the warp leaves
        if (lane == 0) set_device_error(a.err, KVSEL_ERR_TIMEOUT, 6u);
        for (int x = st + 1 < a.stages ? st + 1 : 0; x != lst; x = x + 1 < a.stages ? x + 1 : 0)
          sm100::mbar_wait(bar0 + 8 * x, phase ^ (x < st ? 1 : 0));
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        return;
      }
      uint8_t* stage = stages + st * a.stage_bytes;
      if (slot != -1) {                                         // (else padding)
        const int n = min(r1, a.e4m3 ? all : bv) - r0;          // 16-bit values go through as they are
        // R rows of every lane at once, hb and on: their sums and shuffles overlap.  Units of queries alone, the most of
        // them where there are many heads, share the matrices' reads and know no 8-bit rows.
        auto turn = [&](auto r_const, auto q_const, int hb) {
          constexpr int R = decltype(r_const)::value;
          constexpr bool Q = decltype(q_const)::value;
          bool on[R];
          int kind[R];                                          // a query, key or value row
          float scale[R], held[R];                              // held: what a row of an 8-bit pool is divided by
          F2 x[R][4], y[R][4];
#pragma unroll
          for (int t = 0; t < R; ++t) {
            const int h = hb + t * rows;
            on[t] = live && h < n;
            kind[t] = Q || r0 + h < bk ? 0 : r0 + h < bv ? 1 : 2;
            scale[t] = held[t] = 1.f;
            uint4 r[2];
            r[0] = r[1] = make_uint4(0, 0, 0, 0);
            if (on[t]) {
              r[0] = *reinterpret_cast<const uint4*>(stage + h * row_bytes + 2 * o0);
              r[1] = *reinterpret_cast<const uint4*>(stage + h * row_bytes + 2 * o1);
              if (!Q && kind[t] > 0 && a.e4m3) held[t] = kind[t] == 1 ? a.k_scale[r0 + h - bk] : a.v_scale[r0 + h - bv];
            }
            unpack16<T, HALF>(r, x[t], y[t]);
          }
          if (a.q_weight != nullptr || (!Q && a.k_weight != nullptr)) {
            float ss[R];
#pragma unroll
            for (int t = 0; t < R; ++t) {
              F2 s2 = mul(x[t][0], x[t][0]), t2 = mul(y[t][0], y[t][0]);
#pragma unroll
              for (int m = 1; m < 4; ++m) {
                s2 = fma(x[t][m], x[t][m], s2);
                t2 = fma(y[t][m], y[t][m], t2);
              }
              const float2 sf = get(s2), tf = get(t2);
              ss[t] = (sf.x + sf.y) + (tf.x + tf.y);
            }
            if (GROUP > 0) {
#pragma unroll
              for (int o = GROUP / 2; o > 0; o >>= 1)
#pragma unroll
                for (int t = 0; t < R; ++t) ss[t] += __shfl_xor_sync(0xffffffffu, ss[t], o);
            } else {
              for (int o = group >> 1; o > 0; o >>= 1)
#pragma unroll
                for (int t = 0; t < R; ++t) ss[t] += __shfl_xor_sync(0xffffffffu, ss[t], o);
            }
#pragma unroll
            for (int t = 0; t < R; ++t)
              if (kind[t] < 2 && (kind[t] == 0 ? a.q_weight : a.k_weight) != nullptr) scale[t] *= rsqrtf(fmaf(ss[t], inv_d, a.eps));
          }
          auto apply = [&](int t, int m, float4 ab, float4 cd) {
            const F2 p = x[t][m], q = y[t][m];
            x[t][m] = mul(p, f2(ab.x, ab.y));
            y[t][m] = mul(q, f2(cd.x, cd.y));
            if (rotate) {
              x[t][m] = fma(q, f2(ab.z, ab.w), x[t][m]);
              y[t][m] = fma(p, f2(cd.z, cd.w), y[t][m]);
            }
          };
          if (Q) {
            if (live)
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const float4 ab = mats[2 * m * pitch + j], cd = mats[(2 * m + 1) * pitch + j];
#pragma unroll
                for (int t = 0; t < R; ++t) apply(t, m, ab, cd);
              }
          } else {
#pragma unroll
            for (int t = 0; t < R; ++t) {
              const float4* mt = mats + kind[t] * 8 * pitch + j;
              if (live && kind[t] < 2)
#pragma unroll
                for (int m = 0; m < 4; ++m) apply(t, m, mt[2 * m * pitch], mt[(2 * m + 1) * pitch]);
            }
          }
          if (!Q && a.e4m3) __syncwarp();                             // a row's bytes lie over its lanes' values
#pragma unroll
          for (int t = 0; t < R; ++t) {
            const bool quotient = !Q && kind[t] > 0 && a.e4m3;
            const float s1 = quotient ? -scale[t] : scale[t];
            const F2 s2 = f2(s1, s1);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              x[t][m] = mul(x[t][m], s2);
              y[t][m] = mul(y[t][m], s2);
            }
            if (quotient) {
              const float inv = -1.f / held[t], res = fabsf(held[t]) < 0x1p-60f ? 0.f : inv;
              const Divisor by = {f2(held[t], held[t]), f2(inv, inv), f2(res, res)};
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                x[t][m] = divide_neg(x[t][m], by);
                y[t][m] = divide_neg(y[t][m], by);
              }
            }
            float f[16];
            order16<HALF>(x[t], y[t], f);
            if (!on[t]) continue;
            uint8_t* row = stage + (hb + t * rows) * row_bytes;
            if (quotient) {
              *reinterpret_cast<uint2*>(row + o0) = pack8_e4m3(f);
              *reinterpret_cast<uint2*>(row + o1) = pack8_e4m3(f + 8);
            } else {
              *reinterpret_cast<uint4*>(row + 2 * o0) = pack8<T>(f);
              *reinterpret_cast<uint4*>(row + 2 * o1) = pack8<T>(f + 8);
            }
          }
        };
        auto turn_all = [&](auto q_const) {
          int hb = sub;
          for (; hb - sub + rows < n; hb += 2 * rows) turn(std::integral_constant<int, 2>(), q_const, hb);
          if (hb - sub < n) turn(std::integral_constant<int, 1>(), q_const, hb);
        };
        if (r1 <= bk) turn_all(std::true_type());
        else turn_all(std::false_type());
      }
      sm100::fence_proxy_async_smem();
      __syncwarp();
      if (slot != -1) {
        const uint32_t from = st0 + st * a.stage_bytes;
        const int hi = min(r1, bk);
        if (r0 < hi && lane == 0) bulk_store(static_cast<T*>(a.q_out) + ((int64_t)i * a.h_q + r0) * a.d, from, (hi - r0) * row_bytes);
        const int eb = a.e4m3 ? 1 : 2;
        auto part = [&](void* pool, int base, int end) {
          const int lo = max(r0, base), hi = min(r1, end);
          if (lo >= hi || !cached) return;
          uint8_t* dst = static_cast<uint8_t*>(pool) + (at + (lo - base) * a.head_stride) * eb;
          const uint32_t src = from + (lo - r0) * row_bytes;
          if (a.head_stride == a.d && !a.e4m3) {
            if (lane == 0) bulk_store(dst, src, (hi - lo) * row_bytes);
          } else {
            for (int h = lane; h < hi - lo; h += 32) bulk_store(dst + h * a.head_stride * eb, src + h * row_bytes, a.d * eb);
          }
        };
        part(a.k_cache, bk, bv);
        part(a.v_cache, bv, all);
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      if (++st == a.stages) {
        st = 0;
        phase ^= 1;
      }
    }
    ++r;
    i = next_token(i, r);
    u = r == a.rounds ? rest_u : 0;
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // written before the kernel ends
}

}  // namespace

kvsel_status launch_rope_append(const RopeArgs& in, int32_t dtype, int32_t layout, cudaStream_t s) {
  using Kernel = void (*)(const RopeArgs);
  RopeArgs a = in;
  int group = 1;
  while (group < a.d / 16) group <<= 1;
  // units of equal size, whole steps of `rows` rows where there are several
  const int rows = 32 / group, all = (a.q != nullptr ? a.h_q : 0) + (a.k != nullptr ? 2 * a.h_kv : 0);
  const int fit = std::max(1, kUnitBytes / (2 * a.d) / rows) * rows;
  const int each = (int)ceil_div(all, ceil_div(all, fit));
  a.unit_rows = std::min(fit, (int)ceil_div(each, rows) * rows);
  const int64_t units = ceil_div(all, a.unit_rows);
  a.stage_bytes = std::min(a.unit_rows, all) * 2 * a.d;
  a.stages = std::min(kMaxStages, kRingBytes / a.stage_bytes);
  const bool half = layout == KVSEL_ROPE_HALF;
  auto pick = [&](auto t) -> Kernel {
    using T = decltype(t);
    if (group == 8) return half ? rope_append<T, true, 8> : rope_append<T, false, 8>;
    if (group == 4) return half ? rope_append<T, true, 4> : rope_append<T, false, 4>;
    return half ? rope_append<T, true, 0> : rope_append<T, false, 0>;
  };
  const Kernel kern = dtype == KVSEL_DTYPE_BF16 ? pick(__nv_bfloat16()) : pick(__half());
  const size_t smem = rope_smem(a.d, a.rot);
  const int64_t resident = resident_ctas((const void*)kern, kRopeThreads, smem);
  if (resident <= 0) return KVSEL_ERR_CUDA;
  const int64_t grid = std::min(resident, ceil_div(a.n * units, kWarps));
  const int64_t n_w = grid * kWarps;
  a.rounds = (int32_t)(a.n / n_w);
  a.share = a.n % n_w * units / n_w;
  a.extra = a.n % n_w * units % n_w;
  TraceScope ts("rope_append", s);
  return launch_after(kern, dim3((unsigned)grid), kRopeThreads, smem, s, a);
}

}  // namespace kvsel
