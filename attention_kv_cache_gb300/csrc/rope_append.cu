// RMS norm of every query and key head, rotary positions, and the new K / V rows into the paged pool.
//
// y = x rsqrt(mean(x^2) + eps) (w + bias), then the pairs (a, b) of the first `rot` elements become
// factor (a cos - b sin, b cos + a sin) of the angle position * inv_freq.
//
// The angle is formed in turns as a 64-bit fraction: inv_freq / (2 pi) as a multiple of 2^-64 times the
// position, modulo 2^64, is the fraction of a turn exactly up to position * 2^-65, so a far position loses
// nothing that a 32-bit product of position and frequency would lose; the top 32 bits go to sincospif.
//
// One pass over the data: a head row is d / 16 lanes of 16 elements, chosen so that both elements of a
// pair lie in one lane (elements 8 j .. 8 j + 7 and rot / 2 + 8 j .. of a half layout, 16 j .. 16 j + 15 of
// an interleaved one), so a row is read once, summed by shuffles, turned in registers and written once.
// A warp takes the head rows of one token, 32 / (lanes of a row) at a time, and forms its lanes' 8 angles
// once for all of them; with few tokens the rows of a token are dealt over several warps.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "paged.cuh"

namespace kvsel {
namespace {

constexpr int kRopeThreads = 256;

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

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = Pair<T>::get(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
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

// One lane's 16 elements of a head row, normed and turned.
template <typename T, bool HALF>
__device__ __forceinline__ void turn(float* x, bool norm, const float* w, bool rotate, const float* cs, const float* sn,
                                     float inv_d, float eps, int group) {
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
    for (int o = group >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(fmaf(ss, inv_d, eps));
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
  }
  if (rotate) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ia = HALF ? i : 2 * i, ib = HALF ? i + 8 : 2 * i + 1;
      const float a = x[ia], b = x[ib];
      x[ia] = fmaf(a, cs[i], -(b * sn[i]));
      x[ib] = fmaf(b, cs[i], a * sn[i]);
    }
  }
}

template <typename T, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_append(const __grid_constant__ RopeArgs a, int parts) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t i = w / parts;
  const int part = (int)(w - i * parts);
  if (i >= a.n) return;
  const int64_t slot = a.slots != nullptr ? a.slots[i] : 0;
  if (slot == -1) return;                                       // padding: nothing is written
  bool cached = a.k != nullptr;
  if (cached && (slot < 0 || slot >= a.n_slots)) {
    if (lane == 0 && part == 0) set_device_error(a.err, KVSEL_ERR_DEVICE, (uint32_t)i);
    cached = false;
  }
  // this lane's elements: chunk j of a head row, rows `sub` of every `rows` rows taken at a time
  const int chunks = a.d / 16;
  int group = 1;
  while (group < chunks) group <<= 1;
  const int rows = 32 / group, sub = lane / group, j = lane % group;
  const bool live = j < chunks;
  const bool rotate = j < a.rot / 16;
  const int o0 = HALF && rotate ? 8 * j : 16 * j, o1 = HALF && rotate ? a.rot / 2 + 8 * j : 16 * j + 8;
  const int iq = a.q != nullptr ? (a.h_q + rows - 1) / rows : 0, ik = cached ? (a.h_kv + rows - 1) / rows : 0;
  const int total = iq + 2 * ik;
  const int u0 = (int)((int64_t)total * part / parts), u1 = (int)((int64_t)total * (part + 1) / parts);
  float cs[8], sn[8];
  if (rotate && u0 < iq + ik) {
    const int64_t pos = a.positions[i];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      // turns per position as a signed multiple of 2^-64 (whole turns drop out), times the position
      double f = a.inv_freq[8 * j + p] * 0.15915494309189533577;
      f -= rint(f);
      const int64_t turns = __double2ll_rn(f * 18446744073709551616.0) * pos;
      sincospif((float)(int32_t)(turns >> 32) * 4.656612873077393e-10f, &sn[p], &cs[p]);
      cs[p] *= a.factor;
      sn[p] *= a.factor;
    }
  }
  const float inv_d = 1.f / (float)a.d;
  const int64_t page = slot / a.P;
  const int64_t at = page * a.page_stride + (slot - page * a.P) * a.row_stride;
  for (int u = u0; u < u1; ++u) {
    const int kind = u < iq ? 0 : u < iq + ik ? 1 : 2;          // a query, key or value row
    const int h = (u - (kind == 0 ? 0 : kind == 1 ? iq : iq + ik)) * rows + sub;
    const bool on = live && h < (kind == 0 ? a.h_q : a.h_kv);
    const T* src = kind == 0   ? static_cast<const T*>(a.q) + i * a.q_stride + h * a.q_head
                   : kind == 1 ? static_cast<const T*>(a.k) + i * a.k_stride + h * a.k_head
                               : static_cast<const T*>(a.v) + i * a.v_stride + h * a.v_head;
    float x[16];
    uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
    if (on) {
      r0 = *reinterpret_cast<const uint4*>(src + o0);
      r1 = *reinterpret_cast<const uint4*>(src + o1);
    }
    unpack8<T>(r0, x);
    unpack8<T>(r1, x + 8);
    if (kind < 2) {
      const T* wt = static_cast<const T*>(kind == 0 ? a.q_weight : a.k_weight);
      float wf[16];
      if (wt != nullptr && live) {
        unpack8<T>(*reinterpret_cast<const uint4*>(wt + o0), wf);
        unpack8<T>(*reinterpret_cast<const uint4*>(wt + o1), wf + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e) wf[e] += a.bias;
      }
      turn<T, HALF>(x, wt != nullptr, wf, rotate, cs, sn, inv_d, a.eps, group);
    }
    if (!on) continue;
    if (kind == 0) {
      T* dst = static_cast<T*>(a.q_out) + (i * a.h_q + h) * a.d;
      *reinterpret_cast<uint4*>(dst + o0) = pack8<T>(x);
      *reinterpret_cast<uint4*>(dst + o1) = pack8<T>(x + 8);
    } else {
      const int64_t to = at + h * a.head_stride;
      void* pool = kind == 1 ? a.k_cache : a.v_cache;
      if (a.e4m3) {
        const float s = 1.f / (kind == 1 ? a.k_scale : a.v_scale)[h];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= s;
        uint8_t* dst = static_cast<uint8_t*>(pool) + to;
        *reinterpret_cast<uint2*>(dst + o0) = pack8_e4m3(x);
        *reinterpret_cast<uint2*>(dst + o1) = pack8_e4m3(x + 8);
      } else {
        T* dst = static_cast<T*>(pool) + to;
        *reinterpret_cast<uint4*>(dst + o0) = kind == 1 ? pack8<T>(x) : r0;
        *reinterpret_cast<uint4*>(dst + o1) = kind == 1 ? pack8<T>(x + 8) : r1;
      }
    }
  }
}

}  // namespace

kvsel_status launch_rope_append(const RopeArgs& a, int32_t dtype, int32_t layout, cudaStream_t s) {
  int group = 1;
  while (group < a.d / 16) group <<= 1;
  const int rows = 32 / group;
  const int total = (a.q != nullptr ? (a.h_q + rows - 1) / rows : 0) + (a.k != nullptr ? 2 * ((a.h_kv + rows - 1) / rows) : 0);
  int64_t parts = ceil_div(152 * 16, a.n);
  if (parts > total) parts = total;
  const int64_t grid = ceil_div(a.n * parts, kRopeThreads / 32);
  if (grid >= (int64_t(1) << 31)) return KVSEL_ERR_UNSUPPORTED;
  TraceScope ts("rope_append", s);
  const bool half = layout == KVSEL_ROPE_HALF;
  if (dtype == KVSEL_DTYPE_BF16) {
    if (half) rope_append<__nv_bfloat16, true><<<(unsigned)grid, kRopeThreads, 0, s>>>(a, (int)parts);
    else rope_append<__nv_bfloat16, false><<<(unsigned)grid, kRopeThreads, 0, s>>>(a, (int)parts);
  } else {
    if (half) rope_append<__half, true><<<(unsigned)grid, kRopeThreads, 0, s>>>(a, (int)parts);
    else rope_append<__half, false><<<(unsigned)grid, kRopeThreads, 0, s>>>(a, (int)parts);
  }
  return launch_status();
}

}  // namespace kvsel
