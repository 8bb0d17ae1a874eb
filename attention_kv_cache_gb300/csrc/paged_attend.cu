// Attention over a paged pool: the merge of the requests' pieces, and the launches (the kernels are in paged_attend.cuh).
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "paged_attend.cuh"

namespace kvsel {
namespace {

// o of a request that several lanes hold: sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over its pieces i.
// blockIdx.y is the request (or the lane) whose span says which pieces; blockIdx.x takes `heads` query heads of it.
// A request of few pieces gives a warp to each head; of many, all warps to one head after another, each warp every
// WARPS-th piece.  A warp loads LOADS pieces at once, offsets and rows together, and keeps its own running
// offset: latency is what this costs, so nothing waits for anything but the span.
//
// Launched while the attention runs (its CTAs fit beside it) and waiting for its end, so that no launch lies between.
constexpr int kFewPieces = 16;
template <int D, int WARPS, int LOADS>
__global__ void __launch_bounds__(32 * WARPS) paged_join(const __grid_constant__ PagedArgs a, int nt8, int heads) {
  constexpr int V = D / 32;                         // values of a row per lane
  using Vec = typename std::conditional<V == 4, float4, float2>::type;
  __shared__ Vec red[WARPS][32];
  __shared__ float2 redml[WARPS];
  wait_for_earlier_kernels();
  const int2 span = a.span[blockIdx.y];
  const int b = a.by_lane ? span.x : blockIdx.y, i0 = a.by_lane ? blockIdx.y : span.x, i1 = span.y;
  if (i0 >= i1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int padded = a.h_kv * a.tiles * nt8;
  const bool few = heads > 1 && i1 - i0 < kFewPieces;
  for (int hh = few ? warp : 0; hh < heads; hh += few ? WARPS : 1) {
    const int h = blockIdx.x * heads + hh;
    if (h >= a.h_q) return;                         // (the whole CTA where its warps share a head)
    const int g = h / a.G;
    const int at = g * a.tiles * nt8 + (h - g * a.G);                    // the head among the padded heads
    float M = -INFINITY, den = 0.f, num[V];
#pragma unroll
    for (int e = 0; e < V; ++e) num[e] = 0.f;
    // (offset, sum, row) taken into the warp's own; a piece whose scores were all NaN, or none, has offset -inf
    auto take = [&](float2 ml, const float* v) {
      const float top = fmaxf(M, ml.x);
      const float wo = M == top ? 1.f : exp2f(M - top), wn = ml.x == top ? 1.f : exp2f(ml.x - top);
      M = top;
      den = den * wo + ml.y * wn;
#pragma unroll
      for (int e = 0; e < V; ++e) num[e] = num[e] * wo + v[e] * wn;
    };
    const int step = few ? 1 : WARPS;
    for (int i = i0 + (few ? 0 : warp); i <= i1; i += LOADS * step) {
      float2 ml[LOADS];
      Vec v[LOADS];
#pragma unroll
      for (int k = 0; k < LOADS; ++k)
        if (i + k * step <= i1) {
          const int64_t r = (int64_t)(2 * (i + k * step) + (i + k * step == i0 ? 1 : 0)) * padded + at;
          ml[k] = a.part_ml[r];
          v[k] = reinterpret_cast<const Vec*>(a.part + r * D)[lane];
        }
#pragma unroll
      for (int k = 0; k < LOADS; ++k)
        if (i + k * step <= i1) take(ml[k], reinterpret_cast<const float*>(&v[k]));
    }
    if (!few) {
      __syncthreads();                              // the last head's sums are read
#pragma unroll
      for (int e = 0; e < V; ++e) reinterpret_cast<float*>(&red[warp][lane])[e] = num[e];
      if (lane == 0) redml[warp] = make_float2(M, den);
      __syncthreads();
      if (warp != 0) continue;
#pragma unroll
      for (int i = 1; i < WARPS; ++i) take(redml[i], reinterpret_cast<const float*>(&red[i][lane]));
    }
    const float s = den == 0.f ? 0.f : (a.v_scale != nullptr ? a.v_scale[g] : 1.f) / a.unit / den;
    const int64_t oh = (int64_t)b * a.h_q + h;
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      uint32_t u;
      if (a.out_f16) {
        const __half2 y = __floats2half2_rn(num[e] * s, num[e + 1] * s);
        u = *reinterpret_cast<const uint32_t*>(&y);
      } else {
        const __nv_bfloat162 y = __floats2bfloat162_rn(num[e] * s, num[e + 1] * s);
        u = *reinterpret_cast<const uint32_t*>(&y);
      }
      static_cast<uint32_t*>(a.o)[(oh * D + V * lane + e) / 2] = u;
    }
    if (a.lse != nullptr && lane == 0) a.lse[oh] = (M + log2f(den)) * 0.6931471805599453f;
  }
}

PagedVariant variant(const PagedShape& p, int nt) {
  if (p.cache_dtype == KVSEL_DTYPE_E4M3) return paged_variant_e4m3(p.d, nt);
  return p.dtype == KVSEL_DTYPE_F16 ? paged_variant_f16(p.d, nt) : paged_variant_bf16(p.d, nt);
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
  int sms, nt, tiles, lanes, grid, by_lane, solo;
  size_t span_off, ml_off, part_off, total;
};
// One CTA per SM, fewer when the bound on the steps needs fewer warps.
bool geometry(const PagedShape& p, Geometry* out) {
  const int sms = sm_count();
  if (sms <= 0) return false;
  const int G = p.h_q / p.h_kv;
  Geometry& o = *out;
  o.sms = sms;
  o.nt = G <= 8 ? 1 : 2;
  o.tiles = (int)ceil_div(G, 8 * o.nt);
  const PagedVariant v = variant(p, o.nt);
  const int64_t units = (int64_t)p.h_kv * o.tiles;
  // steps of one request at most, by its table and by the window (whose rows may begin and end inside a step)
  int64_t most = ceil_div((int64_t)p.max_blocks * p.P, kKeys);
  if (p.window > 0) most = std::min<int64_t>(most, ceil_div((int64_t)p.window + kKeys - 1, kKeys));
  const int64_t lanes = std::min<int64_t>(std::max<int64_t>(1, (int64_t)sms * v.warps / units),
                                          std::max<int64_t>(1, most * p.batch));
  o.lanes = (int)lanes;
  o.grid = (int)std::min<int64_t>(sms, ceil_div(lanes * units, v.warps));
  // Short calls, all of whose CTAs run at once.  Lanes use every SM, a CTA per request and unit `ctas` of them, which
  // takes about (most / warps) (1 - ctas / SMs) steps longer; the join and its launch take about as long as 4 (us, by
  // requests x rows, 8 KV heads of 128: 1 x 400 7.0 against 7.3 by lanes, 16 x 400 7.5 / 17, 16 x 800 13.3 / 17.3,
  // 1 x 800 9.9 / 7.5, 1 x 1600 15.2 / 7.9).  kSoloSteps bounds what one long request among short ones can cost.
  const int64_t ctas = units * p.batch;
  o.solo = ctas <= sms && most <= (int64_t)kSoloSteps * v.warps && most * (sms - ctas) <= (int64_t)4 * v.warps * sms;
  if (o.solo) o.grid = (int)ctas;
  const int64_t heads = units * 8 * o.nt;
  auto up = [](size_t x) { return (x + KVSEL_WS_ALIGN - 1) / KVSEL_WS_ALIGN * KVSEL_WS_ALIGN; };
  o.by_lane = !o.solo && p.batch > lanes;
  o.span_off = sizeof(DeviceError);
  o.ml_off = up(o.span_off + sizeof(int2) * (size_t)(o.by_lane ? lanes : p.batch));
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
  const PagedVariant var = variant(p, geo.nt);
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
  a.span = reinterpret_cast<int2*>(base + geo.span_off);
  a.part_ml = reinterpret_cast<float2*>(base + geo.ml_off);
  a.part = reinterpret_cast<float*>(base + geo.part_off);
  a.err = reinterpret_cast<DeviceError*>(ws);
  a.page_stride = p.page_stride;
  a.head_stride = p.head_stride;
  a.row_stride = p.row_stride;
  a.q_stride = p.q_stride;
  a.scale = p.scale;
  a.softcap = p.softcap;
  a.unit = p.cache_dtype == KVSEL_DTYPE_BF16 ? weight_unit<kBf16>() : weight_unit<kF16>();
  a.h_q = p.h_q;
  a.h_kv = p.h_kv;
  a.G = p.h_q / p.h_kv;
  a.P = p.P;
  a.p_shift = 0;
  while ((1 << a.p_shift) < p.P) ++a.p_shift;
  a.p_mul = (uint32_t)((((uint64_t)1 << 32) * ((1u << a.p_shift) - (uint32_t)p.P)) / (uint32_t)p.P + 1);
  a.batch = p.batch;
  a.max_blocks = p.max_blocks;
  a.n_pages = p.n_pages;
  a.window = p.window;
  a.out_f16 = p.dtype == KVSEL_DTYPE_F16;
  a.tiles = geo.tiles;
  a.lanes = geo.lanes;
  a.by_lane = geo.by_lane;
  a.solo = geo.solo;
  const size_t smem = var.smem + sizeof(int2) * (size_t)p.batch;
  if (set_smem((const void*)var.kern, smem) != cudaSuccess) return KVSEL_ERR_CUDA;
  {
    TraceScope ts("paged_attend", s);
    const kvsel_status st = launch_after(var.kern, dim3(geo.grid), 32 * var.warps, smem, s, a);
    if (st != KVSEL_OK || geo.solo) return st;
  }
  TraceScope ts("paged_join", s);
  const int rows = geo.by_lane ? geo.lanes : p.batch;
  // Requests of many pieces: a CTA of 16 warps for each head, while those are at most four to an SM; else a warp per head in
  // CTAs of 4.
  // More requests than lanes have two or three pieces each: few loads at once, few registers, all CTAs at once (256
  // requests of 1-300 rows 33.7 -> 29.7 us, of 1-4095 rows 141 -> 136).
  const bool split = geo.lanes / rows >= kFewPieces && (int64_t)rows * p.h_q <= 4 * geo.sms;
  using Join = void (*)(const PagedArgs, int, int);
  Join join;
  if (p.d == 64) join = split ? paged_join<64, 16, 10> : geo.by_lane ? paged_join<64, 4, 2> : paged_join<64, 4, 10>;
  else join = split ? paged_join<128, 16, 10> : geo.by_lane ? paged_join<128, 4, 2> : paged_join<128, 4, 10>;
  const int warps = split ? 16 : 4, heads = split ? 1 : 4;
  return launch_after(join, dim3((unsigned)ceil_div(p.h_q, heads), (unsigned)rows), 32 * warps, 0, s, a, 8 * geo.nt, heads);
}

}  // namespace kvsel
