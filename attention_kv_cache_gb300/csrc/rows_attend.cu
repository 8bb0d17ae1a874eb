// Attention of many rows over a paged pool: the plan of a call's items, the merge of cut items, and the launches (the kernels
// are in rows_attend.cuh).
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "rows_attend.cuh"

namespace kvsel {
namespace {

constexpr int kPlanThreads = 1024;            // (256 for few jobs and items: what the plan costs is latency)
constexpr int kPlanItems = 4096;              // items whose first steps the plan keeps in shared memory

// Inclusive sum over the CTA's threads; `all`: of all of them.
__device__ int64_t plan_scan(int64_t x, int64_t* warp_sum, int64_t& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int64_t before = 0;
  all = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    all += warp_sum[w];
  }
  return before + x;
}

__device__ __forceinline__ int find_job(const int32_t* first, int n, int x) {
  int lo = 0, hi = n;                         // first[lo] <= x < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// (hi - k0 + 127 may pass 2^31)
__device__ __forceinline__ int steps_of(const RowsItem& it) { return (int)(((uint32_t)(it.hi - it.k0) + kTileKeys - 1) / kTileKeys); }

// The items, `make(i)` for each, with the steps of the items before it; then all steps, and where the CTAs' shares begin.
template <typename Make>
__device__ __forceinline__ void put_items(const RowsArgs& a, int n_items, int64_t* warp_sum, int32_t* step_sm, Make make) {
  int64_t steps = 0;
  for (int i0 = 0; i0 < n_items; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    RowsItem it = {};
    if (i < n_items) it = make(i);
    int64_t all;
    const int64_t upto = plan_scan(it.steps, warp_sum, all);
    if (i < n_items) {
      it.step0 = (int32_t)(steps + upto - it.steps);
      a.items[i] = it;
      if (i < kPlanItems) step_sm[i] = it.step0;
    }
    steps += all;
  }
  __syncthreads();
  const int64_t W = steps * a.h_kv;
  const int N = (int)min((int64_t)a.grid, W);
  if (threadIdx.x == 0) *a.plan = RowsPlan{steps, n_items, N};
  for (int i = threadIdx.x; i < a.grid; i += blockDim.x) {
    RowsStart st = {};
    if (i < N) {
      const int64_t x = lane_begin64(i, W, N);
      const int g = (int)(x / steps), y = (int)(x - g * steps);
      int lo = 0, hi = n_items;               // the last item that begins at or before y (items without steps come before it)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((n_items <= kPlanItems ? step_sm[mid] : a.items[mid].step0) <= y) lo = mid; else hi = mid;
      }
      st.steps = lane_begin64(i + 1, W, N) - x;
      st.g = g;
      st.at = lo;
      st.n_items = n_items;
      st.item = a.items[lo];
      st.step = y - st.item.step0;
    }
    a.starts[i] = st;
  }
}

// Items of a chunk call: the rows of every request's new tokens, 256 at a time.
__global__ void __launch_bounds__(kPlanThreads) chunk_plan(const __grid_constant__ RowsArgs a) {
  extern __shared__ int32_t first[];          // [batch + 1] items before each request, [batch] its tokens, then the items' steps
  __shared__ int64_t warp_sum[kPlanThreads / 32];
  int32_t* n_tok = first + a.jobs + 1;
  wait_for_earlier_kernels();
  let_later_kernels_start();
  const int64_t cap = (int64_t)a.max_blocks * a.P;
  int64_t items = 0;
  for (int b0 = 0; b0 < a.jobs; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int64_t n = 0;
    if (b < a.jobs) {
      const int64_t x = a.first[b], y = a.first[b + 1], len = a.lens[b];
      if (x < 0 || y < x || y > a.max_tokens || len < 0 || len > cap || y - x > len)
        set_device_error(a.err, KVSEL_ERR_INVALID_ARG, (uint32_t)b);
      else
        n = y - x;
      n_tok[b] = (int32_t)n;
    }
    const int64_t t = (n * a.G + kItemRows - 1) / kItemRows;
    int64_t all;
    const int64_t upto = plan_scan(t, warp_sum, all);
    if (b < a.jobs) first[b] = (int32_t)(items + upto - t);
    items += all;
  }
  // (offsets that overlap, which rise nevertheless, cannot give more items than the tokens allow)
  const int n_items = (int)min(items, (int64_t)a.max_items);
  if (threadIdx.x == 0) first[a.jobs] = n_items;
  __syncthreads();
  put_items(a, n_items, warp_sum, n_tok + a.jobs, [&](int i) {
    const int b = find_job(first, a.jobs, i);
    RowsItem it = {};
    const int n = n_tok[b];
    it.table = b;
    it.token0 = (int32_t)a.first[b];
    it.base = (int32_t)a.lens[b] - n;
    it.row0 = (i - first[b]) * kItemRows;
    it.rows = (int)min((int64_t)kItemRows, (int64_t)n * a.G - it.row0);
    const int p0 = it.base + it.row0 / a.G, p1 = it.base + (it.row0 + it.rows - 1) / a.G;    // its first and last token's rows
    it.hi = p1 + 1;
    it.lo = a.window > 0 ? max(0, p0 + 1 - a.window) : 0;
    it.full_hi = p0 + 1;
    it.full_lo = a.window > 0 ? max(0, p1 + 1 - a.window) : 0;
    it.k0 = it.lo / kTileKeys * kTileKeys;
    it.steps = steps_of(it);
    return it;
  });
}

// Shared whole pages of group j, 0 where they cannot be shared; all threads of the CTA call it.
__device__ int shared_pages(const RowsArgs& a, int64_t r0, int64_t r1, int64_t shared) {
  __shared__ int unfit;
  __syncthreads();
  if (threadIdx.x == 0) unfit = 0;
  __syncthreads();
  const int64_t cap = (int64_t)a.max_blocks * a.P;
  for (int64_t r = r0 + threadIdx.x; r < r1; r += blockDim.x) {
    const int64_t len = a.lens[r];
    if (shared < 0 || len < shared || len > cap) unfit = 1;
  }
  __syncthreads();
  return unfit != 0 ? 0 : (int)(shared / a.P);
}
// Whether the groups' offsets run from 0 to batch.
__device__ bool groups_ok(const RowsArgs& a) {
  bool ok = true;
  for (int j = threadIdx.x; j < a.jobs; j += blockDim.x) ok &= a.first[j] >= 0 && a.first[j] <= a.first[j + 1] && a.first[j + 1] <= a.batch;
  if (threadIdx.x == 0) ok &= a.first[0] == 0 && a.first[a.jobs] == a.batch;
  return __syncthreads_and(ok) != 0;
}

// Of the requests (dealt to the CTAs from the second on): their tables behind the shared pages, and their rows left.
// The first CTA makes the items: the rows of every group's requests, 256 at a time, over the shared rows.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan(const __grid_constant__ RowsArgs a) {
  extern __shared__ int32_t first[];          // [groups + 1] items before each group, [groups] its shared rows, then the items' steps
  __shared__ int64_t warp_sum[kPlanThreads / 32];
  int32_t* rows_of = first + a.jobs + 1;
  wait_for_earlier_kernels();
  let_later_kernels_start();
  const bool ok = groups_ok(a);
  if (blockIdx.x > 0) {
    for (int r = blockIdx.x - 1; r < a.batch; r += gridDim.x - 1) {
      int skip = 0;
      if (ok) {
        int lo = 0, hi = a.jobs;              // the group with first[lo] <= r < first[lo + 1]: the last that begins there or before
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (a.first[mid] <= r) lo = mid; else hi = mid;
        }
        skip = shared_pages(a, a.first[lo], a.first[lo + 1], a.shared[lo]);
      }
      const int64_t len = a.lens[r], left = len - (int64_t)skip * a.P;
      if (threadIdx.x == 0) a.own_lens[r] = left;
      const int n = left > 0 && len <= (int64_t)a.max_blocks * a.P ? (int)((left + a.P - 1) / a.P) : 0;
      for (int c = threadIdx.x; c < n; c += blockDim.x)
        a.own_tables[(int64_t)r * a.max_blocks + c] = a.tables[(int64_t)r * a.max_blocks + skip + c];
    }
    return;
  }
  if (!ok && threadIdx.x == 0) set_device_error(a.err, KVSEL_ERR_INVALID_ARG, (uint32_t)a.batch);
  const int jobs = ok ? a.jobs : 1;
  // groups, a warp each: their shared rows; then their items
  const int64_t cap = (int64_t)a.max_blocks * a.P;
  for (int j = threadIdx.x >> 5; j < jobs; j += blockDim.x / 32) {
    const int64_t r0 = ok ? a.first[j] : 0, r1 = ok ? a.first[j + 1] : a.batch, shared = ok ? a.shared[j] : 0;
    bool low = shared < 0, over = false;
    for (int64_t r = r0 + (threadIdx.x & 31); r < r1; r += 32) {
      const int64_t len = a.lens[r];
      low |= len < shared;
      over |= len > cap;
    }
    low = __any_sync(0xffffffffu, low && r1 > r0) && shared != 0;
    over = __any_sync(0xffffffffu, over);
    if ((threadIdx.x & 31) == 0) {
      if (low) set_device_error(a.err, KVSEL_ERR_INVALID_ARG, (uint32_t)r0);
      rows_of[j] = low || over ? 0 : (int32_t)(shared / a.P * a.P);
    }
  }
  __syncthreads();
  int64_t items = 0;
  for (int j0 = 0; j0 < jobs; j0 += blockDim.x) {
    const int j = j0 + threadIdx.x;
    const int64_t n = j < jobs ? (ok ? a.first[j + 1] - a.first[j] : a.batch) : 0;
    const int64_t t = (n * a.G + kItemRows - 1) / kItemRows;
    int64_t all;
    const int64_t upto = plan_scan(t, warp_sum, all);
    if (j < jobs) first[j] = (int32_t)(items + upto - t);
    items += all;
  }
  const int n_items = (int)items;
  if (threadIdx.x == 0) first[jobs] = n_items;
  __syncthreads();
  put_items(a, n_items, warp_sum, rows_of + a.jobs, [&](int i) {
    const int j = find_job(first, jobs, i);
    const int64_t r0 = ok ? a.first[j] : 0, r1 = ok ? a.first[j + 1] : a.batch;
    RowsItem it = {};
    it.table = it.token0 = (int32_t)r0;
    it.row0 = (i - first[j]) * kItemRows;
    it.rows = (int)min((int64_t)kItemRows, (r1 - r0) * a.G - it.row0);
    it.part_row = (int32_t)r0 * a.G + it.row0;
    it.hi = it.full_hi = rows_of[j];
    if (a.window > 0 && it.hi > 0) {
      int64_t least = cap, most = 0;          // lengths of the requests it has rows of
      for (int64_t r = r0 + it.row0 / a.G; r <= r0 + (it.row0 + it.rows - 1) / a.G; ++r) {
        least = min(least, a.lens[r]);
        most = max(most, a.lens[r]);
      }
      it.lo = (int)min((int64_t)it.hi, max((int64_t)0, least - a.window));
      it.full_lo = (int)max((int64_t)0, most - a.window);
    }
    it.k0 = it.lo / kTileKeys * kTileKeys;
    it.steps = it.lo < it.hi ? steps_of(it) : 0;
    return it;
  });
}

// o of an item's rows from its pieces, sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i, and with a prefix from what the decode
// kernel made of the requests' own rows (normalised: a sum of one at the offset lse).
// A CTA takes 8 (32) values of each row of an item, a thread per row, so that neighbouring rows' values lie next to one another; of
// few rows the threads share out the pieces.  Four (two) pieces' loads are in flight at once: latency is what this costs.
// Prefix, many pieces and few items: blockIdx.x is a (KV head, item).  Chunk, two pieces or a few more: blockIdx.x is a cut
// between two CTAs' shares, and the first cut of an item speaks for it.
template <int kJoinValues, int kJoinLoads>
__global__ void __launch_bounds__(kItemRows) rows_join(const __grid_constant__ RowsArgs a) {
  wait_for_earlier_kernels();
  let_later_kernels_start();
  const RowsPlan plan = *a.plan;
  const int64_t W = plan.steps * a.h_kv;
  const int N = plan.n_parts;
  int g, index, first = 0, last = -1;
  if (a.prefix) {
    index = blockIdx.x / a.h_kv;
    g = blockIdx.x - index * a.h_kv;
    if (index >= plan.n_items) return;
  } else {
    const int cut = blockIdx.x + 1;
    if (cut >= N) return;
    const RowsStart& st = a.starts[cut];
    if (st.step == 0) return;
    g = st.g;
    index = st.at;
    if (lane_begin64(cut - 1, W, N) > g * plan.steps + a.items[index].step0) return;     // cut before, too
  }
  const RowsItem it = a.items[index];
  if (it.steps > 0) {
    const int64_t x = g * plan.steps + it.step0;
    first = lane_of64(x, W, N);
    last = lane_of64(x + it.steps - 1, W, N);
  }
  const int rows_p = it.rows > 128 ? 256 : it.rows > 64 ? 128 : it.rows > 32 ? 64 : 32;
  const int i = threadIdx.x & (rows_p - 1), share = threadIdx.x / rows_p, shares = kItemRows / rows_p, c0 = blockIdx.y * kJoinValues;
  const bool live = i < it.rows;
  const int r = it.row0 + i, tok = r / a.G, h = g * a.G + (r - tok * a.G);
  const int64_t out = ((int64_t)it.token0 + tok) * a.h_q + h;
  float own_lse = -INFINITY;
  float4 own_y[kJoinValues / 4] = {};
  if (a.prefix && live && share == 0) {
    own_lse = a.own_lse[out];
#pragma unroll
    for (int e = 0; e < kJoinValues / 4; ++e) own_y[e] = reinterpret_cast<const float4*>(a.own_o + out * a.d + c0)[e];
  }
  float M = -INFINITY, den = 0.f, num[kJoinValues];
#pragma unroll
  for (int e = 0; e < kJoinValues; ++e) num[e] = 0.f;
  // (offset, sum, values) taken in; a piece whose scores were all NaN, or none, has offset -inf
  auto take = [&](float m, float l, const float* y) {
    const float top = fmaxf(M, m);
    const float wo = M == top ? 1.f : exp2f(M - top), wn = m == top ? 1.f : exp2f(m - top);
    M = top;
    den = den * wo + l * wn;
#pragma unroll
    for (int e = 0; e < kJoinValues; ++e) num[e] = num[e] * wo + y[e] * wn;
  };
  for (int c = first + share; c <= last && live; c += kJoinLoads * shares) {
    float2 ml[kJoinLoads];
    float4 y[kJoinLoads][kJoinValues / 4];
#pragma unroll
    for (int k = 0; k < kJoinLoads; ++k)
      if (c + k * shares <= last) {
        const int64_t row = rows_part(a, c + k * shares, c + k * shares == first, g, it);
        const float4* from = reinterpret_cast<const float4*>(a.part + row * a.d) + (int64_t)(c0 / 4) * it.rows + i;
        ml[k] = a.part_ml[row + i];
#pragma unroll
        for (int e = 0; e < kJoinValues / 4; ++e) y[k][e] = from[(int64_t)e * it.rows];
      }
#pragma unroll
    for (int k = 0; k < kJoinLoads; ++k)
      if (c + k * shares <= last) take(ml[k].x, ml[k].y, reinterpret_cast<const float*>(y[k]));
  }
  __shared__ float red[kItemRows][kJoinValues + 3];
  if (shares > 1) {
    float* to = red[threadIdx.x];
    to[0] = M;
    to[1] = den;
#pragma unroll
    for (int e = 0; e < kJoinValues; ++e) to[2 + e] = num[e];
    __syncthreads();
    if (share != 0 || !live) return;
    for (int k = 1; k < shares; ++k) take(red[k * rows_p + i][0], red[k * rows_p + i][1], red[k * rows_p + i] + 2);
  }
  if (!live) return;
  const float vsc = (a.v_scale != nullptr ? a.v_scale[g] : 1.f) / a.unit;
  float own = 0.f;
  if (own_lse != -INFINITY) {
    const float z = own_lse * kLog2e + a.shift, top = fmaxf(M, z);      // (the pieces' sums are 2^shift times as large)
    const float wo = M == top ? 1.f : exp2f(M - top);
    own = z == top ? 1.f : exp2f(z - top);    // (of a NaN, NaN)
    M = top;
    den = den * wo + own;
#pragma unroll
    for (int e = 0; e < kJoinValues; ++e) num[e] *= wo;
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  const float* u = reinterpret_cast<const float*>(own_y);
  float f[kJoinValues];
#pragma unroll
  for (int e = 0; e < kJoinValues; ++e) f[e] = (num[e] * vsc + (own != 0.f ? own * u[e] : 0.f)) * inv;
  alignas(16) uint32_t b[kJoinValues / 2];
#pragma unroll
  for (int e = 0; e < kJoinValues / 2; ++e) b[e] = a.out_f16 ? pack16<kF16>(f[2 * e], f[2 * e + 1]) : pack16<kBf16>(f[2 * e], f[2 * e + 1]);
  uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + out * a.d + c0);
#pragma unroll
  for (int e = 0; e < kJoinValues / 8; ++e) to[e] = *reinterpret_cast<const uint4*>(b + 4 * e);
  if (a.lse != nullptr && c0 == 0) a.lse[out] = (M + log2f(den) - a.shift) * 0.6931471805599453f;
}

// Whether weights are two 16-bit parts (rows_attend.cuh says why).
bool split_weights(const RowsShape& p) { return p.prefix != 0 && p.cache_dtype != KVSEL_DTYPE_E4M3; }

// (scored: with a cap or a bias)
RowsVariant variant(const RowsShape& p, bool scored) {
  const bool split = split_weights(p);
  if (p.cache_dtype == KVSEL_DTYPE_E4M3) return rows_variant_e4m3(p.d, split, scored);
  return p.dtype == KVSEL_DTYPE_F16 ? rows_variant_f16(p.d, split, scored) : rows_variant_bf16(p.d, split, scored);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// A map of a pool [page][head][row][d] in its own strides, in boxes of `rows` rows of one head: 128 bytes wide and swizzled for the
// products, or bytes of whole rows.
bool pool_map(const RowsShape& p, const void* pool, int rows, CUtensorMap* map) {
  const auto fn = encoder();
  if (fn == nullptr) return false;
  const bool bytes = p.cache_dtype == KVSEL_DTYPE_E4M3;
  const cuuint64_t size = bytes ? 1 : 2;
  const cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)p.P, (cuuint64_t)p.h_kv, (cuuint64_t)p.n_pages};
  cuuint64_t strides[3] = {p.row_stride * size, p.head_stride * size, p.page_stride * size};
  for (int i = 0; i < 3; ++i)
    if (strides[i] == 0) {
      if (dims[i + 1] > 1) return false;          // (rows, heads or pages that are one and the same)
      strides[i] = 16;
    }
  const cuuint32_t box[4] = {(cuuint32_t)(bytes ? p.d : 64), (cuuint32_t)rows, 1, 1}, one[4] = {1, 1, 1, 1};
  return fn(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : p.cache_dtype == KVSEL_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void*>(pool), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Rows of a box: the largest power of two up to 32 that divides a page, so that a box lies in one page and in one loader warp's
// rows; pages without a factor of eight, and pools that no map describes, are copied by lanes.
int boxes(const RowsShape& p, const void* k, const void* v, CUtensorMap* tk, CUtensorMap* tv) {
  const int rows = std::min(32, p.P & -p.P);
  memset(tk, 0, sizeof(*tk));
  memset(tv, 0, sizeof(*tv));
  return rows >= 8 && pool_map(p, k, rows, tk) && pool_map(p, v, rows, tv) ? rows : 0;
}

struct Layout {
  int grid;
  int64_t max_items, part_rows;
  size_t plan, starts, items, own_lens, own_tables, own_o, own_lse, ml, part, total;
};
bool layout(const RowsShape& p, size_t front, Layout* out) {
  const RowsVariant v = variant(p, true);      // (all variants: one CTA per SM)
  const int64_t grid = resident_ctas((const void*)v.kern, kRowsThreads, v.smem);     // one per SM
  if (grid <= 0) return false;
  Layout& o = *out;
  const int64_t G = p.h_q / p.h_kv;
  o.grid = (int)grid;
  // every job ends with an item that may be part full
  o.max_items = p.jobs + ceil_div((p.prefix ? p.batch : p.max_tokens) * G, kItemRows);
  auto up = [](size_t x) { return (x + KVSEL_WS_ALIGN - 1) / KVSEL_WS_ALIGN * KVSEL_WS_ALIGN; };
  size_t at = std::max(front, sizeof(DeviceError));
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = up(at + bytes);
    return here;
  };
  o.plan = take(sizeof(RowsPlan));
  o.starts = take(sizeof(RowsStart) * (size_t)grid);
  o.items = take(sizeof(RowsItem) * (size_t)o.max_items);
  o.own_lens = o.own_tables = o.own_o = o.own_lse = 0;
  if (p.prefix) {
    o.own_lens = take(sizeof(int64_t) * (size_t)p.batch);
    o.own_tables = take(sizeof(int32_t) * (size_t)p.batch * p.max_blocks);
    o.own_o = take(sizeof(float) * (size_t)p.batch * p.h_q * p.d);
    o.own_lse = take(sizeof(float) * (size_t)p.batch * p.h_q);
  }
  o.part_rows = p.prefix ? grid * kItemRows + (int64_t)p.batch * p.h_q : 2 * grid * kItemRows;
  o.ml = take(sizeof(float2) * (size_t)o.part_rows);
  o.part = take(sizeof(float) * (size_t)o.part_rows * p.d);
  o.total = at;
  return true;
}

// The arguments of a call's kernels from the caller's and the workspace.
RowsArgs rows_args(const RowsShape& p, const RowsArgs& in, const Layout& lay, void* ws) {
  char* base = static_cast<char*>(ws);
  RowsArgs a = in;
  a.part = reinterpret_cast<float*>(base + lay.part);
  a.part_ml = reinterpret_cast<float2*>(base + lay.ml);
  a.items = reinterpret_cast<RowsItem*>(base + lay.items);
  a.plan = reinterpret_cast<RowsPlan*>(base + lay.plan);
  a.starts = reinterpret_cast<RowsStart*>(base + lay.starts);
  a.err = reinterpret_cast<DeviceError*>(ws);
  a.own_tables = reinterpret_cast<int32_t*>(base + lay.own_tables);
  a.own_lens = reinterpret_cast<int64_t*>(base + lay.own_lens);
  a.own_o = reinterpret_cast<const float*>(base + lay.own_o);
  a.own_lse = reinterpret_cast<const float*>(base + lay.own_lse);
  a.max_tokens = p.max_tokens;
  a.page_stride = p.page_stride;
  a.head_stride = p.head_stride;
  a.row_stride = p.row_stride;
  a.q_stride = p.q_stride;
  a.scale = p.scale;
  a.softcap = p.softcap;
  a.h_q = p.h_q;
  a.h_kv = p.h_kv;
  a.G = p.h_q / p.h_kv;
  a.d = p.d;
  a.P = p.P;
  a.jobs = p.jobs;
  a.batch = p.batch;
  a.max_blocks = p.max_blocks;
  a.n_pages = p.n_pages;
  a.window = p.window;
  a.out_f16 = p.dtype == KVSEL_DTYPE_F16;
  a.prefix = p.prefix;
  page_division(p.P, &a.p_mul, &a.p_shift);
  a.grid = lay.grid;
  a.max_items = (int32_t)lay.max_items;
  a.head_rows = p.batch * (p.h_q / p.h_kv);
  // factor on O against the sums, and binary orders on both
  const bool bf16 = p.cache_dtype == KVSEL_DTYPE_BF16, split = split_weights(p);
  a.unit = !split ? 1.f : bf16 ? weight_unit<kBf16>() : weight_unit<kF16>();
  a.shift = split ? 0.f : bf16 ? -8.f : 13.f;
  return a;
}

}  // namespace

size_t rows_ws(const RowsShape& p, size_t front) {
  Layout lay;
  return layout(p, front, &lay) ? lay.total : 0;
}

kvsel_status launch_chunk_attend(const RowsShape& p, const RowsArgs& in, void* ws, cudaStream_t s) {
  Layout lay;
  if (!layout(p, 0, &lay)) return KVSEL_ERR_CUDA;
  const RowsVariant var = variant(p, p.softcap != 0.f || in.slopes != nullptr);
  RowsArgs a = rows_args(p, in, lay, ws);
  CUtensorMap tk, tv;
  a.box_rows = boxes(p, a.k, a.v, &tk, &tv);
  const size_t smem = sizeof(int32_t) * (2 * (size_t)a.jobs + 1 + kPlanItems);
  const unsigned threads = a.jobs <= 256 && a.max_items <= 256 ? 256 : kPlanThreads;
  if (set_smem((const void*)chunk_plan, smem) != cudaSuccess || set_smem((const void*)var.kern, var.smem) != cudaSuccess) return KVSEL_ERR_CUDA;
  kvsel_status st;
  {
    TraceScope ts("chunk_plan", s);
    if ((st = launch_after(chunk_plan, dim3(1), threads, smem, s, a)) != KVSEL_OK) return st;
  }
  {
    TraceScope ts("rows_attend", s);
    if ((st = launch_after(var.kern, dim3(a.grid), kRowsThreads, var.smem, s, a, tk, tv)) != KVSEL_OK) return st;
  }
  TraceScope ts("rows_join", s);
  return launch_after(rows_join<32, 2>, dim3(std::max(1, a.grid - 1), p.d / 32), kItemRows, 0, s, a);
}

kvsel_status launch_prefix_attend(const RowsShape& p, const PagedShape& own, const RowsArgs& in, void* ws, size_t front, cudaStream_t s) {
  Layout lay;
  if (!layout(p, front, &lay)) return KVSEL_ERR_CUDA;
  const RowsVariant var = variant(p, p.softcap != 0.f || in.slopes != nullptr);
  RowsArgs a = rows_args(p, in, lay, ws);
  CUtensorMap tk, tv;
  a.box_rows = boxes(p, a.k, a.v, &tk, &tv);
  const size_t smem = sizeof(int32_t) * (2 * (size_t)a.jobs + 1 + kPlanItems);
  const unsigned threads = a.jobs <= 256 && a.max_items <= 256 ? 256 : kPlanThreads;
  if (set_smem((const void*)prefix_plan, smem) != cudaSuccess || set_smem((const void*)var.kern, var.smem) != cudaSuccess) return KVSEL_ERR_CUDA;
  kvsel_status st;
  {
    TraceScope ts("prefix_plan", s);
    if ((st = launch_after(prefix_plan, dim3(1 + std::min(a.batch, 2 * a.grid)), threads, smem, s, a)) != KVSEL_OK) return st;
  }
  {
    TraceScope ts("rows_attend", s);
    if ((st = launch_after(var.kern, dim3(a.grid), kRowsThreads, var.smem, s, a, tk, tv)) != KVSEL_OK) return st;
  }
  st = launch_paged_attend(own, a.q, a.k, a.v, a.own_tables, a.own_lens, a.slopes, a.k_scale, a.v_scale, nullptr, const_cast<float*>(a.own_lse), ws, s,
                           const_cast<float*>(a.own_o));
  if (st != KVSEL_OK) return st;
  TraceScope ts("rows_join", s);
  return launch_after(rows_join<8, 4>, dim3((unsigned)(lay.max_items * a.h_kv), p.d / 8), kItemRows, 0, s, a);
}

}  // namespace kvsel
