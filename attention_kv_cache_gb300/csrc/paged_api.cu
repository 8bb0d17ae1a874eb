// C ABI of the calls over a paged cache: argument checks and the kernels' arguments.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>

#include "paged.cuh"

namespace kvsel {

kvsel_status check_cache(const kvsel_cache_desc* c) {
  if (c == nullptr) return KVSEL_ERR_INVALID_ARG;
  if (c->h_kv < 1 || c->h_q < 1 || c->h_q % c->h_kv != 0) return KVSEL_ERR_INVALID_ARG;
  if (c->page_size < 1 || c->page_size > KVSEL_MAX_PAGE) return KVSEL_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->n_pages >= (int64_t(1) << 31)) return KVSEL_ERR_INVALID_ARG;
  if (c->dtype != KVSEL_DTYPE_BF16 && c->dtype != KVSEL_DTYPE_F16) return KVSEL_ERR_INVALID_ARG;
  if (c->cache_dtype != c->dtype && c->cache_dtype != KVSEL_DTYPE_E4M3) return KVSEL_ERR_INVALID_ARG;
  if (c->head_dim < 1) return KVSEL_ERR_INVALID_ARG;
  if (c->head_dim % 16 != 0 || c->head_dim > 256) return KVSEL_ERR_UNSUPPORTED;
  if (c->h_q > (1 << 16)) return KVSEL_ERR_UNSUPPORTED;
  const int64_t unit = c->cache_dtype == KVSEL_DTYPE_E4M3 ? 16 : 8;     // elements of 16 bytes
  for (int64_t s : {c->page_stride, c->head_stride, c->row_stride})
    if (s < 0 || s % unit != 0 || s > (int64_t(1) << 40)) return KVSEL_ERR_INVALID_ARG;
  return KVSEL_OK;
}

bool scales_ok(const kvsel_cache_desc& c, const float* k_scale, const float* v_scale) {
  const bool want = c.cache_dtype == KVSEL_DTYPE_E4M3;
  return (k_scale != nullptr) == want && (v_scale != nullptr) == want && aligned(k_scale, 4) && aligned(v_scale, 4);
}

kvsel_status check_attend(const kvsel_cache_desc* cache, const kvsel_paged_attend_desc* p, PagedShape* out) {
  const kvsel_status st = check_cache(cache);
  if (st != KVSEL_OK) return st;
  const kvsel_cache_desc& c = *cache;
  if (p == nullptr) return KVSEL_ERR_INVALID_ARG;
  if (p->batch < 1 || p->batch > KVSEL_PAGED_MAX_BATCH || p->max_blocks < 1) return KVSEL_ERR_INVALID_ARG;
  if (((int64_t)p->max_blocks + 1) * c.page_size >= (int64_t(1) << 31)) return KVSEL_ERR_INVALID_ARG;
  if (p->q_stride < 0 || p->q_stride % 8 != 0) return KVSEL_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale) || p->scale < 0.f) return KVSEL_ERR_INVALID_ARG;
  // (the kernel divides by the cap and multiplies it by log2 e, in fp32)
  if (!(p->softcap == 0.f || (p->softcap >= FLT_MIN && p->softcap <= 0x1p127f)) || p->window < 0) return KVSEL_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128) return KVSEL_ERR_UNSUPPORTED;
  // the steps of a call are numbered in 32 bits
  if ((((int64_t)p->max_blocks * c.page_size) / 32 + 2) * p->batch >= (int64_t(1) << 31)) return KVSEL_ERR_UNSUPPORTED;
  PagedShape& o = *out;
  o.dtype = c.dtype;
  o.cache_dtype = c.cache_dtype;
  o.h_q = c.h_q;
  o.h_kv = c.h_kv;
  o.d = c.head_dim;
  o.P = c.page_size;
  o.batch = p->batch;
  o.max_blocks = p->max_blocks;
  o.n_pages = (int32_t)c.n_pages;
  o.page_stride = c.page_stride;
  o.head_stride = c.head_stride;
  o.row_stride = c.row_stride;
  o.q_stride = p->q_stride != 0 ? p->q_stride : (int64_t)c.h_q * c.head_dim;
  o.scale = p->scale != 0.f ? p->scale : (float)(1.0 / std::sqrt((double)c.head_dim));
  o.softcap = p->softcap;
  o.window = p->window;
  return KVSEL_OK;
}

int64_t resident_ctas(const void* kern, int threads, size_t smem) {
  struct Entry {
    int dev, threads;
    const void* kern;
    size_t smem;
    int64_t n;
  };
  constexpr int kMost = 128;                // further combinations are asked every time
  static std::mutex mu;
  static Entry known[kMost];
  static int n_known = 0;
  int dev = 0, sms = 0, per_sm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n_known; ++i) {
    const Entry& e = known[i];
    if (e.dev == dev && e.kern == kern && e.threads == threads && e.smem == smem) return e.n;
  }
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || set_smem(kern, smem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  const int64_t n = (int64_t)sms * per_sm;
  if (n_known < kMost) known[n_known++] = {dev, threads, kern, smem, n};
  return n;
}

}  // namespace kvsel

using namespace kvsel;

extern "C" {

kvsel_status kvsel_page_assign_workspace_size(int32_t batch, size_t* bytes) {
  if (batch < 1 || batch > KVSEL_PAGED_MAX_BATCH || bytes == nullptr) return KVSEL_ERR_INVALID_ARG;
  *bytes = page_assign_ws(batch);
  return KVSEL_OK;
}

kvsel_status kvsel_page_assign(int32_t page_size, int64_t n_pages, int32_t batch, int32_t max_blocks,
                               const int64_t* lens, const int64_t* n_new, const int64_t* pos_offset,
                               const int32_t* free_pages, int64_t n_free, const int64_t* free_head,
                               int32_t* block_tables, int64_t* lens_out, int64_t* free_head_out, int64_t* indptr,
                               int64_t max_tokens, int64_t* slots, int64_t* positions, int32_t* seq_ids, void* ws,
                               size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx("kvsel_page_assign");
  if (page_size < 1 || page_size > KVSEL_MAX_PAGE || n_pages < 1 || n_pages >= (int64_t(1) << 31))
    return KVSEL_ERR_INVALID_ARG;
  if (batch < 1 || batch > KVSEL_PAGED_MAX_BATCH || max_blocks < 1) return KVSEL_ERR_INVALID_ARG;
  if (((int64_t)max_blocks + 1) * page_size >= (int64_t(1) << 31)) return KVSEL_ERR_INVALID_ARG;
  if (n_free < 0 || n_free >= (int64_t(1) << 31) || max_tokens < 0 || max_tokens >= (int64_t(1) << 31))
    return KVSEL_ERR_INVALID_ARG;
  if (lens == nullptr || n_new == nullptr || free_head == nullptr || block_tables == nullptr || lens_out == nullptr ||
      free_head_out == nullptr || indptr == nullptr)
    return KVSEL_ERR_INVALID_ARG;
  if ((free_pages == nullptr && n_free > 0) || (slots == nullptr && max_tokens > 0)) return KVSEL_ERR_INVALID_ARG;
  for (const void* p : {(const void*)lens, (const void*)n_new, (const void*)pos_offset, (const void*)free_head,
                        (const void*)lens_out, (const void*)free_head_out, (const void*)indptr, (const void*)slots,
                        (const void*)positions})
    if (!aligned(p, 8)) return KVSEL_ERR_INVALID_ARG;
  if (!aligned(free_pages, 4) || !aligned(block_tables, 4) || !aligned(seq_ids, 4)) return KVSEL_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws, KVSEL_WS_ALIGN) || ws_bytes < page_assign_ws(batch)) return KVSEL_ERR_WORKSPACE;
  AssignArgs a;
  a.P = page_size;
  a.batch = batch;
  a.max_blocks = max_blocks;
  a.n_pages = n_pages;
  a.n_free = n_free;
  a.max_tokens = max_tokens;
  a.lens = lens;
  a.n_new = n_new;
  a.pos_offset = pos_offset;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.block_tables = block_tables;
  a.lens_out = lens_out;
  a.free_head_out = free_head_out;
  a.indptr = indptr;
  a.slots = slots;
  a.positions = positions;
  a.seq_ids = seq_ids;
  a.err = reinterpret_cast<DeviceError*>(ws);
  a.plan = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + sizeof(DeviceError));
  return launch_page_assign(a, stream);
}

kvsel_status kvsel_rope_freqs(int32_t rot_dim, const kvsel_rope_scaling* scaling, double* inv_freq, float* scale) {
  if (scaling == nullptr || inv_freq == nullptr || scale == nullptr) return KVSEL_ERR_INVALID_ARG;
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 256) return KVSEL_ERR_INVALID_ARG;
  const kvsel_rope_scaling& s = *scaling;
  if (s.type < KVSEL_ROPE_PLAIN || s.type > KVSEL_ROPE_RAMP) return KVSEL_ERR_INVALID_ARG;
  if (!(s.base > 1.0) || !std::isfinite(s.base)) return KVSEL_ERR_INVALID_ARG;
  const bool banded = s.type == KVSEL_ROPE_BANDED, ramp = s.type == KVSEL_ROPE_RAMP;
  if (s.type != KVSEL_ROPE_PLAIN && (!(s.factor >= 1.0) || !std::isfinite(s.factor))) return KVSEL_ERR_INVALID_ARG;
  if ((banded || ramp) && (!(s.low > 0.0) || !(s.high > s.low) || !std::isfinite(s.high) || s.original_len < 1))
    return KVSEL_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925, L0 = (double)s.original_len;
  double lo = 0.0, hi = 0.0;
  if (ramp) {
    // the index whose pair turns r times over L0 rows: L0 / (2 pi r) = base^(2 i / rot_dim)
    auto index = [&](double r) { return rot_dim * std::log(L0 / (two_pi * r)) / (2.0 * std::log(s.base)); };
    lo = std::max(0.0, std::floor(index(s.high)));
    hi = std::min((double)(rot_dim - 1), std::ceil(index(s.low)));
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double theta = std::pow(s.base, -2.0 * i / rot_dim);
    double f = theta;
    if (s.type == KVSEL_ROPE_LINEAR) {
      f = theta / s.factor;
    } else if (banded) {
      const double turns = L0 * theta / two_pi;                       // L0 / wavelength
      const double w = std::min(1.0, std::max(0.0, (turns - s.low) / (s.high - s.low)));
      f = (1.0 - w) * theta / s.factor + w * theta;
    } else if (ramp) {
      const double r = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
      f = r * theta / s.factor + (1.0 - r) * theta;
    }
    inv_freq[i] = f;
  }
  *scale = ramp ? (float)(0.1 * std::log(s.factor) + 1.0) : 1.f;
  return KVSEL_OK;
}

kvsel_status kvsel_rope_append(const kvsel_cache_desc* cache, const kvsel_rope_desc* rope, int64_t n_tokens,
                               const void* q, const void* k, const void* v, const int64_t* positions,
                               const int64_t* slots, const void* q_weight, const void* k_weight,
                               const double* inv_freq, void* q_out, void* k_cache, void* v_cache,
                               const float* k_scale, const float* v_scale, void* ws, cudaStream_t stream) {
  NvtxRange nvtx("kvsel_rope_append");
  const kvsel_status st = check_cache(cache);
  if (st != KVSEL_OK) return st;
  const kvsel_cache_desc& c = *cache;
  if (rope == nullptr || n_tokens < 0 || n_tokens >= (int64_t(1) << 31)) return KVSEL_ERR_INVALID_ARG;
  const kvsel_rope_desc& r = *rope;
  if (r.rot_dim < 0 || r.rot_dim > c.head_dim) return KVSEL_ERR_INVALID_ARG;
  if (r.layout != KVSEL_ROPE_HALF && r.layout != KVSEL_ROPE_INTERLEAVED) return KVSEL_ERR_INVALID_ARG;
  if (!std::isfinite(r.factor) || !std::isfinite(r.weight_bias) || !std::isfinite(r.norm_eps) || r.norm_eps < 0.f)
    return KVSEL_ERR_INVALID_ARG;
  if (r.rot_dim % 16 != 0) return KVSEL_ERR_UNSUPPORTED;
  for (int64_t s : {r.q_stride, r.q_head_stride, r.k_stride, r.k_head_stride, r.v_stride, r.v_head_stride})
    if (s < 0 || s % 8 != 0 || s > (int64_t(1) << 40)) return KVSEL_ERR_INVALID_ARG;
  if (n_tokens == 0) return KVSEL_OK;             // (arrays of no tokens may have no address)
  const bool has_q = q != nullptr, has_kv = k != nullptr;
  if (!has_q && !has_kv) return KVSEL_ERR_INVALID_ARG;
  if (has_q != (q_out != nullptr) || has_kv != (v != nullptr) || has_kv != (k_cache != nullptr) ||
      has_kv != (v_cache != nullptr))
    return KVSEL_ERR_INVALID_ARG;
  if (has_kv && (slots == nullptr || !scales_ok(c, k_scale, v_scale) || k_cache == v_cache)) return KVSEL_ERR_INVALID_ARG;
  if (r.rot_dim > 0 && (positions == nullptr || inv_freq == nullptr)) return KVSEL_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, (const void*)q_out, (const void*)k_cache, (const void*)v_cache, q_weight, k_weight})
    if (!aligned(p, 16)) return KVSEL_ERR_INVALID_ARG;
  if (!aligned(positions, 8) || !aligned(slots, 8) || !aligned(inv_freq, 8)) return KVSEL_ERR_INVALID_ARG;
  // in place only where every row is written over itself
  if (has_q && q_out == q && (r.q_head_stride != c.head_dim || r.q_stride != (int64_t)c.h_q * c.head_dim))
    return KVSEL_ERR_INVALID_ARG;
  if (ws != nullptr && !aligned(ws, KVSEL_WS_ALIGN)) return KVSEL_ERR_WORKSPACE;
  RopeArgs a;
  a.h_q = c.h_q;
  a.h_kv = c.h_kv;
  a.d = c.head_dim;
  a.P = c.page_size;
  a.rot = r.rot_dim;
  a.e4m3 = c.cache_dtype == KVSEL_DTYPE_E4M3;
  a.n = n_tokens;
  a.n_slots = c.n_pages * c.page_size;
  a.page_stride = c.page_stride;
  a.head_stride = c.head_stride;
  a.row_stride = c.row_stride;
  a.q_stride = r.q_stride;
  a.q_head = r.q_head_stride;
  a.k_stride = r.k_stride;
  a.k_head = r.k_head_stride;
  a.v_stride = r.v_stride;
  a.v_head = r.v_head_stride;
  a.factor = r.factor;
  a.eps = r.norm_eps;
  a.bias = r.weight_bias;
  a.q = q;
  a.k = k;
  a.v = v;
  a.positions = positions;
  a.slots = slots;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.inv_freq = inv_freq;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.err = reinterpret_cast<DeviceError*>(ws);
  return launch_rope_append(a, c.dtype, r.layout, stream);
}

kvsel_status kvsel_paged_attend_workspace_size(const kvsel_cache_desc* cache, const kvsel_paged_attend_desc* desc,
                                               size_t* bytes) {
  PagedShape p;
  const kvsel_status st = check_attend(cache, desc, &p);
  if (st != KVSEL_OK) return st;
  if (bytes == nullptr) return KVSEL_ERR_INVALID_ARG;
  *bytes = paged_attend_ws(p);
  return *bytes > 0 ? KVSEL_OK : KVSEL_ERR_CUDA;
}

kvsel_status kvsel_paged_attend(const kvsel_cache_desc* cache, const kvsel_paged_attend_desc* desc, const void* q,
                                const void* k_cache, const void* v_cache, const int32_t* block_tables,
                                const int64_t* lens, const float* slopes, const float* k_scale, const float* v_scale,
                                void* o, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx("kvsel_paged_attend");
  PagedShape p;
  const kvsel_status st = check_attend(cache, desc, &p);
  if (st != KVSEL_OK) return st;
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || block_tables == nullptr || lens == nullptr ||
      o == nullptr)
    return KVSEL_ERR_INVALID_ARG;
  if (!scales_ok(*cache, k_scale, v_scale)) return KVSEL_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(lens, 8) ||
      !aligned(block_tables, 4) || !aligned(slopes, 4) || !aligned(lse, 4))
    return KVSEL_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws, KVSEL_WS_ALIGN)) return KVSEL_ERR_WORKSPACE;
  const size_t need = paged_attend_ws(p);
  if (need == 0) return KVSEL_ERR_CUDA;
  if (ws_bytes < need) return KVSEL_ERR_WORKSPACE;
  return launch_paged_attend(p, q, k_cache, v_cache, block_tables, lens, slopes, k_scale, v_scale, o, lse, ws, stream);
}

}  // extern "C"
