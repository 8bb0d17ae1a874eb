// C ABI of the calls with many query rows over the same keys: argument checks and the kernels' arguments.
#include <cfloat>
#include <cmath>

#include "rows.cuh"

namespace kvsel {
namespace {

kvsel_status check_chunk(const kvsel_cache_desc* cache, const kvsel_chunk_attend_desc* p, RowsShape* out) {
  if (p == nullptr) return KVSEL_ERR_INVALID_ARG;
  // (what a chunk call shares with a decode step is checked as that is)
  const kvsel_paged_attend_desc step = {p->batch, p->max_blocks, p->q_stride, p->scale, p->softcap, p->window};
  PagedShape s;
  const kvsel_status st = check_attend(cache, &step, &s);
  if (st != KVSEL_OK) return st;
  if (p->max_tokens < 0 || p->max_tokens >= (int64_t(1) << 31)) return KVSEL_ERR_INVALID_ARG;
  const int64_t G = s.h_q / s.h_kv;
  // an item's rows are numbered in 32 bits, and so are the steps of a KV head
  if (p->max_tokens * G >= (int64_t(1) << 31)) return KVSEL_ERR_UNSUPPORTED;
  const int64_t items = p->batch + ceil_div(p->max_tokens * G, kItemRows);
  if (items * (ceil_div((int64_t)s.max_blocks * s.P, 128) + 1) >= (int64_t(1) << 31)) return KVSEL_ERR_UNSUPPORTED;
  *out = RowsShape{s.dtype, s.cache_dtype, s.h_q, s.h_kv, s.d, s.P, s.batch, s.max_blocks, s.n_pages, s.batch, 0,
                   p->max_tokens, s.page_stride, s.head_stride, s.row_stride, s.q_stride, s.scale, s.softcap, s.window};
  return KVSEL_OK;
}

kvsel_status check_prefix(const kvsel_cache_desc* cache, const kvsel_paged_attend_desc* p, int32_t n_groups, PagedShape* own, RowsShape* out) {
  const kvsel_status st = check_attend(cache, p, own);
  if (st != KVSEL_OK) return st;
  const PagedShape& s = *own;
  if (n_groups < 1 || n_groups > s.batch) return KVSEL_ERR_INVALID_ARG;
  const int64_t G = s.h_q / s.h_kv, items = n_groups + ceil_div(s.batch * G, kItemRows);
  if (items * (ceil_div((int64_t)s.max_blocks * s.P, 128) + 1) >= (int64_t(1) << 31)) return KVSEL_ERR_UNSUPPORTED;
  *out = RowsShape{s.dtype, s.cache_dtype, s.h_q, s.h_kv, s.d, s.P, s.batch, s.max_blocks, s.n_pages, n_groups, 1,
                   0, s.page_stride, s.head_stride, s.row_stride, s.q_stride, s.scale, s.softcap, s.window};
  return KVSEL_OK;
}

}  // namespace
}  // namespace kvsel

using namespace kvsel;

extern "C" {

kvsel_status kvsel_chunk_attend_workspace_size(const kvsel_cache_desc* cache, const kvsel_chunk_attend_desc* desc, size_t* bytes) {
  RowsShape p;
  const kvsel_status st = check_chunk(cache, desc, &p);
  if (st != KVSEL_OK) return st;
  if (bytes == nullptr) return KVSEL_ERR_INVALID_ARG;
  *bytes = rows_ws(p, 0);
  return *bytes > 0 ? KVSEL_OK : KVSEL_ERR_CUDA;
}

kvsel_status kvsel_chunk_attend(const kvsel_cache_desc* cache, const kvsel_chunk_attend_desc* desc, const void* q,
                                const void* k_cache, const void* v_cache, const int32_t* block_tables, const int64_t* lens,
                                const int64_t* indptr, const float* slopes, const float* k_scale, const float* v_scale, void* o,
                                float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx("kvsel_chunk_attend");
  RowsShape p;
  const kvsel_status st = check_chunk(cache, desc, &p);
  if (st != KVSEL_OK) return st;
  if (p.max_tokens == 0) return KVSEL_OK;         // (arrays of no tokens may have no address)
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || block_tables == nullptr || lens == nullptr ||
      indptr == nullptr || o == nullptr)
    return KVSEL_ERR_INVALID_ARG;
  if (!scales_ok(*cache, k_scale, v_scale) || o == q) return KVSEL_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(lens, 8) ||
      !aligned(indptr, 8) || !aligned(block_tables, 4) || !aligned(slopes, 4) || !aligned(lse, 4))
    return KVSEL_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws, KVSEL_WS_ALIGN)) return KVSEL_ERR_WORKSPACE;
  const size_t need = rows_ws(p, 0);
  if (need == 0) return KVSEL_ERR_CUDA;
  if (ws_bytes < need) return KVSEL_ERR_WORKSPACE;
  RowsArgs in = {};
  in.q = q;
  in.k = k_cache;
  in.v = v_cache;
  in.tables = block_tables;
  in.lens = lens;
  in.first = indptr;
  in.slopes = slopes;
  in.k_scale = k_scale;
  in.v_scale = v_scale;
  in.o = o;
  in.lse = lse;
  return launch_chunk_attend(p, in, ws, stream);
}

kvsel_status kvsel_prefix_attend_workspace_size(const kvsel_cache_desc* cache, const kvsel_paged_attend_desc* desc, int32_t n_groups,
                                                size_t* bytes) {
  PagedShape own;
  RowsShape p;
  const kvsel_status st = check_prefix(cache, desc, n_groups, &own, &p);
  if (st != KVSEL_OK) return st;
  if (bytes == nullptr) return KVSEL_ERR_INVALID_ARG;
  const size_t front = paged_attend_ws(own);
  *bytes = front > 0 ? rows_ws(p, front) : 0;
  return *bytes > 0 ? KVSEL_OK : KVSEL_ERR_CUDA;
}

kvsel_status kvsel_prefix_attend(const kvsel_cache_desc* cache, const kvsel_paged_attend_desc* desc, int32_t n_groups, const void* q,
                                 const void* k_cache, const void* v_cache, const int32_t* block_tables, const int64_t* lens,
                                 const int64_t* group_indptr, const int64_t* shared_lens, const float* slopes, const float* k_scale,
                                 const float* v_scale, void* o, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx("kvsel_prefix_attend");
  PagedShape own;
  RowsShape p;
  const kvsel_status st = check_prefix(cache, desc, n_groups, &own, &p);
  if (st != KVSEL_OK) return st;
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || block_tables == nullptr || lens == nullptr ||
      group_indptr == nullptr || shared_lens == nullptr || o == nullptr)
    return KVSEL_ERR_INVALID_ARG;
  if (!scales_ok(*cache, k_scale, v_scale) || o == q) return KVSEL_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(lens, 8) ||
      !aligned(group_indptr, 8) || !aligned(shared_lens, 8) || !aligned(block_tables, 4) || !aligned(slopes, 4) || !aligned(lse, 4))
    return KVSEL_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws, KVSEL_WS_ALIGN)) return KVSEL_ERR_WORKSPACE;
  const size_t front = paged_attend_ws(own), need = front > 0 ? rows_ws(p, front) : 0;
  if (need == 0) return KVSEL_ERR_CUDA;
  if (ws_bytes < need) return KVSEL_ERR_WORKSPACE;
  RowsArgs in = {};
  in.q = q;
  in.k = k_cache;
  in.v = v_cache;
  in.tables = block_tables;
  in.lens = lens;
  in.first = group_indptr;
  in.shared = shared_lens;
  in.slopes = slopes;
  in.k_scale = k_scale;
  in.v_scale = v_scale;
  in.o = o;
  in.lse = lse;
  return launch_prefix_attend(p, own, in, ws, front, stream);
}

}  // extern "C"
