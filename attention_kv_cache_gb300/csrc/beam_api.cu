// C ABI of the beam search calls: argument checks and the kernels' arguments.
#include <algorithm>

#include "beam.cuh"

namespace kvsel {
namespace {

kvsel_status check_select(const kvsel_beam_select_desc* p, SelectArgs* out) {
  if (p == nullptr) return KVSEL_ERR_INVALID_ARG;
  if (p->batch < 1 || p->beams < 1 || p->n_out < 1 || p->vocab < 1) return KVSEL_ERR_INVALID_ARG;
  if (p->dtype != KVSEL_DTYPE_BF16 && p->dtype != KVSEL_DTYPE_F16 && p->dtype != KVSEL_DTYPE_F32) return KVSEL_ERR_INVALID_ARG;
  if (p->pad_token < 0 || p->pad_token >= p->vocab || p->n_out > (int64_t)p->beams * p->vocab) return KVSEL_ERR_INVALID_ARG;
  if (p->row_stride < 0 || p->row_stride > (int64_t(1) << 40)) return KVSEL_ERR_INVALID_ARG;
  if (p->beams > kMaxBeams || p->n_out > kMaxBeamOut) return KVSEL_ERR_UNSUPPORTED;
  const int64_t slices = ceil_div(p->vocab, kSliceKeys);
  if (p->beams * slices > kMaxLists || (int64_t)p->batch * p->beams > KVSEL_PAGED_MAX_BATCH) return KVSEL_ERR_UNSUPPORTED;
  SelectArgs& a = *out;
  a.batch = p->batch;
  a.beams = p->beams;
  a.n_out = p->n_out;
  a.vocab = p->vocab;
  // Segments: slices of their own while there are few rows; of many rows so that the CTAs are some 2048 (each begins a bound and
  // leaves a list: 64 sets of 16 beams over 128256 tokens took 245 us in slices of their own, 131 in four segments, 99 in two).
  const int64_t rows = (int64_t)p->batch * p->beams, most = std::max<int64_t>(1, kSelectCtas / rows);
  a.seg_slices = (int32_t)std::min(kMaxSegSlices, ceil_div(slices, std::min(slices, most)));
  a.segments = (int32_t)ceil_div(slices, a.seg_slices);
  a.pad_token = p->pad_token;
  a.row_stride = p->row_stride != 0 ? p->row_stride : p->vocab;
  return KVSEL_OK;
}

kvsel_status check_reorder(const kvsel_beam_reorder_desc* p) {
  if (p == nullptr) return KVSEL_ERR_INVALID_ARG;
  if (p->batch < 1 || p->beams < 1 || p->max_blocks < 1 || p->n_layers < 1) return KVSEL_ERR_INVALID_ARG;
  if (p->layer_stride < 0 || p->layer_stride > (int64_t(1) << 45)) return KVSEL_ERR_INVALID_ARG;
  if (p->beams > kMaxBeams || (int64_t)p->batch * p->beams > KVSEL_PAGED_MAX_BATCH) return KVSEL_ERR_UNSUPPORTED;
  // freed pages are counted in 32 bits, and a table row's entries are numbered so
  if ((int64_t)p->batch * p->beams * p->max_blocks >= (int64_t(1) << 31)) return KVSEL_ERR_UNSUPPORTED;
  return KVSEL_OK;
}

}  // namespace
}  // namespace kvsel

using namespace kvsel;

extern "C" {

kvsel_status kvsel_beam_select_workspace_size(const kvsel_beam_select_desc* desc, size_t* bytes) {
  SelectArgs a;
  const kvsel_status st = check_select(desc, &a);
  if (st != KVSEL_OK) return st;
  if (bytes == nullptr) return KVSEL_ERR_INVALID_ARG;
  size_t best, sums, tops;
  *bytes = beam_select_ws((int64_t)a.batch * a.beams, a.segments, a.n_out, &best, &sums, &tops);
  return KVSEL_OK;
}

kvsel_status kvsel_beam_select(const kvsel_beam_select_desc* desc, const void* logits, const float* scores,
                               const uint8_t* ended, float* scores_out, int32_t* parents, int32_t* tokens, float* lse,
                               void* ws, size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx("kvsel_beam_select");
  SelectArgs a;
  const kvsel_status st = check_select(desc, &a);
  if (st != KVSEL_OK) return st;
  if (logits == nullptr || scores == nullptr || scores_out == nullptr || parents == nullptr || tokens == nullptr)
    return KVSEL_ERR_INVALID_ARG;
  if (!aligned(logits, desc->dtype == KVSEL_DTYPE_F32 ? 4 : 2)) return KVSEL_ERR_INVALID_ARG;
  for (const void* p : {(const void*)scores, (const void*)scores_out, (const void*)parents, (const void*)tokens, (const void*)lse})
    if (!aligned(p, 4)) return KVSEL_ERR_INVALID_ARG;
  if (scores_out == scores) return KVSEL_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws, KVSEL_WS_ALIGN)) return KVSEL_ERR_WORKSPACE;
  size_t best, sums, tops;
  if (ws_bytes < beam_select_ws((int64_t)a.batch * a.beams, a.segments, a.n_out, &best, &sums, &tops)) return KVSEL_ERR_WORKSPACE;
  a.logits = logits;
  a.scores = scores;
  a.ended = ended;
  a.scores_out = scores_out;
  a.parents = parents;
  a.tokens = tokens;
  a.lse = lse;
  a.best = reinterpret_cast<float2*>(static_cast<char*>(ws) + best);
  a.sums = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + sums);
  a.tops = reinterpret_cast<float*>(static_cast<char*>(ws) + tops);
  return launch_beam_select(a, desc->dtype, stream);
}

kvsel_status kvsel_beam_reorder_workspace_size(const kvsel_beam_reorder_desc* desc, size_t* bytes) {
  const kvsel_status st = check_reorder(desc);
  if (st != KVSEL_OK) return st;
  if (bytes == nullptr) return KVSEL_ERR_INVALID_ARG;
  size_t off[7];
  *bytes = beam_reorder_ws(desc->batch, desc->beams, (int32_t)ceil_div(desc->max_blocks, kReorderCols), off);
  return KVSEL_OK;
}

kvsel_status kvsel_beam_reorder(const kvsel_cache_desc* cache, const kvsel_beam_reorder_desc* desc, const int32_t* parents,
                                const int64_t* lens, const int32_t* block_tables, int32_t* free_pages, int64_t n_free,
                                const int64_t* free_head, int32_t* block_tables_out, int64_t* lens_out,
                                int64_t* free_head_out, void* k_cache, void* v_cache, void* ws, size_t ws_bytes,
                                cudaStream_t stream) {
  NvtxRange nvtx("kvsel_beam_reorder");
  kvsel_status st = check_cache(cache);
  if (st == KVSEL_OK) st = check_reorder(desc);
  if (st != KVSEL_OK) return st;
  const kvsel_cache_desc& c = *cache;
  const int64_t size = c.cache_dtype == KVSEL_DTYPE_E4M3 ? 1 : 2;
  if (((int64_t)desc->max_blocks + 1) * c.page_size >= (int64_t(1) << 31)) return KVSEL_ERR_INVALID_ARG;
  if (desc->layer_stride * size % 16 != 0) return KVSEL_ERR_INVALID_ARG;
  if (n_free < 0 || n_free >= (int64_t(1) << 31)) return KVSEL_ERR_INVALID_ARG;
  for (const void* p : {(const void*)parents, (const void*)lens, (const void*)block_tables, (const void*)free_pages,
                        (const void*)free_head, (const void*)block_tables_out, (const void*)lens_out,
                        (const void*)free_head_out, (const void*)k_cache, (const void*)v_cache})
    if (p == nullptr) return KVSEL_ERR_INVALID_ARG;
  if (k_cache == v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return KVSEL_ERR_INVALID_ARG;
  for (const void* p : {(const void*)lens, (const void*)free_head, (const void*)lens_out, (const void*)free_head_out})
    if (!aligned(p, 8)) return KVSEL_ERR_INVALID_ARG;
  for (const void* p : {(const void*)parents, (const void*)block_tables, (const void*)free_pages, (const void*)block_tables_out})
    if (!aligned(p, 4)) return KVSEL_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws, KVSEL_WS_ALIGN)) return KVSEL_ERR_WORKSPACE;
  ReorderArgs a;
  a.tiles = (int32_t)ceil_div(desc->max_blocks, kReorderCols);
  size_t off[7];
  if (ws_bytes < beam_reorder_ws(desc->batch, desc->beams, a.tiles, off)) return KVSEL_ERR_WORKSPACE;
  a.batch = desc->batch;
  a.beams = desc->beams;
  a.P = c.page_size;
  a.max_blocks = desc->max_blocks;
  a.n_layers = desc->n_layers;
  a.h_kv = c.h_kv;
  a.n_pages = c.n_pages;
  a.n_free = n_free;
  a.page_stride = c.page_stride * size;
  a.head_stride = c.head_stride * size;
  a.row_stride = c.row_stride * size;
  a.layer_stride = desc->layer_stride * size;
  a.row_bytes = (int32_t)(c.head_dim * size);
  a.parents = parents;
  a.lens = lens;
  a.tables = block_tables;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.tables_out = block_tables_out;
  a.lens_out = lens_out;
  a.head_out = free_head_out;
  a.k = static_cast<uint8_t*>(k_cache);
  a.v = static_cast<uint8_t*>(v_cache);
  char* base = static_cast<char*>(ws);
  a.err = reinterpret_cast<DeviceError*>(ws);
  a.plan = reinterpret_cast<ReorderPlan*>(base + off[0]);
  a.parent_of = reinterpret_cast<int32_t*>(base + off[1]);
  a.blocks = reinterpret_cast<int32_t*>(base + off[2]);
  a.twin = reinterpret_cast<int32_t*>(base + off[3]);
  a.copy = reinterpret_cast<ReorderCopy*>(base + off[4]);
  a.count = reinterpret_cast<int32_t*>(base + off[5]);
  a.freed = reinterpret_cast<int32_t*>(base + off[6]);
  return launch_beam_reorder(a, stream);
}

}  // extern "C"
