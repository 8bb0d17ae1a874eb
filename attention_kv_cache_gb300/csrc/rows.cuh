// What the kernels for many query rows over the same keys share: items, their order, partial sums (rows_attend.cu plans and
// merges, rows_attend.cuh computes, rows_api.cu checks).
#pragma once

#include "paged.cuh"

namespace kvsel {

constexpr int kItemRows = 256;        // query rows of an item: two tiles of 128

// Up to 256 query rows (rows row0 .. of a job: token or request r / G, head r % G) and the keys [lo, hi) that they see.
struct RowsItem {
  int32_t table;                      // row of the block tables that the keys are read through
  int32_t token0;                     // the job's first token (chunk) or request (prefix)
  int32_t base;                       // row number of the job's first token (chunk)
  int32_t row0, rows;
  int32_t k0;                         // first key of its first step, a multiple of 128
  int32_t lo, hi, full_lo, full_hi;   // keys [full_lo, full_hi) are seen by all of its rows
  int32_t step0, steps;               // its steps of 128 keys among those of a KV head
  int32_t part_row;                   // its first row among all items' (prefix)
  int32_t pad[3];
};
struct RowsPlan {
  int64_t steps;                      // of a KV head
  int32_t n_items, n_parts;           // items; CTAs that have steps
};
struct RowsStart {                    // where a CTA's steps begin, and how many it has
  int64_t steps;
  int32_t g, at, step, n_items;       // KV head, item, step of it; items of the call
  int32_t pad[2];
  RowsItem item;
};

struct RowsArgs {
  const void *q, *k, *v;
  const int32_t* tables;
  const int64_t *lens, *first;        // first: indptr of the tokens (chunk), of the groups' requests (prefix)
  const int64_t* shared;              // rows of the groups' prefixes (prefix)
  const float *slopes, *k_scale, *v_scale;
  void* o;
  float* lse;
  float* part;                        // partial O: of a piece [d / 4][rows][4]
  float2* part_ml;                    // its rows' offsets (base 2) and sums
  RowsItem* items;
  RowsPlan* plan;
  RowsStart* starts;                  // [grid]
  DeviceError* err;
  // the prefix call's own rows: tables without the shared pages, rows left, and what the decode kernel makes of them
  int32_t* own_tables;
  int64_t* own_lens;
  const float *own_o, *own_lse;
  int64_t max_tokens, page_stride, head_stride, row_stride, q_stride;
  float scale, softcap;
  int32_t h_q, h_kv, G, d, P, jobs, batch, max_blocks, n_pages, window, out_f16, prefix;
  uint32_t p_mul, p_shift;            // division of a row below 2^31 by P
  int32_t grid;                       // CTAs at most
  int32_t box_rows;                   // rows of a box of the pools' tensor maps, 0: they have none
  int32_t max_items;
  int32_t head_rows;                  // query rows of a KV head (prefix)
  float unit, shift;                  // factor on O, and binary orders on sums, of the weights as the kernel holds them
};

// Step x of W at which part i of N begins, and the part that holds step x.
__host__ __device__ __forceinline__ int64_t lane_begin64(int64_t i, int64_t W, int64_t N) { return i * W / N; }
__host__ __device__ __forceinline__ int lane_of64(int64_t x, int64_t W, int64_t N) { return (int)(((x + 1) * N + W - 1) / W - 1); }

// First row of a piece's partial sums.  Chunk: a CTA has at most two pieces that are not whole, one that begins before it and
// one that goes on behind it.  Prefix: all pieces are kept; along a CTA's pieces and from one CTA to the next the rows rise.
__device__ __forceinline__ int64_t rows_part(const RowsArgs& a, int cta, bool starts, int g, const RowsItem& it) {
  return a.prefix ? (int64_t)cta * kItemRows + (int64_t)g * a.head_rows + it.part_row : (int64_t)(2 * cta + (starts ? 1 : 0)) * kItemRows;
}

struct RowsShape {
  int32_t dtype, cache_dtype, h_q, h_kv, d, P, batch, max_blocks, n_pages, jobs, prefix;
  int64_t max_tokens, page_stride, head_stride, row_stride, q_stride;
  float scale, softcap;
  int32_t window;
};
// Workspace bytes behind `front` bytes that belong to others (0: the device cannot be queried).
size_t rows_ws(const RowsShape& p, size_t front);
kvsel_status launch_chunk_attend(const RowsShape& p, const RowsArgs& in, void* ws, cudaStream_t s);
kvsel_status launch_prefix_attend(const RowsShape& p, const PagedShape& own, const RowsArgs& in, void* ws, size_t front, cudaStream_t s);

}  // namespace kvsel
