// Declarations shared by the beam search calls (beam_api.cu checks, the kernels' files launch).
#pragma once

#include "paged.cuh"

namespace kvsel {

constexpr int kSliceKeys = 8192;      // tokens of one row that a CTA takes at a time
constexpr int64_t kSelectCtas = 2048; // segments of all rows, about
constexpr int kMaxBeams = 64, kMaxBeamOut = 64;
constexpr int64_t kMaxLists = 8192;   // slices of a set's rows, and segments at most
constexpr int64_t kMaxSegSlices = 1024;   // of a segment: 2^23 terms of 2^40 at most, whose sum has 64 bits

// ---- beam_select.cu ----------------------------------------------------------------------
struct SelectArgs {
  int32_t batch, beams, n_out, vocab, pad_token;
  int32_t segments, seg_slices;         // of a row, and slices of a segment
  int64_t row_stride;
  const void* logits;
  const float* scores;
  const uint8_t* ended;
  float* scores_out;
  int32_t *parents, *tokens;
  float* lse;
  float2* best;         // [row][segment][n_out]: a segment's best tokens, (logit, token as bits) in order; token -1: none
  float* tops;          // [row][segment]: largest logit
  uint64_t* sums;       // [row][segment]: sum of exp(x - largest), in 2^-40
};
size_t beam_select_ws(int64_t rows, int32_t segments, int32_t n_out, size_t* best_off, size_t* sums_off, size_t* tops_off);
kvsel_status launch_beam_select(const SelectArgs& a, int32_t dtype, cudaStream_t s);

// ---- beam_reorder.cu ---------------------------------------------------------------------
constexpr int kReorderCols = 128;     // table columns of a CTA
struct ReorderCopy {
  int32_t source, page, rows, pad;    // the parent's page, the child's, and its filled rows
};
struct ReorderPlan {
  int64_t head;                       // queue entries taken before the call
  int32_t freed, copies, bad, pad;
};
struct ReorderArgs {
  int32_t batch, beams, P, max_blocks, tiles, n_layers, h_kv;
  int64_t n_pages, n_free, page_stride, head_stride, row_stride, layer_stride;   // strides in bytes
  int32_t row_bytes;
  const int32_t* parents;
  const int64_t* lens;
  const int32_t* tables;
  int32_t* free_pages;
  const int64_t* free_head;
  int32_t* tables_out;
  int64_t *lens_out, *head_out;
  uint8_t *k, *v;
  DeviceError* err;
  ReorderPlan* plan;
  int32_t* parent_of;                 // [batch * beams]: the parents as they were read
  int32_t* blocks;                    // [batch * beams]: pages held before
  int32_t* count;                     // [batch][tiles]: pages freed, then those freed before; negative: refused
  int32_t* twin;                      // [batch * beams]: the page of its own that a child gets, or -1
  int32_t* freed;                     // [batch][tiles][beams * kReorderCols]: pages freed
  ReorderCopy* copy;                  // [batch * beams]
};
size_t beam_reorder_ws(int32_t batch, int32_t beams, int32_t tiles, size_t off[7]);
kvsel_status launch_beam_reorder(const ReorderArgs& a, cudaStream_t s);

}  // namespace kvsel
