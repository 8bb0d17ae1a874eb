// Declarations shared by the calls over a paged cache (paged_api.cu checks, the kernels' files launch).
#pragma once

#include "internal.cuh"

namespace kvsel {

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A launch whose CTAs may start while the stream's last kernel drains; the kernel calls wait_for_earlier_kernels()
// before it touches memory that others write or read.
template <typename... Params, typename... Args>
kvsel_status launch_after(void (*kern)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  const bool ok = cudaLaunchKernelEx(&c, kern, static_cast<Params>(args)...) == cudaSuccess;
  count_launch();
  return ok && cudaGetLastError() == cudaSuccess ? KVSEL_OK : KVSEL_ERR_CUDA;
}
// Everything the stream's earlier kernels wrote is there, and what they read may be overwritten.
__device__ __forceinline__ void wait_for_earlier_kernels() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The stream's next kernel may be launched (it still waits for this grid's end before it touches memory).
__device__ __forceinline__ void let_later_kernels_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// CTAs of a kernel resident at once on the current device (0: it cannot be queried), asked once per device,
// kernel and shared-memory size (paged_api.cu).
int64_t resident_ctas(const void* kern, int threads, size_t smem);

// ---- page_assign.cu ----------------------------------------------------------------------
struct AssignArgs {
  int32_t P, batch, max_blocks;
  int64_t n_pages, n_free, max_tokens;
  const int64_t *lens, *n_new, *pos_offset;
  const int32_t* free_pages;
  const int64_t* free_head;
  int32_t* block_tables;
  int64_t *lens_out, *free_head_out, *indptr, *slots, *positions;
  int32_t* seq_ids;
  int32_t* plan;        // [3 * batch + kAssignPlanHead] in the workspace, after the error word
  DeviceError* err;
};
constexpr int kAssignPlanHead = 8;
inline size_t page_assign_ws(int32_t batch) {
  const size_t n = sizeof(DeviceError) + sizeof(int32_t) * (3 * (size_t)batch + kAssignPlanHead + 2);
  return (n + KVSEL_WS_ALIGN - 1) / KVSEL_WS_ALIGN * KVSEL_WS_ALIGN;
}
kvsel_status launch_page_assign(const AssignArgs& a, cudaStream_t s);

// ---- rope_append.cu ----------------------------------------------------------------------
struct RopeArgs {
  int32_t h_q, h_kv, d, P, rot, e4m3;
  int32_t unit_rows, stage_bytes, stages;   // head rows of a unit, a warp's ring (set by the launcher)
  int32_t rounds;       // whole tokens of every warp; then its units of the rest, and the warps with one more (the same)
  int64_t share, extra;
  int64_t n, n_slots, page_stride, head_stride, row_stride;
  int64_t q_stride, q_head, k_stride, k_head, v_stride, v_head;
  float factor, eps, bias;
  const void *q, *k, *v;
  const int64_t *positions, *slots;
  const void *q_weight, *k_weight;
  const double* inv_freq;
  void *q_out, *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  DeviceError* err;
};
kvsel_status launch_rope_append(const RopeArgs& a, int32_t dtype, int32_t layout, cudaStream_t s);

// ---- paged_attend.cu ---------------------------------------------------------------------
struct PagedShape {
  int32_t dtype, cache_dtype, h_q, h_kv, d, P, batch, max_blocks, n_pages;
  int64_t page_stride, head_stride, row_stride, q_stride;
  float scale, softcap;
  int32_t window;
};
// Workspace bytes of a call on the current device (0: the device cannot be queried).
size_t paged_attend_ws(const PagedShape& p);
kvsel_status launch_paged_attend(const PagedShape& p, const void* q, const void* k, const void* v,
                                 const int32_t* tables, const int64_t* lens, const float* slopes,
                                 const float* k_scale, const float* v_scale, void* o, float* lse, void* ws,
                                 cudaStream_t s);

}  // namespace kvsel
