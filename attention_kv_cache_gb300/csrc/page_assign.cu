// Pages, slots, positions and block tables of a step's new rows, from the requests' lengths.
//
// With have_b = ceil(lens_b / P) pages and want_b = ceil((lens_b + new_b) / P), request b takes
// want_b - have_b pages of the free queue; the exclusive sums over the requests of those counts and of
// new_b give every request its place in the queue and among the step's tokens.  Everything is integer.
//
// Latency is what this costs: a step reads and writes a few KB to a few MB.  So a CTA forms the sums of all requests
// itself (a batch is at most 4096: a few requests per thread and a shuffle scan), and every CTA of the step does so,
// which takes one launch and no exchange between CTAs.  The tokens and pages are then dealt to the threads, which find
// their request by bisection in shared memory.
//
// Lengths and queue head that are updated in place must not be written while another CTA still reads them: a step small
// enough for one CTA writes them after its own reads; a larger one in place takes two launches, one CTA that leaves
// the sums in the workspace and a grid that reads them there.
//
// Measured (GB300, device time): 8 requests of one new row each 2.6 us, 1024 requests 4.2 us, 262144 rows of 64 requests
// 6.8 us; in place 1061 rows 3.9 us by one CTA, 3970 rows 4.7 us and 262144 rows 5.9 us by two launches (3970 by one CTA 6.6).
#include <algorithm>

#include "paged.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 1024;
constexpr int64_t kOneCta = 2048;     // a step in place of up to so many tokens is one CTA's

// The sums of a step: where request b's tokens and new pages begin, and the rows it held.
struct Sums {
  const int32_t *tok, *pg, *old;      // [batch + 1], [batch + 1], [batch]
  int32_t n_tok, n_pg;
  int64_t head;
};

// The last of `batch` requests whose first token (page) is at most x: `first` rises, with equal entries where a request
// has none.
__device__ __forceinline__ int find_request(const int32_t* first, int batch, int x) {
  int lo = 0, hi = batch;                        // first[lo] <= x < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Forms the sums in shared memory; with `write`, puts out offsets, lengths and queue head.  A step that cannot be
// carried out has no tokens and no pages.
__device__ Sums form_sums(const AssignArgs& a, int32_t* sm, bool write) {
  __shared__ int64_t warp_tok[32], warp_pg[32];
  __shared__ int bad;
  int32_t *tok = sm, *pg = tok + a.batch + 1, *old = pg + a.batch + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
  const int64_t head = *a.free_head;
  const int64_t cap = (int64_t)a.max_blocks * a.P;             // < 2^31
  if (tid == 0) bad = 0x7fffffff;
  if (tid < 32) warp_tok[tid] = warp_pg[tid] = 0;
  __syncthreads();
  // this thread's requests: counts and their sums
  const int per = (a.batch + blockDim.x - 1) / blockDim.x;
  const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
  int64_t st = 0, sp = 0;
  for (int b = b0; b < b1; ++b) {
    int64_t L = a.lens[b], m = a.n_new[b];
    if (L < 0 || L > cap || m < 0 || m > cap - L) {
      atomicMin(&bad, b);
      L = m = 0;
    }
    const int need = ((int)(L + m) + (a.P - 1)) / a.P - ((int)L + (a.P - 1)) / a.P;
    old[b] = (int)L;
    tok[b] = (int)m;
    pg[b] = need;
    st += m;
    sp += need;
  }
  auto scan = [&](int64_t& x, int64_t& y) {                    // inclusive, over the warp's lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t ux = __shfl_up_sync(0xffffffffu, x, o), uy = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x += ux;
        y += uy;
      }
    }
  };
  int64_t it = st, ip = sp;
  scan(it, ip);
  if (lane == 31) {
    warp_tok[warp] = it;
    warp_pg[warp] = ip;
  }
  __syncthreads();
  int64_t bt = warp_tok[lane], bp = warp_pg[lane];             // every warp scans the warps' sums
  scan(bt, bp);
  const int64_t n_tok = __shfl_sync(0xffffffffu, bt, n_warps - 1), n_pg = __shfl_sync(0xffffffffu, bp, n_warps - 1);
  const int64_t before_t = __shfl_sync(0xffffffffu, bt, max(warp - 1, 0)), before_p = __shfl_sync(0xffffffffu, bp, max(warp - 1, 0));
  const bool sums_ok = n_tok <= a.max_tokens && head >= 0 && head <= a.n_free && n_pg <= a.n_free - head;
  const bool ok = bad == 0x7fffffff && sums_ok;
  if (ok) {
    int64_t t = (warp > 0 ? before_t : 0) + it - st, p = (warp > 0 ? before_p : 0) + ip - sp;
    for (int b = b0; b < b1; ++b) {
      const int m = tok[b], need = pg[b];
      tok[b] = (int)t;
      pg[b] = (int)p;
      if (write) {
        a.indptr[b] = t;
        a.lens_out[b] = (int64_t)old[b] + m;
      }
      t += m;
      p += need;
    }
    if (tid == 0) {
      tok[a.batch] = (int)n_tok;
      pg[a.batch] = (int)n_pg;
      if (write) {
        a.indptr[a.batch] = n_tok;
        *a.free_head_out = head + n_pg;
      }
    }
  } else if (write) {
    if (tid == 0) {
      set_device_error(a.err, KVSEL_ERR_INVALID_ARG, (uint32_t)(bad != 0x7fffffff ? bad : a.batch));
      *a.free_head_out = head;
      a.indptr[a.batch] = 0;
    }
    for (int b = b0; b < b1; ++b) {
      a.indptr[b] = 0;
      a.lens_out[b] = a.lens[b];
    }
  }
  __syncthreads();
  return Sums{tok, pg, old, ok ? (int32_t)n_tok : 0, ok ? (int32_t)n_pg : 0, head};
}

// This thread's tokens and pages of the step.
__device__ __forceinline__ void fill(const AssignArgs& a, const Sums& p) {
  const int64_t step = (int64_t)gridDim.x * blockDim.x, first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t t = first; t < a.max_tokens; t += step) {
    int64_t slot = -1, pos = 0;                                 // (of padding)
    int b = -1;
    if (t < p.n_tok) {
      b = find_request(p.tok, a.batch, (int)t);
      const int row = p.old[b] + ((int)t - p.tok[b]);
      const int at = row / a.P, held = (p.old[b] + a.P - 1) / a.P;
      const int32_t page = at < held ? a.block_tables[(int64_t)b * a.max_blocks + at] : a.free_pages[p.head + p.pg[b] + (at - held)];
      if (page >= 0 && page < a.n_pages) slot = (int64_t)page * a.P + (row - at * a.P);
      else set_device_error(a.err, KVSEL_ERR_DEVICE, (uint32_t)b);
      pos = row + (a.pos_offset != nullptr ? a.pos_offset[b] : 0);
    }
    a.slots[t] = slot;
    if (a.positions != nullptr) a.positions[t] = pos;
    if (a.seq_ids != nullptr) a.seq_ids[t] = b;
  }
  // new page j goes behind the pages its request held
  for (int64_t j = first; j < p.n_pg; j += step) {
    const int b = find_request(p.pg, a.batch, (int)j);
    const int held = (p.old[b] + a.P - 1) / a.P;
    a.block_tables[(int64_t)b * a.max_blocks + held + ((int)j - p.pg[b])] = a.free_pages[p.head + j];
  }
}

// A whole step: any grid where nothing is updated in place, else one CTA.
__global__ void __launch_bounds__(kThreads) page_assign(const __grid_constant__ AssignArgs a) {
  extern __shared__ int32_t sm[];
  wait_for_earlier_kernels();
  fill(a, form_sums(a, sm, blockIdx.x == 0));
}

// The sums of a step in place, into the workspace.
__global__ void __launch_bounds__(kThreads) page_assign_plan(const __grid_constant__ AssignArgs a) {
  extern __shared__ int32_t sm[];
  wait_for_earlier_kernels();
  let_later_kernels_start();                                   // (the fill: it waits for this grid's end)
  const Sums p = form_sums(a, sm, true);
  if (threadIdx.x == 0) {
    a.plan[0] = p.n_tok;
    a.plan[1] = p.n_pg;
    *reinterpret_cast<int64_t*>(a.plan + 2) = p.head;
  }
  for (int x = threadIdx.x; x < 3 * a.batch + 2; x += blockDim.x) a.plan[kAssignPlanHead + x] = sm[x];
}

// The tokens and table entries of a planned step.
__global__ void __launch_bounds__(kThreads) page_assign_fill(const __grid_constant__ AssignArgs a) {
  extern __shared__ int32_t sm[];
  wait_for_earlier_kernels();
  for (int x = threadIdx.x; x < 3 * a.batch + 2; x += blockDim.x) sm[x] = a.plan[kAssignPlanHead + x];
  const int32_t n_tok = a.plan[0], n_pg = a.plan[1];
  const int64_t head = *reinterpret_cast<const int64_t*>(a.plan + 2);
  __syncthreads();
  fill(a, Sums{sm, sm + a.batch + 1, sm + 2 * (a.batch + 1), n_tok, n_pg, head});
}

}  // namespace

kvsel_status launch_page_assign(const AssignArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(int32_t) * (3 * (size_t)a.batch + 2);
  const bool in_place = a.lens_out == a.lens || a.free_head_out == a.free_head;
  const bool one = in_place && a.max_tokens <= kOneCta;
  const unsigned threads = std::max<int64_t>(a.max_tokens, a.batch) <= 256 ? 256 : kThreads;
  const unsigned grid = one ? 1 : (unsigned)std::min<int64_t>(std::max<int64_t>(1, ceil_div(a.max_tokens, threads)), 1 << 12);
  if (one || !in_place) {
    if (set_smem((const void*)page_assign, smem) != cudaSuccess) return KVSEL_ERR_CUDA;
    TraceScope ts("page_assign", s);
    return launch_after(page_assign, dim3(grid), threads, smem, s, a);
  }
  if (set_smem((const void*)page_assign_plan, smem) != cudaSuccess || set_smem((const void*)page_assign_fill, smem) != cudaSuccess)
    return KVSEL_ERR_CUDA;
  {
    TraceScope ts("page_assign", s);
    const kvsel_status st = launch_after(page_assign_plan, dim3(1), kThreads, smem, s, a);
    if (st != KVSEL_OK) return st;
  }
  TraceScope ts("page_assign_fill", s);
  return launch_after(page_assign_fill, dim3(grid), kThreads, smem, s, a);
}

}  // namespace kvsel
