// Pages, slots, positions and block tables of a step's new rows, from the requests' lengths.
//
// With have_b = ceil(lens_b / P) pages and want_b = ceil((lens_b + new_b) / P), request b takes
// want_b - have_b pages of the free queue; the exclusive sums over the requests of those counts and of
// new_b give every request its place in the queue and among the step's tokens.  Everything is integer.
//
// One CTA forms the two sums (a request per thread and a shuffle scan: a batch is at most 4096), so the
// lengths and the queue's head may be updated in place: they are read before anything is written.  A
// decode step's tokens are written by the same CTA; a prefill step's by a second grid that reads the
// sums from the workspace.
#include "paged.cuh"

namespace kvsel {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kTokensPerThread = 4;

// The sums of a step: where request b's tokens and new pages begin, and the rows it held.
struct Plan {
  const int32_t *tok, *pg, *old;
  int32_t n_tok, n_pg;
  int64_t head;
};

// The last request whose first token (page) is at most x; requests without one are passed over.
__device__ __forceinline__ int find_request(const int32_t* first, int batch, int x) {
  int lo = 0, hi = batch;                        // first[lo] <= x < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Tokens [t0, t0 + 4) of the step: slot, position and request, or the padding's values.
__device__ __forceinline__ void fill_tokens(const AssignArgs& a, const Plan& p, const int32_t* tok, int64_t t0) {
  int b = t0 < p.n_tok ? find_request(tok, a.batch, (int)t0) : 0;
#pragma unroll
  for (int i = 0; i < kTokensPerThread; ++i) {
    const int64_t t = t0 + i;
    if (t >= a.max_tokens) return;
    int64_t slot = -1, pos = 0;
    int32_t id = -1;
    if (t < p.n_tok) {
      while (tok[b + 1] <= t) ++b;
      const int row = p.old[b] + ((int)t - tok[b]);
      const int page_at = row / a.P, held = (p.old[b] + a.P - 1) / a.P;
      const int32_t page = page_at < held ? a.block_tables[(int64_t)b * a.max_blocks + page_at]
                                          : a.free_pages[p.head + p.pg[b] + (page_at - held)];
      if (page >= 0 && page < a.n_pages) slot = (int64_t)page * a.P + (row - page_at * a.P);
      else set_device_error(a.err, KVSEL_ERR_DEVICE, (uint32_t)b);
      pos = row + (a.pos_offset != nullptr ? a.pos_offset[b] : 0);
      id = b;
    }
    a.slots[t] = slot;
    if (a.positions != nullptr) a.positions[t] = pos;
    if (a.seq_ids != nullptr) a.seq_ids[t] = id;
  }
}

// New page j of the step: its id goes behind the pages its request held.
__device__ __forceinline__ void fill_page(const AssignArgs& a, const Plan& p, const int32_t* pg, int j) {
  const int b = find_request(pg, a.batch, j);
  const int held = (p.old[b] + a.P - 1) / a.P;
  a.block_tables[(int64_t)b * a.max_blocks + held + (j - pg[b])] = a.free_pages[p.head + j];
}

// The step's sums, lengths and queue head; with `fill`, its tokens and table entries too.
__global__ void __launch_bounds__(kPlanThreads) page_assign_plan(const __grid_constant__ AssignArgs a, int fill) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t warp_tok[32], warp_pg[32];
  __shared__ int bad;
  int32_t* tok = sm;
  int32_t* pg = tok + a.batch + 1;
  int32_t* old = pg + a.batch + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
  wait_for_earlier_kernels();
  if (!fill) let_later_kernels_start();                        // (the fill: it waits for this grid's end)
  const int64_t head = *a.free_head;
  const int64_t cap = (int64_t)a.max_blocks * a.P;             // < 2^31
  if (tid == 0) bad = 0x7fffffff;
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
  int64_t it = st, ip = sp;                                    // inclusive over the warp's threads
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ut = __shfl_up_sync(0xffffffffu, it, o), up = __shfl_up_sync(0xffffffffu, ip, o);
    if (lane >= o) {
      it += ut;
      ip += up;
    }
  }
  if (lane == 31) {
    warp_tok[warp] = it;
    warp_pg[warp] = ip;
  }
  __syncthreads();
  int64_t bt = 0, bp = 0, n_tok = 0, n_pg = 0;                 // before this warp; in all
  for (int w = 0; w < n_warps; ++w) {
    if (w == warp) {
      bt = n_tok;
      bp = n_pg;
    }
    n_tok += warp_tok[w];
    n_pg += warp_pg[w];
  }
  const bool sums_ok = n_tok <= a.max_tokens && head >= 0 && head <= a.n_free && n_pg <= a.n_free - head;
  const bool ok = bad == 0x7fffffff && sums_ok;
  if (!ok) {
    if (tid == 0) {
      set_device_error(a.err, KVSEL_ERR_INVALID_ARG, (uint32_t)(bad != 0x7fffffff ? bad : a.batch));
      *a.free_head_out = head;
      a.indptr[a.batch] = 0;
    }
    for (int b = b0; b < b1; ++b) {
      a.indptr[b] = 0;
      a.lens_out[b] = a.lens[b];
    }
    n_tok = n_pg = 0;
  } else {
    int64_t t = bt + it - st, p = bp + ip - sp;
    for (int b = b0; b < b1; ++b) {
      const int m = tok[b], need = pg[b];
      tok[b] = (int)t;
      pg[b] = (int)p;
      a.indptr[b] = t;
      a.lens_out[b] = (int64_t)old[b] + m;
      t += m;
      p += need;
    }
    if (tid == 0) {
      tok[a.batch] = (int)n_tok;
      pg[a.batch] = (int)n_pg;
      a.indptr[a.batch] = n_tok;
      *a.free_head_out = head + n_pg;
    }
  }
  __syncthreads();
  if (fill) {
    const Plan p{tok, pg, old, (int32_t)n_tok, (int32_t)n_pg, head};
    for (int64_t t0 = (int64_t)tid * kTokensPerThread; t0 < a.max_tokens; t0 += (int64_t)blockDim.x * kTokensPerThread)
      fill_tokens(a, p, tok, t0);
    for (int j = tid; j < (int)n_pg; j += blockDim.x) fill_page(a, p, pg, j);
    return;
  }
  if (tid == 0) {
    a.plan[0] = (int32_t)n_tok;
    a.plan[1] = (int32_t)n_pg;
    *reinterpret_cast<int64_t*>(a.plan + 2) = head;
  }
  for (int x = tid; x < 3 * a.batch + 2; x += blockDim.x) a.plan[kAssignPlanHead + x] = sm[x];
}

// The tokens and table entries of a planned step.
__global__ void __launch_bounds__(kFillThreads) page_assign_fill(const __grid_constant__ AssignArgs a) {
  extern __shared__ int32_t tok[];
  wait_for_earlier_kernels();
  Plan p;
  p.n_tok = a.plan[0];
  p.n_pg = a.plan[1];
  p.head = *reinterpret_cast<const int64_t*>(a.plan + 2);
  p.tok = a.plan + kAssignPlanHead;
  p.pg = p.tok + a.batch + 1;
  p.old = p.pg + a.batch + 1;
  const int64_t t0 = ((int64_t)blockIdx.x * kFillThreads + threadIdx.x) * kTokensPerThread;
  const int64_t first = (int64_t)blockIdx.x * kFillThreads * kTokensPerThread;
  if (first < p.n_tok)                                          // (a failed step has no sums)
    for (int x = threadIdx.x; x <= a.batch; x += kFillThreads) tok[x] = p.tok[x];
  __syncthreads();
  if (t0 < a.max_tokens) fill_tokens(a, p, tok, t0);
  for (int64_t j = (int64_t)blockIdx.x * kFillThreads + threadIdx.x; j < p.n_pg; j += (int64_t)gridDim.x * kFillThreads)
    fill_page(a, p, p.pg, (int)j);
}

}  // namespace

kvsel_status launch_page_assign(const AssignArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(int32_t) * (3 * (size_t)a.batch + 2);
  const bool one = a.max_tokens <= 4096;
  const int64_t items = a.max_tokens > a.batch ? a.max_tokens : a.batch;
  const int threads = items <= 256 ? 256 : kPlanThreads;
  if (set_smem((const void*)page_assign_plan, smem) != cudaSuccess) return KVSEL_ERR_CUDA;
  {
    TraceScope ts("page_assign", s);
    const kvsel_status st = launch_after(page_assign_plan, dim3(1), threads, smem, s, a, one ? 1 : 0);
    if (st != KVSEL_OK || one) return st;
  }
  TraceScope ts("page_assign_fill", s);
  const int64_t grid = ceil_div(a.max_tokens, (int64_t)kFillThreads * kTokensPerThread);
  return launch_after(page_assign_fill, dim3((unsigned)grid), kFillThreads, sizeof(int32_t) * (a.batch + 1), s, a);
}

}  // namespace kvsel
