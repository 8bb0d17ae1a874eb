// Block tables of a set's beams after a selection: child j takes its parent's pages, pages that no child names are freed,
// and a second child of a parent gets its own copy of the last page if that is part full.
//
// Beams of a set that share a page name it in the same column, so a column's pages are judged by themselves: a page is freed
// if none of its beams goes on, once, for the first beam that names it.  Freed pages go onto the queue in front of its head
// in the order (set, column, beam), copies then take pages from the new head on in the order (set, child): the freed ones
// first.  Integer work, the same result every time.
//
// Bound: the copies (rows x layers x heads, read and written); small calls by the chain of launches.  Three of them, since
// a page's place in the queue needs the count of all sets' freed pages before it: the freed pages by (set, 128 columns); one
// CTA's sums, checks, lengths and list of copies with the pages they take; tables, queue and copies.  Each starts while the one
// before it drains.  A refused call stops at the second: nothing of its outputs is written.  (One set of 4: 12 us, 24 of 5: 14;
// 64 of 8 with 378 MB to read and write: 77 us, 4.9 TB/s.)
#include <algorithm>

#include "beam.cuh"
#include "sm100.cuh"

namespace kvsel {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int64_t kPlanEntries = 8192;       // (set, tile)s whose sums the plan keeps in shared memory
constexpr int kCopyThreads = 256;

// What a CTA of (set, column tile) knows of its set: parents, which beams go on, pages held; false: refused (bad gives why).
struct Set {
  int32_t parent[kMaxBeams], blocks[kMaxBeams], twin[kMaxBeams];   // twin: the page of its own that a child gets, or -1
  uint64_t goes_on;                           // beams that have a child
};

__device__ __forceinline__ int blocks_of(int64_t len, int P) { return (int)((len + P - 1) / P); }

// The freed pages of this thread's column: bit k for the first beam that names such a page.  `bad`: a held page outside the pool.
__device__ __forceinline__ uint64_t freed_of(const ReorderArgs& a, const Set& set, const int32_t* tile, int x, int column, bool& bad) {
  uint64_t freed = 0;
  for (int k = 0; k < a.beams; ++k) {
    if (column >= set.blocks[k]) continue;
    const int32_t page = tile[k * kReorderCols + x];
    bad |= page < 0 || page >= a.n_pages;
    if ((set.goes_on >> k) & 1) continue;
    bool kept = false;
    for (int j = 0; j < a.beams && !kept; ++j)
      kept = j != k && column < set.blocks[j] && tile[j * kReorderCols + x] == page && (j < k || ((set.goes_on >> j) & 1));
    if (!kept) freed |= uint64_t(1) << k;     // (named by an earlier beam: judged there)
  }
  return freed;
}

__device__ __forceinline__ void load_tile(const ReorderArgs& a, const Set& set, int s, int first, int32_t* tile) {
  const int column = first + threadIdx.x;
  for (int k = 0; k < a.beams; ++k)
    if (column < set.blocks[k]) tile[k * kReorderCols + threadIdx.x] = a.tables[((int64_t)s * a.beams + k) * a.max_blocks + column];
}

__global__ void __launch_bounds__(kReorderCols) reorder_count(const __grid_constant__ ReorderArgs a) {
  extern __shared__ int32_t tile[];
  __shared__ Set set;
  __shared__ int refused;
  const int s = blockIdx.y, first = blockIdx.x * kReorderCols;
  wait_for_earlier_kernels();
  let_later_kernels_start();
  if (threadIdx.x == 0) refused = 0, set.goes_on = 0;
  __syncthreads();
  if (threadIdx.x < a.beams) {
    const int k = threadIdx.x;
    const int64_t len = a.lens[(int64_t)s * a.beams + k];
    const int32_t p = a.parents[(int64_t)s * a.beams + k];
    const bool len_ok = len >= 0 && len <= (int64_t)a.max_blocks * a.P, p_ok = p >= 0 && p < a.beams;
    if (!len_ok || !p_ok) atomicOr(&refused, 1);
    set.parent[k] = p;
    set.blocks[k] = len_ok ? blocks_of(len, a.P) : 0;
    if (p_ok) atomicOr(reinterpret_cast<unsigned long long*>(&set.goes_on), 1ull << p);
  }
  __syncthreads();
  load_tile(a, set, s, first, tile);          // (a thread reads its own column alone)
  bool bad = false;
  uint64_t freed = freed_of(a, set, tile, threadIdx.x, first + threadIdx.x, bad);
  if (bad) atomicOr(&refused, 2);
  // the tile's freed pages, by column and beam
  __shared__ int sum[kReorderCols / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, own = __popcll(freed);
  int at = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += u;
  }
  if (lane == 31) sum[warp] = at;
  __syncthreads();
  for (int w = 0; w < warp; ++w) at += sum[w];
  const int64_t entry = (int64_t)s * a.tiles + blockIdx.x;
  int32_t* list = a.freed + entry * (a.beams * kReorderCols);
  if (threadIdx.x == kReorderCols - 1) a.count[entry] = refused != 0 ? -refused : at;
  for (at -= own; freed != 0; freed &= freed - 1) list[at++] = tile[(__ffsll((long long)freed) - 1) * kReorderCols + threadIdx.x];
}

// Inclusive sum over the CTA's threads; `all`: of all of them.
__device__ __forceinline__ int scan(int x, int* warp_sum, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int before = 0;
  all = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    all += warp_sum[w];
  }
  return before + x;
}

__global__ void __launch_bounds__(kPlanThreads) reorder_plan(const __grid_constant__ ReorderArgs a) {
  extern __shared__ int32_t before_sm[];      // freed pages before every (set, tile), where they fit
  __shared__ int warp_sum[kPlanThreads / 32];
  __shared__ int bad;                         // the first refused request, the kind of its fault in the low two bits
  const int tid = threadIdx.x, n = a.batch * a.beams;
  wait_for_earlier_kernels();
  let_later_kernels_start();
  if (tid == 0) bad = 0x7fffffff;
  const int64_t head = *a.free_head;
  __syncthreads();
  // freed pages before every (set, tile)
  const int64_t entries = (int64_t)a.batch * a.tiles;
  int freed = 0;
  for (int64_t i0 = 0; i0 < entries; i0 += kPlanThreads) {
    const int64_t i = i0 + tid;
    int c = i < entries ? a.count[i] : 0;
    if (c < 0) {
      atomicMin(&bad, (int)(i / a.tiles) * a.beams * 4 + -c);
      c = 0;
    }
    int all;
    const int upto = scan(c, warp_sum, all);
    if (i < entries) {
      a.count[i] = freed + upto - c;
      if (entries <= kPlanEntries) before_sm[i] = freed + upto - c;
    }
    freed += all;
  }
  __syncthreads();
  bool ok = bad == 0x7fffffff;
  // requests, a run of them per thread: what they held, and which of them are copies
  const int per = (n + kPlanThreads - 1) / kPlanThreads, r0 = min(n, tid * per), r1 = min(n, r0 + per);
  int mine = 0;
  if (ok) {
    for (int r = r0; r < r1; ++r) {
      const int p = a.parents[r];
      a.parent_of[r] = p;
      a.blocks[r] = blocks_of(a.lens[r], a.P);
      const int set0 = r / a.beams * a.beams;
      bool twin = false;
      for (int j = set0; j < r && !twin; ++j) twin = a.parents[j] == p;
      mine += twin && a.lens[set0 + p] % a.P != 0;
    }
  }
  int copies;
  int at = scan(mine, warp_sum, copies) - mine;
  int fault = 0;
  if (ok) {
    // the pages left behind the head, the freed ones among them, must do for the copies
    if (head < freed || head > a.n_free || copies - freed > a.n_free - head) fault = 1;
    else
      for (int c = freed + tid; c < copies; c += kPlanThreads) {
        const int32_t page = a.free_pages[head - freed + c];
        if (page < 0 || page >= a.n_pages) fault = 2;
      }
    if (fault) atomicMin(&bad, n * 4 + fault);
  }
  __syncthreads();
  ok = bad == 0x7fffffff;
  if (!ok) {
    if (tid == 0) {
      set_device_error(a.err, (bad & 3) == 2 ? KVSEL_ERR_DEVICE : KVSEL_ERR_INVALID_ARG, (uint32_t)(bad >> 2));
      a.plan->bad = 1;
    }
    return;
  }
  int64_t len[4];                             // (n <= 4096, 1024 threads: up to four requests each)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + i;
    if (r >= r1) continue;
    const int set0 = r / a.beams * a.beams, p = a.parents[r];
    len[i] = a.lens[set0 + p];
    bool twin = false;
    for (int j = set0; j < r && !twin; ++j) twin = a.parents[j] == p;
    const int rest = (int)(len[i] % a.P);
    int32_t page = -1;
    if (twin && rest != 0) {
      const int column = blocks_of(len[i], a.P) - 1, c = at++;
      if (c < freed) {
        // the c-th freed page: of the last (set, tile) with at most c before it
        int64_t lo = 0, hi = entries;
        while (hi - lo > 1) {
          const int64_t mid = (lo + hi) >> 1;
          if ((entries <= kPlanEntries ? before_sm[mid] : a.count[mid]) <= c) lo = mid; else hi = mid;
        }
        page = a.freed[lo * (a.beams * kReorderCols) + (c - (entries <= kPlanEntries ? before_sm[lo] : a.count[lo]))];
      } else {
        page = a.free_pages[head - freed + c];
      }
      a.copy[c] = ReorderCopy{a.tables[((int64_t)set0 + p) * a.max_blocks + column], page, rest, 0};
    }
    a.twin[r] = page;
  }
  __syncthreads();                            // every length is read: they may be written over
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r0 + i < r1) a.lens_out[r0 + i] = len[i];
  if (tid == 0) {
    *a.plan = ReorderPlan{head, freed, copies, 0, 0};
    *a.head_out = head - freed + copies;
  }
}

// The first `table_ctas` CTAs take (set, tile)s: the children's entries, and the tile's freed pages into the queue.  The others take
// units of the copies, one copy's rows in one layer of K or V: 16 bytes per thread and turn, heads and rows in the pool's
// own strides.
__global__ void __launch_bounds__(kCopyThreads) reorder_apply(const __grid_constant__ ReorderArgs a, int table_ctas) {
  extern __shared__ int32_t tile[];
  __shared__ Set set;
  wait_for_earlier_kernels();
  const ReorderPlan plan = *a.plan;
  if (plan.bad) return;
  if ((int)blockIdx.x < table_ctas) {
    const int64_t entries = (int64_t)a.batch * a.tiles;
    for (int64_t entry = blockIdx.x; entry < entries; entry += table_ctas) {
      const int s = (int)(entry / a.tiles), first = (int)(entry - (int64_t)s * a.tiles) * kReorderCols;
      __syncthreads();                        // (the last tile is done with)
      if (threadIdx.x < a.beams) {
        set.parent[threadIdx.x] = a.parent_of[s * a.beams + threadIdx.x];
        set.blocks[threadIdx.x] = a.blocks[s * a.beams + threadIdx.x];
        set.twin[threadIdx.x] = a.twin[s * a.beams + threadIdx.x];
      }
      __syncthreads();
      // rows by halves of the CTA; all of a tile is read before any of it is written (the tables may be updated in place)
      const int x = threadIdx.x & (kReorderCols - 1), k0 = threadIdx.x / kReorderCols, column = first + x;
      for (int k = k0; k < a.beams; k += kCopyThreads / kReorderCols)
        if (column < set.blocks[k]) tile[k * kReorderCols + x] = a.tables[((int64_t)s * a.beams + k) * a.max_blocks + column];
      __syncthreads();
      for (int j = k0; j < a.beams; j += kCopyThreads / kReorderCols) {
        const int p = set.parent[j], n = set.blocks[p];
        if (column < n)
          a.tables_out[((int64_t)s * a.beams + j) * a.max_blocks + column] =
              column == n - 1 && set.twin[j] >= 0 ? set.twin[j] : tile[p * kReorderCols + x];
      }
      const int before = a.count[entry], upto = entry + 1 < entries ? a.count[entry + 1] : plan.freed;
      const int32_t* list = a.freed + entry * (a.beams * kReorderCols);
      for (int i = before + threadIdx.x; i < upto; i += kCopyThreads) a.free_pages[plan.head - plan.freed + i] = list[i - before];
    }
    return;
  }
  const int64_t units = (int64_t)plan.copies * a.n_layers * 2;
  const int chunks = a.row_bytes / 16;
  // consecutive chunks are consecutive memory: rows inside heads or heads inside rows
  const bool heads_inside = a.head_stride < a.row_stride;
  for (int64_t u = blockIdx.x - table_ctas; u < units; u += gridDim.x - table_ctas) {
    const int c = (int)(u / (a.n_layers * 2)), part = (int)(u - (int64_t)c * a.n_layers * 2);
    const ReorderCopy y = a.copy[c];
    uint8_t* base = ((part & 1) ? a.v : a.k) + (part >> 1) * a.layer_stride;
    const uint8_t* from = base + y.source * a.page_stride;
    uint8_t* to = base + y.page * a.page_stride;
    const int inner = heads_inside ? a.h_kv : y.rows, n = a.h_kv * y.rows * chunks;
    for (int i0 = threadIdx.x; i0 < n; i0 += 4 * kCopyThreads) {
      uint4 v[4];
      int64_t at[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + e * kCopyThreads;
        if (i >= n) continue;
        const int row = i / chunks, o = row / inner, in = row - o * inner;
        at[e] = (heads_inside ? in * a.head_stride + o * a.row_stride : o * a.head_stride + in * a.row_stride) + (i - row * chunks) * 16;
        v[e] = *reinterpret_cast<const uint4*>(from + at[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i0 + e * kCopyThreads < n) *reinterpret_cast<uint4*>(to + at[e]) = v[e];
    }
  }
}

}  // namespace

size_t beam_reorder_ws(int32_t batch, int32_t beams, int32_t tiles, size_t off[7]) {
  auto up = [](size_t x) { return (x + KVSEL_WS_ALIGN - 1) / KVSEL_WS_ALIGN * KVSEL_WS_ALIGN; };
  const size_t n = (size_t)batch * beams;
  off[0] = sizeof(DeviceError);                                // the plan
  off[1] = off[0] + KVSEL_WS_ALIGN;                            // parents
  off[2] = up(off[1] + sizeof(int32_t) * n);                   // pages held
  off[3] = up(off[2] + sizeof(int32_t) * n);                   // twins' pages
  off[4] = up(off[3] + sizeof(int32_t) * n);                   // copies
  off[5] = up(off[4] + sizeof(ReorderCopy) * n);               // counts
  off[6] = up(off[5] + sizeof(int32_t) * (size_t)batch * tiles);                        // freed pages by (set, tile)
  return up(off[6] + sizeof(int32_t) * n * (size_t)tiles * kReorderCols);
}

kvsel_status launch_beam_reorder(const ReorderArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(int32_t) * (size_t)a.beams * kReorderCols;
  const int64_t entries = (int64_t)a.batch * a.tiles;
  kvsel_status st;
  {
    TraceScope ts("reorder_count", s);
    if ((st = launch_after(reorder_count, dim3((unsigned)a.tiles, (unsigned)a.batch), kReorderCols, smem, s, a)) != KVSEL_OK) return st;
  }
  {
    TraceScope ts("reorder_plan", s);
    const size_t sums = entries <= kPlanEntries ? sizeof(int32_t) * (size_t)entries : 0;
    if ((st = launch_after(reorder_plan, dim3(1), kPlanThreads, sums, s, a)) != KVSEL_OK) return st;
  }
  TraceScope ts("reorder_apply", s);
  const int64_t resident = resident_ctas((const void*)reorder_apply, kCopyThreads, smem);
  if (resident <= 0) return KVSEL_ERR_CUDA;
  // (every set keeps a beam)
  const int64_t units = (int64_t)a.batch * (a.beams - 1) * a.n_layers * 2, table_ctas = std::min(entries, resident);
  return launch_after(reorder_apply, dim3((unsigned)(table_ctas + std::min(resident, units))), kCopyThreads, smem, s, a, (int)table_ctas);
}

}  // namespace kvsel
