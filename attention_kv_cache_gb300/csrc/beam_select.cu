// The best continuations of a set of beams: score(k, v) = s_k + x_kv - log sum_u exp x_ku, the first n of beams x vocab.
//
// Bound: the logits, read once.  A CTA takes a slice of 8192 tokens of one row into registers and leaves the slice's largest
// logit, its sum of exponentials and its n best tokens in order; a second kernel, a CTA per set, forms the rows' log-sums,
// finds the n lists whose heads are best (an entry of any other list comes behind n heads) and ranks what they hold.
//
// A slice's n best: of 64 (or 256) groups of threads the n-th largest group maximum is found bit by bit by one warp, and is
// a lower bound of the n-th largest logit; the few tokens at or above it (n to 1.4 n of independent logits) are ranked by
// counting.  Where more than kCandidates reach it (equal logits), the exact n-th (logit, token) is found by bisection over
// the slice.
//
// Ties are the rule with 16-bit logits, and scores of different beams may lie within a rounding of each other, so scores are
// formed and compared in 64 bits.  A slice's exponentials are ex2.approx (2^-22 of each, of either sign) summed in fp32 by
// thread and then as 64-bit whole multiples of 2^-40: the sum is off by the mean of its terms' errors and the same for equal
// rows, whatever CTA forms it.
#include <cuda_fp16.h>

#include "beam.cuh"
#include "sm100.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 256, kEach = kSliceKeys / kThreads;
constexpr int kCandidates = 1024;
constexpr int kMergeThreads = 1024;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  return (b >> 63) ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float no_nan(float x) { return x == x ? x + 0.f : -INFINITY; }   // (-0 becomes 0: they are equal)
__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Element i of a thread's kEach is token `first + place(tid, i)` of its slice; places rise with i.  Vectors of 16 bytes where
// all rows are aligned to them, else single elements, neighbours on neighbouring threads.
template <typename T, bool VEC>
__device__ __forceinline__ int place(int tid, int i) {
  constexpr int V = 16 / (int)sizeof(T);
  return VEC ? (i / V * kThreads + tid) * V + i % V : i * kThreads + tid;
}

template <typename T, bool VEC, int KEYS>
__global__ void __launch_bounds__(kThreads) beam_slice(const __grid_constant__ SelectArgs a) {
  __shared__ uint32_t group_key[32 * KEYS];
  __shared__ float warp_max[kThreads / 32];
  __shared__ uint64_t warp_sum[kThreads / 32];
  __shared__ uint32_t edge;
  __shared__ int n_cand;
  __shared__ uint64_t cand[kCandidates];      // (ordered logit, all ones less the place in the slice)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slice = blockIdx.x % a.slices;
  const int64_t row = blockIdx.x / a.slices;
  const int first = slice * kSliceKeys, n_here = min(kSliceKeys, a.vocab - first);
  wait_for_earlier_kernels();
  let_later_kernels_start();                  // (the merge: it waits for this grid's end)
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride + first;
  constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
  alignas(16) T val[kEach];
#pragma unroll
  for (int i = 0; i < kEach; i += V) {
    const int p = place<T, VEC>(tid, i);
    if (p + V <= n_here) {
      if constexpr (VEC) *reinterpret_cast<uint4*>(&val[i]) = __ldcs(reinterpret_cast<const uint4*>(x + p));
      else val[i] = x[p];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) val[i + e] = p + e < n_here ? x[p + e] : T(-INFINITY);
    }
  }
  float mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < kEach; ++i) mine = fmaxf(mine, to_float(val[i]));         // (fmaxf passes over NaN)
  mine += 0.f;
  // group maxima: 8 KEYS lanes of a warp's 32 leave a key each
  float grp = mine;
  if (KEYS == 2) {
    grp = fmaxf(grp, __shfl_xor_sync(0xffffffffu, grp, 1));
    grp = fmaxf(grp, __shfl_xor_sync(0xffffffffu, grp, 2));
    if ((lane & 3) == 0) group_key[tid / 4] = ordered(grp);
  } else {
    group_key[tid] = ordered(grp);
  }
  float top = grp;
#pragma unroll
  for (int o = KEYS == 2 ? 4 : 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) warp_max[warp] = top;
  if (tid == 0) n_cand = 0;
  __syncthreads();
  top = warp_max[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) top = fmaxf(top, warp_max[w]);
  // sum of exponentials (0 where every logit is -inf; of +inf the merge makes an infinite log-sum)
  const float off = isinf(top) ? 0.f : top;
  float part[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const float y = to_float(val[i]);
    const float e = ex2f((y - off) * kLog2e);
    part[i & 1] += y == y ? e : 0.f;
  }
  uint64_t sum = isinf(top) ? 0ull : __float2ull_rn((part[0] + part[1]) * 0x1p40f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) warp_sum[warp] = sum;
  // the n-th largest group maximum
  const int n = min(a.n_out, n_here);
  if (warp == 0) {
    uint32_t key[KEYS], found = 0;
#pragma unroll
    for (int k = 0; k < KEYS; ++k) key[k] = group_key[lane + 32 * k];
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t probe = found | (1u << bit);
      int c = 0;
#pragma unroll
      for (int k = 0; k < KEYS; ++k) c += __popc(__ballot_sync(0xffffffffu, key[k] >= probe));
      if (c >= a.n_out) found = probe;
    }
    if (lane == 0) edge = found;
  }
  __syncthreads();
  if (tid == 0) {
    uint64_t all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) all += warp_sum[w];
    a.sums[row * a.slices + slice] = make_double2((double)top, (double)all * 0x1p-40);
  }
  auto key_of = [&](float y, int p) {
    return (uint64_t)ordered(no_nan(y)) << 32 | (0xffffffffu - (uint32_t)p);
  };
  const float least = unordered(edge);
  if (!(mine < least)) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const float y = to_float(val[i]);
      const int p = place<T, VEC>(tid, i);
      if (!(y < least) && p < n_here) {       // (a NaN too: its key is the lowest)
        const int c = atomicAdd(&n_cand, 1);
        if (c < kCandidates) cand[c] = key_of(y, p);
      }
    }
  }
  __syncthreads();
  int c_all = n_cand;
  if (c_all > kCandidates) {
    // many equal logits: the n-th key itself, from the top bit down, from the logits as they lie
    auto again = [&](int i) -> uint64_t {
      const int p = i * kThreads + tid;
      return p < n_here ? key_of(to_float(x[p]), p) : 0ull;
    };
    uint64_t found = 0;
    for (int bit = 63; bit >= 0; --bit) {
      if (bit == 31) {                        // places are below 2^13: the bits between are ones
        found |= 0xffffe000ull;
        bit = 12;
      }
      const uint64_t probe = found | (uint64_t(1) << bit);
      int c = 0;
#pragma unroll 4
      for (int i = 0; i < kEach; ++i) c += again(i) >= probe;
      c = __reduce_add_sync(0xffffffffu, c);
      __syncthreads();
      if (lane == 0) group_key[warp] = c;
      __syncthreads();
      c = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) c += group_key[w];
      if (c >= n) found = probe;
    }
    if (tid == 0) n_cand = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = 0; i < kEach; ++i) {
      const uint64_t k = again(i);
      if (k >= found) cand[atomicAdd(&n_cand, 1)] = k;        // exactly n: keys are distinct
    }
    __syncthreads();
    c_all = n_cand;
  }
  float2* out = a.best + (row * a.slices + slice) * a.n_out;
  for (int c = tid; c < c_all; c += kThreads) {
    const uint64_t k = cand[c];
    int rank = 0;
    for (int j = 0; j < c_all; ++j) rank += cand[j] > k;
    if (rank < n) out[rank] = make_float2(unordered((uint32_t)(k >> 32)), __int_as_float(first + (int)(0xffffffffu - (uint32_t)k)));
  }
  for (int c = n + tid; c < a.n_out; c += kThreads) out[c] = make_float2(-INFINITY, __int_as_float(-1));
}

// A beam's row for the merge: its log-sum, its score, and whether its order is that of the logits.
struct Beam {
  double lse, score;
  int kind;             // 0: by logit; 1: ended, the pad token and then every other one at -inf; 2: every token at -inf
};

// Entry i of list (beam k, slice): its token, or -1, and its score.
__device__ __forceinline__ int entry(const SelectArgs& a, const Beam& b, int64_t row, int slice, int i, double& score) {
  score = -INFINITY;
  if (b.kind == 0) {
    const float2 e = a.best[(row * a.slices + slice) * a.n_out + i];
    const int token = __float_as_int(e.y);
    if (token >= 0) {
      const double z = b.score + ((double)e.x - b.lse);
      score = z == z ? z : -INFINITY;
    }
    return token;
  }
  if (slice != 0) return -1;
  int token = i;
  if (b.kind == 1) {
    if (i == 0) score = b.score;
    token = i == 0 ? a.pad_token : i - 1 < a.pad_token ? i - 1 : i;
  }
  return token < a.vocab ? token : -1;
}

__global__ void __launch_bounds__(kMergeThreads) beam_merge(const __grid_constant__ SelectArgs a) {
  extern __shared__ uint64_t sm[];
  __shared__ Beam beam[kMaxBeams];
  __shared__ int n_cand;
  constexpr int kMost = kMaxBeamOut * kMaxBeamOut;
  const int lists = a.beams * a.slices, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t* key = sm;                                          // [kMost] candidates' scores
  int2* what = reinterpret_cast<int2*>(key + kMost);           // [kMost] (list, entry)
  uint64_t* head = reinterpret_cast<uint64_t*>(what + kMost);  // [lists]
  const int64_t set = blockIdx.x, row0 = set * a.beams;
  wait_for_earlier_kernels();
  // the rows' log-sums, a warp each: lanes take slices in turn, whatever the launch
  for (int k = warp; k < a.beams; k += kMergeThreads / 32) {
    const double2* s = a.sums + (row0 + k) * a.slices;
    double top = -INFINITY, sum = 0.0;
    for (int i = lane; i < a.slices; i += 32) top = fmax(top, s[i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int i = lane; i < a.slices; i += 32) {
      const double2 p = s[i];
      if (p.y > 0.0) sum += p.y * exp(p.x - top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      const double lse = isinf(top) ? top : top + log(sum);
      const double score = a.scores[row0 + k];
      const bool ended = a.ended != nullptr && a.ended[row0 + k] != 0;
      beam[k] = Beam{lse, score, !isfinite(score) ? 2 : ended ? 1 : isinf(lse) ? 2 : 0};
      if (a.lse != nullptr) a.lse[row0 + k] = (float)lse;
    }
  }
  if (tid == 0) n_cand = 0;
  __syncthreads();
  for (int l = tid; l < lists; l += kMergeThreads) {
    const int k = l / a.slices;
    double z;
    head[l] = entry(a, beam[k], row0 + k, l - k * a.slices, 0, z) >= 0 ? ordered(z) : 0ull;   // (a real key is not 0)
  }
  __syncthreads();
  // the n-th largest head, and of the lists equal to it those before the place `upto`
  const int n = a.n_out;
  uint64_t found = 0;
  int upto = lists;
  if (lists <= kMergeThreads) {
    const uint64_t h = tid < lists ? head[tid] : 0ull;
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t probe = found | (uint64_t(1) << bit);
      if (__syncthreads_count(h >= probe) >= n) found = probe;
    }
    if (__syncthreads_count(h >= found && tid < lists) > n) {
      int lo = 0;                                              // fewer than n before lo
      for (int bit = 1 << 12; bit > 0; bit >>= 1)
        if (__syncthreads_count(tid < lists && (h > found || (h == found && tid < lo + bit))) < n) lo += bit;
      upto = lo + 1;
    }
  } else {
    __shared__ int total;
    auto all = [&](uint64_t least, int before) {               // heads above `least`, or equal to it and before `before`
      if (tid == 0) total = 0;
      __syncthreads();
      int c = 0;
      for (int l = tid; l < lists; l += kMergeThreads) c += head[l] > least || (head[l] == least && l < before);
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0 && c != 0) atomicAdd(&total, c);
      __syncthreads();
      const int r = total;
      __syncthreads();
      return r;
    };
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t probe = found | (uint64_t(1) << bit);
      if (all(probe, lists) >= n) found = probe;
    }
    if (all(found, lists) > n) {
      int lo = 0;
      for (int bit = 1 << 12; bit > 0; bit >>= 1)
        if (all(found, lo + bit) < n) lo += bit;
      upto = lo + 1;
    }
  }
  // what those lists (at most n) hold at or above it
  for (int l = tid; l < lists; l += kMergeThreads) {
    if (head[l] == 0 || head[l] < found || (head[l] == found && l >= upto)) continue;
    const int k = l / a.slices;
    for (int i = 0; i < n; ++i) {
      double z;
      if (entry(a, beam[k], row0 + k, l - k * a.slices, i, z) < 0 || ordered(z) < found) break;
      const int c = atomicAdd(&n_cand, 1);
      if (c < kMost) {
        key[c] = ordered(z);
        what[c] = make_int2(l, i);
      }
    }
  }
  __syncthreads();
  const int c_all = min(n_cand, kMost);
  // equal scores: the earlier list (beam, then slice), then the earlier entry
  for (int c = tid; c < c_all; c += kMergeThreads) {
    const uint64_t z = key[c];
    const int2 w = what[c];
    int rank = 0;
    for (int j = 0; j < c_all; ++j) {
      const int2 u = what[j];
      rank += key[j] > z || (key[j] == z && (u.x < w.x || (u.x == w.x && u.y < w.y)));
    }
    if (rank >= n) continue;
    const int k = w.x / a.slices;
    double score;
    const int token = entry(a, beam[k], row0 + k, w.x - k * a.slices, w.y, score);
    a.scores_out[set * n + rank] = (float)score;
    a.parents[set * n + rank] = k;
    a.tokens[set * n + rank] = token;
  }
}

template <typename T, bool VEC>
kvsel_status launch_slices(const SelectArgs& a, cudaStream_t s) {
  const int64_t grid = (int64_t)a.batch * a.beams * a.slices;
  TraceScope ts("beam_slice", s);
  // 64 groups of four threads hold the n-th maximum near the n-th logit up to n = 32; beyond, every thread is a group
  if (a.n_out <= 32) return launch_after(beam_slice<T, VEC, 2>, dim3((unsigned)grid), kThreads, 0, s, a);
  return launch_after(beam_slice<T, VEC, 8>, dim3((unsigned)grid), kThreads, 0, s, a);
}

}  // namespace

size_t beam_select_ws(int64_t rows, int32_t slices, int32_t n_out, size_t* best_off, size_t* sums_off) {
  auto up = [](size_t x) { return (x + KVSEL_WS_ALIGN - 1) / KVSEL_WS_ALIGN * KVSEL_WS_ALIGN; };
  *sums_off = sizeof(DeviceError);
  *best_off = up(*sums_off + sizeof(double2) * (size_t)(rows * slices));
  return up(*best_off + sizeof(float2) * (size_t)(rows * slices) * n_out);
}

kvsel_status launch_beam_select(const SelectArgs& a, int32_t dtype, cudaStream_t s) {
  const size_t size = dtype == KVSEL_DTYPE_F32 ? 4 : 2;
  const bool vec = ((uintptr_t)a.logits & 15) == 0 && a.row_stride * size % 16 == 0;
  kvsel_status st;
  if (dtype == KVSEL_DTYPE_BF16) st = vec ? launch_slices<__nv_bfloat16, true>(a, s) : launch_slices<__nv_bfloat16, false>(a, s);
  else if (dtype == KVSEL_DTYPE_F16) st = vec ? launch_slices<__half, true>(a, s) : launch_slices<__half, false>(a, s);
  else st = vec ? launch_slices<float, true>(a, s) : launch_slices<float, false>(a, s);
  if (st != KVSEL_OK) return st;
  const size_t smem = (size_t)kMaxBeamOut * kMaxBeamOut * 16 + sizeof(uint64_t) * (size_t)a.beams * a.slices;
  if (set_smem((const void*)beam_merge, smem) != cudaSuccess) return KVSEL_ERR_CUDA;
  TraceScope ts("beam_merge", s);
  return launch_after(beam_merge, dim3((unsigned)a.batch), kMergeThreads, smem, s, a);
}

}  // namespace kvsel
