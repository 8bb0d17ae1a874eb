// The best continuations of a set of beams: score(k, v) = s_k + x_kv - log sum_u exp x_ku, the first n of beams x vocab.
//
// Bound: the logits, read once.  A CTA streams a segment of one row, 8192 tokens at a time in registers, and leaves the
// segment's largest logit, its sum of exponentials and its n best tokens in order; a second kernel, a CTA per set, forms the
// rows' log-sums, finds the n lists whose heads are best (an entry of any other list comes behind n heads) and ranks what they
// hold.
//
// A segment's n best: of 64 (or 256) groups of threads the n-th largest group maximum over the first 8192 tokens is found bit
// by bit by one warp, and is a lower bound of their n-th largest logit.  The tokens at or above it (n to 1.4 n of independent
// logits) are collected and ranked by counting, and the n-th of them is the bound for what follows, renewed when n more have
// passed it (half as many tokens of the next slice do then): a token is compared once and hardly ever more.  Where too many reach
// the bound at once (equal logits, rising ones, masks of one finite value over most of a row) they are taken 256 at a time: with
// 99.9 % of 128256 tokens at -1e30 64 sets of 16 take 524 us.  Tokens at -inf, of which constrained decoding has most of a
// vocabulary, are left out and fill a short list by their order.
//
// 64 sets of 16 beams over 128256 bf16 logits: 97 us, 2.7 TB/s (fp16 97); the same read alone runs at 6 TB/s.  What bounds it is
// latency between barriers: a CTA loads a slice, sums it, collects its candidates, and only then loads the next.  52 % of the issue
// slots and 39 % of DRAM are busy; of 13.7 cycles between a warp's instructions 3.9 wait for memory, 3.6 at barriers.  A slice
// costs a warp 400 instructions, a third of them the exponentials (without them 12 us less), as much the candidates (14).  A
// slice ahead by cp.async, one barrier a slice or ranks by four lanes left the time as it is.
//
// The merge ranks what it collects by counting.  Where few scores of a set are above -inf (the first step of many beams) that is
// up to n entries of as many lists: 4 sets of 32 beams of which one has a score, 64 outputs, take 1170 us.
//
// Ties are the rule with 16-bit logits, and scores of different beams may lie within a rounding of each other, so scores are
// formed and compared in 64 bits.  Exponentials are ex2.approx (2^-22 of each, of either sign) summed in fp32 by thread and
// then as 64-bit whole multiples of 2^-40: the sum is off by the mean of its terms' errors and the same for equal rows
// of a call, whatever CTA forms it.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "beam.cuh"
#include "sm100.cuh"

namespace kvsel {
namespace {

constexpr int kThreads = 256, kEach = kSliceKeys / kThreads;
constexpr int kCandidates = 1024;              // room for candidates
constexpr int kMergeThreads = 256;
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

// A thread's kEach tokens of a slice, as they lie: kEach * sizeof(T) / 4 words.  Vector v of 16 bytes holds the tokens from
// place V * (v * kThreads + tid) of the slice on, whatever the row's alignment: rows that lie equal are summed alike.
template <typename T>
struct Tokens {
  static constexpr int V = 16 / (int)sizeof(T), WORDS = kEach * (int)sizeof(T) / 4;
  alignas(16) uint32_t w[WORDS];
  static __device__ __forceinline__ int place(int tid, int i) { return (i / V * kThreads + tid) * V + i % V; }

  // Two aligned vectors and a shift by the row's offset of WORD words and `bits`.  (The words before the first token, and behind
  // the last, are of vectors that hold tokens.)
  template <int WORD>
  __device__ __forceinline__ void shifted(const uint4* from, uint32_t bits) {
#pragma unroll
    for (int v = 0; v < WORDS / 4; ++v) {
      const uint4 a = __ldg(from + v * kThreads), b = __ldg(from + v * kThreads + 1);
      const uint32_t y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) w[4 * v + k] = sizeof(T) == 2 ? __funnelshift_r(y[WORD + k], y[WORD + k + 1], bits) : y[WORD + k];
    }
  }
  // x: the slice's first token; tokens from n on are -inf.
  __device__ __forceinline__ void load(const T* x, int n, int tid) {
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(x) & 15);
    if (n == kSliceKeys) {
      if (off == 0) {
#pragma unroll
        for (int v = 0; v < WORDS / 4; ++v)
          *reinterpret_cast<uint4*>(w + 4 * v) = __ldcs(reinterpret_cast<const uint4*>(x) + v * kThreads + tid);
      } else {
        const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(x) - off) + tid;
        const uint32_t bits = (off & 2) * 8;
        if (off < 4) shifted<0>(from, bits);
        else if (off < 8) shifted<1>(from, bits);
        else if (off < 12) shifted<2>(from, bits);
        else shifted<3>(from, bits);
      }
    } else {
#pragma unroll
      for (int v = 0; v < WORDS / 4; ++v) {
        const int p = V * (v * kThreads + tid);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[4 * v + k] = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
        if (p < n) {                          // (single elements: the row's last slice alone)
          alignas(16) T y[V];
          *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(w + 4 * v);
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (p + e < n) y[e] = x[p + e];
          *reinterpret_cast<uint4*>(w + 4 * v) = *reinterpret_cast<const uint4*>(y);
        }
      }
    }
  }
  // tokens 2 i and 2 i + 1
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    else return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  // The largest, NaN passed over; -0 as 0.
  __device__ __forceinline__ float largest() const {
    float r;
    if constexpr (sizeof(T) == 4) {
      r = __uint_as_float(w[0]);
#pragma unroll
      for (int i = 1; i < WORDS; ++i) r = fmaxf(r, __uint_as_float(w[i]));
    } else {
      using P = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
      P m = *reinterpret_cast<const P*>(&w[0]);
#pragma unroll
      for (int i = 1; i < WORDS; ++i) m = __hmax2(m, *reinterpret_cast<const P*>(&w[i]));
      r = fmaxf(to_float(T(m.x)), to_float(T(m.y)));
    }
    return (r == r ? r : -INFINITY) + 0.f;
  }
  // Sum of exp(x - top), a NaN as none.  With c the rounded product top log2 e and r what that leaves, exp(x - top) is
  // 2^(x log2 e - c) 2^-r: one fused multiply-add per logit, rounded at its distance.  r is up to half a unit of c's last place, so
  // that holds while the largest is moderate; beyond 2^20 (masks of large finite values are) the difference is taken first.
  __device__ __forceinline__ float exp_sum(float top) const {
    const float c = top * kLog2e, r = fmaf(top, kLog2e, -c);
    const float2 c2 = make_float2(-c, -c), l2 = make_float2(kLog2e, kLog2e);
    float sum = NAN;
    if (fabsf(top) < 0x1p20f) {
      float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < kEach / 2; ++i) {
        const float2 z = __ffma2_rn(pair(i), l2, c2);
        part[i & 1] = __fadd2_rn(part[i & 1], make_float2(ex2f(z.x), ex2f(z.y)));
      }
      const float2 s = __fadd2_rn(part[0], part[1]);
      sum = (s.x + s.y) * ex2f(-r);
    }
    if (sum != sum) {                         // (or a NaN among them: once more without it)
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < kEach / 2; ++i) {
        const float2 y = pair(i);
        sum += (y.x == y.x ? ex2f((y.x - top) * kLog2e) : 0.f) + (y.y == y.y ? ex2f((y.y - top) * kLog2e) : 0.f);
      }
    }
    return sum;
  }
  // The tokens above `least` (one of the logits, or -inf), or equal to it and not -inf where `equal` ones count: bit i for
  // token i, or in pairs bit i for token 2 i and bit 16 + i for token 2 i + 1.
  static __device__ __forceinline__ int token_of(int bit) { return sizeof(T) == 4 ? bit : 2 * (bit & 15) + (bit >> 4); }
  __device__ __forceinline__ uint32_t above(float least, bool equal) const {
    uint32_t r = 0;
    const bool ge = equal && least != -INFINITY;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const float y = __uint_as_float(w[i]);
        r |= ((ge ? y >= least : y > least) ? 1u : 0u) << i;
      }
    } else {
      using P = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
      const P b = P(T(least), T(least));
      if (ge) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) r |= __hge2_mask(*reinterpret_cast<const P*>(&w[i]), b) & (0x00010001u << i);
      } else {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) r |= __hgt2_mask(*reinterpret_cast<const P*>(&w[i]), b) & (0x00010001u << i);
      }
    }
    return r;
  }
};

template <typename T, int KEYS>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3) beam_slice(const __grid_constant__ SelectArgs a) {
  __shared__ uint32_t group_key[32 * KEYS];
  __shared__ float warp_max[kThreads / 32];
  __shared__ uint64_t warp_sum[kThreads / 32];
  __shared__ uint32_t edge;
  __shared__ int n_cand;
  __shared__ uint64_t cand[kCandidates], kept[kMaxBeamOut];     // (ordered logit, all ones less the token)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seg = blockIdx.x % a.segments;
  const int64_t row = blockIdx.x / a.segments;
  const int s0 = seg * a.seg_slices * kSliceKeys, s1 = min(a.vocab, s0 + a.seg_slices * kSliceKeys);
  wait_for_earlier_kernels();
  let_later_kernels_start();                  // (the merge: it waits for this grid's end)
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
  const int n = a.n_out;
  if (tid == 0) n_cand = 0;
  auto key_of = [&](float y, int p) { return (uint64_t)ordered(no_nan(y)) << 32 | (0xffffffffu - (uint32_t)p); };
  // the n best of the candidates, in order; the bound for what follows is the n-th (none while there are fewer)
  float bound = -INFINITY;                    // of tokens behind those seen: only larger logits count
  uint64_t bound_key = 0;
  auto renew = [&]() {
    __syncthreads();
    const int c_all = n_cand, m = min(n, c_all);
    for (int c = tid; c < c_all; c += kThreads) {
      const uint64_t k = cand[c];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < c_all; ++j) rank += cand[j] > k;
      if (rank < n) kept[rank] = k;
    }
    __syncthreads();
    if (tid < m) cand[tid] = kept[tid];
    if (tid == 0) n_cand = m;
    if (m == n) {
      bound_key = kept[n - 1];
      bound = unordered((uint32_t)(bound_key >> 32));
    }
    __syncthreads();
  };
  float mine_m = -INFINITY, mine_s = 0.f;     // this thread's largest logit and sum of exponentials
#pragma unroll 1
  for (int first = s0; first < s1; first += kSliceKeys) {
    const int n_here = min(kSliceKeys, s1 - first);
    Tokens<T> val;
    val.load(x + first, n_here, tid);
    const float mine = val.largest();
    if (first == s0) {
      // group maxima: 8 KEYS lanes of a warp's 32 leave a key each; the n-th largest is the first bound
      float grp = mine;
      if (KEYS == 2) {
        grp = fmaxf(grp, __shfl_xor_sync(0xffffffffu, grp, 1));
        grp = fmaxf(grp, __shfl_xor_sync(0xffffffffu, grp, 2));
        if ((lane & 3) == 0) group_key[tid / 4] = ordered(grp);
      } else {
        group_key[tid] = ordered(grp);
      }
      __syncthreads();
      if (warp == 0) {
        uint32_t key[KEYS], found = 0;
#pragma unroll
        for (int k = 0; k < KEYS; ++k) key[k] = group_key[lane + 32 * k];
        // (16-bit logits differ in the top 16 bits, bf16, or the top 19; the others are all ones in a negative one's key)
        constexpr int last = sizeof(T) == 4 ? 0 : std::is_same<T, __half>::value ? 13 : 16;
        for (int bit = 31; bit >= last; --bit) {
          const uint32_t probe = found | (1u << bit);
          int c = 0;
#pragma unroll
          for (int k = 0; k < KEYS; ++k) c += __popc(__ballot_sync(0xffffffffu, key[k] >= probe));
          if (c >= n) found = probe;
        }
        if ((found >> 31) == 0) found |= (1u << last) - 1u;
        if (lane == 0) edge = found;
      }
    }
    // sums of exponentials, to this thread's largest
    const float top = fmaxf(mine_m, mine);
    if (isfinite(top)) {
      if (top > mine_m) mine_s *= ex2f((mine_m - top) * kLog2e);
      mine_s += val.exp_sum(top);
    }
    mine_m = top;
    if (first == s0) __syncthreads();
    // candidates: at or above the first bound in the first tokens, above the n-th so far in later ones (an equal one comes
    // behind n); never -inf
    const int before = n_cand;
    const float least = first == s0 ? unordered(edge) : bound;
    __syncthreads();                          // (`before` is read)
    if (mine >= least && mine != -INFINITY) {
      uint32_t hits = val.above(least, first == s0);
      while (hits != 0) {
        const int p = first + Tokens<T>::place(tid, Tokens<T>::token_of(__ffs((int)hits) - 1));
        hits &= hits - 1;
        const int c = atomicAdd(&n_cand, 1);
        if (c < kCandidates) cand[c] = key_of(to_float(x[p]), p);           // (in L1 or L2 still)
      }
    }
    __syncthreads();
    const int c_all = n_cand;
    if (c_all > kCandidates) {
      // too many at once: 256 at a time, as they lie, against the n-th key so far
      __syncthreads();
      if (tid == 0) n_cand = before;
      renew();
#pragma unroll 1
      for (int p = tid; p < kSliceKeys; p += kThreads) {
        const float y = p < n_here ? to_float(x[first + p]) : -INFINITY;
        const uint64_t k = key_of(y, first + p);
        if (p < n_here && y > -INFINITY && k > bound_key) cand[atomicAdd(&n_cand, 1)] = k;
        __syncthreads();
        const int c = n_cand;
        __syncthreads();
        if (c > kCandidates - kThreads) renew();
      }
      renew();
    } else if (c_all >= 2 * n || first == s0 || first + kSliceKeys >= s1) {
      renew();
    }
  }
  // the row's part of the log-sum
  float top = mine_m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) warp_max[warp] = top;
  __syncthreads();
  top = warp_max[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) top = fmaxf(top, warp_max[w]);
  // (0 where every logit is -inf; of +inf the merge makes an infinite log-sum)
  uint64_t sum = isinf(top) || mine_m == -INFINITY ? 0ull : __float2ull_rn(mine_s * ex2f((mine_m - top) * kLog2e) * 0x1p40f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) warp_sum[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    uint64_t all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) all += warp_sum[w];
    a.tops[row * a.segments + seg] = top;
    a.sums[row * a.segments + seg] = all;
  }
  const int c_all = n_cand;
  float2* out = a.best + (row * a.segments + seg) * n;
  if (tid < c_all) {
    const uint64_t k = cand[tid];
    out[tid] = make_float2(unordered((uint32_t)(k >> 32)), __int_as_float((int)(0xffffffffu - (uint32_t)k)));
  }
  if (c_all < n && warp == 0) {
    // the first tokens at -inf (and NaN) fill the list
    int at = c_all;
    for (int p0 = s0; p0 < s1 && at < n; p0 += 32) {
      const int p = p0 + lane;
      const bool low = p < s1 && !(to_float(x[p]) > -INFINITY);
      const uint32_t b = __ballot_sync(0xffffffffu, low);
      const int to = at + __popc(b & ((1u << lane) - 1u));
      if (low && to < n) out[to] = make_float2(-INFINITY, __int_as_float(p));
      at += __popc(b);
    }
    for (int c = at + lane; c < n; c += 32) out[c] = make_float2(-INFINITY, __int_as_float(-1));
  }
}

// e^x in 64 bits for x in [-700, 1]: the Taylor series to the 12th power within half a binary order, off by at most 2^-52 of the
// value there.  (Few fused multiply-adds in line: the merge runs once a step, and its code is fetched as it goes.)
__device__ __forceinline__ double exp64(double x) {
  const double k = rint(x * 1.4426950408889634074), g = fma(-k, 0.69314718055994530942, x);
  double y = 1.0 / 479001600.0;
  const double c[12] = {1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0, 1.0 / 5040.0, 1.0 / 720.0,
                        1.0 / 120.0,      1.0 / 24.0,      1.0 / 6.0,      0.5,           1.0,          1.0};
#pragma unroll
  for (int i = 0; i < 12; ++i) y = fma(y, g, c[i]);
  return y * __longlong_as_double((long long)(1023 + (int)k) << 52);
}
// log x for x in [1, 2^40]: the 32-bit one and a step of Newton's, x e^-y - 1 further.
__device__ __forceinline__ double log64(double x) {
  const double y = (double)logf((float)x);
  return y + fma(x, exp64(-y), -1.0);
}

// Whether candidate a comes before b: as numbers of 128 bits, a > b.
__device__ __forceinline__ int precedes(ulonglong2 a, ulonglong2 b) {
  uint32_t r;
  asm("{\n\t.reg .b64 t;\n\tsub.cc.u64 t, %1, %2;\n\tsubc.cc.u64 t, %3, %4;\n\tsubc.u32 %0, 0, 0;\n\t}" : "=r"(r) : "l"(b.x), "l"(a.x), "l"(b.y), "l"(a.y));
  return -(int)r;
}

// A beam's row for the merge: its log-sum, its score, and whether its order is that of the logits.
struct Beam {
  double lse, score;
  int kind;             // 0: by logit; 1: ended, the pad token and then every other one at -inf; 2: every token at -inf
};

// Entry i of list (beam k, segment): its token, or -1, its score, and its place among equal scores (the larger comes first): the
// smaller beam, the larger logit (where the score is not -inf), the smaller token.
constexpr int kTokenBits = 26;
static_assert(kMaxLists * kSliceKeys <= int64_t(1) << kTokenBits && kMaxBeams <= 1 << (32 - kTokenBits), "beam, logit and token fill 64 bits");
__device__ __forceinline__ int entry(const SelectArgs& a, const Beam& b, int64_t row, int k, int segment, int i, double& score, uint64_t& place) {
  score = -INFINITY;
  uint32_t logit = 0;
  int token = -1;
  if (b.kind == 0) {
    const float2 e = a.best[(row * a.segments + segment) * a.n_out + i];
    token = __float_as_int(e.y);
    if (token >= 0) {
      const double z = b.score + ((double)e.x - b.lse);
      score = z == z ? z : -INFINITY;
      if (score != -INFINITY) logit = ordered(e.x);
    }
  } else if (segment == 0) {
    token = i;
    if (b.kind == 1) {
      if (i == 0) score = b.score;
      token = i == 0 ? a.pad_token : i - 1 < a.pad_token ? i - 1 : i;
    }
    if (token >= a.vocab) token = -1;
  }
  place = (uint64_t)(kMaxBeams - 1 - k) << (32 + kTokenBits) | (uint64_t)logit << kTokenBits | (uint32_t)((1 << kTokenBits) - 1 - token);
  return token;
}

__global__ void __launch_bounds__(kMergeThreads) beam_merge(const __grid_constant__ SelectArgs a) {
  extern __shared__ uint64_t sm[];
  __shared__ Beam beam[kMaxBeams];
  __shared__ float row_top[kMaxBeams];
  __shared__ int n_cand, n_lists, total;
  __shared__ int16_t chosen[kMaxBeamOut];
  constexpr int kMost = kMaxBeamOut * kMaxBeamOut;
  const int lists = a.beams * a.segments, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  ulonglong2* cand = reinterpret_cast<ulonglong2*>(sm);        // [kMost] candidates: place among equal scores, score
  uint64_t* head = sm + 2 * kMost;                             // [lists]
  const int64_t set = blockIdx.x, row0 = set * a.beams;
  wait_for_earlier_kernels();
  // The rows' log-sums.  A 64-bit operation takes a warp 16 cycles of the SM whatever its lanes do (two lanes a clock), so lanes
  // are filled: a thread for a segment's term, then one for a row's sum, in the order of its segments.
  double* term = reinterpret_cast<double*>(head);              // [lists], read before the heads are written
  for (int k = warp; k < a.beams; k += kMergeThreads / 32) {
    float top = -INFINITY;
    for (int i = lane; i < a.segments; i += 32) top = fmaxf(top, a.tops[(row0 + k) * a.segments + i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) row_top[k] = top;
  }
  __syncthreads();
  for (int l = tid; l < lists; l += kMergeThreads) {
    const float top = row_top[l / a.segments], mine = a.tops[row0 * a.segments + l];
    const uint64_t sum = a.sums[row0 * a.segments + l];
    const float less = mine - top;                             // (to tell 0 and what is nothing beside the largest; -inf - -inf is NaN)
    term[l] = sum == 0 ? 0.0 : less == 0.f ? (double)sum : less > -700.f ? (double)sum * exp64((double)mine - (double)top) : 0.0;
  }
  __syncthreads();
  if (tid < a.beams) {
    const int k = tid;
    double sum = 0.0;
    for (int i = 0; i < a.segments; ++i) sum += term[k * a.segments + i];
    const float top = row_top[k], score = a.scores[row0 + k];
    const double lse = isinf(top) ? (double)top : (double)top + log64(sum * 0x1p-40);
    const bool ended = a.ended != nullptr && a.ended[row0 + k] != 0;
    beam[k] = Beam{lse, (double)score, !isfinite(score) ? 2 : ended ? 1 : isinf(top) ? 2 : 0};
    if (a.lse != nullptr) a.lse[row0 + k] = (float)lse;
  }
  if (tid == 0) n_cand = n_lists = 0;
  __syncthreads();
  // The n-th largest of the lists' first entries (of as many as make 2 n, where there are few lists), by its upper half, which is
  // enough unless more lists than there is room for reach it; then by all of it, and of the lists equal to it those whose first
  // entries' places are `from` or larger.
  const int n = a.n_out, depth = lists > n ? 1 : min(n, (2 * n + lists - 1) / lists), values = lists * depth;
  for (int v = tid; v < values; v += kMergeThreads) {
    const int l = v / depth, k = l / a.segments;
    double z;
    uint64_t w;
    head[v] = entry(a, beam[k], row0 + k, k, l - k * a.segments, v - l * depth, z, w) >= 0 ? ordered(z) : 0ull;   // (a real key is not 0)
  }
  __syncthreads();
  auto count = [&](auto test) {
    int c = 0;
    if (values <= kMergeThreads) return (int)__syncthreads_count(tid < values && test(head[tid], tid));
    if (tid == 0) total = 0;
    __syncthreads();
    for (int v = tid; v < values; v += kMergeThreads) c += test(head[v], v) ? 1 : 0;
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0 && c != 0) atomicAdd(&total, c);
    __syncthreads();
    c = total;
    __syncthreads();
    return c;
  };
  auto place_of = [&](int l) {                                 // of a list's first entry
    const int k = l / a.segments;
    double z;
    uint64_t w;
    (void)entry(a, beam[k], row0 + k, k, l - k * a.segments, 0, z, w);
    return w;
  };
  uint64_t found = 0, from = 0;
  if (values <= kMergeThreads) {
    // few values: the one that n - 1 others precede
    if (tid == 0) total = 0;
    __syncthreads();
    if (tid < values) {
      const uint64_t h = head[tid];
      int before = 0;
#pragma unroll 8
      for (int v = 0; v < values; ++v) before += (head[v] > h) | ((head[v] == h) & (v < tid));
      if (before == n - 1) total = tid;
    }
    __syncthreads();
    found = values >= n ? head[total] >> 32 << 32 : 0ull;
  } else {
    for (int bit = 63; bit >= 32; --bit) {
      const uint64_t probe = found | (uint64_t(1) << bit);
      if (count([&](uint64_t h, int) { return h >= probe; }) >= n) found = probe;
    }
  }
  if (lists > kMaxBeamOut) {                                   // (depth 1: a value is a list)
    if (count([&](uint64_t h, int) { return h != 0 && h >= found; }) > kMaxBeamOut) {
      for (int bit = 31; bit >= 0; --bit) {
        const uint64_t probe = found | (uint64_t(1) << bit);
        if (count([&](uint64_t h, int) { return h >= probe; }) >= n) found = probe;
      }
      if (count([&](uint64_t h, int) { return h != 0 && h >= found; }) > n) {
        for (int bit = 63; bit >= 0; --bit) {
          const uint64_t probe = from | (uint64_t(1) << bit);
          if (count([&](uint64_t h, int l) { return h > found || (h == found && h != 0 && place_of(l) >= probe); }) >= n) from = probe;
        }
      }
    }
  }
  for (int l = tid; l < lists; l += kMergeThreads) {
    const uint64_t h = head[l * depth];
    if (h > found || (h == found && h != 0 && (from == 0 || place_of(l) >= from))) chosen[atomicAdd(&n_lists, 1)] = (int16_t)l;
  }
  __syncthreads();
  // what those lists hold at or above it, a warp each
  for (int i = warp; i < n_lists; i += kMergeThreads / 32) {
    const int l = chosen[i], k = l / a.segments;
    for (int e = lane; e < n; e += 32) {
      double z;
      uint64_t w;
      if (entry(a, beam[k], row0 + k, k, l - k * a.segments, e, z, w) < 0 || ordered(z) < found) break;
      const int c = atomicAdd(&n_cand, 1);
      cand[c] = make_ulonglong2(w, ordered(z));
    }
  }
  __syncthreads();
  const int c_all = n_cand;
  for (int c = tid; c < c_all; c += kMergeThreads) {
    const ulonglong2 mine = cand[c];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < c_all; ++j) rank += precedes(cand[j], mine);
    if (rank >= n) continue;
    const uint64_t z = mine.y, w = mine.x;
    a.scores_out[set * n + rank] = (float)__longlong_as_double((long long)(z >> 63 ? z & ~(uint64_t(1) << 63) : ~z));
    a.parents[set * n + rank] = kMaxBeams - 1 - (int)(w >> (32 + kTokenBits));
    a.tokens[set * n + rank] = (1 << kTokenBits) - 1 - (int)(w & ((1u << kTokenBits) - 1));
  }
}

template <typename T>
kvsel_status launch_slices(const SelectArgs& a, cudaStream_t s) {
  const int64_t grid = (int64_t)a.batch * a.beams * a.segments;
  TraceScope ts("beam_slice", s);
  // 64 groups of four threads hold the n-th maximum near the n-th logit up to n = 32; beyond, every thread is a group
  if (a.n_out <= 32) return launch_after(beam_slice<T, 2>, dim3((unsigned)grid), kThreads, 0, s, a);
  return launch_after(beam_slice<T, 8>, dim3((unsigned)grid), kThreads, 0, s, a);
}

}  // namespace

size_t beam_select_ws(int64_t rows, int32_t segments, int32_t n_out, size_t* best_off, size_t* sums_off, size_t* tops_off) {
  auto up = [](size_t x) { return (x + KVSEL_WS_ALIGN - 1) / KVSEL_WS_ALIGN * KVSEL_WS_ALIGN; };
  *sums_off = sizeof(DeviceError);
  *tops_off = up(*sums_off + sizeof(uint64_t) * (size_t)(rows * segments));
  *best_off = up(*tops_off + sizeof(float) * (size_t)(rows * segments));
  return up(*best_off + sizeof(float2) * (size_t)(rows * segments) * n_out);
}

kvsel_status launch_beam_select(const SelectArgs& a, int32_t dtype, cudaStream_t s) {
  const kvsel_status st = dtype == KVSEL_DTYPE_BF16  ? launch_slices<__nv_bfloat16>(a, s)
                          : dtype == KVSEL_DTYPE_F16 ? launch_slices<__half>(a, s)
                                                     : launch_slices<float>(a, s);
  if (st != KVSEL_OK) return st;
  const size_t smem = (size_t)kMaxBeamOut * kMaxBeamOut * 16 + sizeof(uint64_t) * (size_t)std::max<int64_t>((int64_t)a.beams * a.segments, 4 * kMaxBeamOut);
  if (set_smem((const void*)beam_merge, smem) != cudaSuccess) return KVSEL_ERR_CUDA;
  TraceScope ts("beam_merge", s);
  return launch_after(beam_merge, dim3((unsigned)a.batch), kMergeThreads, smem, s, a);
}

}  // namespace kvsel
