// Attention of many query rows over one request's cached rows, on the 5th-generation tensor cores.
//
// Both calls that have many rows for the same keys run this kernel: the new tokens of a request (kvsel_chunk_attend) and the
// requests of a group over the prefix they share (kvsel_prefix_attend).  The query rows of a KV head are its G query heads of
// every token (request), laid end to end; an item is up to 256 of them and the keys that they see, in steps of 128.  All
// items' steps of all KV heads, laid end to end, are dealt evenly to one CTA per SM; a piece is what a CTA has of an item.
// Pieces that are not a whole item leave partial sums, which rows_join merges.
//
// Roles of the 16 warps: 0-3 and 4-7 softmax of tile A and B, a thread per row of the tile; 8-11 load K and V; 12 issues
// the products S, 13 P V.  S = Q K^T goes to TMEM; the softmax reads it, keeps an exponent offset that moves only when a row's largest
// score passes it by 2^lag (so O is rescaled rarely) and writes the weights over S as 16-bit values, which O += P V takes from
// TMEM with V as it lies.  (16-bit pools: the weights' sum bounds the largest of them, which is looked for only where that does
// not do.)
//
// An item of more than 128 rows has them in both tiles, which share every step; P V of one and S of the other are issued in
// alternation, as the prefill kernel does.  A smaller item has its rows in both: the tiles take steps in turn, so
// that two chains S -> softmax -> P V -> S run at once (one alone takes 4000 cycles a step and more; HBM brings one in 2800,
// which is what the two in turn take).  Items of up to 32 rows fill the tile's 128 rows with four copies, which take 32 keys
// of a step each: the softmax of a step is a thread's loop over its keys, 2000 cycles for 128.  What tiles and copies hold is
// merged when the piece ends.
//
// Bound: with full items the chain of a tile's step, 2000 cycles of softmax and as many of S and P V with the waits between them;
// TMEM holds S and O of two tiles, at d = 128 with no room for a third S that could be formed meanwhile (at 64 a tile leaves 64 of
// its 256 columns unused).  4096 tokens behind 12288, 32 / 8 heads
// of 128, bf16: 791 us, 1.2 PFLOP/s, a step of both tiles in 4000 cycles where its products take 2048.  (Halves of a step told
// of apart, to start P V early: 912; steps of 64 keys: 1127.)  With few rows HBM, and what a piece costs beside its
// steps (queries, a first step alone, the merge of tiles and copies: 11 us): 16 requests of 5 tokens behind up to 8191: 101 us,
// 2.8 TB/s; of CTAs with 29 steps each, those with one piece take 50 us, with two 63, the slowest, with four, 83.
//
// SCORED: kernels for capped or biased scores, which are formed in the registers that hold them for the softmax; a step with
// a mask has them formed in TMEM first.  (8 chunks behind up to 7000 rows, 8-bit, capped, a window: 415 us when all were
// formed in TMEM, 396 now.)
//
// SPLIT (the shared prefix over 16-bit pools): weights are a high and a low 16-bit part, as in the decode kernel whose results it
// must match; the steps wait for HBM there, so the third product is free up to 128 rows.  Without it (chunks, bound by the tensor
// cores, and 8-bit pools) a weight is rounded once, by at most 2^-8 of it over bf16 and 2^-11 over fp16 products (or 2^-33 of the
// row's largest: those below 2^-22 of it are subnormal): what the outputs' own rounding is, and far below a row's in 8 bits.
// (64 requests behind 32768 e4m3 rows take 166 us; the low parts would add 26.)
// Factors on the weights as in paged_attend.cuh: 2^-8 over bf16 and 2^13 over fp16 products; without SPLIT it is taken by the
// exponent, whose rounding at 13 (2^-21 of a weight) is far below the weight's own.
//
// K and V come into the 128-byte swizzled layout of the products, a warp per 32 rows of a step: by TMA boxes of 8 to 32 rows
// where pages are made of such, else by cp.async, whole rows at a time: any page size, order and stride.  An e4m3 pool's rows
// (boxes of bytes in a ring of their own, or rows by plain loads) pass through registers, where they become fp16.
//
// Rows that some token of the item does not see may hold anything: their scores are replaced, and where a V row in such a
// step is not finite its bad values are zeros in shared memory (0 times infinity is no number) and are added to the rows that
// do see it by hand.
#pragma once

#include <type_traits>

#include "paged_attend.cuh"
#include "rows.cuh"

namespace kvsel {

constexpr int kRowsThreads = 512;
constexpr int kTileRows = 128, kTileKeys = 128;
constexpr uint32_t kHalf = 16384;                // bytes of 128 rows of 64 16-bit values
template <int D>
__host__ __device__ constexpr uint32_t rows_tile_bytes() { return D / 64 * kHalf; }
// K and V tiles of the steps, in turn, as the products read them: as many as shared memory holds.  An e4m3 pool's bytes land
// in a ring of their own, four tiles.
template <int D, int KIND>
__host__ __device__ constexpr int rows_slots() { return D == 64 ? 8 : KIND == kE4m3 ? 3 : 5; }
constexpr int kRawTiles = 4;
// shared memory: Q_A | Q_B (and the merge's buffers) | slots | bytes of an e4m3 pool | barriers and the steps' words
template <int D, int KIND>
__host__ __device__ constexpr uint32_t rows_raw_off() { return (2 + rows_slots<D, KIND>()) * rows_tile_bytes<D>(); }
template <int D, int KIND>
__host__ __device__ constexpr uint32_t rows_bar_off() { return rows_raw_off<D, KIND>() + (KIND == kE4m3 ? kRawTiles * kTileKeys * D : 0); }
template <int D, int KIND>
constexpr size_t rows_smem() { return rows_bar_off<D, KIND>() + 1024 + 1024; }
// barriers: full and empty of the slots, then of the tiles s_full, p_full, pv_done and q_full, the merge's, of the loader
// warps one each for rows that are looked at before they count, and one each per raw tile
constexpr int kBarEmpty = 8, kBarTiles = 16, kBarMerge = 24, kBarDrain = 25, kBarLand = 27, kBarRaw = 31, kRowsBars = kBarRaw + 4 * kRawTiles;
constexpr uint32_t kWordsOff = 512;              // behind the barriers: misc, then the words of 8 steps twice
static_assert(kRowsBars * 8 <= kWordsOff, "barriers lie before the words");

enum : uint32_t { kRowsLoader = 21, kRowsMma = 22, kRowsSoftmax = 23, kRowsDrain = 24 };

// Instruction descriptor of kind::f16 with 16-bit operands of the products' type.
template <int KIND>
__host__ __device__ constexpr uint32_t rows_idesc(uint32_t M, uint32_t N) {
  return (1u << 4) | (KIND == kBf16 ? (1u << 7) | (1u << 10) : 0u) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ bool rows_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred P1;\n\tmbarrier.test_wait.parity.shared::cta.b64 P1, [%1], %2;\n\tselp.b32 %0, 1, 0, P1;\n\t}"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// A bounded wait that also ends when another role has given up.
__device__ __forceinline__ bool rows_wait(uint32_t bar, uint32_t parity, const volatile uint32_t* flag) {
  for (uint32_t i = 0; i < sm100::kSpinLimit; ++i) {
    if (sm100::mbar_try_wait(bar, parity)) return true;
    if ((i & 255) == 255 && *flag != 0) return false;
  }
  return false;
}
__device__ __forceinline__ void rows_fail(const RowsArgs& a, volatile uint32_t* flag, uint32_t where) {
  set_device_error(a.err, KVSEL_ERR_TIMEOUT, where);
  *flag = 1;
}

// A box of `rows` rows of one head of one page (the map says how many, and 128 bytes or all of a row) from element x of the rows.
__device__ __forceinline__ void rows_box(uint32_t dst, const CUtensorMap* map, int x, int row, int head, int page, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(head), "r"(page), "r"(bar)
               : "memory");
}

// The pieces of a CTA, in order: every role walks them by itself.
struct RowsPiece {
  const RowsItem* item;
  int32_t g, s0, s1;             // KV head, the item's steps [s0, s1) here
  __device__ bool starts() const { return s0 == 0; }
  __device__ bool ends() const { return s1 == item->steps; }
};
struct RowsWalk {
  int64_t left;
  int32_t g, at, s, n_items;
  const RowsItem* item;          // the first piece's is kept with the CTA's start
  __device__ void begin(const RowsStart& st) {
    left = st.steps;
    n_items = st.n_items;
    g = st.g;
    at = st.at;
    s = st.step;
    item = &st.item;
  }
  __device__ bool next(const RowsArgs& a, RowsPiece& p) {
    if (left <= 0) return false;
    while (item == nullptr) {
      if (at == n_items) at = 0, ++g;
      if (a.items[at].steps > 0) item = a.items + at;       // (the steps left say that there is one)
      else ++at;
    }
    p.item = item;
    p.g = g;
    p.s0 = s;
    p.s1 = (int)min((int64_t)item->steps, s + left);
    left -= p.s1 - s;
    s = 0;
    ++at;
    item = nullptr;
    return true;
  }
};

// Whether a step's keys that are loaded include one that some row of the item does not see.  (t0 + kTileKeys may be 2^31.)
__device__ __forceinline__ bool rows_partial(int lo, int hi, int full_lo, int full_hi, int t0) {
  return max(t0, lo) < full_lo || min(kTileKeys, hi - t0) > full_hi - t0;
}
// Adds to this thread's O (TMEM at `o`) the values of V rows that are not finite and that the thread's row sees.
template <int D, int KIND>
__device__ __forceinline__ void add_bad_rows(const RowsArgs& a, const uint8_t* vbase, int table, int t0, int pos, uint4 bad, uint32_t o,
                                          bool fresh) {
  const uint32_t word[4] = {bad.x, bad.y, bad.z, bad.w};
  const int low = a.window > 0 ? pos + 1 - a.window : 0;
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 32) {
    float v[32];
    if (fresh) {
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = 0.f;
    } else {
      sm100::tmem_ld32(o + c0, v);
    }
    for (int w = 0; w < 4; ++w)
      for (uint32_t bits = word[w]; bits != 0; bits &= bits - 1) {
        const int t = t0 + 32 * w + __ffs((int)bits) - 1;
        if (t < low || t > pos) continue;
        const int blk = (int)((__umulhi(a.p_mul, (uint32_t)t) + (uint32_t)t) >> a.p_shift);
        const int64_t id = a.tables[(int64_t)table * a.max_blocks + blk];      // (in range: its row was loaded)
        const uint8_t* row = vbase + (id * a.page_stride + (int64_t)(t - blk * a.P) * a.row_stride) * elem_bytes<KIND>();
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float y;
          if constexpr (KIND == kBf16) y = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[c0 + e]);
          else if constexpr (KIND == kF16) y = __half2float(reinterpret_cast<const __half*>(row)[c0 + e]);
          else y = (row[c0 + e] & 0x7f) == 0x7f ? NAN : 0.f;
          if (!isfinite(y)) v[e] += y;
        }
      }
    uint32_t r[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(v[e]);
    __syncwarp();
    sm100::tmem_st32(o + c0, r);
  }
  sm100::tmem_wait_st();
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int N>
__device__ __forceinline__ float rows_max(const float* v) {
  float m[N / 8];
#pragma unroll
  for (int k = 0; k < N / 8; ++k) {
    const float* c = v + 8 * k;
    m[k] = fmaxf(max3(max3(c[0], c[1], c[2]), c[3], c[4]), max3(c[5], c[6], c[7]));
  }
#pragma unroll
  for (int k = N / 16; k > 0; k /= 2)
#pragma unroll
    for (int i = 0; i < k; ++i) m[i] = fmaxf(m[i], m[i + k]);
  return m[0];
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int N>
__device__ __forceinline__ float rows_min(const float* v) {
  float m[N / 16];
#pragma unroll
  for (int k = 0; k < N / 16; ++k) {
    const float* c = v + 16 * k;
    m[k] = min3(min3(min3(c[0], c[1], c[2]), c[3], c[4]), min3(min3(c[5], c[6], c[7]), c[8], c[9]), min3(min3(c[10], c[11], c[12]), c[13], c[14]));
    m[k] = fminf(m[k], c[15]);
  }
  static_assert(N == 64, "four parts");
  return min3(fminf(m[0], m[1]), m[2], m[3]);
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
               "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t at, float* v) {
  uint32_t r[16];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
                 "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(at));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
template <int KIND>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
  float a, b;
  return pack_hi<KIND>(x, y, a, b);
}

// Weights of N scores, 2^(mul z - m) times the factor, as 16-bit pairs: hi (and lo with SPLIT); returns their sum.
// Without SPLIT the factor is in `nm` and the sum, and `hi` may be the scores' own registers (word c is written after v[2 c]
// and v[2 c + 1] are read).
template <int KIND, bool SPLIT, int N>
__device__ __forceinline__ float rows_weights(const float* v, float mul, float nm, uint32_t* hi, uint32_t* lo) {
  const float2 m2 = make_float2(mul, mul), n2 = make_float2(nm, nm);
  float2 sp[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) sp[k] = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < N / 2; ++c) {
    const float2 t = __ffma2_rn(make_float2(v[2 * c], v[2 * c + 1]), m2, n2);
    const float2 p = make_float2(ex2(t.x), ex2(t.y));
    sp[c & 3] = __fadd2_rn(sp[c & 3], p);
    if constexpr (SPLIT) {
      constexpr float unit = weight_unit<KIND>();
      const float2 w = __fmul2_rn(p, make_float2(unit, unit));
      float r0, r1;
      hi[c] = pack_hi<KIND>(w.x, w.y, r0, r1);
      lo[c] = pack16<KIND>(r0, r1);
    } else {
      hi[c] = pack16<KIND>(p.x, p.y);
    }
  }
  const float2 s = __fadd2_rn(__fadd2_rn(sp[0], sp[1]), __fadd2_rn(sp[2], sp[3]));
  return s.x + s.y;
}

// A row's scores as they are compared, from the products: with a cap c z' = c tanh(z / c), a bias slope (t - p), in base 2.
struct RowsScore {
  float sc, icap, cap2, slope;        // sc: scale with log2 e; icap: scale / cap
  bool capped, biased;                // biased: with a bias, or a factor that is not positive
};
// With the bias, and the factor `by` on what stands there.
template <int N>
__device__ __forceinline__ void rows_bias(float* z, float by, float slope, float d0) {
  const float2 s2 = make_float2(by, by), sl = make_float2(slope, slope), dd = make_float2(d0, d0 + 1.f);
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const float2 y = __ffma2_rn(sl, __fadd2_rn(dd, make_float2((float)c, (float)c)), __fmul2_rn(make_float2(z[c], z[c + 1]), s2));
    z[c] = y.x;
    z[c + 1] = y.y;
  }
}
// N products as their scores: capped, biased (d0: distance of the first key to the row's own), and those not seen (by 32, where not
// all are) as -inf.
template <int N>
__device__ __forceinline__ void rows_scores(float* z, const RowsScore& k, float d0, bool whole, const uint32_t* see) {
  if (k.capped) {
    const float2 ic = make_float2(k.icap, k.icap), cp = make_float2(k.cap2, k.cap2);
    float big = 0.f;
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const float2 x = __fmul2_rn(make_float2(z[c], z[c + 1]), ic);
      z[c] = x.x;
      z[c + 1] = x.y;
      big = max3(big, fabsf(x.x), fabsf(x.y));
    }
    // (scores far below the cap are the rule: the series alone, as tanh_fast has it below 1/4)
    if (__all_sync(0xffffffffu, big < 0.25f)) {
      const float2 c3 = make_float2(-17.f / 315.f, -17.f / 315.f), c2 = make_float2(2.f / 15.f, 2.f / 15.f),
                   c1 = make_float2(-1.f / 3.f, -1.f / 3.f), one = make_float2(1.f, 1.f);
#pragma unroll
      for (int c = 0; c < N; c += 2) {
        const float2 x = make_float2(z[c], z[c + 1]), x2 = __fmul2_rn(x, x);
        const float2 y = __fmul2_rn(__fmul2_rn(x, cp), __ffma2_rn(x2, __ffma2_rn(x2, __ffma2_rn(x2, c3, c2), c1), one));
        z[c] = y.x;
        z[c + 1] = y.y;
      }
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c) z[c] = k.cap2 * tanh_fast(z[c]);
    }
  }
  if (k.biased) {                                 // (and where the factor is not positive: the bias is 0 then)
    rows_bias<N>(z, k.capped ? 1.f : k.sc, k.slope, d0);
  }
  if (!whole) {
#pragma unroll
    for (int c = 0; c < N; ++c) z[c] = (see[c / 32] >> (c & 31)) & 1u ? z[c] : -INFINITY;
  }
}
// What a cap does to products that stay far below it (|x| < 1/4 of it, the series of tanh_fast), but for the factor scale log2 e:
// z (1 + w (a1 + w (a2 + w a3))) with w = z^2 and the powers of 1 / cap^2 in the constants.
struct RowsSeries {
  float a1, a2, a3;
  __device__ explicit RowsSeries(float icap) {
    const float i2 = icap * icap;
    a1 = -1.f / 3.f * i2;
    a2 = 2.f / 15.f * i2 * i2;
    a3 = -17.f / 315.f * i2 * i2 * i2;
  }
  __device__ float operator()(float z) const {
    const float w = z * z;
    return fmaf(z * w, fmaf(w, fmaf(w, a3, a2), a1), z);
  }
};
template <int N>
__device__ __forceinline__ void rows_series(float* z, const RowsSeries& k) {
  const float2 a1 = make_float2(k.a1, k.a1), a2 = make_float2(k.a2, k.a2), a3 = make_float2(k.a3, k.a3);
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const float2 x = make_float2(z[c], z[c + 1]), w = __fmul2_rn(x, x);
    const float2 y = __ffma2_rn(__fmul2_rn(x, w), __ffma2_rn(w, __ffma2_rn(w, a3, a2), a1), x);
    z[c] = y.x;
    z[c + 1] = y.y;
  }
}
// The same for a step's 128 keys, in TMEM.
__device__ __forceinline__ void rows_scores_tmem(uint32_t s, const RowsScore& k, float d0, bool whole, uint4 see) {
#pragma unroll 1
  for (int j = 0; j < 2; ++j) {
    uint32_t r[64];
    sm100::tmem_ld64_async(s + 64 * j, r);
    sm100::tmem_wait_ld64(r);
    const uint32_t word[2] = {j ? see.z : see.x, j ? see.w : see.y};
    rows_scores<64>(reinterpret_cast<float*>(r), k, d0 + 64.f * j, whole, word);
    sm100::tmem_st64(s + 64 * j, r);
  }
  sm100::tmem_wait_st();
}

// One step of a thread's row: weights of its keys, written over S: all 128 of the step (COPIES 1), or the 32 of copy `copy` with
// zeros in the other copies' places; updates the offset m, mo, the sum l; returns the factor on what O holds.  The scores
// of all 128 are in TMEM as they are compared, but for the factor `mul`; a copy forms its own here.
template <int KIND, bool SPLIT, bool SCORED, int COPIES>
__device__ __forceinline__ float rows_step(uint32_t s, int copy, float mul, const RowsScore& k, float d0, bool whole, uint32_t see, float& m, float& mo,
                                           float& l) {
  using namespace sm100;
  constexpr float kShift = SPLIT ? 0.f : (KIND == kBf16 ? -8.f : 13.f), kLag = weight_lag<KIND>();
  float alpha = 1.f, sum;
  auto offset = [&](float mt) {                         // where a score passes the lag, the offset moves to the largest
    if (mt > m + kLag) {
      if (m != -INFINITY) alpha = ex2(m - mt);          // (nothing to rescale before the first)
      m = mo = mt;
    }
  };
  if constexpr (COPIES == 1 && SPLIT) {
    // the first half is read twice, so that a thread never holds both and their parts
    uint32_t r[64], hi[32], lo[32];
    float* z = reinterpret_cast<float*>(r);
    tmem_ld64_async(s, r);
    tmem_wait_ld64(r);
    const float m0 = rows_max<64>(z);
    tmem_ld64_async(s + 64, r);
    tmem_wait_ld64(r);
    offset(fmaxf(m0, rows_max<64>(z)) * mul);           // (mul > 0: the largest stays the largest)
    sum = rows_weights<KIND, true, 64>(z, mul, kShift - mo, hi, lo);
    tmem_st32(s + 96, lo);
    tmem_ld64_async(s, r);
    tmem_wait_ld64(r);
    tmem_st32(s + 32, hi);
    sum += rows_weights<KIND, true, 64>(z, mul, kShift - mo, hi, lo);
    tmem_st32(s + 64, lo);
    tmem_st32(s, hi);
  } else if constexpr (COPIES == 1) {
    uint32_t rv[64], rw[64];
    float* v = reinterpret_cast<float*>(rv);
    float* u = reinterpret_cast<float*>(rw);
    if constexpr (!SCORED && KIND != kE4m3) {
      // No weight is above their sum: the largest score is looked for only where a row has no offset yet or the sum passes what
      // the products' type holds (both rare), and the weights are formed again.  Over fp16 products the offset is then put 5
      // binary orders above the largest, where 128 weights of that size stay within 2^15: what is lost of a weight is
      // below 2^-32 of the row's largest.  (4096 tokens behind 12288, 32 / 8 heads of 128: bf16 867 -> 791 us, fp16 931 -> 796; over an
      // e4m3 pool, whose softmax has fewer registers, 1072 -> 1112 when it was tried: not there.)
      constexpr float kMost = KIND == kBf16 ? 1.f : 0x1p15f, kAbove = KIND == kBf16 ? 0.f : 5.f;
      bool look = __any_sync(0xffffffffu, m == -INFINITY);
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        tmem_ld64_async(s + 64, rv);
        tmem_ld64_async(s, rw);
        tmem_wait_ld64(rv);
        reg_tie64(rw);
        if (look) {
          const float mt = fmaxf(rows_max<64>(u), rows_max<64>(v)) * mul + kAbove;
          if (mt > m) {                                 // (any row's: none is above the bound behind this)
            if (m != -INFINITY) alpha = ex2(m - mt);
            m = mo = mt;
          }
        }
        sum = rows_weights<KIND, false, 64>(u, mul, kShift - mo, rw, nullptr);
        sum += rows_weights<KIND, false, 64>(v, mul, kShift - mo, rv, nullptr);
        if (look || !__any_sync(0xffffffffu, sum > kMost)) break;
        look = true;
      }
      tmem_st32(s, rw);
      tmem_st32(s + 32, rv);
      l = l * alpha + sum;
      return alpha;
    }
    tmem_ld64_async(s + 64, rv);
    tmem_ld64_async(s, rw);
    tmem_wait_ld64(rv);                                 // one wait covers both loads
    reg_tie64(rw);
    float top = fmaxf(rows_max<64>(u), rows_max<64>(v)), by = mul;
    if constexpr (SCORED) {
      if (!whole) {                                     // not yet as they are compared (`whole`: they are)
        bool fit = true;
        if (k.capped) {
          // (scores far below the cap are the rule; constants of the series stay finite)
          const float low = fminf(rows_min<64>(u), rows_min<64>(v));
          fit = __all_sync(0xffffffffu, fmaxf(top, -low) * k.icap < 0.25f && k.icap < 0x1p20f && k.sc > 0.f);
          if (fit) {
            const RowsSeries f(k.icap);
            rows_series<64>(u, f);
            rows_series<64>(v, f);
            top = f(top);                               // (the series rises with its argument)
            by = k.sc;
          }
        }
        if (!fit) {
          rows_scores_tmem(s, k, d0, true, make_uint4(0, 0, 0, 0));
          tmem_ld64_async(s + 64, rv);
          tmem_ld64_async(s, rw);
          tmem_wait_ld64(rv);
          reg_tie64(rw);
        } else if (k.biased) {
          rows_bias<64>(u, k.sc, k.slope, d0);
          rows_bias<64>(v, k.sc, k.slope, d0 + 64.f);
          by = 1.f;
        }
        if (!fit || k.biased) top = fmaxf(rows_max<64>(u), rows_max<64>(v));
      }
    }
    offset(top * by);
    sum = rows_weights<KIND, false, 64>(u, by, kShift - mo, rw, nullptr);
    tmem_st32(s, rw);
    sum += rows_weights<KIND, false, 64>(v, by, kShift - mo, rv, nullptr);
    tmem_st32(s + 32, rv);
  } else {
    float z[32];
    uint32_t hi[16], lo[16], zero[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) zero[c] = 0u;
    tmem_ld32(s + 32 * copy, z);
    rows_scores<32>(z, k, d0, whole, &see);
    offset(rows_max<32>(z) * mul);
    sum = rows_weights<KIND, SPLIT, 32>(z, mul, kShift - mo, hi, lo);
#pragma unroll
    for (int part = 0; part < (SPLIT ? 2 : 1); ++part)
#pragma unroll
      for (int j = 0; j < 4; ++j) tmem_st16(s + 64 * part + 16 * ((copy + j) & 3), j != 0 ? zero : part ? lo : hi);
  }
  l = l * alpha + sum;
  return alpha;
}

template <int D, int KIND, bool SPLIT, bool SCORED>
__global__ void __launch_bounds__(kRowsThreads, 1) rows_attend(const __grid_constant__ RowsArgs a, const __grid_constant__ CUtensorMap tk,
                                                               const __grid_constant__ CUtensorMap tv) {
  using namespace sm100;
  constexpr uint32_t TB = rows_tile_bytes<D>();
  constexpr int RB = row_bytes<D, KIND>(), CPR = RB / 16, NS = rows_slots<D, KIND>();
  // TMEM: tile X in {0, 1}: S (the weights over it) at 256 X, O at 256 X + 128
  constexpr uint32_t kSCol = 0, kOCol = 128, kTileCols = 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_addr(sbase), bars = base + rows_bar_off<D, KIND>(), slots = base + 2 * TB;
  auto bar = [&](int i) { return bars + 8u * i; };
  // tile q (K of step q / 2, V after it) of the CTA: its slot's barriers and the parity of its use
  auto full = [&](uint32_t q) { return bar(q % NS); };
  auto empty = [&](uint32_t q) { return bar(kBarEmpty + q % NS); };
  auto use = [&](uint32_t q) { return (q / NS) & 1; };
  auto s_full = [&](int x) { return bar(kBarTiles + x); };
  auto p_full = [&](int x) { return bar(kBarTiles + 2 + x); };
  auto pv_done = [&](int x) { return bar(kBarTiles + 4 + x); };
  auto q_full = [&](int x) { return bar(kBarTiles + 6 + x); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(sbase + rows_bar_off<D, KIND>() + kWordsOff);
  uint32_t* tslot = misc;
  volatile uint32_t* flag = misc + 1;
  volatile uint32_t* o_begun = misc + 2;           // [2]: O of the piece holds values before its first product
  // [8][4] each, by steps of the CTA modulo 8: rows that were loaded and are seen by some row; rows whose V is not finite, where
  // that matters
  uint32_t *seen_w = misc + 16, *bad_w = misc + 48;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // (what needs nothing of the earlier kernels, while they run)
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar(i), 4);                        // one arrival per loader warp
      mbar_init(bar(kBarEmpty + i), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full(x), 1);
      mbar_init(p_full(x), 4);                     // one arrival per softmax warp of the tile
      mbar_init(pv_done(x), 1);
      mbar_init(q_full(x), 4);
    }
    mbar_init(bar(kBarMerge), 8);
    for (int i = kBarDrain; i < kRowsBars; ++i) mbar_init(bar(i), 1);
    *flag = 0;
    o_begun[0] = o_begun[1] = 0;
    fence_barrier_init();
  }
  if (warp == 12) tmem_alloc(smem_addr(tslot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  wait_for_earlier_kernels();
  let_later_kernels_start();
  const RowsStart& start = a.starts[cta];         // (a CTA without steps walks none)

  // registers: 512 x 128 at the launch; the rows' threads hold 128 scores
  constexpr int kRegRows = KIND == kE4m3 ? 168 : 184, kRegLoad = KIND == kE4m3 ? 112 : 80, kRegMma = 64;
  static_assert(256 * kRegRows + 128 * kRegLoad + 128 * kRegMma <= 512 * 128, "the shares fit what the block was launched with");
  RowsWalk walk;
  RowsPiece p;

  if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegLoad));
    walk.begin(start);
    // ---------------------------------------------------------------- loaders: rows 32 w .. 32 w + 31 of every step
    const int w = warp - 8;
    constexpr int KPI = 32 / CPR;                  // rows that 32 lanes take 16 bytes of
    const int c = lane % CPR;
    const int R = a.box_rows;                      // rows of a box, 0: the pool's pages do not fall into boxes
    // a step to load: this lane's row of it; the page's entry is read ahead, nothing waits for it here
    struct Row {
      int32_t id, within, g, table;
      uint32_t flags;                              // there is a step; this row is needed; its box is; some row needs looking at
    };
    enum : uint32_t { kMore = 1, kNeed = 2, kBox = 4, kPartial = 8 };
    bool have = walk.next(a, p);
    int s = have ? p.s0 : 0;
    auto look = [&]() -> Row {
      Row r{0, 0, 0, 0, 0};
      if (!have) return r;
      const RowsItem& it = *p.item;
      const int t0 = it.k0 + kTileKeys * s, t = t0 + 32 * w + lane, tb = R != 0 ? t & ~(R - 1) : t;
      r.flags = kMore | (t >= it.lo && t < it.hi ? kNeed : 0u) | (tb < it.hi && tb > it.lo - max(R, 1) ? kBox : 0u) |
                (t0 < it.lo || it.hi - t0 < kTileKeys || rows_partial(it.lo, it.hi, it.full_lo, it.full_hi, t0) ? kPartial : 0u);
      r.g = p.g;
      r.table = it.table;
      if (r.flags & kBox) {
        const int blk = (int)((__umulhi(a.p_mul, (uint32_t)t) + (uint32_t)t) >> a.p_shift);
        r.within = t - blk * a.P;
        r.id = a.tables[(int64_t)it.table * a.max_blocks + blk];
      }
      if (++s == p.s1) {
        have = walk.next(a, p);
        s = p.s0;
      }
      return r;
    };
    // the row's entry names a page of the pool
    auto known = [&](const Row& r) {
      const bool in = r.id >= 0 && r.id < a.n_pages;
      if ((r.flags & kNeed) && !in) set_device_error(a.err, KVSEL_ERR_DEVICE, (uint32_t)r.table);
      return in;
    };
    auto await = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, rows_wait(b, parity, flag)); };
    auto slot_chunk = [&](uint32_t q, int x, int cc) {         // of row x of this warp's, 16-byte chunk cc of 16-bit values
      return 2 * TB + (q % NS) * TB + (cc >> 3) * kHalf + (32 * w + x) * 128 + (((cc & 7) ^ (x & 7)) << 4);
    };
    // the boxes of a tile's rows (those of `boxes`, by first row), 128 bytes of them at a time into a slot, or whole into `dst`
    auto load_boxes = [&](const Row& r, uint32_t boxes, const CUtensorMap* map, uint32_t dst, uint32_t b) {
      constexpr int HALVES = KIND == kE4m3 ? 1 : D / 64;
      const uint32_t bytes = __popc(boxes) * R * RB;
      if (lane == 0) {
        if (bytes != 0) mbar_expect_tx(b, bytes);
        else mbar_arrive(b);
      }
      __syncwarp();
      if ((boxes >> lane) & 1u)
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
          rows_box(dst + h * kHalf + lane * (KIND == kE4m3 ? RB : 128), map, 64 * h, r.within, r.g, r.id, b);
    };
    // 16-bit rows in a slot: those not in `rows` become zeros, and values that are not finite do in the others; which rows had such
    auto clean = [&](uint32_t q, uint32_t rows) -> uint32_t {
      uint32_t bad = 0;
#pragma unroll 1
      for (int i = 0; i < 32 / KPI; ++i) {
        const int x = i * KPI + lane / CPR;
        uint4* at = reinterpret_cast<uint4*>(sbase + slot_chunk(q, x, c));
        uint4 y = *at;
        uint32_t* h = reinterpret_cast<uint32_t*>(&y);
        constexpr uint32_t ex = KIND == kBf16 ? 0x7f80u : 0x7c00u;
        bool hit = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((h[e] & ex) == ex) h[e] &= 0xffff0000u, hit = true;
          if ((h[e] & (ex << 16)) == (ex << 16)) h[e] &= 0xffffu, hit = true;
        }
        if (!((rows >> x) & 1u)) *at = make_uint4(0, 0, 0, 0);
        else if (hit) *at = y, bad |= 1u << x;
      }
      return __reduce_or_sync(0xffffffffu, bad);
    };
    auto told = [&](uint32_t q) {                  // this warp's rows of tile q are there
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(q));
    };
    bool ok = true;
    uint32_t boxed = 0, n_land = 0;                // tiles whose boxes were asked for, and those that were looked at first
    constexpr int AHEAD = 2;                       // steps whose pages are looked up ahead
    Row rows[AHEAD + 1];
#pragma unroll
    for (int i = 0; i <= AHEAD; ++i) rows[i] = look();
    auto shift = [&]() {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) rows[i] = rows[i + 1];
      rows[AHEAD] = look();
    };
    if (KIND != kE4m3 && R != 0) {
      for (uint32_t step = 0; (rows[0].flags & kMore) && ok; ++step) {
        const Row& r = rows[0];
        const bool in = known(r), partial = r.flags & kPartial;
        const uint32_t fine = __ballot_sync(0xffffffffu, in && (r.flags & kNeed));
        const uint32_t boxes = __ballot_sync(0xffffffffu, in && (r.flags & kBox) && (lane & (R - 1)) == 0);
        ok = await(empty(2 * step), use(2 * step) ^ 1);
        if (!ok) break;
        if (lane == 0) seen_w[(step & 7) * 4 + w] = fine;
        load_boxes(r, boxes, &tk, slots + (2 * step) % NS * TB + 32 * w * 128, full(2 * step));
        const uint32_t q = 2 * step + 1;
        boxed = q;
        ok = await(empty(q), use(q) ^ 1);
        if (!ok) break;
        const uint32_t dst = slots + q % NS * TB + 32 * w * 128;
        boxed = q + 1;
        if (partial) {
          load_boxes(r, boxes, &tv, dst, bar(kBarLand + w));
          ok = await(bar(kBarLand + w), n_land++ & 1);
          if (!ok) break;
          const uint32_t bad = clean(q, fine);
          if (lane == 0) bad_w[(step & 7) * 4 + w] = bad;
          told(q);
        } else {
          if (fine != 0xffffffffu) {               // (pages outside the pool)
            clean(q, 0u);
            fence_proxy_async_smem();
            __syncwarp();
          }
          load_boxes(r, boxes, &tv, dst, full(q));
        }
        shift();
      }
    } else if (KIND != kE4m3) {
      // cp.async, whole rows at a time, rows without a source as zeros
      uint32_t issued = 0, done = 0, check = 0;    // tiles; bit i & 7: V to be looked at
      auto tell = [&]() {                          // the oldest tile not told of is there (copies end in order only)
        switch (issued - done) {
          case 1: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
          case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
          case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
          default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        }
        if ((done & 1) && ((check >> (done & 7)) & 1)) {
          const uint32_t bad = clean(done, 0xffffffffu);
          if (lane == 0) bad_w[((done >> 1) & 7) * 4 + w] = bad;
        }
        told(done);
        ++done;
      };
      while ((rows[0].flags & kMore) && ok) {
        const Row& r = rows[0];
        const bool fine = known(r) && (r.flags & kNeed);
        const int64_t off = (fine ? (int64_t)r.id * a.page_stride + (int64_t)r.within * a.row_stride : 0) * 2;
        const uint32_t there = __ballot_sync(0xffffffffu, fine);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          while (issued - done == 4 || !__all_sync(0xffffffffu, rows_test(empty(issued), use(issued) ^ 1))) {
            if (issued != done) tell();
            else if (!(ok = await(empty(issued), use(issued) ^ 1))) break;
          }
          if (!ok) break;
          if (kv == 0 && lane == 0) seen_w[((issued >> 1) & 7) * 4 + w] = there;
          const uint8_t* from = static_cast<const uint8_t*>(kv ? a.v : a.k) + (int64_t)r.g * a.head_stride * 2;
#pragma unroll
          for (int i = 0; i < 32 / KPI; ++i) {
            const int x = i * KPI + lane / CPR;
            const int64_t ox = __shfl_sync(0xffffffffu, off, x) + c * 16;
            cp_async16(base + slot_chunk(issued, x, c), from + ox, (there >> x) & 1u);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          check &= ~(1u << (issued & 7));
          if (kv && (r.flags & kPartial)) check |= 1u << (issued & 7);
          ++issued;
        }
        shift();
      }
      while (ok && done != issued) tell();
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
      // 16 e4m3 values become two chunks of 8 fp16 values; values that are no numbers become zeros where they are looked for
      auto widen = [&](uint4 y, uint32_t q, int x, bool look_at) -> uint32_t {
        uint32_t* h = reinterpret_cast<uint32_t*>(&y);
        uint32_t bad = 0, o[8];
        if (look_at) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t nan = __vcmpeq4(h[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
            if (nan) h[e] &= ~nan, bad |= 1u << x;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) e4m3x4_to_f16(h[e], o[2 * e], o[2 * e + 1]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(base + slot_chunk(q, x, 2 * c + e)), "r"(o[4 * e]), "r"(o[4 * e + 1]),
                       "r"(o[4 * e + 2]), "r"(o[4 * e + 3]) : "memory");
        return bad;
      };
      constexpr int NI = 32 / KPI;
      if (R != 0) {
        // boxes of bytes, four tiles ahead, into this warp's part of a ring
        const uint32_t raw = rows_raw_off<D, KIND>() + 32 * w * RB;
        auto raw_bar = [&](uint32_t q) { return bar(kBarRaw + 4 * (q % kRawTiles) + w); };
        auto request = [&](const Row& r, uint32_t q) {         // K (even q) or V of the step
          if (!(r.flags & kMore)) return;
          const uint32_t boxes = __ballot_sync(0xffffffffu, known(r) && (r.flags & kBox) && (lane & (R - 1)) == 0);
          load_boxes(r, boxes, (q & 1) ? &tv : &tk, base + raw + (q % kRawTiles) * kTileKeys * RB, raw_bar(q));
          boxed = q + 1;
        };
        static_assert(kRawTiles == 2 * AHEAD, "the tiles ahead are those of the steps looked up");
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          request(rows[i], 2 * i);
          request(rows[i], 2 * i + 1);
        }
        for (uint32_t step = 0; (rows[0].flags & kMore) && ok; ++step) {
          const Row& r = rows[0];
          const uint32_t fine = __ballot_sync(0xffffffffu, known(r) && (r.flags & kNeed));
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t q = 2 * step + kv;
            ok = ok && await(raw_bar(q), (q / kRawTiles) & 1) && await(empty(q), use(q) ^ 1);
            if (!ok) break;
            if (kv == 0 && lane == 0) seen_w[(step & 7) * 4 + w] = fine;
            uint32_t bad = 0;
            const uint8_t* from = sbase + raw + (q % kRawTiles) * kTileKeys * RB;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              const int x = i * KPI + lane / CPR;
              const uint4 y = *reinterpret_cast<const uint4*>(from + x * RB + c * 16);
              bad |= widen((fine >> x) & 1u ? y : make_uint4(0, 0, 0, 0), q, x, kv && (r.flags & kPartial));
            }
            if (kv && (r.flags & kPartial)) {
              bad = __reduce_or_sync(0xffffffffu, bad);
              if (lane == 0) bad_w[(step & 7) * 4 + w] = bad;
            }
            told(q);                               // (and the warp is done with the raw tile)
            request(rows[AHEAD], q + kRawTiles);
          }
          shift();
        }
      } else {
        // rows through registers, a tile ahead
        uint4 y[2][NI];
        struct Fetch {
          int64_t off;
          uint32_t rows;
        };
        auto resolve = [&](const Row& r) -> Fetch {
          const bool fine = known(r) && (r.flags & kNeed);
          return {fine ? (int64_t)r.id * a.page_stride + (int64_t)r.within * a.row_stride : 0, __ballot_sync(0xffffffffu, fine)};
        };
        auto fetch = [&](const Fetch& f, int g, const void* pool, uint4* to) {
          const uint8_t* from = static_cast<const uint8_t*>(pool) + (int64_t)g * a.head_stride + c * 16;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const int x = i * KPI + lane / CPR;
            const int64_t ox = __shfl_sync(0xffffffffu, f.off, x);
            to[i] = (f.rows >> x) & 1u ? *reinterpret_cast<const uint4*>(from + ox) : make_uint4(0, 0, 0, 0);
          }
        };
        Fetch f{0, 0};
        if (rows[0].flags & kMore) {
          f = resolve(rows[0]);
          fetch(f, rows[0].g, a.k, y[0]);
        }
        for (uint32_t step = 0; (rows[0].flags & kMore) && ok; ++step) {
          const bool partial = rows[0].flags & kPartial;
          fetch(f, rows[0].g, a.v, y[1]);
          const uint32_t there = f.rows;
          shift();
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t q = 2 * step + kv;
            ok = ok && await(empty(q), use(q) ^ 1);
            if (!ok) break;
            if (kv == 0 && lane == 0) seen_w[(step & 7) * 4 + w] = there;
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < NI; ++i) bad |= widen(y[kv][i], q, i * KPI + lane / CPR, kv && partial);
            if (kv && partial) {
              bad = __reduce_or_sync(0xffffffffu, bad);
              if (lane == 0) bad_w[(step & 7) * 4 + w] = bad;
            }
            told(q);
            if (kv == 0 && (rows[0].flags & kMore)) {
              f = resolve(rows[0]);
              fetch(f, rows[0].g, a.k, y[0]);
            }
          }
        }
      }
    }
    if (!ok && lane == 0) rows_fail(a, flag, kRowsLoader);
    // Boxes in flight land before the CTA ends.  (Without a failure every tile's barrier was waited for by those who read it.)
    if (!ok && R != 0) {
      constexpr uint32_t kPolls = 1u << 14;
      if constexpr (KIND == kE4m3) {
        for (uint32_t q = boxed < kRawTiles ? 0 : boxed - kRawTiles; q < boxed; ++q) (void)mbar_wait_n(bar(kBarRaw + 4 * (q % kRawTiles) + w), (q / kRawTiles) & 1, kPolls);
      } else {
        for (uint32_t q = boxed < NS ? 0 : boxed - NS; q < boxed; ++q) (void)mbar_wait_n(full(q), use(q), kPolls);
        if (n_land > 0) (void)mbar_wait_n(bar(kBarLand + w), (n_land - 1) & 1, kPolls);
      }
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegMma));
    // ---------------------------------------------------------------- products, a thread for S and one for P V: each of
    // them spends as long on waits and commits as the tensor cores on its products
    if (warp <= 13 && lane == 0) {
      walk.begin(start);
      const bool pv = warp == 13;
      constexpr uint32_t idesc_s = rows_idesc<KIND>(128, 128), idesc_o = rows_idesc<KIND>(128, D) | kUmmaBMajorMN;
      constexpr int KS = D / 16, KP = kTileKeys / 16 * (SPLIT ? 2 : 1);
      const uint64_t vdesc = umma_desc_sw128_mn(slots, kHalf), kdesc = umma_desc_sw128(slots), qdesc = umma_desc_sw128(base);
      uint32_t q = pv ? 1 : 0, slot = q, turn = 0;  // the step's K (V) tile, its slot, the tile whose turn it is
      uint32_t phase = 0;                           // of the slot
      uint32_t at = 0, last_pv = 3, was_pv = 0;     // by tile: parity of the next queries (weights), of the last P V; whether there was one
      bool ok = true, any = false;
      while (ok && walk.next(a, p)) {
        const bool two = p.item->rows > kTileRows;
        const int s0 = p.s0, s1 = p.s1;
        for (int s = s0; s < s1 && ok; ++s) {
          const bool first = s < s0 + (two ? 1 : 2);
          const uint32_t x0 = two ? 0 : turn, x1 = two ? 1 : turn;
          ok = rows_wait(bar(slot), phase, flag);   // the tile has landed
          for (uint32_t x = x0; x <= x1 && ok; ++x) {
            if (pv) {
              // P V once the weights are written
              if (!(ok = rows_wait(p_full(x), (at >> x) & 1, flag))) break;
              at ^= 1u << x;
              tc_fence_after();
              const bool keep = !first || o_begun[x] != 0;
              const uint64_t vd = vdesc + slot * (TB >> 4);
              const uint32_t to = tmem + x * kTileCols + kOCol, from = tmem + x * kTileCols + kSCol;
#pragma unroll
              for (int kk = 0; kk < KP; ++kk) umma_bf16_ta(to, from + kk * 8, vd + ((kk & 7) * 2048 >> 4), idesc_o, (keep || kk > 0) ? 1u : 0u);
              umma_commit(pv_done(x));
            } else {
              // S once the tile's queries are there and its last P V (which reads the same TMEM columns) is done
              if (first) {
                if (!(ok = rows_wait(q_full(x), (at >> x) & 1, flag))) break;
                at ^= 1u << x;
              }
              if ((was_pv >> x) & 1) {
                if (!(ok = rows_wait(pv_done(x), (last_pv >> x) & 1, flag))) break;
              }
              was_pv |= 1u << x;
              last_pv ^= 1u << x;                   // (0 for the first: what the tile's second S waits for)
              tc_fence_after();
              const uint64_t qd = qdesc + x * (TB >> 4), kd = kdesc + slot * (TB >> 4);
              const uint32_t to = tmem + x * kTileCols + kSCol;
#pragma unroll
              for (int kk = 0; kk < KS; ++kk)
                umma_bf16(to, qd + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4), kd + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
              umma_commit(s_full(x));
            }
            any = true;
          }
          if (!ok) break;
          umma_commit(bar(kBarEmpty + slot));       // (a commit covers every product of its thread before it)
          turn ^= 1;
          q += 2;
          slot += 2;
          if (slot >= NS) slot -= NS;
          phase = (q / NS) & 1;
        }
      }
      if (!ok) rows_fail(a, flag, kRowsMma);
      if (any) {
        umma_commit(bar(kBarDrain + (pv ? 1 : 0)));
        if (!mbar_wait(bar(kBarDrain + (pv ? 1 : 0)), 0)) set_device_error(a.err, KVSEL_ERR_TIMEOUT, kRowsDrain);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegRows));
    walk.begin(start);
    // ---------------------------------------------------------------- softmax, a thread per query row
    const int x = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t tm = tmem + ((uint32_t)(quarter * 32) << 16) + x * kTileCols;
    constexpr float kShift = SPLIT ? 0.f : (KIND == kBf16 ? -8.f : 13.f);
    uint32_t n = 0, n_merged = 0;                   // steps of this tile, meetings of the softmax warps so far
    bool ok = true;
    // small: a piece's rows are one block of 32 in a tile, with four copies; whether the tile has a step of a piece
    auto has_steps = [&](const RowsPiece& t, int i0) {
      return t.item->rows > kTileRows || t.s1 - t.s0 > 1 || (i0 & 1) == x;
    };
    // this thread's query row of a piece: into shared memory, swizzled; returns the factor taken out of it
    auto load_q = [&](const RowsPiece& t) -> float {
      const int rows = t.item->rows;
      const int i = rows > kTileRows ? x * kTileRows + row : rows <= 32 ? lane : row, r = t.item->row0 + i;
      const bool live = i < rows;
      uint4 y[D / 8];
      const int tok = r / a.G, h = r - tok * a.G;
      const uint16_t* from = static_cast<const uint16_t*>(a.q) + (live ? ((int64_t)t.item->token0 + tok) * a.q_stride + (int64_t)(t.g * a.G + h) * D : 0);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) y[c] = live ? reinterpret_cast<const uint4*>(from)[c] : make_uint4(0, 0, 0, 0);
      float by = 1.f;
      if constexpr (KIND == kE4m3) {
        if (!a.out_f16) {                           // bf16 queries over fp16 products: divided by the power of two at their largest
          uint32_t* hw = reinterpret_cast<uint32_t*>(y);
          float mx = 0.f;
#pragma unroll
          for (int e = 0; e < D / 2; ++e)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(hw[e] << 16)), fabsf(__uint_as_float(hw[e] & 0xffff0000u))));
          // powers 2^-100 .. 2^100 keep both the factor and its inverse normal
          const int ex = min(100, max(-100, (int)((__float_as_uint(mx) >> 23) & 0xff) - 127));
          by = __uint_as_float((uint32_t)(ex + 127) << 23);
          const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
          for (int e = 0; e < D / 2; ++e) {
            const __half2 hh = __floats2half2_rn(__uint_as_float(hw[e] << 16) * inv, __uint_as_float(hw[e] & 0xffff0000u) * inv);
            hw[e] = *reinterpret_cast<const uint32_t*>(&hh);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<uint4*>(sbase + x * TB + (c >> 3) * kHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = y[c];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(x));
      return by;
    };
    // the eight softmax warps meet; false where one does not come
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarMerge));
      return __all_sync(0xffffffffu, rows_wait(bar(kBarMerge), n_merged++ & 1, flag));
    };
    RowsPiece cur{nullptr, 0, 0, 0};                // (none before the first)
    int i0 = 0;                                     // the piece's first step among the CTA's
    float by = 1.f;
    do {
      const bool now = cur.item != nullptr;
      const RowsItem& it = now ? *cur.item : start.item;
      const int rows = now ? it.rows : 0;
      const bool two = rows > kTileRows, small = rows <= 32;
      const int i = two ? x * kTileRows + row : small ? lane : row, copy = small ? quarter : 0;
      const int r = it.row0 + i, tok = r / a.G, h = cur.g * a.G + (r - tok * a.G);
      const bool live = i < rows;
      const bool idle = __all_sync(0xffffffffu, !live);         // a warp of padding alone
      float m = -INFINITY, mo = 0.f, l = 0.f;
      bool had = false;
      if (now) {
        const int k0 = it.k0, k_lo = it.lo, k_hi = it.hi, full_lo = it.full_lo, full_hi = it.full_hi;
        const int pos = !live ? -1 : a.prefix ? (int)a.lens[it.token0 + tok] - 1 : it.base + tok;
        const int low = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
        const float head_scale = a.k_scale != nullptr ? a.k_scale[cur.g] : 1.f, ksc = a.scale * head_scale * by;
        RowsScore score;
        score.capped = SCORED && a.softcap != 0.f;
        score.sc = ksc * kLog2e;
        // (a factor that ended at 0 would make no number of the rows not seen, at -inf; 2^-126 leaves nothing of the others either)
        if (KIND == kE4m3 && head_scale > 0.f) score.sc = fmaxf(score.sc, 0x1p-126f);
        score.icap = score.capped ? ksc / a.softcap : 0.f;
        score.cap2 = a.softcap * kLog2e;
        score.slope = SCORED && a.slopes != nullptr && live ? a.slopes[h] * kLog2e : 0.f;
        score.biased = (SCORED && a.slopes != nullptr) || (!score.capped && !(head_scale > 0.f));
        const bool plain = !score.capped && !score.biased;
        const float mul = plain ? score.sc : 1.f;
        bool begun = false;
        if (lane == 0 && quarter == 0) o_begun[x] = 0;          // (before the piece's first weights are told of)
        uint32_t step = i0;
#pragma unroll 1
        for (int s = cur.s0; s < cur.s1; ++s, ++step) {
          if (!two && (int)(step & 1) != x) continue;
          const int t0 = k0 + kTileKeys * s;
          const bool within = t0 >= full_lo && full_hi - t0 >= kTileKeys, partial = rows_partial(k_lo, k_hi, full_lo, full_hi, t0);
          ok = __all_sync(0xffffffffu, rows_wait(s_full(x), n & 1, flag));
          if (!ok) break;
          ++n;
          tc_fence_after();
          const uint4 there = *reinterpret_cast<const uint4*>(&seen_w[(step & 7) * 4]);
          const bool whole = within && (there.x & there.y & there.z & there.w) == 0xffffffffu;
          if (partial) {
            ok = __all_sync(0xffffffffu, rows_wait(full(2 * step + 1), use(2 * step + 1), flag));
            if (!ok) break;
            uint4 bad = *reinterpret_cast<const uint4*>(&bad_w[(step & 7) * 4]);
            if ((bad.x | bad.y | bad.z | bad.w) != 0) {
              if (small) bad = make_uint4(copy == 0 ? bad.x : 0, copy == 1 ? bad.y : 0, copy == 2 ? bad.z : 0, copy == 3 ? bad.w : 0);
              add_bad_rows<D, KIND>(a, static_cast<const uint8_t*>(a.v) + (int64_t)cur.g * a.head_stride * elem_bytes<KIND>(), it.table, t0, pos,
                                    bad, tm + kOCol, !had);
              if (!had) begun = true;
              if (!had && lane == 0 && quarter == 0) o_begun[x] = 1;
            }
          }
          if (!idle) {
            uint32_t word[4] = {there.x, there.y, there.z, there.w};
            if (!whole) {
              const int from = low - t0, to = pos + 1 - t0;     // keys of the step that the row sees: [from, to)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int lo = min(32, max(0, from - 32 * k)), hi = min(32, max(0, to - 32 * k));
                const uint32_t below_hi = hi >= 32 ? 0xffffffffu : (1u << hi) - 1u, below_lo = lo >= 32 ? 0xffffffffu : (1u << lo) - 1u;
                word[k] = live ? word[k] & below_hi & ~below_lo : 0u;
              }
            }
            float alpha;
            if (small) {
              const uint32_t see = copy == 0 ? word[0] : copy == 1 ? word[1] : copy == 2 ? word[2] : word[3];
              alpha = rows_step<KIND, SPLIT, SCORED, 4>(tm + kSCol, copy, mul, score, (float)(t0 + 32 * copy - pos), whole, see, m, mo, l);
            } else {
              // with a mask they are brought to what is compared in TMEM, else in the registers that hold them for the softmax
              const bool before = !whole || (!plain && (SPLIT || !SCORED));
              if (before) rows_scores_tmem(tm + kSCol, score, (float)(t0 - pos), whole, make_uint4(word[0], word[1], word[2], word[3]));
              alpha = rows_step<KIND, SPLIT, SCORED, 1>(tm + kSCol, 0, mul, score, (float)(t0 - pos), before || plain, 0u, m, mo, l);
            }
            // O of the tile's step before is final (this step's S was issued behind its P V)
            if ((had || begun) && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float f[32];
                uint32_t y[32];
                tmem_ld32(tm + kOCol + c, f);
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(f[e] * alpha);
                tmem_st32(tm + kOCol + c, y);
              }
            }
            tmem_wait_st();
          }
          had = true;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(x));
        }
        if (ok && had) {
          // the piece's last P V; its queries are read by then
          ok = __all_sync(0xffffffffu, rows_wait(pv_done(x), (n - 1) & 1, flag));
          tc_fence_after();
        }
        if (!ok) break;
      }
      const bool final = now && !a.prefix && cur.starts() && cur.ends();
      const float vsc = a.v_scale != nullptr ? a.v_scale[cur.g] : 1.f;
      const int64_t out = ((int64_t)it.token0 + tok) * a.h_q + h;
      const int64_t prow = rows_part(a, cta, cur.starts(), cur.g, it);
      const bool f16 = KIND == kE4m3 ? a.out_f16 != 0 : KIND == kF16;
      auto pack = [&](float u, float v) { return f16 ? pack16<kF16>(u, v) : pack16<kBf16>(u, v); };
      // factor on O: to the output, or none to the partial sums
      auto factor = [&](float sum) { return !final ? 1.f : sum == 0.f ? 0.f : (SPLIT ? vsc / weight_unit<KIND>() : vsc) / sum; };
      if (now && !two) {
        // What the tiles and copies hold of a row, in the queries' room once both tiles' products are done with them: offsets and
        // sums meet first, then D / 4 columns at a time in one of two buffers, where every warp sums its share of its rows'
        // columns, each part times 2^(m - M).  With copies all warps hold parts of the same 32 rows, else two.
        if (!(ok = meet())) break;
        constexpr int COLS = D / 4;
        float* buf = reinterpret_cast<float*>(sbase);
        float2* ml = reinterpret_cast<float2*>(buf + 8 * COLS * 32);
        ml[warp * 32 + lane] = make_float2(m, l);
        auto merge = [&](auto parts_c) {
          constexpr int PARTS = decltype(parts_c)::value, OWN = COLS / PARTS;      // parts of a row, columns of a warp
          const int first = PARTS == 8 ? 0 : quarter, c0 = (PARTS == 8 ? warp : x) * OWN;        // warps first + k * (8 / PARTS)
          float f[PARTS];
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            float* b = buf + (q & 1) * 8 * COLS * 32;
            float y[COLS];
            __syncwarp();
            if (had && !idle) {
              if constexpr (COLS == 32) tmem_ld32(tm + kOCol + q * COLS, y);
              else tmem_ld16(tm + kOCol + q * COLS, y);
            } else {
#pragma unroll
              for (int e = 0; e < COLS; ++e) y[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < COLS; ++e) b[(warp * COLS + e) * 32 + lane] = y[e];
            if (!(ok = meet())) return;
            if (q == 0) {
              float M = -INFINITY, L = 0.f;
#pragma unroll
              for (int k = 0; k < PARTS; ++k) M = fmaxf(M, ml[(first + 8 / PARTS * k) * 32 + lane].x);
#pragma unroll
              for (int k = 0; k < PARTS; ++k) {
                const float2 z = ml[(first + 8 / PARTS * k) * 32 + lane];
                f[k] = z.x == M ? 1.f : exp2f(z.x - M);
                L += z.y * f[k];
              }
              if (!(ok = meet())) return;           // (the second buffer is read)
              m = M;
              l = L;
              const float g = factor(L);
#pragma unroll
              for (int k = 0; k < PARTS; ++k) f[k] *= g;
            }
            float r[OWN];
#pragma unroll
            for (int e = 0; e < OWN; ++e) {
              r[e] = 0.f;
#pragma unroll
              for (int k = 0; k < PARTS; ++k) r[e] = fmaf(b[((first + 8 / PARTS * k) * COLS + c0 + e) * 32 + lane], f[k], r[e]);
            }
            const int col = q * COLS + c0;
            if (live && final) {
#pragma unroll
              for (int e = 0; e < OWN; e += 2) static_cast<uint32_t*>(a.o)[(out * D + col + e) / 2] = pack(r[e], r[e + 1]);
            } else if (live) {
#pragma unroll
              for (int e = 0; e < OWN; e += 2)
                *reinterpret_cast<float2*>(a.part + prow * D + ((int64_t)((col + e) / 4) * rows + i) * 4 + ((col + e) & 2)) = make_float2(r[e], r[e + 1]);
            }
          }
          ok = meet();                              // the buffers are read
        };
        if (small) merge(std::integral_constant<int, 8>{});
        else merge(std::integral_constant<int, 2>{});
        if (!ok) break;
      }
      // the next piece's queries, then what is left of this one's result
      RowsPiece nxt{nullptr, 0, 0, 0};
      (void)walk.next(a, nxt);
      const int i_next = i0 + cur.s1 - cur.s0;
      float by_next = 1.f;
      if (nxt.item != nullptr && has_steps(nxt, i_next)) by_next = load_q(nxt);
      if (now && two && !idle) {
        const float f = factor(l);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float y[32];
          __syncwarp();
          tmem_ld32(tm + kOCol + c, y);
          if (!live) continue;
          if (final) {
            uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + out * D + c);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              to[e] = make_uint4(pack(y[8 * e] * f, y[8 * e + 1] * f), pack(y[8 * e + 2] * f, y[8 * e + 3] * f), pack(y[8 * e + 4] * f, y[8 * e + 5] * f),
                                 pack(y[8 * e + 6] * f, y[8 * e + 7] * f));
          } else {
            // four values of a row next to those of the next row
            float4* to = reinterpret_cast<float4*>(a.part + prow * D) + (int64_t)(c / 4) * rows + i;
#pragma unroll
            for (int e = 0; e < 8; ++e) to[(int64_t)e * rows] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          }
        }
      }
      if (live && (two || (small ? warp == 0 : x == 0))) {
        if (!final) a.part_ml[prow + i] = make_float2(m, l);
        else if (a.lse != nullptr) a.lse[out] = (m + log2f(l) - kShift) * 0.6931471805599453f;
      }
      tc_fence_before();
      cur = nxt;
      by = by_next;
      i0 = i_next;
    } while (cur.item != nullptr);
    if (!ok && lane == 0) rows_fail(a, flag, kRowsSoftmax);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

using RowsKernel = void (*)(const RowsArgs, const CUtensorMap, const CUtensorMap);
struct RowsVariant {
  RowsKernel kern;
  size_t smem;
};
// (SPLIT kernels wait for HBM: one for all scores)
template <int D, int KIND>
RowsVariant rows_variant(bool split, bool scored) {
  RowsKernel kern = scored ? rows_attend<D, KIND, false, true> : rows_attend<D, KIND, false, false>;
  if constexpr (KIND != kE4m3)
    if (split) kern = rows_attend<D, KIND, true, true>;
  return {kern, rows_smem<D, KIND>()};
}
// The kernels of a pool type, each in a file of its own (rows_attend_*.cu).
RowsVariant rows_variant_bf16(int d, bool split, bool scored);
RowsVariant rows_variant_f16(int d, bool split, bool scored);
RowsVariant rows_variant_e4m3(int d, bool split, bool scored);

}  // namespace kvsel
