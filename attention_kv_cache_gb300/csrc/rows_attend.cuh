// Attention of many query rows over one request's cached rows, on the 5th-generation tensor cores.
//
// Both calls that have many rows for the same keys run this kernel: the new tokens of a request (kvsel_chunk_attend) and the
// requests of a group over the prefix they share (kvsel_prefix_attend).  The query rows of a KV head are its G query heads of
// every token (request), laid end to end; an item is up to 256 of them, two tiles of 128 that share every K and V tile, and
// the keys that they see, in steps of 128.  All items' steps of all KV heads, laid end to end, are dealt evenly to one CTA per
// SM; a piece is what a CTA has of an item.  Pieces that are not a whole item leave partial sums, which rows_join merges.
//
// Roles of the 16 warps: 0-3 and 4-7 softmax of tile A and B, a thread per query row; 8-11 load K and V; 12 issues the
// products.  S = Q K^T goes to TMEM; the softmax reads it, keeps an exponent offset that moves only when a row's largest
// score passes it by 2^lag (so O is rescaled rarely) and writes the weights over S as 16-bit values, which O += P V takes from
// TMEM with V as it lies.  P V of one tile and S of the other are issued in alternation, as the prefill kernel does.
//
// SPLIT (the shared prefix): weights are a high and a low 16-bit part, as in the decode kernel whose results it must match;
// the steps wait for HBM there, so the third product is free up to 256 rows.  Without it (chunks, bound by the tensor
// cores) a weight is rounded once, 2^-9 of it over bf16 and 2^-12 over fp16 products.
// Factors on the weights as in paged_attend.cuh: 2^-8 over bf16 and 2^13 over fp16 products; without SPLIT it is taken by the
// exponent, whose rounding at 13 (2^-21 of a weight) is far below the weight's own.
//
// K and V come by cp.async, a warp per 32 rows, whole rows at a time, into the 128-byte swizzled layout of the products: any
// page size, order and stride.  An e4m3 pool's rows pass through registers, where they become fp16.
//
// Rows that some token of the item does not see may hold anything: their scores are replaced, and where a V row in such a
// step is not finite its bad values are zeros in shared memory (0 times infinity is no number) and are added to the rows that
// do see it by hand.
#pragma once

#include "paged_attend.cuh"
#include "rows.cuh"

namespace kvsel {

constexpr int kRowsThreads = 512;
constexpr int kTileRows = 128, kTileKeys = 128;
constexpr uint32_t kHalf = 16384;                // bytes of 128 rows of 64 16-bit values
template <int D>
__host__ __device__ constexpr uint32_t rows_tile_bytes() { return D / 64 * kHalf; }
// shared memory: Q_A | Q_B | K stages | V stages, then barriers and the steps' words
template <int D>
__host__ __device__ constexpr uint32_t rows_bar_off() { return 6 * rows_tile_bytes<D>(); }
constexpr uint32_t kRowsBars = 16;
template <int D>
constexpr size_t rows_smem() { return rows_bar_off<D>() + kRowsBars * 8 + 64 + 2 * 4 * 16 + 1024; }

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

// The pieces of a CTA, in order: every role walks them by itself.
struct RowsPiece {
  const RowsItem* item;
  int32_t g, s0, s1;             // KV head, the item's steps [s0, s1) here
  __device__ bool starts() const { return s0 == 0; }
  __device__ bool ends() const { return s1 == item->steps; }
};
struct RowsWalk {
  int64_t x, x1;
  int32_t g, at, s, n_items;
  __device__ void begin(const RowsArgs& a, int cta, int64_t W, int N) {
    n_items = a.plan->n_items;
    x = lane_begin64(cta, W, N);
    x1 = lane_begin64(cta + 1, W, N);
    const RowsStart st = a.starts[cta];
    g = st.g;
    at = st.item;
    s = st.step;
  }
  __device__ bool next(const RowsArgs& a, RowsPiece& p) {
    if (x >= x1) return false;
    for (;;) {
      if (at == n_items) at = 0, ++g;
      p.item = a.items + at;
      if (p.item->steps > 0) break;            // (the x left says that there is one)
      ++at;
    }
    p.g = g;
    p.s0 = s;
    p.s1 = (int)min((int64_t)p.item->steps, s + (x1 - x));
    x += p.s1 - s;
    s = 0;
    ++at;
    return true;
  }
};

// Whether a step's keys that are loaded include one that some row of the item does not see.
__device__ __forceinline__ bool rows_partial(int lo, int hi, int full_lo, int full_hi, int t0) {
  return max(t0, lo) < full_lo || min(t0 + kTileKeys, hi) > full_hi;
}
// Adds to this thread's O (TMEM at `o`) the values of V rows that are not finite and that the thread's row sees.
template <int D, int KIND>
__device__ __noinline__ void add_bad_rows(const RowsArgs& a, const uint8_t* vbase, int table, int t0, int pos, uint4 bad, uint32_t o,
                                          bool fresh) {
  const uint32_t word[4] = {bad.x, bad.y, bad.z, bad.w};
  const int low = a.window > 0 ? pos + 1 - a.window : 0;
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
__device__ __forceinline__ float rows_max64(const float* v) {
  float mp[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float* c = v + 8 * k;
    mp[k] = fmaxf(max3(max3(c[0], c[1], c[2]), c[3], c[4]), max3(c[5], c[6], c[7]));
  }
  return max3(max3(mp[0], mp[1], mp[2]), max3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
}
template <int KIND>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
  float a, b;
  return pack_hi<KIND>(x, y, a, b);
}

// Weights of 64 scores, 2^(mul z - m) times the factor, as 16-bit pairs: hi (and lo with SPLIT); returns their sum.
// Without SPLIT the factor is in `nm` and the sum, and `hi` may be the scores' own registers (word c is written after v[2 c]
// and v[2 c + 1] are read).
template <int KIND, bool SPLIT>
__device__ __forceinline__ float rows_weights(const float* v, float mul, float nm, uint32_t* hi, uint32_t* lo) {
  const float2 m2 = make_float2(mul, mul), n2 = make_float2(nm, nm);
  float2 sp[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) sp[k] = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    const float2 t = __ffma2_rn(make_float2(v[2 * c], v[2 * c + 1]), m2, n2);
    const float2 p = make_float2(ex2(t.x), ex2(t.y));
    sp[c & 3] = __fadd2_rn(sp[c & 3], p);
    if constexpr (SPLIT) {
      constexpr float unit = weight_unit<KIND>();
      float r0, r1;
      hi[c] = pack_hi<KIND>(p.x * unit, p.y * unit, r0, r1);
      lo[c] = pack16<KIND>(r0, r1);
    } else {
      hi[c] = pack16<KIND>(p.x, p.y);
    }
  }
  const float2 s = __fadd2_rn(__fadd2_rn(sp[0], sp[1]), __fadd2_rn(sp[2], sp[3]));
  return s.x + s.y;
}

template <int D, int KIND, bool SPLIT>
__global__ void __launch_bounds__(kRowsThreads, 1) rows_attend(const __grid_constant__ RowsArgs a) {
  using namespace sm100;
  constexpr uint32_t TB = rows_tile_bytes<D>();
  constexpr int RB = row_bytes<D, KIND>(), CPR = RB / 16;
  // TMEM: tile X in {0, 1}: S (the weights over it) at 256 X, O at 256 X + 128
  constexpr uint32_t kSCol = 0, kOCol = 128, kTileCols = 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_addr(sbase), bars = base + rows_bar_off<D>();
  const uint32_t kOff = 2 * TB, vOff = 4 * TB;
  auto k_full = [&](int s) { return bars + 8u * s; };
  auto k_empty = [&](int s) { return bars + 8u * (2 + s); };
  auto v_full = [&](int s) { return bars + 8u * (4 + s); };
  auto v_empty = [&](int s) { return bars + 8u * (6 + s); };
  auto s_full = [&](int x) { return bars + 8u * (8 + x); };
  auto p_full = [&](int x) { return bars + 8u * (10 + x); };
  auto pv_done = [&](int x) { return bars + 8u * (12 + x); };
  auto q_full = [&](int x) { return bars + 8u * (14 + x); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(sbase + rows_bar_off<D>() + kRowsBars * 8);
  uint32_t* tslot = misc;
  volatile uint32_t* flag = misc + 1;
  volatile uint32_t* o_begun = misc + 2;           // [2]: O of the piece holds values before its first product
  const uint32_t drain = smem_addr(misc + 4);      // (8-byte aligned)
  uint32_t* seen_w = misc + 16;                    // [4][4]: rows of a step that were loaded, by steps of the CTA modulo 4
  uint32_t* bad_w = misc + 32;                     // [4][4]: rows whose V is not finite, where that matters
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  wait_for_earlier_kernels();
  let_later_kernels_start();
  const int64_t W = a.plan->steps * a.h_kv;
  const int N = (int)min((int64_t)a.grid, W), cta = blockIdx.x;
  if (cta >= N) return;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(k_full(s), 4);                     // one arrival per loader warp
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), 4);
      mbar_init(v_empty(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), 4);                     // one arrival per softmax warp of the tile
      mbar_init(pv_done(s), 1);
      mbar_init(q_full(s), 4);
    }
    mbar_init(drain, 1);
    *flag = 0;
    o_begun[0] = o_begun[1] = 0;
    fence_barrier_init();
  }
  if (warp == 12) tmem_alloc(smem_addr(tslot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  // registers: 512 x 128 at the launch; the rows' threads hold 128 scores
  constexpr int kRegRows = KIND == kE4m3 ? 168 : 184, kRegLoad = KIND == kE4m3 ? 112 : 80, kRegMma = 64;
  static_assert(256 * kRegRows + 128 * kRegLoad + 128 * kRegMma <= 512 * 128, "the shares fit what the block was launched with");
  RowsWalk walk;
  RowsPiece p;

  if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegLoad));
    walk.begin(a, cta, W, N);
    // ---------------------------------------------------------------- loaders: rows 32 w .. 32 w + 31 of every step
    const int w = warp - 8;
    // a step to load: this lane's row of it
    struct Row {
      int32_t id, within, g, table, t0;
      bool need, check, more;
    };
    bool have = walk.next(a, p);
    int s = have ? p.s0 : 0;
    auto look = [&]() -> Row {
      Row r{0, 0, 0, 0, 0, false, false, false};
      if (!have) return r;
      const RowsItem& it = *p.item;
      r.more = true;
      r.t0 = it.k0 + kTileKeys * s;
      const int t = r.t0 + 32 * w + lane;
      r.need = t >= it.lo && t < it.hi;
      r.g = p.g;
      r.table = it.table;
      r.check = rows_partial(it.lo, it.hi, it.full_lo, it.full_hi, r.t0);
      if (r.need) {
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
    bool ok = true;
    Row next = look();
    if constexpr (KIND != kE4m3) {
      uint32_t issued = 0, told = 0, check = 0;      // tiles (K and V of every step in turn); bit i & 7: V to be checked
      // the oldest tile not told of is there: fence, arrive
      auto tell = [&]() {
        switch (issued - told) {                     // (cp.async groups may end in order only)
          case 1: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
          case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
          case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
          default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        }
        const uint32_t step = told >> 1, stage = step & 1;
        if ((told & 1) && ((check >> (told & 7)) & 1)) {
          // what this lane copied is searched for values that are not finite, 0 in their place
          constexpr int KPI = 32 / CPR;
          const int c = lane % CPR;
          uint32_t bad = 0;
#pragma unroll 1
          for (int i = 0; i < 32 / KPI; ++i) {
            const int x = i * KPI + lane / CPR;
            uint4* at = reinterpret_cast<uint4*>(sbase + vOff + stage * TB + (c >> 3) * kHalf + (32 * w + x) * 128 + (((c & 7) ^ (x & 7)) << 4));
            uint4 y = *at;
            uint32_t* h = reinterpret_cast<uint32_t*>(&y);
            constexpr uint32_t ex = KIND == kBf16 ? 0x7f80u : 0x7c00u;
            bool hit = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((h[e] & ex) == ex) h[e] &= 0xffff0000u, hit = true;
              if ((h[e] & (ex << 16)) == (ex << 16)) h[e] &= 0xffffu, hit = true;
            }
            if (hit) *at = y, bad |= 1u << x;
          }
          bad = __reduce_or_sync(0xffffffffu, bad);
          if (lane == 0) bad_w[(step & 3) * 4 + w] = bad;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive((told & 1) ? v_full(stage) : k_full(stage));
        ++told;
      };
      while (next.more && ok) {
        const Row r = next;
        const bool fine = r.need && r.id >= 0 && r.id < a.n_pages;
        if (r.need && !fine) set_device_error(a.err, KVSEL_ERR_DEVICE, (uint32_t)r.table);
        const int64_t off = (fine ? (int64_t)r.id * a.page_stride + (int64_t)r.within * a.row_stride : 0) * 2;
        const uint32_t rows = __ballot_sync(0xffffffffu, fine);
        next = look();
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t step = issued >> 1, stage = step & 1, parity = ((step >> 1) & 1) ^ 1;
          const uint32_t empty = kv ? v_empty(stage) : k_empty(stage);
          while (!__all_sync(0xffffffffu, rows_test(empty, parity))) {
            if (issued != told) tell();
            else {
              ok = __all_sync(0xffffffffu, rows_wait(empty, parity, flag));
              if (!ok) break;
            }
          }
          if (!ok) break;
          if (kv == 0 && lane == 0) {
            seen_w[(step & 3) * 4 + w] = rows;
            bad_w[(step & 3) * 4 + w] = 0;
          }
          const uint8_t* from = static_cast<const uint8_t*>(kv ? a.v : a.k) + (int64_t)r.g * a.head_stride * 2;
          const uint32_t dst = base + (kv ? vOff : kOff) + stage * TB;
          constexpr int KPI = 32 / CPR;
          const int c = lane % CPR;
#pragma unroll
          for (int i = 0; i < 32 / KPI; ++i) {
            const int x = i * KPI + lane / CPR;
            const int64_t ox = __shfl_sync(0xffffffffu, off, x) + c * 16;
            cp_async16(dst + (c >> 3) * kHalf + (32 * w + x) * 128 + (((c & 7) ^ (x & 7)) << 4), from + ox, (rows >> x) & 1u);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (kv && r.check) check |= 1u << (issued & 7);
          else check &= ~(1u << (issued & 7));
          ++issued;
        }
      }
      while (ok && told != issued) tell();
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
      // rows through registers, a tile ahead: 16 e4m3 values become two chunks of 8 fp16 values
      constexpr int KPI = 32 / CPR, NI = 32 / KPI;
      uint4 kr[NI], vr[NI];
      const int c = lane % CPR;
      struct Fetch {
        int64_t off;
        uint32_t rows;
        int g;
      };
      auto resolve = [&](const Row& r) -> Fetch {
        const bool fine = r.need && r.id >= 0 && r.id < a.n_pages;
        if (r.need && !fine) set_device_error(a.err, KVSEL_ERR_DEVICE, (uint32_t)r.table);
        return {fine ? (int64_t)r.id * a.page_stride + (int64_t)r.within * a.row_stride : 0, __ballot_sync(0xffffffffu, fine), r.g};
      };
      auto fetch = [&](const Fetch& f, const void* pool, uint4* to) {
        const uint8_t* from = static_cast<const uint8_t*>(pool) + (int64_t)f.g * a.head_stride + c * 16;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int x = i * KPI + lane / CPR;
          const int64_t ox = __shfl_sync(0xffffffffu, f.off, x);
          to[i] = (f.rows >> x) & 1u ? *reinterpret_cast<const uint4*>(from + ox) : make_uint4(0, 0, 0, 0);
        }
      };
      uint32_t step = 0;
      auto store = [&](uint4* y, uint32_t dst, bool check) -> uint32_t {
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int x = i * KPI + lane / CPR;
          uint32_t* h = reinterpret_cast<uint32_t*>(&y[i]);
          if (check) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t nan = __vcmpeq4(h[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
              if (nan) h[e] &= ~nan, bad |= 1u << x;
            }
          }
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) e4m3x4_to_f16(h[e], o[2 * e], o[2 * e + 1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int cc = 2 * c + e;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (cc >> 3) * kHalf + (32 * w + x) * 128 + (((cc & 7) ^ (x & 7)) << 4)),
                         "r"(o[4 * e]), "r"(o[4 * e + 1]), "r"(o[4 * e + 2]), "r"(o[4 * e + 3]) : "memory");
          }
        }
        return bad;
      };
      Row r = next;
      Fetch f{0, 0, 0};
      if (r.more) {
        f = resolve(r);
        fetch(f, a.k, kr);
      }
      while (r.more && ok) {
        fetch(f, a.v, vr);
        next = look();
        const uint32_t stage = step & 1, parity = ((step >> 1) & 1) ^ 1;
        ok = __all_sync(0xffffffffu, rows_wait(k_empty(stage), parity, flag));
        if (!ok) break;
        if (lane == 0) seen_w[(step & 3) * 4 + w] = f.rows;
        store(kr, base + kOff + stage * TB, false);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full(stage));
        const bool check = r.check;
        r = next;
        if (r.more) {
          f = resolve(r);
          fetch(f, a.k, kr);
        }
        ok = __all_sync(0xffffffffu, rows_wait(v_empty(stage), parity, flag));
        if (!ok) break;
        const uint32_t bad = __reduce_or_sync(0xffffffffu, store(vr, base + vOff + stage * TB, check));
        if (lane == 0) bad_w[(step & 3) * 4 + w] = bad;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full(stage));
        ++step;
      }
    }
    if (!ok && lane == 0) rows_fail(a, flag, kRowsLoader);
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegMma));
    // ---------------------------------------------------------------- products
    if (warp == 12 && lane == 0) {
      walk.begin(a, cta, W, N);
      constexpr uint32_t idesc_s = rows_idesc<KIND>(128, 128), idesc_o = rows_idesc<KIND>(128, D) | kUmmaBMajorMN;
      constexpr int KS = D / 16, KP = kTileKeys / 16 * (SPLIT ? 2 : 1);
      bool ok = true, any = false;
      // a step: its number among the CTA's, whether tile B has rows, first of its piece
      struct Step {
        int i;
        bool two, first, more;
      };
      bool have = walk.next(a, p);
      int s = have ? p.s0 : 0, count = 0;
      auto advance = [&]() -> Step {
        Step r{count, false, false, have};
        if (!have) return r;
        r.two = p.item->rows > kTileRows;
        r.first = s == p.s0;
        ++count;
        if (++s == p.s1) {
          have = walk.next(a, p);
          s = p.s0;
        }
        return r;
      };
      uint32_t nq[2] = {0, 0}, npv[2] = {0, 0}, np[2] = {0, 0};      // phases waited for, by tile
      // S of a step may start once K has landed, the tile's queries are there, and its last P V (which reads the same TMEM
      // columns) is done; P V once V has landed and the weights are written
      auto s_ready = [&](int x, const Step& t) {
        if (!rows_wait(k_full(t.i & 1), (t.i >> 1) & 1, flag)) return false;
        if (t.first) {
          if (!rows_wait(q_full(x), nq[x] & 1, flag)) return false;
          ++nq[x];
        }
        return npv[x] == 0 || rows_wait(pv_done(x), (npv[x] - 1) & 1, flag);
      };
      auto pv_ready = [&](int x, const Step& t) {
        if (!rows_wait(v_full(t.i & 1), (t.i >> 1) & 1, flag) || !rows_wait(p_full(x), np[x] & 1, flag)) return false;
        ++np[x];
        return true;
      };
      auto s_step = [&](int x, const Step& t, int kk) {
        const uint32_t sq = base + x * TB, sk = base + kOff + (t.i & 1) * TB, off = (kk >> 2) * kHalf + (kk & 3) * 32;
        umma_bf16(tmem + x * kTileCols + kSCol, umma_desc_sw128(sq + off), umma_desc_sw128(sk + off), idesc_s, kk > 0);
      };
      auto pv_step = [&](int x, const Step& t, int kk, bool keep) {
        const uint32_t sv = base + vOff + (t.i & 1) * TB;
        umma_bf16_ta(tmem + x * kTileCols + kOCol, tmem + x * kTileCols + kSCol + kk * 8,
                     umma_desc_sw128_mn(sv + (kk & 7) * 2048, kHalf), idesc_o, (keep || kk > 0) ? 1u : 0u);
      };
      // a commit covers every product before it
      auto s_done = [&](int x, const Step& t) {
        umma_commit(s_full(x));
        if (x == 1 || !t.two) umma_commit(k_empty(t.i & 1));
        any = true;
      };
      auto pv_end = [&](int x, const Step& t) {
        umma_commit(pv_done(x));
        if (x == 1 || !t.two) umma_commit(v_empty(t.i & 1));
        ++npv[x];
      };
      auto s_alone = [&](int x, const Step& t) {
        if (!s_ready(x, t)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) s_step(x, t, kk);
        s_done(x, t);
        return true;
      };
      Step cur = advance();
      ok = cur.more && s_alone(0, cur) && (!cur.two || s_alone(1, cur));
      while (cur.more && ok) {
        const Step nxt = advance();
        if (!(ok = pv_ready(0, cur))) break;
        tc_fence_after();
        const bool keep0 = !cur.first || o_begun[0] != 0;
#pragma unroll
        for (int kk = 0; kk < KP; ++kk) pv_step(0, cur, kk, keep0);
        pv_end(0, cur);
        const bool pvb = cur.two, sa = nxt.more;
        if (pvb && !(ok = pv_ready(1, cur))) break;
        if (sa && !(ok = s_ready(0, nxt))) break;
        tc_fence_after();
        if (pvb && sa) {
          const bool keep1 = !cur.first || o_begun[1] != 0;
#pragma unroll
          for (int kk = 0; kk < (KP > KS ? KP : KS); ++kk) {
            if (kk < KP) pv_step(1, cur, kk, keep1);
            if (kk < KS) s_step(0, nxt, kk);
          }
        } else if (pvb) {
          const bool keep1 = !cur.first || o_begun[1] != 0;
#pragma unroll
          for (int kk = 0; kk < KP; ++kk) pv_step(1, cur, kk, keep1);
        } else if (sa) {
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) s_step(0, nxt, kk);
        }
        if (pvb) pv_end(1, cur);
        if (sa) s_done(0, nxt);
        if (sa && nxt.two) ok = s_alone(1, nxt);
        cur = nxt;
      }
      if (!ok) rows_fail(a, flag, kRowsMma);
      if (any) {
        umma_commit(drain);
        if (!mbar_wait(drain, 0)) set_device_error(a.err, KVSEL_ERR_TIMEOUT, kRowsDrain);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegRows));
    walk.begin(a, cta, W, N);
    // ---------------------------------------------------------------- softmax, a thread per query row
    const int x = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t tm = tmem + ((uint32_t)(quarter * 32) << 16) + x * kTileCols;
    const float kShift = SPLIT ? 0.f : (KIND == kBf16 ? -8.f : 13.f);
    constexpr float kLag = weight_lag<KIND>();
    auto live_piece = [&](RowsPiece& to) {          // the next piece in which this tile has rows
      while (walk.next(a, to))
        if (x == 0 || to.item->rows > kTileRows) return true;
      return false;
    };
    // this thread's query row of a piece: into shared memory, swizzled; returns the factor taken out of it
    auto load_q = [&](const RowsPiece& t) -> float {
      const int i = x * kTileRows + row, r = t.item->row0 + i;
      const bool live = i < t.item->rows;
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
    const int64_t x_begin = walk.x;                 // steps are numbered as the loaders number them
    RowsPiece cur;
    bool more = live_piece(cur);
    float by = more ? load_q(cur) : 1.f;
    uint32_t n = 0;                                 // steps of this tile so far
    bool ok = true;
    int64_t x_end = walk.x;                         // step number behind the current piece
    while (more && ok) {
      const RowsItem& it = *cur.item;
      const int k0 = it.k0, k_lo = it.lo, k_hi = it.hi, full_lo = it.full_lo, full_hi = it.full_hi;
      const int i = x * kTileRows + row, r = it.row0 + i, tok = r / a.G, h = cur.g * a.G + (r - tok * a.G);
      const bool live = i < it.rows;
      const int pos = !live ? -1 : a.prefix ? (int)a.lens[it.token0 + tok] - 1 : it.base + tok;
      const int low = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
      const float ksc = a.scale * (a.k_scale != nullptr ? a.k_scale[cur.g] : 1.f);
      const float sc = ksc * by * (a.softcap != 0.f ? 1.f : kLog2e);
      const float slope = a.slopes != nullptr && live ? a.slopes[h] * kLog2e : 0.f;
      const float cap2 = a.softcap * kLog2e, icap = a.softcap != 0.f ? 1.f / a.softcap : 0.f;
      const bool general = a.softcap != 0.f || a.slopes != nullptr || !(ksc > 0.f);
      const bool idle = __all_sync(0xffffffffu, !live);         // a warp of padding alone
      float m = -INFINITY, mo = 0.f, l = 0.f;
      bool begun = false;
      if (lane == 0 && quarter == 0) o_begun[x] = 0;            // (before the piece's first weights are told of)
      int step = (int)(x_end - x_begin) - (cur.s1 - cur.s0);    // its number among the CTA's steps
      for (int s = cur.s0; s < cur.s1; ++s, ++step, ++n) {
        ok = __all_sync(0xffffffffu, rows_wait(s_full(x), n & 1, flag));
        if (!ok) break;
        tc_fence_after();
        const int t0 = k0 + kTileKeys * s;
        const uint4 there = *reinterpret_cast<const uint4*>(&seen_w[(step & 3) * 4]);
        const bool whole = t0 >= full_lo && t0 + kTileKeys <= full_hi && (there.x & there.y & there.z & there.w) == 0xffffffffu;
        if (rows_partial(k_lo, k_hi, full_lo, full_hi, t0)) {
          ok = __all_sync(0xffffffffu, rows_wait(v_full(step & 1), (step >> 1) & 1, flag));
          if (!ok) break;
          const uint4 bad = *reinterpret_cast<const uint4*>(&bad_w[(step & 3) * 4]);
          if ((bad.x | bad.y | bad.z | bad.w) != 0) {
            const bool fresh = s == cur.s0;
            add_bad_rows<D, KIND>(a, static_cast<const uint8_t*>(a.v) + (int64_t)cur.g * a.head_stride * elem_bytes<KIND>(), it.table, t0, pos,
                                  bad, tm + kOCol, fresh);
            if (fresh) begun = true;
            if (fresh && lane == 0 && quarter == 0) o_begun[x] = 1;
          }
        }
        if (!idle) {
          // keys of the step that the row sees, by 32
          uint32_t see[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
          if (!whole) {
            const int from = low - t0, to = pos + 1 - t0;
            const uint32_t word[4] = {there.x, there.y, there.z, there.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int lo = min(32, max(0, from - 32 * k)), hi = min(32, max(0, to - 32 * k));
              const uint32_t below_hi = hi >= 32 ? 0xffffffffu : (1u << hi) - 1u, below_lo = lo >= 32 ? 0xffffffffu : (1u << lo) - 1u;
              see[k] = live ? word[k] & below_hi & ~below_lo : 0u;
            }
          }
          const float mul = general ? 1.f : sc;
          // 64 scores of the step (its half H) as they are compared: capped and biased, those not seen at -inf
          auto scores = [&](float* z, int half) {
            if (general) {
              const float d0 = (float)(t0 + 64 * half - pos);
#pragma unroll
              for (int c = 0; c < 64; ++c) {
                float y = z[c] * sc;
                if (a.softcap != 0.f) y = cap2 * tanh_fast(y * icap);
                z[c] = fmaf(slope, d0 + (float)c, y);
              }
            }
            if (!whole) {
              const uint32_t w0 = half ? see[2] : see[0], w1 = half ? see[3] : see[1];
#pragma unroll
              for (int c = 0; c < 64; ++c) z[c] = ((c < 32 ? w0 : w1) >> (c & 31)) & 1u ? z[c] : -INFINITY;
            }
          };
          float alpha = 1.f, sum;
          auto offset = [&](float mt) {                         // where a score passes the lag, the offset moves to the largest
            if (mt > m + kLag) {
              if (m != -INFINITY) alpha = ex2(m - mt);          // (nothing to rescale before the first)
              m = mo = mt;
            }
          };
          if constexpr (SPLIT) {
            // the first half is read twice, so that a thread never holds both and their parts
            uint32_t r[64], hi[32], lo[32];
            float* z = reinterpret_cast<float*>(r);
            tmem_ld64_async(tm + kSCol, r);
            tmem_wait_ld64(r);
            scores(z, 0);
            const float m0 = rows_max64(z);
            tmem_ld64_async(tm + kSCol + 64, r);
            tmem_wait_ld64(r);
            scores(z, 1);
            offset(fmaxf(m0, rows_max64(z)) * mul);             // (mul > 0: the largest stays the largest)
            sum = rows_weights<KIND, true>(z, mul, kShift - mo, hi, lo);
            tmem_st32(tm + kSCol + 96, lo);
            tmem_ld64_async(tm + kSCol, r);
            tmem_wait_ld64(r);
            tmem_st32(tm + kSCol + 32, hi);
            scores(z, 0);
            sum += rows_weights<KIND, true>(z, mul, kShift - mo, hi, lo);
            tmem_st32(tm + kSCol + 64, lo);
            tmem_st32(tm + kSCol, hi);
          } else {
            uint32_t rv[64], rw[64];
            tmem_ld64_async(tm + kSCol + 64, rv);
            tmem_ld64_async(tm + kSCol, rw);
            tmem_wait_ld64(rv);                                 // one wait covers both loads
            reg_tie64(rw);
            float* v = reinterpret_cast<float*>(rv);
            float* u = reinterpret_cast<float*>(rw);
            scores(u, 0);
            scores(v, 1);
            offset(fmaxf(rows_max64(u), rows_max64(v)) * mul);
            sum = rows_weights<KIND, false>(u, mul, kShift - mo, rw, nullptr);
            tmem_st32(tm + kSCol, rw);
            sum += rows_weights<KIND, false>(v, mul, kShift - mo, rv, nullptr);
            tmem_st32(tm + kSCol + 32, rv);
          }
          l = l * alpha + sum;
          // O of the step before is final (this step's S was issued behind its P V)
          if ((s > cur.s0 || begun) && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
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
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(x));
      }
      if (!ok) break;
      // the next piece's queries (this piece's last S is done with them), then this one's result
      RowsPiece nxt;
      const bool has_next = live_piece(nxt);
      float by_next = 1.f;
      const int64_t nx_end = walk.x;
      if (has_next) by_next = load_q(nxt);
      ok = __all_sync(0xffffffffu, rows_wait(pv_done(x), (n - 1) & 1, flag));
      if (!ok) break;
      tc_fence_after();
      if (!idle) {
        const bool final = !a.prefix && cur.starts() && cur.ends();
        const float vsc = a.v_scale != nullptr ? a.v_scale[cur.g] : 1.f;
        const float f = !final ? 1.f : l == 0.f ? 0.f : (SPLIT ? vsc / weight_unit<KIND>() : vsc) / l;
        const int64_t out = ((int64_t)it.token0 + tok) * a.h_q + h;
        const int64_t prow = rows_part(a, cta, cur.starts(), cur.g, it);
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float y[32];
          tmem_ld32(tm + kOCol + c, y);
          if (!live) continue;
          if (final) {
            uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + out * D + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t b[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float y0 = y[8 * e + 2 * k] * f, y1 = y[8 * e + 2 * k + 1] * f;
                b[k] = a.out_f16 ? pack16<kF16>(y0, y1) : pack16<kBf16>(y0, y1);
              }
              to[e] = make_uint4(b[0], b[1], b[2], b[3]);
            }
          } else {
            // four values of a row next to those of the next row
            float4* to = reinterpret_cast<float4*>(a.part + prow * D) + (int64_t)(c / 4) * it.rows + i;
#pragma unroll
            for (int e = 0; e < 8; ++e) to[(int64_t)e * it.rows] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          }
        }
        if (live) {
          if (!final) a.part_ml[prow + i] = make_float2(m, l);
          else if (a.lse != nullptr) a.lse[out] = (m + log2f(l) - kShift) * 0.6931471805599453f;
        }
      }
      tc_fence_before();
      cur = nxt;
      more = has_next;
      by = by_next;
      x_end = nx_end;
    }
    if (!ok && lane == 0) rows_fail(a, flag, kRowsSoftmax);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

using RowsKernel = void (*)(const RowsArgs);
struct RowsVariant {
  RowsKernel kern;
  size_t smem;
};
template <int D, int KIND>
RowsVariant rows_variant(bool split) {
  return {split ? rows_attend<D, KIND, true> : rows_attend<D, KIND, false>, rows_smem<D>()};
}
// The kernels of a pool type, each in a file of its own (rows_attend_*.cu).
RowsVariant rows_variant_bf16(int d, bool split);
RowsVariant rows_variant_f16(int d, bool split);
RowsVariant rows_variant_e4m3(int d, bool split);

}  // namespace kvsel
