// softmax_tc.cuh -- one key tile's step of an online softmax over scores in tensor memory, one
// query row per thread (TMEM lane): what the window attention's forward and the attention behind a
// shared prefix have in common.
#pragma once

#include <math.h>

#include "window_tc.cuh"

namespace psa {

constexpr float kLn2 = 0.69314718055994530942f;

// The running maximum m (log2 units) takes in a tile's, mx; O (at tO) and the sum l are rescaled
// if it grew by more than 2^8 in a row of the warp.
template <int D>
__device__ __forceinline__ void new_maximum(uint32_t tO, float mx, bool first, float& m, float& l) {
  float alpha = 1.f;
  if (mx > m + 8.f || first) {
    // -inf - -inf: a row that has seen nothing yet has nothing to rescale
    alpha = m == -INFINITY ? 0.f : fast_exp2(m - mx);
    m = mx;
  }
  if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
    l *= alpha;
    // s_full says that every product issued before this S is done, O's among them
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float o[32];
      tmem_load32(tO + c, o);
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] *= alpha;
      tmem_store32(tO + c, o);
    }
  }
}

__device__ __forceinline__ float max32(const uint32_t* x, float mx) {
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    m0 = fmax3(m0, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
    m1 = fmax3(m1, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
  }
  return fmax3(mx, m0, m1);
}

// 2^(x sl - base) of 32 scores, packed into the first half of `to`, and their sum.
__device__ __forceinline__ void exp32(const uint32_t* x, uint32_t* to, float2 sl, float2 nm, float2& l01,
                                      float2& l23) {
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    const float2 x01 = __ffma2_rn(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), sl, nm);
    const float2 x23 = __ffma2_rn(make_float2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3])), sl, nm);
    const float2 p01 = make_float2(fast_exp2(x01.x), fast_exp2(x01.y));
    const float2 p23 = make_float2(fast_exp2(x23.x), fast_exp2(x23.y));
    l01 = __fadd2_rn(l01, p01);
    l23 = __fadd2_rn(l23, p23);
    to[k / 2] = pack2(p01.x, p01.y);
    to[k / 2 + 1] = pack2(p23.x, p23.y);
  }
}

// One tile's step of the online softmax, for one row per thread: scores from tensor memory at tS,
// probabilities in bf16 back over the first half of their columns.  Tiles that every row sees
// whole keep all 128 scores in registers.
template <int D>
__device__ __forceinline__ void whole_step(uint32_t tS, uint32_t tO, float sl2, bool first, float& m, float& l) {
  using Chunk = uint32_t[32];
  uint32_t x[128];
#pragma unroll
  for (int c = 0; c < 128; c += 32) tmem_load32_async(tS + c, *reinterpret_cast<Chunk*>(x + c));
  tmem_wait_ld();
#pragma unroll
  for (int c = 0; c < 128; c += 32) tmem_pin(*reinterpret_cast<Chunk*>(x + c));
  float mx = -INFINITY;
#pragma unroll
  for (int c = 0; c < 128; c += 32) mx = max32(x + c, mx);
  new_maximum<D>(tO, mx * sl2, first, m, l);
  const float2 sl = make_float2(sl2, sl2), nm = make_float2(-m, -m);
  float2 l01 = make_float2(0.f, 0.f), l23 = l01;
#pragma unroll
  for (int c = 0; c < 128; c += 32) exp32(x + c, x + c / 2, sl, nm, l01, l23);
  l += (l01.x + l01.y) + (l23.x + l23.y);
#pragma unroll
  for (int c = 0; c < 64; c += 16) tmem_store16_async(tS + c, x + c);
}

// The others: the columns in use, 32 at a time, once for the maximum and once for the
// exponentials (holding them all costs the step above its registers: 732 -> 969 us at 16384
// causal).  lo, hi, sk: the row's limits relative to the tile (visible32).
template <int D>
__device__ __forceinline__ void masked_step(uint32_t tS, uint32_t tO, int cols, int lo, int hi, int sk, float sl2,
                                            bool first, float& m, float& l) {
  uint32_t x[32];
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < cols; c += 32) {
    tmem_load32_async(tS + c, x);
    tmem_wait_ld();
    tmem_pin(x);
    hide(x, visible32(lo - c, hi - c, sk - c));
    mx = max32(x, mx);
  }
  new_maximum<D>(tO, mx * sl2, first, m, l);
  const float base = m == -INFINITY ? 0.f : m;
  const float2 sl = make_float2(sl2, sl2), nm = make_float2(-base, -base);
  float2 l01 = make_float2(0.f, 0.f), l23 = l01;
#pragma unroll 1
  for (int c = 0; c < cols; c += 32) {
    tmem_load32_async(tS + c, x);
    tmem_wait_ld();
    tmem_pin(x);
    hide(x, visible32(lo - c, hi - c, sk - c));
    exp32(x, x, sl, nm, l01, l23);
    tmem_store16_async(tS + c / 2, x);  // over columns that have been read
  }
  l += (l01.x + l01.y) + (l23.x + l23.y);
}

}  // namespace psa
