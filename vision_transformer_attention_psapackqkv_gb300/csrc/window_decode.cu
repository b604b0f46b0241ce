// window_decode.cu -- attention of one query token per sequence over a cache, with a sliding
// window and first tokens that stay visible; the cache in bf16, or in 4 bits (kv_cache.cu
// has the format).
//
//   o_h = sum_j softmax_j(scale q_h . k_j) v_j over the visible rows j of the cache
//
// Bound by memory: every visible row of K and V is read once, for all query heads that
// share it.  So the heads of a group are the 16 rows of a tensor-core tile (m16n8k16; the
// work is at most a fifth of what those units can do at this rate, and there is nothing a
// larger instruction could fill), and the cache goes from memory straight into registers as
// the B operand of the products, without shared memory or a barrier between a load and its
// use.  That works because the order of the inner index of Q K^T (channels), and the column
// order of P V (channels), are free: each lane takes 16 neighbouring bytes of a row and
// Q's fragment (the output's columns) is permuted to match.  For P V the two keys of a
// pair sit in two registers of one lane, and one byte permute per product register puts
// them side by side.
//
// Keys are cut into blocks of 16; the visible blocks (the sinks', then the window's) are
// dealt to gridDim.x CTAs in contiguous parts and inside a CTA to its warps in turn.  Every
// warp keeps its own running maximum, sum and output; they are joined in shared memory, and
// the parts of a sequence by a second small kernel from fp32 partial results.  The number
// of parts goes by the problem's sizes alone: enough CTAs for every SM.
//
// 4 bits: a code n becomes the bf16 number 128 + n by setting the exponent bits around it
// (0x4300 | n), and 136 is subtracted: two values in two instructions, exact.  A key's
// scale multiplies its fp32 partial score of each group of 32 channels (two products); a
// value's scale multiplies the probability before it is rounded to bf16.
#include <algorithm>

#include "lm.cuh"
#include "ptx.cuh"

namespace psa {
namespace {

constexpr int kWarps = 4;        // per CTA
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;        // query heads of a tile
constexpr int kBlock = 16;       // keys of a block
constexpr float kLog2eD = 1.4426950408889634074f;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (128 + n, 128 + n') - 136 for the nibbles n, n' at bits i4 and i4 + 16
__device__ __forceinline__ uint32_t nibbles_bf16(uint32_t x, int i4) {
  const uint32_t u = ((x >> i4) & 0x000F000Fu) | 0x43004300u;
  const uint32_t k136 = 0x43084308u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                   *reinterpret_cast<const __nv_bfloat162*>(&k136));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// cache reads: each byte is used once
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load4(const void* p) {
  uint32_t v;
  asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// The visible rows of sequence b: blocks 0 .. sink - 1, then first .. (count in all).
struct Blocks {
  int len, lo, sink, first, count;
  __device__ __forceinline__ Blocks(const Window& w, int b) {
    len = w.len(b);
    lo = max(0, len - 1 - w.left);
    first = lo / kBlock;
    sink = min(first, (min(w.sinks, len) + kBlock - 1) / kBlock);
    count = len > 0 ? sink + (len - 1) / kBlock - first + 1 : 0;
  }
  __device__ __forceinline__ int block(int t) const { return t < sink ? t : first + t - sink; }
};

// One lane's part of a block of 16 keys of K (lane = 4 key + t of an 8-key half) and of V
// (lane = 4 a + t: keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9; channels by a).
template <int D, bool kKv4>
struct Cache;

template <int D>
struct Cache<D, false> {
  static constexpr int NT = D / 8;  // column tiles of the output
  uint4 k[2][D / 32], v[4][D / 64];

  __device__ __forceinline__ void load_k(const DecodeArgs& a, int b, int h, int j0, int lane) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int j = min(j0 + 8 * half + (lane >> 2), a.w.nk - 1);
      const __nv_bfloat16* p = a.k.row(b, h, j) + 8 * (lane & 3);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) k[half][i] = load16(p + 32 * i);
    }
  }
  __device__ __forceinline__ void load_v(const DecodeArgs& a, int b, int h, int j0, int lane) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int j = min(j0 + 2 * (lane & 3) + (x & 1) + 8 * (x >> 1), a.w.nk - 1);
      const __nv_bfloat16* p = a.v.row(b, h, j) + 8 * (lane >> 2);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) v[x][i] = load16(p + 64 * i);
    }
  }
  // channels 32 i + 8 t + 2 s', + 1 are the lane's pair s' of products 2 i and 2 i + 1
  static __device__ __forceinline__ void load_q(const __nv_bfloat16* row, int t, uint32_t (&q)[D / 8]) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 u = row ? *reinterpret_cast<const uint4*>(row + 32 * i + 8 * t) : make_uint4(0, 0, 0, 0);
      q[4 * i] = u.x;
      q[4 * i + 1] = u.y;
      q[4 * i + 2] = u.z;
      q[4 * i + 3] = u.w;
    }
  }
  __device__ __forceinline__ void scores(const uint32_t (&q0)[D / 8], const uint32_t (&q1)[D / 8],
                                         float (&s)[2][4]) const {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      s[half][0] = s[half][1] = s[half][2] = s[half][3] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 u = k[half][i];
        const uint32_t a0[4] = {q0[4 * i], q1[4 * i], q0[4 * i + 1], q1[4 * i + 1]};
        const uint32_t a1[4] = {q0[4 * i + 2], q1[4 * i + 2], q0[4 * i + 3], q1[4 * i + 3]};
        mma16816(s[half], a0, u.x, u.y);
        mma16816(s[half], a1, u.z, u.w);
      }
    }
  }
  // rows that are not visible may hold anything (NaN times a probability of 0)
  __device__ __forceinline__ void drop_v(int x) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) v[x][i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void mix(const float (&p)[2][4], float (&o)[NT][4]) const {
    const uint32_t a[4] = {pack2(p[0][0], p[0][1]), pack2(p[0][2], p[0][3]), pack2(p[1][0], p[1][1]),
                           pack2(p[1][2], p[1][3])};
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint32_t w[4][4] = {{v[0][i].x, v[0][i].y, v[0][i].z, v[0][i].w},
                                {v[1][i].x, v[1][i].y, v[1][i].z, v[1][i].w},
                                {v[2][i].x, v[2][i].y, v[2][i].z, v[2][i].w},
                                {v[3][i].x, v[3][i].y, v[3][i].z, v[3][i].w}};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t sel = (e & 1) ? 0x7632 : 0x5410;
        mma16816(o[8 * i + e], a, __byte_perm(w[0][e / 2], w[1][e / 2], sel),
                 __byte_perm(w[2][e / 2], w[3][e / 2], sel));
      }
    }
  }
  // channel of column tile nt, column `col`
  static __device__ __forceinline__ int channel(int nt, int col) {
    return 64 * (nt / 8) + 8 * col + nt % 8;
  }
};

template <int D>
struct Cache<D, true> {
  static constexpr int NT = D / 8, G = D / 32;
  uint32_t k[2][G], v[4][G / 2];  // codes
  uint32_t ks[2][2][G / 2];       // scales of keys 8 half + 2 t, + 1: two bf16 in each word
  uint32_t vs[4][G / 2];

  static __device__ __forceinline__ void load_scales(const void* scales, long long row,
                                                     uint32_t (&s)[G / 2]) {
    const char* p = static_cast<const char*>(scales) + row * (2 * G);
    if constexpr (G == 4) {
      const uint2 u = load8(p);
      s[0] = u.x;
      s[1] = u.y;
    } else {
      s[0] = load4(p);
    }
  }
  __device__ __forceinline__ void load_k(const DecodeArgs& a, int b, int h, int j0, int lane) {
    const long long base = ((long long)b * a.w.nkv + h) * a.w.nk;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int j = min(j0 + 8 * half + (lane >> 2), a.w.nk - 1);
      const char* p = static_cast<const char*>(a.kcodes) + (base + j) * (D / 2) + (D / 8) * (lane & 3);
      if constexpr (G == 4) {
        const uint4 u = load16(p);
        k[half][0] = u.x;
        k[half][1] = u.y;
        k[half][2] = u.z;
        k[half][3] = u.w;
      } else {
        const uint2 u = load8(p);
        k[half][0] = u.x;
        k[half][1] = u.y;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        load_scales(a.kscales, base + min(j0 + 8 * half + 2 * (lane & 3) + x, a.w.nk - 1), ks[half][x]);
    }
  }
  __device__ __forceinline__ void load_v(const DecodeArgs& a, int b, int h, int j0, int lane) {
    const long long base = ((long long)b * a.w.nkv + h) * a.w.nk;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int j = min(j0 + 2 * (lane & 3) + (x & 1) + 8 * (x >> 1), a.w.nk - 1);
      const char* p = static_cast<const char*>(a.vcodes) + (base + j) * (D / 2) + (D / 16) * (lane >> 2);
      if constexpr (G == 4) {
        const uint2 u = load8(p);
        v[x][0] = u.x;
        v[x][1] = u.y;
      } else {
        v[x][0] = load4(p);
      }
      load_scales(a.vscales, base + j, vs[x]);
    }
  }
  // channels 32 g + 8 t + i and 32 g + 8 t + 4 + i are pair i of group g
  static __device__ __forceinline__ void load_q(const __nv_bfloat16* row, int t, uint32_t (&q)[D / 8]) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint4 u = row ? *reinterpret_cast<const uint4*>(row + 32 * g + 8 * t) : make_uint4(0, 0, 0, 0);
      q[4 * g] = __byte_perm(u.x, u.z, 0x5410);
      q[4 * g + 1] = __byte_perm(u.x, u.z, 0x7632);
      q[4 * g + 2] = __byte_perm(u.y, u.w, 0x5410);
      q[4 * g + 3] = __byte_perm(u.y, u.w, 0x7632);
    }
  }
  static __device__ __forceinline__ float scale_of(const uint32_t (&s)[G / 2], int g) {
    return __uint_as_float((g & 1) ? s[g / 2] & 0xffff0000u : s[g / 2] << 16);
  }
  __device__ __forceinline__ void scores(const uint32_t (&q0)[D / 8], const uint32_t (&q1)[D / 8],
                                         float (&s)[2][4]) const {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      s[half][0] = s[half][1] = s[half][2] = s[half][3] = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        // words of a = 2 t come first, those of a = 2 t + 1 after them
        const uint32_t x = __byte_perm(k[half][g / 2], k[half][G / 2 + g / 2], (g & 1) ? 0x7632 : 0x5410);
        const uint32_t a0[4] = {q0[4 * g], q1[4 * g], q0[4 * g + 1], q1[4 * g + 1]};
        const uint32_t a1[4] = {q0[4 * g + 2], q1[4 * g + 2], q0[4 * g + 3], q1[4 * g + 3]};
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        mma16816(c, a0, nibbles_bf16(x, 0), nibbles_bf16(x, 4));
        mma16816(c, a1, nibbles_bf16(x, 8), nibbles_bf16(x, 12));
        const float s0 = scale_of(ks[half][0], g), s1 = scale_of(ks[half][1], g);
        s[half][0] += c[0] * s0;
        s[half][1] += c[1] * s1;
        s[half][2] += c[2] * s0;
        s[half][3] += c[3] * s1;
      }
    }
  }
  __device__ __forceinline__ void drop_v(int x) {
#pragma unroll
    for (int i = 0; i < G / 2; ++i) vs[x][i] = 0;
  }
  __device__ __forceinline__ void mix(const float (&p)[2][4], float (&o)[NT][4]) const {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float s0 = scale_of(vs[0], g), s1 = scale_of(vs[1], g), s2 = scale_of(vs[2], g),
                  s3 = scale_of(vs[3], g);
      const uint32_t a[4] = {pack2(p[0][0] * s0, p[0][1] * s1), pack2(p[0][2] * s0, p[0][3] * s1),
                             pack2(p[1][0] * s2, p[1][1] * s3), pack2(p[1][2] * s2, p[1][3] * s3)};
      const uint32_t sel = (g & 1) ? 0x7632 : 0x5410;
      const uint32_t x = __byte_perm(v[0][g / 2], v[1][g / 2], sel);
      const uint32_t y = __byte_perm(v[2][g / 2], v[3][g / 2], sel);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma16816(o[4 * g + i], a, nibbles_bf16(x, 4 * i), nibbles_bf16(y, 4 * i));
    }
  }
  static __device__ __forceinline__ int channel(int nt, int col) {
    return 32 * (nt / 4) + 4 * col + nt % 4;
  }
};

template <int D, bool kKv4>
__global__ void __launch_bounds__(kThreads) window_decode_kernel(const DecodeArgs a) {
  using C = Cache<D, kKv4>;
  constexpr int NT = C::NT;
  __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
  __shared__ float sm_o[kRows][D + 4];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3, r = lane >> 2;
  const int group = a.w.nh / a.w.nkv, tiles = (group + kRows - 1) / kRows;
  const int b = blockIdx.z, h = blockIdx.y / tiles, g0 = (blockIdx.y % tiles) * kRows;
  const int heads = min(kRows, group - g0), h0 = h * group + g0;
  const Blocks bl(a.w, b);
  const int from = (int)((long long)bl.count * blockIdx.x / gridDim.x);
  const int to = (int)((long long)bl.count * (blockIdx.x + 1) / gridDim.x);

  uint32_t q0[D / 8], q1[D / 8];
  C::load_q(r < heads ? a.q.row(b, h0 + r, 0) : nullptr, t, q0);
  C::load_q(r + 8 < heads ? a.q.row(b, h0 + r + 8, 0) : nullptr, t, q1);
  float o[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows r, r + 8 (log2 units)
  const float sl2 = a.scale * kLog2eD;

  C c;
  int blk = from + warp;
  if (blk < to) c.load_k(a, b, h, bl.block(blk) * kBlock, lane);
  for (; blk < to; blk += kWarps) {
    const int j0 = bl.block(blk) * kBlock;
    c.load_v(a, b, h, j0, lane);
    float s[2][4];
    c.scores(q0, q1, s);
    if (blk + kWarps < to) c.load_k(a, b, h, bl.block(blk + kWarps) * kBlock, lane);
    // all 16 keys visible: inside the window, or among the sinks
    const bool whole = j0 + kBlock <= bl.len && (j0 >= bl.lo || j0 + kBlock <= a.w.sinks);
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = j0 + 8 * half + 2 * t + x;
        const bool see = whole || (j < bl.len && (j >= bl.lo || j < a.w.sinks));
        s[half][x] = see ? s[half][x] * sl2 : -INFINITY;
        s[half][2 + x] = see ? s[half][2 + x] * sl2 : -INFINITY;
        if (!see) c.drop_v(2 * half + x);
      }
    float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
    float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, m));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, m));
    }
    // the running maximum moves only when it grows by more than 2^8: output and sum share
    // the stale one, so the result is the same
    const bool grow = x0 > m0 + 8.f || x1 > m1 + 8.f;
    if (__any_sync(0xffffffffu, grow)) {
      const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
      const float f0 = n0 == -INFINITY ? 1.f : fast_exp2(m0 - n0);
      const float f1 = n1 == -INFINITY ? 1.f : fast_exp2(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        o[i][0] *= f0;
        o[i][1] *= f0;
        o[i][2] *= f1;
        o[i][3] *= f1;
      }
    }
    const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      s[half][0] = fast_exp2(s[half][0] - b0);
      s[half][1] = fast_exp2(s[half][1] - b0);
      s[half][2] = fast_exp2(s[half][2] - b1);
      s[half][3] = fast_exp2(s[half][3] - b1);
      l0 += s[half][0] + s[half][1];
      l1 += s[half][2] + s[half][3];
    }
    c.mix(s, o);
  }
  // the four lanes of a row each summed their own columns
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, m);
    l1 += __shfl_xor_sync(0xffffffffu, l1, m);
  }
  if (t == 0) {
    sm_m[warp][r] = m0;
    sm_m[warp][r + 8] = m1;
    sm_l[warp][r] = l0;
    sm_l[warp][r + 8] = l1;
  }
  __syncthreads();
  float n0 = -INFINITY, n1 = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    n0 = fmaxf(n0, sm_m[w][r]);
    n1 = fmaxf(n1, sm_m[w][r + 8]);
  }
  const float f0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - n0);
  const float f1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - n1);
  // the warps add their outputs one after another: a fixed order
  for (int w = 0; w < kWarps; ++w) {
    if (warp == w) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* d0 = &sm_o[r][C::channel(i, 2 * t + e)];
          float* d1 = &sm_o[r + 8][C::channel(i, 2 * t + e)];
          *d0 = (w == 0 ? 0.f : *d0) + o[i][e] * f0;
          *d1 = (w == 0 ? 0.f : *d1) + o[i][2 + e] * f1;
        }
    }
    __syncthreads();
  }
  for (int u = threadIdx.x; u < heads * D; u += kThreads) {
    const int row = u / D, ch = u % D;
    float n = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) n = fmaxf(n, sm_m[w][row]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      l += sm_m[w][row] == -INFINITY ? 0.f : sm_l[w][row] * fast_exp2(sm_m[w][row] - n);
    if (gridDim.x == 1) {
      a.o.row(b, h0 + row, 0)[ch] = __float2bfloat16_rn(l > 0.f ? sm_o[row][ch] / l : 0.f);
    } else {
      // partial result: D outputs relative to the maximum n, then n and the sum
      float* dst = a.ws + (((long long)b * a.w.nh + h0 + row) * gridDim.x + blockIdx.x) * (D + 2);
      dst[ch] = sm_o[row][ch];
      if (ch == 0) {
        dst[D] = n;
        dst[D + 1] = l;
      }
    }
  }
}

// Joins a row's partial results.
template <int D>
__global__ void __launch_bounds__(D) window_join_kernel(const DecodeArgs a, int splits) {
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x, b = blockIdx.y;
  const float* src = a.ws + ((long long)b * a.w.nh + h) * splits * (D + 2);
  float n = -INFINITY;
  for (int s = 0; s < splits; ++s) n = fmaxf(n, src[s * (D + 2) + D]);
  float l = 0.f, o = 0.f;
  for (int s = 0; s < splits; ++s) {
    const float m = src[s * (D + 2) + D];
    const float f = m == -INFINITY ? 0.f : fast_exp2(m - n);
    l += src[s * (D + 2) + D + 1] * f;
    o += src[s * (D + 2) + threadIdx.x] * f;
  }
  a.o.row(b, h, 0)[threadIdx.x] = __float2bfloat16_rn(l > 0.f ? o / l : 0.f);
}

template <int D, bool kKv4>
cudaError_t decode(const DecodeArgs& a, cudaStream_t st) {
  const int group = a.w.nh / a.w.nkv, tiles = (group + kRows - 1) / kRows;
  const int splits = decode_splits(a.w);
  cudaError_t e = launch_pdl(window_decode_kernel<D, kKv4>, dim3(splits, a.w.nkv * tiles, a.w.B),
                             dim3(kThreads), 0, st, a);
  if (e != cudaSuccess || splits == 1) return e;
  return launch_pdl(window_join_kernel<D>, dim3(a.w.nh, a.w.B), dim3(D), 0, st, a, splits);
}

}  // namespace

int decode_splits(const Window& w) {
  const int group = w.nh / w.nkv, tiles = (group + kRows - 1) / kRows;
  // the most blocks a sequence can see
  const long long rows = std::min<long long>(w.nk, (long long)w.left + 1 + w.sinks);
  const long long blocks = (rows + kBlock - 1) / kBlock + 1;
  const long long ctas = (long long)w.B * w.nkv * tiles;
  // six CTAs per SM between them, but at least four blocks for each warp
  const long long want = (6LL * 152 + ctas - 1) / ctas, most = std::max<long long>(1, blocks / (4 * kWarps));
  return (int)std::min<long long>(std::min(want, most), 256);
}

size_t decode_ws_bytes(const Window& w, int d) {
  const int s = decode_splits(w);
  return s == 1 ? 256 : ((size_t)w.B * w.nh * s * (d + 2) * 4 + 255) / 256 * 256;
}

cudaError_t launch_window_decode(const DecodeArgs& a, int d, bool kv4, cudaStream_t st) {
  if (d == 64) return kv4 ? decode<64, true>(a, st) : decode<64, false>(a, st);
  return kv4 ? decode<128, true>(a, st) : decode<128, false>(a, st);
}

}  // namespace psa
