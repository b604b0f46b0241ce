// window_decode.cu -- attention of one query token per sequence over a cache, with a sliding
// window and first tokens that stay visible; the cache in bf16, or in 4 bits (kv_cache.cu
// has the format).
//
//   o_h = sum_j softmax_j(scale q_h . k_j) v_j over the visible rows j of the cache
//
// Bound by memory: every visible row of K and V is read once, for all query heads that
// share it.  The products run on m16n8k16 tensor instructions (a fifth of their rate is
// enough here, and nothing could fill a larger one): 16 keys by 8 query heads for S^T = K Q^T,
// 16 channels by 8 heads for O^T = V^T P^T, so the cache is the A operand and goes from memory
// straight into registers, without shared memory or a barrier between a load and its use.
// That works because the order of the inner index of K Q^T (channels) and the row order of
// V^T P^T (channels) are free: each lane takes 16 neighbouring bytes of a row, and Q's fragment
// (the output's channels) is permuted to match.  For V the two keys of a pair sit in two
// registers of one lane, and a byte permute puts them side by side; P, whose rows are keys,
// becomes the B operand by an 8 x 8 transposition inside the warp.
//
// Keys are cut into blocks of 16 or 32; the visible blocks (the sinks', then the window's) are
// dealt to gridDim.x CTAs in contiguous parts and inside a CTA to its warps in turn.  Every
// warp keeps its own running maximum, sum and output; the maximum moves only when a score
// exceeds it by more than 2^8 (output and sum share the stale one, so the result is the
// same), and only then do lanes exchange anything.  The warps' results are joined in shared
// memory, and the parts of a sequence by a second small kernel from fp32 partial results.
// The number of parts goes by the problem's sizes alone: enough CTAs for every SM.
//
// 4 bits: what bounds the kernel there is the integer work of widening codes, so it is kept
// small.  K: a code at bits 0-3 or 4-7 of a 16-bit half becomes the fp16 number 1024 + n or
// 64 + n by one masked OR, without a shift, and n - 8 by an exact subtraction of two at once.
// (Sums that start at minus 1032 and 72 times the query's sums would do without it, but lose 8 of
// their 24 bits: large keys that differ little then stand off by more than P's rounding.)  The
// query is in fp16 too, each group of 32 channels scaled by a power of two of its own to a
// maximum of 1 .. 2, so that what is lost is at most 2^-25 of the group's largest channel; bf16's
// 8 bits fit down to 2^-17 of it.  V: 128 + n in bf16 (P times a scale needs its range), shifted on
// the multipliers, less 136, exactly.  A key's scale, times the query's power of two, multiplies
// its fp32 partial score of each group; a value's scale multiplies the probability before it is
// rounded to bf16.
//
// Measured: bf16, 32 sequences of up to 8192 keys, 4096 visible, 32 heads of 128 on 8: 85 us (5.9
// TB/s, 0.88 of the copy bandwidth); 4 bits, 16 sequences of up to 32768 keys: 113 us (3.4 TB/s,
// 0.51; the integer pipe is busy 62 % of the time, tensor instructions 18 %).  One sequence of
// 1024 visible keys: 5.5 us with the join.
#include <algorithm>

#include <cuda_fp16.h>

#include "lm.cuh"
#include "ptx_tiles4d.cuh"

namespace psa {
namespace {

constexpr int kWarps = 4;        // per CTA
constexpr int kThreads = 32 * kWarps;
constexpr int kLongBlock = 32;   // most keys that a warp takes at a time
constexpr float kLog2eD = 1.4426950408889634074f;

// An 8 x 8 matrix of 16-bit values, two neighbours of a row per lane, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// n - 8, n' - 8 in fp16 for the nibbles n, n' at bits 0 and 16 (High: 4 and 20)
template <bool High>
__device__ __forceinline__ uint32_t nibbles_fp16(uint32_t x) {
  const uint32_t u = High ? (x & 0x00F000F0u) | 0x54005400u : (x & 0x000F000Fu) | 0x64006400u;
  const uint32_t k = High ? 0x54805480u : 0x64086408u;  // 72, 1032
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&k));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// n - 8, n' - 8 in bf16 for the nibbles n, n' at bits 4 i and 4 i + 16
template <int i>
__device__ __forceinline__ uint32_t nibbles_bf16(uint32_t x) {
  const uint32_t u = ((x >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
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

// reads of this lane's own place that stay where they are (kept out of registers)
__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ float2 shared8(uint32_t at) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at));
  return v;
}

// The visible rows of sequence b: blocks 0 .. sink - 1, then first .. (count in all).
template <int kBlock>
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

// One lane's part of a block of 16 keys, lane = 4 g + t: of K the keys g and g + 8, every
// fourth 16 bytes of their channels by t; of V the keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9,
// channels by g.  HT: tiles of 8 query heads.
// kShort: the cache has fewer rows than a block, so rows behind the last are read as that one
// (they are hidden); otherwise the last block starts early enough to end inside the cache.
template <int D, int HT, bool kKv4, bool kShort>
struct Cache;

template <int D, int HT, bool kShort>
struct Cache<D, HT, false, kShort> {
  static constexpr int U = 1;  // blocks of 16 keys at a time
  const __nv_bfloat16 *kp, *vp;
  long long kn, vn;
  int last;
  uint4 k[U][2][D / 32], v[U][4][D / 64];

  __device__ __forceinline__ Cache(const DecodeArgs& a, int b, int h, int lane) {
    kp = a.k.row(b, h, 0) + 8 * (lane & 3);
    vp = a.v.row(b, h, 0) + 8 * (lane >> 2);
    kn = a.k.sn;
    vn = a.v.sn;
    last = a.w.nk - 1;
  }
  uint32_t q[HT][D / 8];
  struct Shared {};
  __device__ __forceinline__ void prepare(const uint32_t (&q_)[HT][D / 8], int, Shared&) {
#pragma unroll
    for (int ht = 0; ht < HT; ++ht)
#pragma unroll
      for (int i = 0; i < D / 8; ++i) q[ht][i] = q_[ht][i];
  }
  __device__ __forceinline__ int row(int j) const { return kShort ? min(j, last) : j; }
  __device__ __forceinline__ void load_k(int j0, int lane) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const __nv_bfloat16* p = kp + row(j0 + 16 * u + 8 * x + (lane >> 2)) * kn;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) k[u][x][i] = load16(p + 32 * i);
      }
  }
  __device__ __forceinline__ void load_v(int j0, int lane) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const __nv_bfloat16* p = vp + row(j0 + 16 * u + 2 * (lane & 3) + (x & 1) + 8 * (x >> 1)) * vn;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) v[u][x][i] = load16(p + 64 * i);
      }
  }
  // channels 32 i + 8 t + 2 s, + 1 are the lane's pair s of products 2 i and 2 i + 1
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
  __device__ __forceinline__ void scores(float (&s)[U][HT][4]) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        // two chains of products, added at the end
        float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 x = k[u][0][i], y = k[u][1][i];
          mma16816(c[0], x.x, y.x, x.y, y.y, q[ht][4 * i], q[ht][4 * i + 1]);
          mma16816(c[1], x.z, y.z, x.w, y.w, q[ht][4 * i + 2], q[ht][4 * i + 3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[u][ht][e] = c[0][e] + c[1][e];
      }
  }
  // rows that are not visible may hold anything (NaN times a probability of 0)
  __device__ __forceinline__ void drop_v(int u, const bool (&see)[4]) {
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        if (!see[x]) v[u][x][i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void drop_scales(int, const bool (&)[2]) {}
  __device__ __forceinline__ void mix(int u, const float (&p)[HT][4], float (&o)[HT][D / 16][4]) const {
    uint32_t b0[HT], b1[HT];
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
      b0[ht] = transpose8x8(pack2(p[ht][0], p[ht][1]));
      b1[ht] = transpose8x8(pack2(p[ht][2], p[ht][3]));
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint32_t w[4][4] = {{v[u][0][i].x, v[u][0][i].y, v[u][0][i].z, v[u][0][i].w},
                                {v[u][1][i].x, v[u][1][i].y, v[u][1][i].z, v[u][1][i].w},
                                {v[u][2][i].x, v[u][2][i].y, v[u][2][i].z, v[u][2][i].w},
                                {v[u][3][i].x, v[u][3][i].y, v[u][3][i].z, v[u][3][i].w}};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a0 = __byte_perm(w[0][e], w[1][e], 0x5410), a1 = __byte_perm(w[0][e], w[1][e], 0x7632);
        const uint32_t a2 = __byte_perm(w[2][e], w[3][e], 0x5410), a3 = __byte_perm(w[2][e], w[3][e], 0x7632);
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) mma16816(o[ht][4 * i + e], a0, a1, a2, a3, b0[ht], b1[ht]);
      }
    }
  }
  // channel of output tile m, row g (low) or g + 8 (high)
  static __device__ __forceinline__ int channel(int m, int g, int high) {
    return 64 * (m / 4) + 8 * g + 2 * (m % 4) + high;
  }
};

template <int D, int HT, bool kShort>
struct Cache<D, HT, true, kShort> {
  static constexpr int G = D / 32, W = G / 2;  // groups, and words that hold a value for each
  // two blocks of 16 keys at a time: twice the bytes in flight and half the steps' overhead
  // (16 x 32768 keys 123 -> 112 us)
  static constexpr int U = 2;
  const char *kp, *vp, *ksp, *vsp;
  int last;
  uint32_t k[U][2][G], v[U][4][W], ks[U][2][W], vs[U][2][W];  // codes; scales of keys g and g + 8
  // The query, and what each of its groups has been scaled down by for heads 2 t and 2 t + 1, lie in
  // shared memory, each lane's at its place: they are read once per step, and the registers
  // hold more loads instead.
  struct Shared {
    uint4 q[HT][G][32];
    float2 up[HT][G][32];
  };
  uint32_t q_at, up_at;

  __device__ __forceinline__ Cache(const DecodeArgs& a, int b, int h, int lane) {
    const long long base = ((long long)b * a.w.nkv + h) * a.w.nk;
    const int g = lane >> 2, t = lane & 3;
    kp = static_cast<const char*>(a.kcodes) + (base + g) * (D / 2) + (D / 8) * t;
    vp = static_cast<const char*>(a.vcodes) + (base + 2 * t) * (D / 2) + (D / 16) * g;
    ksp = static_cast<const char*>(a.kscales) + (base + g) * (2 * G);
    vsp = static_cast<const char*>(a.vscales) + (base + g) * (2 * G);
    last = a.w.nk - 1;
  }
  // The query in fp16, each group scaled to a maximum of 1 .. 2, and what that has to be undone by.
  // (every warp writes the same values)
  __device__ __forceinline__ void prepare(const uint32_t (&q)[HT][D / 8], int lane, Shared& sh) {
    q_at = smem_addr(&sh.q[0][0][lane]);
    up_at = smem_addr(&sh.up[0][0][lane]);
#pragma unroll
    for (int ht = 0; ht < HT; ++ht)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float m = 0.f;  // of this lane's 8 channels of head lane / 4, then of its four lanes'
#pragma unroll
        for (int i = 0; i < 4; ++i)
          m = fmaxf(m, fmaxf(fabsf(__uint_as_float(q[ht][4 * g + i] << 16)),
                             fabsf(__uint_as_float(q[ht][4 * g + i] & 0xffff0000u))));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        // powers of two: 2^-e and 2^e for m in 2^e .. 2^(e + 1), both normal numbers
        const uint32_t e = min(max(__float_as_uint(m) >> 23, 1u), 253u);
        const float down = __uint_as_float((254u - e) << 23);
        const float mine = __uint_as_float(e << 23);
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = q[ht][4 * g + i];
          const __half2 h = __floats2half2_rn(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xffff0000u) * down);
          y[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        sh.q[ht][g][lane] = make_uint4(y[0], y[1], y[2], y[3]);
        sh.up[ht][g][lane] = make_float2(__shfl_sync(0xffffffffu, mine, 8 * (lane & 3)),
                                         __shfl_sync(0xffffffffu, mine, 8 * (lane & 3) + 4));
      }
  }
  static __device__ __forceinline__ void load_words(const char* p, uint32_t (&w)[W]) {
    if constexpr (W == 2) {
      const uint2 u = load8(p);
      w[0] = u.x;
      w[1] = u.y;
    } else {
      w[0] = load4(p);
    }
  }
  // row of a block relative to its first: the lane's own is in the pointers already
  __device__ __forceinline__ int row(int n, int j0, int own) const {
    return kShort ? min(n, last - j0 - own) : n;
  }
  __device__ __forceinline__ void load_k(int j0, int lane) {
    const char *p = kp + (long long)j0 * (D / 2), *sp = ksp + (long long)j0 * (2 * G);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int n = row(16 * u + 8 * x, j0, lane >> 2);
        if constexpr (G == 4) {
          const uint4 w = load16(p + n * (D / 2));
          k[u][x][0] = w.x;
          k[u][x][1] = w.y;
          k[u][x][2] = w.z;
          k[u][x][3] = w.w;
        } else {
          const uint2 w = load8(p + n * (D / 2));
          k[u][x][0] = w.x;
          k[u][x][1] = w.y;
        }
        load_words(sp + n * (2 * G), ks[u][x]);
      }
  }
  __device__ __forceinline__ void load_v(int j0, int lane) {
    const char *p = vp + (long long)j0 * (D / 2), *sp = vsp + (long long)j0 * (2 * G);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        load_words(p + row(16 * u + (x & 1) + 8 * (x >> 1), j0, 2 * (lane & 3)) * (D / 2), v[u][x]);
#pragma unroll
      for (int x = 0; x < 2; ++x) load_words(sp + row(16 * u + 8 * x, j0, lane >> 2) * (2 * G), vs[u][x]);
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
  static __device__ __forceinline__ float scale_of(const uint32_t (&s)[W], int g) {
    return __uint_as_float((g & 1) ? s[g / 2] & 0xffff0000u : s[g / 2] << 16);
  }
  __device__ __forceinline__ void scores(float (&s)[U][HT][4]) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) s[u][ht][0] = s[u][ht][1] = s[u][ht][2] = s[u][ht][3] = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      uint4 q[HT];
      float2 up[HT];
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        q[ht] = shared16(q_at + (ht * G + g) * 512);
        up[ht] = shared8(up_at + (ht * G + g) * 256);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // words of a = 2 t come first, those of a = 2 t + 1 after them
        const uint32_t sel = (g & 1) ? 0x7632 : 0x5410;
        const uint32_t x = __byte_perm(k[u][0][g / 2], k[u][0][W + g / 2], sel);
        const uint32_t y = __byte_perm(k[u][1][g / 2], k[u][1][W + g / 2], sel);
        const uint32_t x8 = x >> 8, y8 = y >> 8;
        const uint32_t a[8] = {nibbles_fp16<false>(x),  nibbles_fp16<false>(y),  nibbles_fp16<true>(x),  nibbles_fp16<true>(y),
                               nibbles_fp16<false>(x8), nibbles_fp16<false>(y8), nibbles_fp16<true>(x8), nibbles_fp16<true>(y8)};
        const float s0 = scale_of(ks[u][0], g), s1 = scale_of(ks[u][1], g);
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
          mma16816_f16(c, a[0], a[1], a[2], a[3], q[ht].x, q[ht].y);
          mma16816_f16(c, a[4], a[5], a[6], a[7], q[ht].z, q[ht].w);
          const float2 f0 = __fmul2_rn(make_float2(s0, s0), up[ht]), f1 = __fmul2_rn(make_float2(s1, s1), up[ht]);
          const float2 r0 = __ffma2_rn(make_float2(c[0], c[1]), f0, make_float2(s[u][ht][0], s[u][ht][1]));
          const float2 r1 = __ffma2_rn(make_float2(c[2], c[3]), f1, make_float2(s[u][ht][2], s[u][ht][3]));
          s[u][ht][0] = r0.x;
          s[u][ht][1] = r0.y;
          s[u][ht][2] = r1.x;
          s[u][ht][3] = r1.y;
        }
      }
    }
  }
  // codes are finite whatever they are: only the scales of hidden keys may be NaN
  __device__ __forceinline__ void drop_v(int, const bool (&)[4]) {}
  __device__ __forceinline__ void drop_scales(int u, const bool (&see)[2]) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (!see[x]) vs[u][x][i] = 0;
  }
  __device__ __forceinline__ void mix(int u, const float (&p)[HT][4], float (&o)[HT][D / 16][4]) const {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float s0 = scale_of(vs[u][0], g), s1 = scale_of(vs[u][1], g);
      uint32_t b0[HT], b1[HT];
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        b0[ht] = transpose8x8(pack2(p[ht][0] * s0, p[ht][1] * s0));
        b1[ht] = transpose8x8(pack2(p[ht][2] * s1, p[ht][3] * s1));
      }
      const uint32_t sel = (g & 1) ? 0x7632 : 0x5410;
      const uint32_t x = __byte_perm(v[u][0][g / 2], v[u][1][g / 2], sel);
      const uint32_t y = __byte_perm(v[u][2][g / 2], v[u][3][g / 2], sel);
      const uint32_t a[8] = {nibbles_bf16<0>(x), nibbles_bf16<1>(x), nibbles_bf16<0>(y), nibbles_bf16<1>(y),
                             nibbles_bf16<2>(x), nibbles_bf16<3>(x), nibbles_bf16<2>(y), nibbles_bf16<3>(y)};
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        mma16816(o[ht][2 * g], a[0], a[1], a[2], a[3], b0[ht], b1[ht]);
        mma16816(o[ht][2 * g + 1], a[4], a[5], a[6], a[7], b0[ht], b1[ht]);
      }
    }
  }
  static __device__ __forceinline__ int channel(int m, int g, int high) {
    return 32 * (m / 2) + 4 * g + 2 * (m % 2) + high;
  }
};

template <int D, int HT, bool kKv4, bool kShort>
__global__ void __launch_bounds__(kThreads, HT == 2 ? 2 : D == 128 && !kKv4 ? 3 : 4)
    window_decode_kernel(const DecodeArgs a) {
  using C = Cache<D, HT, kKv4, kShort>;
  constexpr int MT = D / 16, kHeads = 8 * HT, U = C::U, kBlock = 16 * U;
  __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads];
  __shared__ float sm_o[kHeads][D + 4];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3, r = lane >> 2;
  const int group = a.w.nh / a.w.nkv, tiles = (group + kHeads - 1) / kHeads;
  const int b = blockIdx.z, h = blockIdx.y / tiles, g0 = (blockIdx.y % tiles) * kHeads;
  const int heads = min(kHeads, group - g0), h0 = h * group + g0;
  const Blocks<kBlock> bl(a.w, b);
  const int from = (int)((long long)bl.count * blockIdx.x / gridDim.x);
  const int to = (int)((long long)bl.count * (blockIdx.x + 1) / gridDim.x);

  C c(a, b, h, lane);
  int blk = from + warp;
  // where a block's 16 rows are read from: the cache's last block reaches back into the one
  // before it (whose keys are hidden there)
  const int top = max(0, a.w.nk - kBlock);
  auto start = [&](int i) { return min(bl.block(i) * kBlock, top); };
  if (blk < to) {
    c.load_k(start(blk), lane);
    c.load_v(start(blk), lane);
  }
  uint32_t q[HT][D / 8];
#pragma unroll
  for (int ht = 0; ht < HT; ++ht)
    C::load_q(8 * ht + r < heads ? a.q.row(b, h0 + 8 * ht + r, 0) : nullptr, t, q[ht]);
  __shared__ typename C::Shared sh;
  c.prepare(q, lane, sh);
  __syncthreads();
  const float sl2 = a.scale * kLog2eD;
  float o[HT][MT][4];
  float m[HT][2], l[HT][2];  // heads 8 ht + 2 t, + 1; maxima in log2 units
#pragma unroll
  for (int ht = 0; ht < HT; ++ht) {
    m[ht][0] = m[ht][1] = -INFINITY;
    l[ht][0] = l[ht][1] = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i) o[ht][i][0] = o[ht][i][1] = o[ht][i][2] = o[ht][i][3] = 0.f;
  }
  for (; blk < to; blk += kWarps) {
    const int first = bl.block(blk) * kBlock, j0 = min(first, top);
    float s[U][HT][4];
    c.scores(s);
    const int next = blk + kWarps < to ? start(blk + kWarps) : -1;
    if (next >= 0) c.load_k(next, lane);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int ht = 0; ht < HT; ++ht)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[u][ht][e] *= sl2;
    // not all keys inside the window, or among the sinks?
    if (j0 < first || j0 + kBlock > bl.len || (j0 < bl.lo && j0 + kBlock > a.w.sinks)) {
      auto sees = [&](int j) { return j >= first && j < bl.len && (j >= bl.lo || j < a.w.sinks); };
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = j0 + 16 * u, v = k + 2 * t;
        const bool mine[2] = {sees(k + r), sees(k + 8 + r)};
        const bool value[4] = {sees(v), sees(v + 1), sees(v + 8), sees(v + 9)};
#pragma unroll
        for (int ht = 0; ht < HT; ++ht)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!mine[e / 2]) s[u][ht][e] = -INFINITY;
        c.drop_v(u, value);
        c.drop_scales(u, mine);
      }
    }
    bool grow = false;
    float top2[HT][2];
#pragma unroll
    for (int ht = 0; ht < HT; ++ht)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top2[ht][e] = fmaxf(s[0][ht][e], s[0][ht][2 + e]);
#pragma unroll
        for (int u = 1; u < U; ++u) top2[ht][e] = fmax3(top2[ht][e], s[u][ht][e], s[u][ht][2 + e]);
        grow |= top2[ht][e] > m[ht][e] + 8.f;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float n = top2[ht][e];
          n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 4));
          n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 8));
          n = fmaxf(m[ht][e], fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 16)));
          const float f = n == -INFINITY ? 1.f : fast_exp2(m[ht][e] - n);
          m[ht][e] = n;
          l[ht][e] *= f;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[ht][i][e] *= f;
            o[ht][i][2 + e] *= f;
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int ht = 0; ht < HT; ++ht)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float base = m[ht][e] == -INFINITY ? 0.f : m[ht][e];
          s[u][ht][e] = fast_exp2(s[u][ht][e] - base);
          s[u][ht][2 + e] = fast_exp2(s[u][ht][2 + e] - base);
          l[ht][e] += s[u][ht][e] + s[u][ht][2 + e];
        }
      c.mix(u, s[u], o);
    }
    if (next >= 0) c.load_v(next, lane);
  }
  // the eight lanes of a head each summed their own keys
#pragma unroll
  for (int ht = 0; ht < HT; ++ht)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int x = 4; x <= 16; x <<= 1) l[ht][e] += __shfl_xor_sync(0xffffffffu, l[ht][e], x);
      if (r == 0) {
        sm_m[warp][8 * ht + 2 * t + e] = m[ht][e];
        sm_l[warp][8 * ht + 2 * t + e] = l[ht][e];
      }
    }
  __syncthreads();
  float f[HT][2];
#pragma unroll
  for (int ht = 0; ht < HT; ++ht)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float n = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) n = fmaxf(n, sm_m[w][8 * ht + 2 * t + e]);
      f[ht][e] = m[ht][e] == -INFINITY ? 0.f : fast_exp2(m[ht][e] - n);
    }
  // the warps add their outputs one after another: a fixed order
  for (int w = 0; w < kWarps; ++w) {
    if (warp == w) {
#pragma unroll
      for (int ht = 0; ht < HT; ++ht)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* d = &sm_o[8 * ht + 2 * t + (e & 1)][C::channel(i, r, e >> 1)];
            *d = (w == 0 ? 0.f : *d) + o[ht][i][e] * f[ht][e & 1];
          }
    }
    __syncthreads();
  }
  for (int u = threadIdx.x; u < heads * D; u += kThreads) {
    // a sum of 0 is a row that sees nothing; a NaN among the scores stays one
    const int row = u / D, ch = u % D;
    float n = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) n = fmaxf(n, sm_m[w][row]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      sum += sm_l[w][row] * (sm_m[w][row] == -INFINITY ? 0.f : fast_exp2(sm_m[w][row] - n));
    if (gridDim.x == 1) {
      a.o.row(b, h0 + row, 0)[ch] = __float2bfloat16_rn(sum != 0.f ? sm_o[row][ch] / sum : 0.f);
    } else {
      // partial result: D outputs relative to the maximum n, then n and the sum
      float* dst = a.ws + (((long long)b * a.w.nh + h0 + row) * gridDim.x + blockIdx.x) * (D + 2);
      dst[ch] = sm_o[row][ch];
      if (ch == 0) {
        dst[D] = n;
        dst[D + 1] = sum;
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
  a.o.row(b, h, 0)[threadIdx.x] = __float2bfloat16_rn(l != 0.f ? o / l : 0.f);
}

// Query heads of a tile: eight where a group has no more (half the registers), else sixteen.
int head_tile(const Window& w) { return w.nh / w.nkv <= 8 ? 8 : 16; }

template <int D, bool kKv4>
cudaError_t decode(const DecodeArgs& a, cudaStream_t st) {
  const int group = a.w.nh / a.w.nkv, tile = head_tile(a.w), tiles = (group + tile - 1) / tile;
  const int splits = decode_splits(a.w);
  auto kern = a.w.nk < kLongBlock
                  ? (tile == 8 ? window_decode_kernel<D, 1, kKv4, true> : window_decode_kernel<D, 2, kKv4, true>)
                  : (tile == 8 ? window_decode_kernel<D, 1, kKv4, false> : window_decode_kernel<D, 2, kKv4, false>);
  cudaError_t e = launch_pdl(kern, dim3(splits, a.w.nkv * tiles, a.w.B), dim3(kThreads), 0, st, a);
  if (e != cudaSuccess || splits == 1) return e;
  return launch_pdl(window_join_kernel<D>, dim3(a.w.nh, a.w.B), dim3(D), 0, st, a, splits);
}

}  // namespace

int decode_splits(const Window& w) {
  const int group = w.nh / w.nkv, tiles = (group + head_tile(w) - 1) / head_tile(w);
  // the most blocks a sequence can see
  const long long rows = std::min<long long>(w.nk, (long long)w.left + 1 + w.sinks);
  const long long blocks = (rows + 15) / 16 + 1;
  const long long ctas = (long long)w.B * w.nkv * tiles;
  // eight CTAs per SM between them, but at least four blocks of 16 for each warp
  const long long want = (8LL * 152 + ctas - 1) / ctas, most = std::max<long long>(1, blocks / (4 * kWarps));
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
