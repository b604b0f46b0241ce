// kv_cache.cu -- rows into a cache: as they are (psa_kv_append), or in 4 bits
// (psa_kv4_append) and back (psa_kv4_read).
//
// 4 bits: for each group g of 32 channels of a row, scale = bf16(max|x| (1 / 7)) and
// code(x) = round(x / scale) + 8 (ties to even, clamped to 1 .. 15), which stands for
// (code - 8) * scale: 4.5 bits a value.  The code of channel 32 g + 4 a + i (a < 8, i < 4)
// is nibble (a * G + g) * 4 + i of the row's d / 2 bytes, G = d / 32.  In this order a
// lane of the decoding kernel finds all its channels of a row, of every group, in one
// load: two neighbouring a for keys (channels are the product's inner dimension there),
// one a for values.
//
// Bound by memory.  Four lanes share a row: lane t holds channels 8 t .. 8 t + 7 of each
// group, whose codes are the row's bytes [t d / 8, (t + 1) d / 8).  So a group's maximum is
// two shuffles, codes leave in one store of 8 or 16 bytes per lane, and the lanes' reads of
// bf16 rows are 64 neighbouring bytes.  Measured, 4 sequences of 8 heads of 128: 2048 rows into
// 4 bits 12.5 us (3.4 TB/s; instructions bound it, 8 a value), 4096 rows back 14.4 us (6.0 TB/s).
#include "lm.cuh"
#include "ptx.cuh"

namespace psa {
namespace {

constexpr int kThreads = 256;

// Cache row of row n of sequence b, or -1.
__device__ __forceinline__ int cache_row(const CacheArgs& c, int b, int n) {
  if (n >= c.N || (c.counts && n >= c.counts[b])) return -1;
  const long long r = (long long)c.starts[b] + n;
  return r >= 0 && r < c.max_len ? (int)r : -1;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    kv_append_kernel(const CacheArgs c, View<const T> k, View<const T> v, View<T> kc, View<T> vc) {
  constexpr int LANES = D / kVec<T>;
  pdl_launch_dependents();
  pdl_wait();
  const int col = (threadIdx.x % LANES) * kVec<T>;
  const int n = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const int b = blockIdx.y / c.nkv, h = blockIdx.y % c.nkv;
  const int r = cache_row(c, b, n);
  if (r < 0) return;
  const uint4 x = *reinterpret_cast<const uint4*>(k.row(b, h, n) + col);
  const uint4 y = *reinterpret_cast<const uint4*>(v.row(b, h, n) + col);
  *reinterpret_cast<uint4*>(kc.row(b, h, r) + col) = x;
  *reinterpret_cast<uint4*>(vc.row(b, h, r) + col) = y;
}

// Eight channels of one group.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  unpack_vec(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = pack_vec(x);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Quantises lane t's channels of one row (any row where it is not live).  Every lane of the
// warp calls it.  A group that
// holds a NaN or an infinity gets a scale that is not finite, and does not read back as finite.
template <typename T, int D>
__device__ __forceinline__ void quantise_row(const T* src, uint8_t* codes, __nv_bfloat16* scales,
                                             int t, bool live) {
  constexpr int G = D / 32;
  uint32_t lo[G], hi[G];  // four nibbles of a = 2 t and of a = 2 t + 1, for each group
  uint32_t sc[G];
  float all[G][8];
#pragma unroll
  for (int g = 0; g < G; ++g) load8(src + 32 * g + 8 * t, all[g]);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const float(&x)[8] = all[g];
    // magnitudes compare as integers do, a NaN above all
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const __nv_bfloat16 s = __float2bfloat16_rn(__fmul_rn(__uint_as_float(top), 1.f / 7.f));
    const float step = __bfloat162float(s);
    sc[g] = *reinterpret_cast<const uint16_t*>(&s);
    // The format's quotient is rounded to fp32, then to a whole number.  With the correctly
    // rounded reciprocal, one correction by the exact remainder makes a quotient within a unit of
    // the last place the correctly rounded one (Markstein, "Computation of elementary functions
    // on the IBM RISC System/6000 processor", 1990); x times the reciprocal may be a unit and a
    // half off, so there is a correction before it.  Below 2^-100, where the reciprocal may overflow and a bf16 scale may
    // be far from a seventh of the maximum, it is the division itself, clamped; elsewhere |q| < 7.5.
    // Adding 1.5 2^23 + 8 rounds (ties to even) and leaves the code in the lowest four bits; the
    // constant's low 16 bits are those of the 8 alone, so four such sums shifted by multiplication
    // add up to four codes in the low half.
    const float inv = __fdiv_rn(1.f, step);
    constexpr float kRound = 12582920.f;
    float q[8];
    if (step >= 7.9e-31f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = x[e] * inv, z = fmaf(fmaf(-y, step, x[e]), inv, y);
        q[e] = fmaf(fmaf(-z, step, x[e]), inv, z);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = step > 0.f ? fminf(fmaxf(__fdiv_rn(x[e], step), -7.f), 7.f) : 0.f;
    }
    lo[g] = hi[g] = 0;
#pragma unroll
    for (int e = 3; e >= 0; --e) {
      lo[g] = lo[g] * 16u + __float_as_uint(q[e] + kRound);
      hi[g] = hi[g] * 16u + __float_as_uint(q[4 + e] + kRound);
    }
    lo[g] &= 0xffffu;
    hi[g] &= 0xffffu;
  }
  if (!live) return;
  if constexpr (G == 4) {
    *reinterpret_cast<uint4*>(codes + 16 * t) = make_uint4(
        lo[0] | lo[1] << 16, lo[2] | lo[3] << 16, hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
    if (t == 0) *reinterpret_cast<uint2*>(scales) = make_uint2(sc[0] | sc[1] << 16, sc[2] | sc[3] << 16);
  } else {
    *reinterpret_cast<uint2*>(codes + 8 * t) = make_uint2(lo[0] | lo[1] << 16, hi[0] | hi[1] << 16);
    if (t == 0) *reinterpret_cast<uint32_t*>(scales) = sc[0] | sc[1] << 16;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    kv4_append_kernel(const CacheArgs c, View<const T> k, View<const T> v, uint8_t* kcodes,
                      __nv_bfloat16* kscales, uint8_t* vcodes, __nv_bfloat16* vscales) {
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x & 3, n = blockIdx.x * (kThreads / 4) + threadIdx.x / 4;
  const int b = blockIdx.y / c.nkv, h = blockIdx.y % c.nkv;
  const int r = cache_row(c, b, n);
  const bool live = r >= 0;
  const long long at = (long long)blockIdx.y * c.max_len + max(r, 0);
  const bool is_v = blockIdx.z;
  const View<const T> src = is_v ? v : k;
  quantise_row<T, D>(src.row(b, h, live ? n : 0), (is_v ? vcodes : kcodes) + at * (D / 2),
                     (is_v ? vscales : kscales) + at * (D / 32), t, live);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(const CacheArgs c, const uint8_t* kcodes, const __nv_bfloat16* kscales,
                    const uint8_t* vcodes, const __nv_bfloat16* vscales, View<T> k, View<T> v) {
  constexpr int G = D / 32;
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x & 3, n = blockIdx.x * (kThreads / 4) + threadIdx.x / 4;
  if (n >= c.N) return;
  const int b = blockIdx.y / c.nkv, h = blockIdx.y % c.nkv;
  const long long at = (long long)blockIdx.y * c.max_len + n;
  const bool is_v = blockIdx.z;
  const uint8_t* codes = (is_v ? vcodes : kcodes) + at * (D / 2) + t * (D / 8);
  const __nv_bfloat16* scales = (is_v ? vscales : kscales) + at * G;
  uint32_t w[G];  // words of a = 2 t, then of a = 2 t + 1, two groups in each
  float sc[G];
  if constexpr (G == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(codes);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(codes);
    w[0] = u.x; w[1] = u.y;
  }
#pragma unroll
  for (int g = 0; g < G; ++g) sc[g] = __bfloat162float(scales[g]);
  T* dst = (is_v ? v : k).row(b, h, n) + 8 * t;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const uint32_t lo = w[g / 2] >> (16 * (g & 1)), hi = w[G / 2 + g / 2] >> (16 * (g & 1));
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = ((float)((lo >> (4 * e)) & 15) - 8.f) * sc[g];
      x[4 + e] = ((float)((hi >> (4 * e)) & 15) - 8.f) * sc[g];
    }
    store8(dst + 32 * g, x);
  }
}

}  // namespace

template <typename T>
cudaError_t launch_kv_append(const CacheArgs& c, View<const T> k, View<const T> v, View<T> kc,
                             View<T> vc, int d, cudaStream_t st) {
  const int rows = kThreads / (d / kVec<T>);
  const dim3 grid((c.N + rows - 1) / rows, c.B * c.nkv);
  return launch_pdl(d == 64 ? kv_append_kernel<T, 64> : kv_append_kernel<T, 128>, grid,
                    dim3(kThreads), 0, st, c, k, v, kc, vc);
}

template <typename T>
cudaError_t launch_kv4_append(const CacheArgs& c, View<const T> k, View<const T> v, void* kcodes,
                              void* kscales, void* vcodes, void* vscales, int d, cudaStream_t st) {
  const dim3 grid((c.N + kThreads / 4 - 1) / (kThreads / 4), c.B * c.nkv, 2);
  return launch_pdl(d == 64 ? kv4_append_kernel<T, 64> : kv4_append_kernel<T, 128>, grid,
                    dim3(kThreads), 0, st, c, k, v, (uint8_t*)kcodes, (__nv_bfloat16*)kscales,
                    (uint8_t*)vcodes, (__nv_bfloat16*)vscales);
}

template <typename T>
cudaError_t launch_kv4_read(const CacheArgs& c, const void* kcodes, const void* kscales,
                            const void* vcodes, const void* vscales, View<T> k, View<T> v, int d,
                            cudaStream_t st) {
  const dim3 grid((c.N + kThreads / 4 - 1) / (kThreads / 4), c.B * c.nkv, 2);
  return launch_pdl(d == 64 ? kv4_read_kernel<T, 64> : kv4_read_kernel<T, 128>, grid,
                    dim3(kThreads), 0, st, c, (const uint8_t*)kcodes, (const __nv_bfloat16*)kscales,
                    (const uint8_t*)vcodes, (const __nv_bfloat16*)vscales, k, v);
}

#define PSA_CACHE(T)                                                                             \
  template cudaError_t launch_kv_append(const CacheArgs&, View<const T>, View<const T>, View<T>, \
                                        View<T>, int, cudaStream_t);                             \
  template cudaError_t launch_kv4_append(const CacheArgs&, View<const T>, View<const T>, void*,  \
                                         void*, void*, void*, int, cudaStream_t);                \
  template cudaError_t launch_kv4_read(const CacheArgs&, const void*, const void*, const void*,  \
                                       const void*, View<T>, View<T>, int, cudaStream_t);
PSA_CACHE(float)
PSA_CACHE(__nv_bfloat16)
#undef PSA_CACHE

}  // namespace psa
