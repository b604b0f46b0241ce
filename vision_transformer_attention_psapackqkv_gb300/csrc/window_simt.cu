// window_simt.cu -- attention with a sliding window and first tokens that stay visible, on
// CUDA cores in fp32: forward, and the dQ and dK/dV kernels of the backward.
//
//   S = scale Q K^T over the visible keys, P = exp(S - lse), O = P V;
//   dV = P^T dO, dP = dO V^T, dS = P o (dP - delta), delta = rowsum(dO o O),
//   dQ = scale dS K, dK = scale dS^T Q.
//
// A CTA owns 64 query rows (64 key rows in dK/dV) and goes through the 64-row tiles of the
// other side that its rows see, so a score exists only in registers and shared memory.
// 256 threads as 16 x 16: a thread holds the 4 x 4 scores of rows ty + 16 i and columns
// tx + 16 j, and of each product with V (K, dO, Q) its rows' channels 4 tx + 64 c .. + 3.
// Measured, fp32: 4 maps of 400 positions, 4 heads of 64, 121 keys a query: 31 us; 2 x 1024
// causal, 8 heads of 128: 237 us forward, 780 us backward.
// Tiles lie row by row in shared memory with 4 floats of padding: 16-byte reads of eight
// neighbouring rows then fall into different banks.  Every key/value head's gradient is
// summed by one CTA over its query heads and tiles in order, so reruns are bitwise equal.
#include <math.h>

#include "lm.cuh"
#include "ptx.cuh"

namespace psa {
namespace {

constexpr int kB = 64;  // rows of a tile, on either side
constexpr int kThreads = 256;  // 16 threads a row, 4 rows a thread, kGap rows between them
constexpr int kR = 4, kGap = kB / kR;
constexpr int kLdP = kB + 4;  // row pitch of a tile of scores

template <int D>
constexpr int kLd = D + 4;

// Rows i0 .. i0 + 63 of one head into shared memory in fp32; rows outside [lo, hi) as 0.
template <int D, typename T, int kN = kThreads>
__device__ __forceinline__ void load_rows(float* dst, const T* base, long long sn, int i0, int lo,
                                          int hi) {
  constexpr int VEC = kVec<T>, PER = D / VEC;
  for (int u = threadIdx.x; u < kB * PER; u += kN) {
    const int r = u / PER, c = (u % PER) * VEC, i = i0 + r;
    float x[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = 0.f;
    if (i >= lo && i < hi) unpack_vec(*reinterpret_cast<const uint4*>(base + i * sn + c), x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) dst[r * kLd<D> + c + e] = x[e];
  }
}

// acc[i][j] = sum over d of A[ty + (64 / R) i][d] B[tx + 16 j][d]
template <int D, int R>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ty, int tx,
                                         float (&acc)[R][4]) {
  constexpr int kR = R, kGap = kB / R;
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
  for (int k = 0; k < D; k += 4) {
    float4 x[kR], y[4];
#pragma unroll
    for (int i = 0; i < kR; ++i) x[i] = *reinterpret_cast<const float4*>(A + (ty + kGap * i) * kLd<D> + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * kLd<D> + k);
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] += x[i].x * y[j].x + x[i].y * y[j].y + x[i].z * y[j].z + x[i].w * y[j].w;
  }
}

// acc[i][4 c + e] += sum over the 64 rows m of P[ty + (64 / R) i][m] B[m][4 tx + 64 c + e]
template <int D, int R>
__device__ __forceinline__ void mix_tile(const float* P, const float* B, int ty, int tx,
                                         float (&acc)[R][D / 16]) {
  constexpr int kR = R, kGap = kB / R;
#pragma unroll 4
  for (int m = 0; m < kB; m += 4) {
    float4 p[kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty + kGap * i) * kLdP + m);
#pragma unroll
    for (int mm = 0; mm < 4; ++mm) {
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float4 y = *reinterpret_cast<const float4*>(B + (m + mm) * kLd<D> + 4 * tx + 64 * c);
#pragma unroll
        for (int i = 0; i < kR; ++i) {
          const float w = mm == 0 ? p[i].x : mm == 1 ? p[i].y : mm == 2 ? p[i].z : p[i].w;
          acc[i][4 * c] += w * y.x;
          acc[i][4 * c + 1] += w * y.y;
          acc[i][4 * c + 2] += w * y.z;
          acc[i][4 * c + 3] += w * y.w;
        }
      }
    }
  }
}

__device__ __forceinline__ bool sees(const Window& w, int len, int p, int j) {
  return p >= 0 && p < len && j < len && j <= p + w.right && (j >= p - w.left || j < w.sinks);
}

// Reduction over the 16 lanes that share ty.
template <bool kMax>
__device__ __forceinline__ float row_reduce(float v) {
#pragma unroll
  for (int m = 8; m > 0; m >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, m);
    v = kMax ? fmaxf(v, o) : v + o;
  }
  return v;
}

template <int D, typename T>
__device__ __forceinline__ void store4(T* dst, float a, float b, float c, float d) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4*>(dst) = make_float4(a, b, c, d);
  else
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2(a, b), pack2(c, d));
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(16 * kB / R) window_fwd_simt_kernel(const WindowArgs<T> a) {
  constexpr int kR = R, kGap = kB / R, kN = 16 * kGap;
  extern __shared__ float sm[];
  float *Q = sm, *K = Q + kB * kLd<D>, *V = K + kB * kLd<D>, *P = V + kB * kLd<D>;
  pdl_launch_dependents();
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = blockIdx.y / a.w.nh, h = blockIdx.y % a.w.nh, hk = h / (a.w.nh / a.w.nkv);
  const int len = a.w.len(b), off = a.w.nk - a.w.nq;
  // the last tiles of a causal problem see the most keys: they start first
  const int i0 = (gridDim.x - 1 - blockIdx.x) * kB;
  const int p0 = i0 + off;
  const KeyTiles<kB> tiles(a.w, len, max(p0, 0), min(min(p0 + kB, a.w.nk) - 1, len - 1));
  load_rows<D, T, kN>(Q, a.q.row(b, h, 0), a.q.sn, i0, max(0, -off), min(a.w.nq, len - off));

  float o[kR][D / 16], m[kR], l[kR];
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
  }
  for (int t = 0; t < tiles.count; ++t) {
    const int j0 = tiles.tile(t) * kB;
    __syncthreads();
    load_rows<D, T, kN>(K, a.k.row(b, hk, 0), a.k.sn, j0, 0, len);
    load_rows<D, T, kN>(V, a.v.row(b, hk, 0), a.v.sn, j0, 0, len);
    __syncthreads();
    float s[kR][4];
    dot_tile<D>(Q, K, ty, tx, s);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int p = p0 + ty + kGap * i;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = sees(a.w, len, p, j0 + tx + 16 * j) ? s[i][j] * a.scale : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      mx = fmaxf(m[i], row_reduce<true>(mx));
      // a row that has seen nothing yet keeps m = -inf and p = 0
      const float base = mx == -INFINITY ? 0.f : mx;
      const float alpha = expf(m[i] - base);
      m[i] = mx;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = expf(s[i][j] - base);
        sum += e;
        P[(ty + kGap * i) * kLdP + tx + 16 * j] = e;
      }
      l[i] = l[i] * alpha + row_reduce<false>(sum);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[i][c] *= alpha;
    }
    __syncthreads();
    mix_tile<D>(P, V, ty, tx, o);
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int q = i0 + ty + kGap * i;
    if (q >= a.w.nq) continue;
    // a sum of 0 is a row that sees nothing; a NaN among the scores stays one
    const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;
    T* dst = a.out.row(b, h, q) + 4 * tx;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      store4<D>(dst + 64 * c, o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv,
                o[i][4 * c + 3] * inv);
    if (a.lse && tx == 0)
      a.lse[(long long)blockIdx.y * a.w.nq + q] = l[i] != 0.f ? m[i] + logf(l[i]) : -INFINITY;
  }
}

// delta = rowsum(dO o O), one row per 16 lanes; 0 for rows that see nothing (whose dO and
// O may hold anything).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) window_delta_kernel(const WindowArgs<T> a) {
  constexpr int VEC = kVec<T>, PER = D / VEC, LANES = PER < 16 ? PER : 16;
  pdl_launch_dependents();
  pdl_wait();
  const int lr = threadIdx.x % LANES;
  const int i = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const int b = blockIdx.y / a.w.nh, h = blockIdx.y % a.w.nh;
  const int p = i + a.w.nk - a.w.nq;
  const bool live = i < a.w.nq && p >= 0 && p < a.w.len(b);
  float s = 0.f;
#pragma unroll
  for (int c = lr * VEC; c < D; c += LANES * VEC) {
    if (!live) continue;
    float x[VEC], y[VEC];
    unpack_vec(*reinterpret_cast<const uint4*>(a.dO.row(b, h, i) + c), x);
    unpack_vec(*reinterpret_cast<const uint4*>(a.o.row(b, h, i) + c), y);
#pragma unroll
    for (int e = 0; e < VEC; ++e) s += x[e] * y[e];
  }
#pragma unroll
  for (int m = LANES / 2; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  if (lr == 0 && i < a.w.nq) a.delta[(long long)blockIdx.y * a.w.nq + i] = s;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) window_dq_simt_kernel(const WindowArgs<T> a) {
  extern __shared__ float sm[];
  float *Q = sm, *dO = Q + kB * kLd<D>, *K = dO + kB * kLd<D>, *V = K + kB * kLd<D>,
        *S = V + kB * kLd<D>;
  pdl_launch_dependents();
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = blockIdx.y / a.w.nh, h = blockIdx.y % a.w.nh, hk = h / (a.w.nh / a.w.nkv);
  const int len = a.w.len(b), off = a.w.nk - a.w.nq;
  const int i0 = (gridDim.x - 1 - blockIdx.x) * kB;
  const int p0 = i0 + off;
  const KeyTiles<kB> tiles(a.w, len, max(p0, 0), min(min(p0 + kB, a.w.nk) - 1, len - 1));
  const int lo = max(0, -off), hi = min(a.w.nq, len - off);
  load_rows<D>(Q, a.q.row(b, h, 0), a.q.sn, i0, lo, hi);
  load_rows<D>(dO, a.dO.row(b, h, 0), a.dO.sn, i0, lo, hi);
  float acc[kR][D / 16], lse[kR], delta[kR];
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int q = i0 + ty + kGap * i;
    const bool in = q >= lo && q < hi;
    lse[i] = in ? a.lse[(long long)blockIdx.y * a.w.nq + q] : 0.f;
    delta[i] = in ? a.delta[(long long)blockIdx.y * a.w.nq + q] : 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
  }
  for (int t = 0; t < tiles.count; ++t) {
    const int j0 = tiles.tile(t) * kB;
    __syncthreads();
    load_rows<D>(K, a.k.row(b, hk, 0), a.k.sn, j0, 0, len);
    load_rows<D>(V, a.v.row(b, hk, 0), a.v.sn, j0, 0, len);
    __syncthreads();
    float s[kR][4], dp[kR][4];
    dot_tile<D>(Q, K, ty, tx, s);
    dot_tile<D>(dO, V, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = p0 + ty + kGap * i;
        const bool see = sees(a.w, len, p, j0 + tx + 16 * j) && !sees_one(a.w, len, p);
        S[(ty + kGap * i) * kLdP + tx + 16 * j] =
            see ? expf(s[i][j] * a.scale - lse[i]) * (dp[i][j] - delta[i]) : 0.f;
      }
    __syncthreads();
    mix_tile<D>(S, K, ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int q = i0 + ty + kGap * i;
    if (q >= a.w.nq) continue;
    T* dst = a.dq.row(b, h, q) + 4 * tx;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      store4<D>(dst + 64 * c, acc[i][4 * c] * a.scale, acc[i][4 * c + 1] * a.scale,
                acc[i][4 * c + 2] * a.scale, acc[i][4 * c + 3] * a.scale);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) window_dkdv_simt_kernel(const WindowArgs<T> a) {
  extern __shared__ float sm[];
  float *K = sm, *V = K + kB * kLd<D>, *Q = V + kB * kLd<D>, *dO = Q + kB * kLd<D>,
        *P = dO + kB * kLd<D>, *S = P + kB * kLdP;
  __shared__ float lse[kB], delta[kB];
  pdl_launch_dependents();
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = blockIdx.y / a.w.nkv, hk = blockIdx.y % a.w.nkv, group = a.w.nh / a.w.nkv;
  const int len = a.w.len(b), off = a.w.nk - a.w.nq;
  const int j0 = blockIdx.x * kB;
  int i0, nq;
  query_range(a.w, len, j0, min(j0 + kB, a.w.nk) - 1, i0, nq);
  load_rows<D>(K, a.k.row(b, hk, 0), a.k.sn, j0, 0, len);
  load_rows<D>(V, a.v.row(b, hk, 0), a.v.sn, j0, 0, len);
  float dk[kR][D / 16], dv[kR][D / 16];
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) dk[i][c] = dv[i][c] = 0.f;
  for (int h = hk * group; h < (hk + 1) * group; ++h) {
    for (int i1 = i0; i1 < i0 + nq; i1 += kB) {
      __syncthreads();
      load_rows<D>(Q, a.q.row(b, h, 0), a.q.sn, i1, i1, i0 + nq);
      load_rows<D>(dO, a.dO.row(b, h, 0), a.dO.sn, i1, i1, i0 + nq);
      if (threadIdx.x < kB) {
        const int i = i1 + threadIdx.x;
        const long long at = ((long long)b * a.w.nh + h) * a.w.nq + i;
        lse[threadIdx.x] = i < i0 + nq ? a.lse[at] : 0.f;
        delta[threadIdx.x] = i < i0 + nq ? a.delta[at] : 0.f;
      }
      __syncthreads();
      float s[kR][4], dp[kR][4];  // rows: keys, columns: queries
      dot_tile<D>(K, Q, ty, tx, s);
      dot_tile<D>(V, dO, ty, tx, dp);
#pragma unroll
      for (int i = 0; i < kR; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = tx + 16 * j;
          const bool see = i1 + c < i0 + nq && sees(a.w, len, i1 + c + off, j0 + ty + kGap * i);
          const float p = see ? expf(s[i][j] * a.scale - lse[c]) : 0.f;
          P[(ty + kGap * i) * kLdP + c] = p;
          S[(ty + kGap * i) * kLdP + c] = see && !sees_one(a.w, len, i1 + c + off) ? p * (dp[i][j] - delta[c]) : 0.f;
        }
      __syncthreads();
      mix_tile<D>(P, dO, ty, tx, dv);
      mix_tile<D>(S, Q, ty, tx, dk);
    }
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int j = j0 + ty + kGap * i;
    if (j >= a.w.nk) continue;
    T *dkr = a.dk.row(b, hk, j) + 4 * tx, *dvr = a.dv.row(b, hk, j) + 4 * tx;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      store4<D>(dkr + 64 * c, dk[i][4 * c] * a.scale, dk[i][4 * c + 1] * a.scale,
                dk[i][4 * c + 2] * a.scale, dk[i][4 * c + 3] * a.scale);
      store4<D>(dvr + 64 * c, dv[i][4 * c], dv[i][4 * c + 1], dv[i][4 * c + 2], dv[i][4 * c + 3]);
    }
  }
}

template <typename T, int D, int R>
cudaError_t fwd(const WindowArgs<T>& a, cudaStream_t st) {
  constexpr int smem = (3 * kB * kLd<D> + kB * kLdP) * 4;
  auto kern = window_fwd_simt_kernel<T, D, R>;
  const cudaError_t e = set_max_dynamic_smem((const void*)kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((a.w.nq + kB - 1) / kB, a.w.B * a.w.nh), dim3(16 * kB / R), smem, st, a);
}

template <typename T, int D>
cudaError_t fwd(const WindowArgs<T>& a, cudaStream_t st) {
  const long long ctas = (long long)((a.w.nq + kB - 1) / kB) * a.w.B * a.w.nh;
  return ctas <= device_sm_count() ? fwd<T, D, 2>(a, st) : fwd<T, D, 4>(a, st);
}

template <typename T, int D>
cudaError_t bwd(const WindowArgs<T>& a, cudaStream_t st) {
  constexpr int smem_dq = (4 * kB * kLd<D> + kB * kLdP) * 4, smem_kv = smem_dq + kB * kLdP * 4;
  constexpr int PER = D / kVec<T>, LANES = PER < 16 ? PER : 16;
  auto dq = window_dq_simt_kernel<T, D>;
  auto dkdv = window_dkdv_simt_kernel<T, D>;
  cudaError_t e = set_max_dynamic_smem((const void*)dq, smem_dq);
  if (e == cudaSuccess) e = set_max_dynamic_smem((const void*)dkdv, smem_kv);
  const int rows = kThreads / LANES;
  if (e == cudaSuccess)
    e = launch_pdl(window_delta_kernel<T, D>, dim3((a.w.nq + rows - 1) / rows, a.w.B * a.w.nh),
                   dim3(kThreads), 0, st, a);
  if (e == cudaSuccess)
    e = launch_pdl(dq, dim3((a.w.nq + kB - 1) / kB, a.w.B * a.w.nh), dim3(kThreads), smem_dq, st, a);
  if (e == cudaSuccess)
    e = launch_pdl(dkdv, dim3((a.w.nk + kB - 1) / kB, a.w.B * a.w.nkv), dim3(kThreads), smem_kv, st, a);
  return e;
}

}  // namespace

template <typename T>
cudaError_t launch_window_fwd_simt(const WindowArgs<T>& a, int d, cudaStream_t st) {
  return d == 64 ? fwd<T, 64>(a, st) : fwd<T, 128>(a, st);
}
template <typename T>
cudaError_t launch_window_bwd_simt(const WindowArgs<T>& a, int d, cudaStream_t st) {
  return d == 64 ? bwd<T, 64>(a, st) : bwd<T, 128>(a, st);
}
template cudaError_t launch_window_fwd_simt(const WindowArgs<float>&, int, cudaStream_t);
template cudaError_t launch_window_bwd_simt(const WindowArgs<float>&, int, cudaStream_t);

}  // namespace psa
