// window_simt.cu -- attention with a sliding window and first tokens that stay visible, on
// CUDA cores in fp32: forward, and the dQ and dK/dV kernels of the backward.
//
//   S = scale Q K^T over the visible keys, P = exp(S - lse), O = P V;
//   dV = P^T dO, dP = dO V^T, dS = P o (dP - delta), delta = rowsum(dO o O),
//   dQ = scale dS K, dK = scale dS^T Q.
//
// A CTA owns 32 or 16 query rows (key rows in dK/dV) and goes through the 64-row tiles of the
// other side that its rows see, so a score exists only in registers and shared memory.  16
// threads share a row: a thread holds the scores of 4 (or 2) rows, kGap apart, and columns
// tx + 16 j, and of each product with V (K, dO, Q) its rows' channels 4 tx + 64 c .. + 3.  What
// bounds it is reads of shared memory (busy 66 to 78 % of the time, the FMA pipe 20 to 33 %,
// each of its instructions two products).  Few rows in a CTA waste less at a window's or a
// triangle's edge and balance better: 2 x 1024 causal, 8 heads of 128, forward 196 us with 64
// rows, 187 with 32, backward 670 and 629; eight rows a thread would read less, but leave too
// few warps (214).  Tiles come asynchronously, the forward's V during the scores and K's next
// during P V (4 maps of 400: 31 -> 28 us with 64 rows), dQ's next V during dS K.
// Measured, fp32: 4 maps of 400 positions, 4 heads of 64, 121 keys a query: 22 us forward, 80
// backward; 2 x 1024 causal, 8 heads of 128: 187 and 629 us.
// Tiles lie row by row in shared memory with 4 floats of padding: 16-byte reads of eight
// neighbouring rows then fall into different banks.  Every key/value head's gradient is
// summed by one CTA over its query heads and tiles in order, so reruns are bitwise equal.
#include <math.h>

#include "lm.cuh"
#include "ptx.cuh"

namespace psa {
namespace {

constexpr int kB = 64;  // rows of a tile, on either side
constexpr int kThreads = 256;  // of the kernel of delta
constexpr int kLdP = kB + 4;  // row pitch of a tile of scores

template <int D>
constexpr int kLd = D + 4;

// Rows i0 .. i0 + kRows - 1 of one head into shared memory; rows outside [lo, hi) as 0.
// Asynchronously: to be waited for with fetched(), then a barrier.
template <int D, int kN, int kRows>
__device__ __forceinline__ void fetch_rows(float* dst, const float* base, long long sn, int i0, int lo,
                                           int hi) {
  for (int u = threadIdx.x; u < kRows * (D / 4); u += kN) {
    const int r = u / (D / 4), c = u % (D / 4) * 4, i = i0 + r;
    const bool in = i >= lo && i < hi;
    // no byte is read for a row outside, its 16 are zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst + r * kLd<D> + c)),
                 "l"(base + (in ? i * sn + c : 0)), "r"(in ? 16 : 0)
                 : "memory");
  }
}
__device__ __forceinline__ void fetched() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// acc[i][j] = sum over d of A[ty + kGap i][d] B[tx + 16 j][d]
template <int D, int R, int kGap>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ty, int tx,
                                         float (&acc)[R][4]) {
  constexpr int kR = R;
  float2 sum[kR][4];  // of the even and of the odd channels: two products per instruction
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[i][j] = make_float2(0.f, 0.f);
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
      for (int j = 0; j < 4; ++j) {
        sum[i][j] = __ffma2_rn(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), sum[i][j]);
        sum[i][j] = __ffma2_rn(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), sum[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = sum[i][j].x + sum[i][j].y;
}

// acc[i][4 c + e] += sum over the 64 rows m of P[ty + kGap i][m] B[m][4 tx + 64 c + e]
template <int D, int R, int kGap>
__device__ __forceinline__ void mix_tile(const float* P, const float* B, int ty, int tx,
                                         float (&acc)[R][D / 16]) {
  constexpr int kR = R;
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
          float* o = acc[i] + 4 * c;
          const float2 lo = __ffma2_rn(make_float2(w, w), make_float2(y.x, y.y), make_float2(o[0], o[1]));
          const float2 hi = __ffma2_rn(make_float2(w, w), make_float2(y.z, y.w), make_float2(o[2], o[3]));
          o[0] = lo.x;
          o[1] = lo.y;
          o[2] = hi.x;
          o[3] = hi.y;
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

__device__ __forceinline__ void store4(float* dst, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(dst) = make_float4(a, b, c, d);
}

template <int D, int kRows, int R>
__global__ void __launch_bounds__(16 * kRows / R) window_fwd_simt_kernel(const WindowArgs<float> a) {
  constexpr int kR = R, kGap = kRows / R, kN = 16 * kGap;
  extern __shared__ float sm[];
  float *Q = sm, *K = Q + kRows * kLd<D>, *V = K + kB * kLd<D>, *P = V + kB * kLd<D>;
  pdl_launch_dependents();
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = blockIdx.y / a.w.nh, h = blockIdx.y % a.w.nh, hk = h / (a.w.nh / a.w.nkv);
  const int len = a.w.len(b), off = a.w.nk - a.w.nq;
  // the last tiles of a causal problem see the most keys: they start first
  const int i0 = (gridDim.x - 1 - blockIdx.x) * kRows;
  const int p0 = i0 + off;
  const KeyTiles<kB> tiles(a.w, len, max(p0, 0), min(min(p0 + kRows, a.w.nk) - 1, len - 1));
  fetch_rows<D, kN, kRows>(Q, a.q.row(b, h, 0), a.q.sn, i0, max(0, -off), min(a.w.nq, len - off));
  const float *k = a.k.row(b, hk, 0), *v = a.v.row(b, hk, 0);
  if (tiles.count > 0) fetch_rows<D, kN, kB>(K, k, a.k.sn, tiles.tile(0) * kB, 0, len);

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
    // K's tile is there and V's is free; V's comes during the scores, K's next during P V
    fetched();
    __syncthreads();
    fetch_rows<D, kN, kB>(V, v, a.v.sn, j0, 0, len);
    float s[kR][4];
    dot_tile<D, kR, kGap>(Q, K, ty, tx, s);
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
    fetched();
    __syncthreads();
    if (t + 1 < tiles.count) fetch_rows<D, kN, kB>(K, k, a.k.sn, tiles.tile(t + 1) * kB, 0, len);
    mix_tile<D, kR, kGap>(P, V, ty, tx, o);
  }
  fetched();  // (a block without keys still has Q on its way)
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int q = i0 + ty + kGap * i;
    if (q >= a.w.nq) continue;
    // a sum of 0 is a row that sees nothing; a NaN among the scores stays one
    const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;
    float* dst = a.out.row(b, h, q) + 4 * tx;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      store4(dst + 64 * c, o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv,
             o[i][4 * c + 3] * inv);
    if (a.lse && tx == 0)
      a.lse[(long long)blockIdx.y * a.w.nq + q] = l[i] != 0.f ? m[i] + logf(l[i]) : -INFINITY;
  }
}

// delta = rowsum(dO o O), one row per 16 lanes; 0 for rows that see nothing (whose dO and
// O may hold anything).
template <int D>
__global__ void __launch_bounds__(kThreads) window_delta_kernel(const WindowArgs<float> a) {
  constexpr int LANES = 16;
  pdl_launch_dependents();
  pdl_wait();
  const int lr = threadIdx.x % LANES;
  const int i = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const int b = blockIdx.y / a.w.nh, h = blockIdx.y % a.w.nh;
  const int p = i + a.w.nk - a.w.nq;
  const bool live = i < a.w.nq && p >= 0 && p < a.w.len(b);
  float s = 0.f;
#pragma unroll
  for (int c = 4 * lr; c < D; c += 4 * LANES) {
    if (!live) continue;
    const float4 x = *reinterpret_cast<const float4*>(a.dO.row(b, h, i) + c);
    const float4 y = *reinterpret_cast<const float4*>(a.o.row(b, h, i) + c);
    s += x.x * y.x;
    s += x.y * y.y;
    s += x.z * y.z;
    s += x.w * y.w;
  }
#pragma unroll
  for (int m = LANES / 2; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  if (lr == 0 && i < a.w.nq) a.delta[(long long)blockIdx.y * a.w.nq + i] = s;
}

template <int D, int kRows, int R>
__global__ void __launch_bounds__(16 * kRows / R) window_dq_simt_kernel(const WindowArgs<float> a) {
  constexpr int kR = R, kGap = kRows / R, kN = 16 * kGap;
  extern __shared__ float sm[];
  float *Q = sm, *dO = Q + kRows * kLd<D>, *K = dO + kRows * kLd<D>, *V = K + kB * kLd<D>,
        *S = V + kB * kLd<D>;
  pdl_launch_dependents();
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = blockIdx.y / a.w.nh, h = blockIdx.y % a.w.nh, hk = h / (a.w.nh / a.w.nkv);
  const int len = a.w.len(b), off = a.w.nk - a.w.nq;
  const int i0 = (gridDim.x - 1 - blockIdx.x) * kRows;
  const int p0 = i0 + off;
  const KeyTiles<kB> tiles(a.w, len, max(p0, 0), min(min(p0 + kRows, a.w.nk) - 1, len - 1));
  const int lo = max(0, -off), hi = min(a.w.nq, len - off);
  fetch_rows<D, kN, kRows>(Q, a.q.row(b, h, 0), a.q.sn, i0, lo, hi);
  fetch_rows<D, kN, kRows>(dO, a.dO.row(b, h, 0), a.dO.sn, i0, lo, hi);
  const float* v = a.v.row(b, hk, 0);
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
    fetch_rows<D, kN, kB>(K, a.k.row(b, hk, 0), a.k.sn, j0, 0, len);
    if (t == 0) fetch_rows<D, kN, kB>(V, v, a.v.sn, j0, 0, len);
    fetched();
    __syncthreads();
    float s[kR][4], dp[kR][4];
    dot_tile<D, kR, kGap>(Q, K, ty, tx, s);
    dot_tile<D, kR, kGap>(dO, V, ty, tx, dp);
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
    // V's next tile comes during dS K
    if (t + 1 < tiles.count) fetch_rows<D, kN, kB>(V, v, a.v.sn, tiles.tile(t + 1) * kB, 0, len);
    mix_tile<D, kR, kGap>(S, K, ty, tx, acc);
  }
  fetched();
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int q = i0 + ty + kGap * i;
    if (q >= a.w.nq) continue;
    float* dst = a.dq.row(b, h, q) + 4 * tx;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      store4(dst + 64 * c, acc[i][4 * c] * a.scale, acc[i][4 * c + 1] * a.scale,
             acc[i][4 * c + 2] * a.scale, acc[i][4 * c + 3] * a.scale);
  }
}

template <int D, int kRows, int R>
__global__ void __launch_bounds__(16 * kRows / R) window_dkdv_simt_kernel(const WindowArgs<float> a) {
  constexpr int kR = R, kGap = kRows / R, kN = 16 * kGap;
  extern __shared__ float sm[];
  float *K = sm, *V = K + kRows * kLd<D>, *Q = V + kRows * kLd<D>, *dO = Q + kB * kLd<D>,
        *P = dO + kB * kLd<D>, *S = P + kRows * kLdP;
  __shared__ float lse[kB], delta[kB];
  pdl_launch_dependents();
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = blockIdx.y / a.w.nkv, hk = blockIdx.y % a.w.nkv, group = a.w.nh / a.w.nkv;
  const int len = a.w.len(b), off = a.w.nk - a.w.nq;
  const int j0 = blockIdx.x * kRows;
  int i0, nq;
  query_range(a.w, len, j0, min(j0 + kRows, a.w.nk) - 1, i0, nq);
  fetch_rows<D, kN, kRows>(K, a.k.row(b, hk, 0), a.k.sn, j0, 0, len);
  fetch_rows<D, kN, kRows>(V, a.v.row(b, hk, 0), a.v.sn, j0, 0, len);
  float dk[kR][D / 16], dv[kR][D / 16];
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) dk[i][c] = dv[i][c] = 0.f;
  for (int h = hk * group; h < (hk + 1) * group; ++h) {
    for (int i1 = i0; i1 < i0 + nq; i1 += kB) {
      __syncthreads();
      fetch_rows<D, kN, kB>(Q, a.q.row(b, h, 0), a.q.sn, i1, i1, i0 + nq);
      fetch_rows<D, kN, kB>(dO, a.dO.row(b, h, 0), a.dO.sn, i1, i1, i0 + nq);
      for (int u = threadIdx.x; u < kB; u += kN) {
        const int i = i1 + u;
        const long long at = ((long long)b * a.w.nh + h) * a.w.nq + i;
        lse[u] = i < i0 + nq ? a.lse[at] : 0.f;
        delta[u] = i < i0 + nq ? a.delta[at] : 0.f;
      }
      fetched();
      __syncthreads();
      float s[kR][4], dp[kR][4];  // rows: keys, columns: queries
      dot_tile<D, kR, kGap>(K, Q, ty, tx, s);
      dot_tile<D, kR, kGap>(V, dO, ty, tx, dp);
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
      mix_tile<D, kR, kGap>(P, dO, ty, tx, dv);
      mix_tile<D, kR, kGap>(S, Q, ty, tx, dk);
    }
  }
  fetched();  // (a block that no query sees still has K and V on their way)
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int j = j0 + ty + kGap * i;
    if (j >= a.w.nk) continue;
    float *dkr = a.dk.row(b, hk, j) + 4 * tx, *dvr = a.dv.row(b, hk, j) + 4 * tx;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      store4(dkr + 64 * c, dk[i][4 * c] * a.scale, dk[i][4 * c + 1] * a.scale,
             dk[i][4 * c + 2] * a.scale, dk[i][4 * c + 3] * a.scale);
      store4(dvr + 64 * c, dv[i][4 * c], dv[i][4 * c + 1], dv[i][4 * c + 2], dv[i][4 * c + 3]);
    }
  }
}

// Tiles of 16 rows, with twice the threads a score, rather than 32, where that leaves no more
// than three CTAs per SM, which all run at once (heads of 64).  4 x 4 heads of 400 positions, 121
// visible: forward 22 us against 27, backward 80 against 98; 4 x 8 heads: 40 against 30, 128
// against 122.  Heads of 128 fill shared memory: 4 x 4 heads 47 against 37, 154 against 148.
template <int D>
bool few_rows(int rows, int heads) {
  return D == 64 && (long long)((rows + 15) / 16) * heads <= 3LL * device_sm_count();
}

template <int D, int kRows, int R>
cudaError_t fwd(const WindowArgs<float>& a, cudaStream_t st) {
  constexpr int smem = ((2 * kB + kRows) * kLd<D> + kRows * kLdP) * 4;
  auto kern = window_fwd_simt_kernel<D, kRows, R>;
  const cudaError_t e = set_max_dynamic_smem((const void*)kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((a.w.nq + kRows - 1) / kRows, a.w.B * a.w.nh), dim3(16 * kRows / R), smem, st, a);
}

template <int D>
cudaError_t fwd(const WindowArgs<float>& a, cudaStream_t st) {
  return few_rows<D>(a.w.nq, a.w.B * a.w.nh) ? fwd<D, 16, 2>(a, st) : fwd<D, 32, 4>(a, st);
}

template <int D, int kRows, int R>
cudaError_t dq(const WindowArgs<float>& a, cudaStream_t st) {
  constexpr int smem = ((2 * kB + 2 * kRows) * kLd<D> + kRows * kLdP) * 4;
  auto kern = window_dq_simt_kernel<D, kRows, R>;
  const cudaError_t e = set_max_dynamic_smem((const void*)kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((a.w.nq + kRows - 1) / kRows, a.w.B * a.w.nh), dim3(16 * kRows / R), smem, st, a);
}

template <int D, int kRows, int R>
cudaError_t dkdv(const WindowArgs<float>& a, cudaStream_t st) {
  constexpr int smem = ((2 * kB + 2 * kRows) * kLd<D> + 2 * kRows * kLdP) * 4;
  auto kern = window_dkdv_simt_kernel<D, kRows, R>;
  const cudaError_t e = set_max_dynamic_smem((const void*)kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3((a.w.nk + kRows - 1) / kRows, a.w.B * a.w.nkv), dim3(16 * kRows / R), smem, st, a);
}

template <int D>
cudaError_t bwd(const WindowArgs<float>& a, cudaStream_t st) {
  const int rows = kThreads / 16;
  cudaError_t e = launch_pdl(window_delta_kernel<D>, dim3((a.w.nq + rows - 1) / rows, a.w.B * a.w.nh),
                             dim3(kThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  e = few_rows<D>(a.w.nq, a.w.B * a.w.nh) ? dq<D, 16, 2>(a, st) : dq<D, 32, 4>(a, st);
  if (e != cudaSuccess) return e;
  return few_rows<D>(a.w.nk, a.w.B * a.w.nkv) ? dkdv<D, 16, 2>(a, st) : dkdv<D, 32, 4>(a, st);
}

}  // namespace

cudaError_t launch_window_fwd_simt(const WindowArgs<float>& a, int d, cudaStream_t st) {
  return d == 64 ? fwd<64>(a, st) : fwd<128>(a, st);
}
cudaError_t launch_window_bwd_simt(const WindowArgs<float>& a, int d, cudaStream_t st) {
  return d == 64 ? bwd<64>(a, st) : bwd<128>(a, st);
}

}  // namespace psa
