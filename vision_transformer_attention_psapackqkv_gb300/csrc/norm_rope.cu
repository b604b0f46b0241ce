// norm_rope.cu -- norms of queries and keys for each head with the position rotation, one
// pass over the data, and its backward.
//
//   xhat = x r, r = (mean(x^2) + eps)^(-1/2);  y = R (w o xhat), R the rotation by the
//   token's angles.  With g' = R^T g (the rotation by the negative angles) the backward is
//     dx = r (w o g' - xhat mean(w o g' o xhat)),   dw = sum over rows of g' o xhat.
//
// Bound by memory: a row is read once and written once, nothing else is large.  A row of d
// channels lies in d / kVec neighbouring lanes, 16 bytes in each, so every access is a
// whole sector and the sums are shuffles inside a warp.  A group of lanes keeps one
// token's angles in registers and goes through several heads of it, so the tables (8 bytes
// of table for 2 bytes of bf16 data) are read once for kHeads heads; few tokens (decoding)
// take one head per group instead, where the latency of one row is the whole time.
#include <algorithm>

#include "lm.cuh"
#include "ptx.cuh"

namespace psa {
namespace {

constexpr int kThreads = 256;

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = LANES / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// One lane's part of a token's rotation: y = c o x + s o x', where x' is the partner
// channel of each (in this lane, interleaved; in lane `partner`, split halves).
template <int VEC>
struct Turn {
  float c[VEC], s[VEC];
  int partner;

  // sign: +1 forward, -1 the inverse rotation
  template <typename T>
  __device__ __forceinline__ void load(const NormRopeArgs<T>& a, int pos, int lane_in_row,
                                       int lanes, float sign) {
    const int c0 = lane_in_row * VEC, half = a.rot / 2;
    const int lane = threadIdx.x & 31;
    partner = lane;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      c[e] = 1.f;
      s[e] = 0.f;
    }
    if (c0 >= a.rot) return;
    const float* ct = a.cos + (long long)pos * half;
    const float* st = a.sin + (long long)pos * half;
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        const float2 cc = *reinterpret_cast<const float2*>(ct + (c0 + e) / 2);
        const float2 ss = *reinterpret_cast<const float2*>(st + (c0 + e) / 2);
        c[e] = c[e + 1] = cc.x;
        c[e + 2] = c[e + 3] = cc.y;
        s[e] = -sign * ss.x;
        s[e + 1] = sign * ss.x;
        s[e + 2] = -sign * ss.y;
        s[e + 3] = sign * ss.y;
      }
    } else {
      const bool low = c0 < half;
      const int i0 = low ? c0 : c0 - half;
      const float sg = low ? -sign : sign;
      partner = low ? lane + half / VEC : lane - half / VEC;
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        const float4 cc = *reinterpret_cast<const float4*>(ct + i0 + e);
        const float4 ss = *reinterpret_cast<const float4*>(st + i0 + e);
        c[e] = cc.x;
        c[e + 1] = cc.y;
        c[e + 2] = cc.z;
        c[e + 3] = cc.w;
        s[e] = sg * ss.x;
        s[e + 1] = sg * ss.y;
        s[e + 2] = sg * ss.z;
        s[e + 3] = sg * ss.w;
      }
    }
  }

  // every lane of the warp takes part (shuffles)
  __device__ __forceinline__ void apply(bool interleaved, float (&x)[VEC]) const {
    float y[VEC];
    if (interleaved) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[e] = x[e ^ 1];
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = c[e] * x[e] + s[e] * y[e];
  }
};

template <int VEC>
__device__ __forceinline__ void load_weight(const float* w, int c0, float (&x)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] = w ? w[c0 + e] : 1.f;
}

// A group takes HEADS heads of its token: blockIdx.y counts the chunks of q's heads (nqc of
// them), then those of k's, so that no chunk holds heads of both.
template <typename T, int D, int HEADS>
__global__ void __launch_bounds__(kThreads) norm_rope_fwd_kernel(const NormRopeArgs<T> a, int nqc) {
  constexpr int VEC = kVec<T>, LANES = D / VEC, GROUPS = kThreads / LANES;
  pdl_launch_dependents();
  pdl_wait();
  const int lr = threadIdx.x % LANES, c0 = lr * VEC;
  const long long token = (long long)blockIdx.x * GROUPS + threadIdx.x / LANES;
  const bool live = token < (long long)a.B * a.N;
  const int b = live ? (int)(token / a.N) : 0, n = live ? (int)(token % a.N) : 0;
  const bool is_q = (int)blockIdx.y < nqc;
  const int h0 = (is_q ? blockIdx.y : blockIdx.y - nqc) * HEADS;
  const int heads = is_q ? a.nh : a.nkv;
  const View<const T> in = is_q ? a.q : a.k;
  const View<T> out = is_q ? a.oq : a.ok;

  uint4 raw[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i)
    raw[i] = live && h0 + i < heads ? *reinterpret_cast<const uint4*>(in.row(b, h0 + i, n) + c0)
                                    : make_uint4(0, 0, 0, 0);
  int pos = n;
  if (a.positions && live) pos = a.positions[token];
  const bool valid = live && pos >= 0 && pos < a.max_pos;
  Turn<VEC> turn;
  turn.load(a, valid ? pos : 0, lr, LANES, 1.f);
  float w[VEC];
  load_weight(is_q ? a.wq : a.wk, c0, w);
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    float x[VEC];
    unpack_vec(raw[i], x);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) ss += x[e] * x[e];
    const float r = rsqrtf(group_sum<LANES>(ss) * (1.f / D) + a.eps);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = x[e] * r * w[e];
    turn.apply(a.interleaved, x);
    if (valid && h0 + i < heads)
      *reinterpret_cast<uint4*>(out.row(b, h0 + i, n) + c0) = pack_vec(x);
  }
}

// A CTA goes through tokens blockIdx.x * GROUPS + group, + gridDim.x * GROUPS, ... and a
// chunk of heads of q or of k; its sum of g' o xhat is one row of partial sums.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    norm_rope_bwd_kernel(const NormRopeArgs<T> a, int nqc, int heads_per) {
  constexpr int VEC = kVec<T>, LANES = D / VEC, GROUPS = kThreads / LANES;
  __shared__ float part[GROUPS][D];
  pdl_launch_dependents();
  pdl_wait();
  const int lr = threadIdx.x % LANES, grp = threadIdx.x / LANES, c0 = lr * VEC;
  const long long tokens = (long long)a.B * a.N;
  const bool is_q = (int)blockIdx.y < nqc;
  const int chunk = is_q ? blockIdx.y : blockIdx.y - nqc;
  const int heads = is_q ? a.nh : a.nkv;
  const int h0 = chunk * heads_per, h1 = min(heads, h0 + heads_per);
  const View<const T> in = is_q ? a.q : a.k, gin = is_q ? a.gq : a.gk;
  const View<T> out = is_q ? a.oq : a.ok;
  float w[VEC], dw[VEC];
  load_weight(is_q ? a.wq : a.wk, c0, w);
#pragma unroll
  for (int e = 0; e < VEC; ++e) dw[e] = 0.f;

  for (long long t0 = (long long)blockIdx.x * GROUPS; t0 < tokens; t0 += (long long)gridDim.x * GROUPS) {
    const long long token = t0 + grp;
    const bool live = token < tokens;
    const int b = live ? (int)(token / a.N) : 0, n = live ? (int)(token % a.N) : 0;
    int pos = n;
    if (a.positions && live) pos = a.positions[token];
    const bool valid = live && pos >= 0 && pos < a.max_pos;
    Turn<VEC> turn;
    turn.load(a, valid ? pos : 0, lr, LANES, -1.f);
    for (int h = h0; h < h1; ++h) {
      uint4 rx = make_uint4(0, 0, 0, 0), rg = rx;
      if (valid) {
        rx = *reinterpret_cast<const uint4*>(in.row(b, h, n) + c0);
        rg = *reinterpret_cast<const uint4*>(gin.row(b, h, n) + c0);
      }
      float x[VEC], g[VEC];
      unpack_vec(rx, x);
      unpack_vec(rg, g);
      turn.apply(a.interleaved, g);
      float ss = 0.f, gx = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        ss += x[e] * x[e];
        gx += g[e] * w[e] * x[e];
      }
      ss = group_sum<LANES>(ss);
      gx = group_sum<LANES>(gx);
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const float back = gx * r * r * (1.f / D);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        // rows of padding hold zeros here: their share is 0 and their dx is 0
        dw[e] += g[e] * (x[e] * r);
        x[e] = r * (g[e] * w[e] - x[e] * back);
      }
      if (live) *reinterpret_cast<uint4*>(out.row(b, h, n) + c0) = pack_vec(x);
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) part[grp][c0 + e] = dw[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) s += part[i][threadIdx.x];
    const int row = chunk * gridDim.x + blockIdx.x;
    a.ws[((is_q ? 0 : kNormRopeParts) + row) * D + threadIdx.x] = s;
  }
}

// Sums the partial rows of 32 channels of one weight: warp w takes rows w, w + 32, ...,
// then the warps' sums are added in order.
__global__ void __launch_bounds__(1024)
    norm_rope_dw_kernel(const float* ws, float* dwq, float* dwk, int rows_q, int rows_k, int D) {
  __shared__ float part[32][33];
  pdl_launch_dependents();
  pdl_wait();
  float* dw = blockIdx.y == 0 ? dwq : dwk;
  if (!dw) return;
  const int rows = blockIdx.y == 0 ? rows_q : rows_k;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
  const float* src = ws + (blockIdx.y == 0 ? 0 : kNormRopeParts * D) + c;
  float s = 0.f;
#pragma unroll 4
  for (int r = warp; r < rows; r += 32) s += src[r * D];
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += part[i][lane];
    dw[c] = s;
  }
}

int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

template <typename T, int D, int HEADS>
cudaError_t fwd(const NormRopeArgs<T>& a, cudaStream_t st) {
  constexpr int GROUPS = kThreads / (D / kVec<T>);
  const int nqc = cdiv(a.nh, HEADS), nkc = cdiv(a.nkv, HEADS);
  return launch_pdl(norm_rope_fwd_kernel<T, D, HEADS>,
                    dim3(cdiv((long long)a.B * a.N, GROUPS), nqc + nkc), dim3(kThreads), 0, st, a, nqc);
}

template <typename T, int D>
cudaError_t fwd(const NormRopeArgs<T>& a, cudaStream_t st) {
  // four heads per group once that still fills the device's threads
  const long long rows = (long long)a.B * a.N * (a.nh + a.nkv);
  return rows * (D / kVec<T>) / 4 >= 152 * 2048LL ? fwd<T, D, 4>(a, st) : fwd<T, D, 1>(a, st);
}

template <typename T, int D>
cudaError_t bwd(const NormRopeArgs<T>& a, cudaStream_t st) {
  constexpr int GROUPS = kThreads / (D / kVec<T>);
  // at most kNormRopeParts partial rows for each weight: chunks of at least 4 heads, and
  // as many token blocks as fit
  const int most = std::max(a.nh, a.nkv);
  const int heads_per = std::max(4, cdiv(most, 256));
  const int nqc = cdiv(a.nh, heads_per), nkc = cdiv(a.nkv, heads_per);
  const int gx = std::max(1, std::min(cdiv((long long)a.B * a.N, GROUPS), kNormRopeParts / std::max(nqc, nkc)));
  cudaError_t e = launch_pdl(norm_rope_bwd_kernel<T, D>, dim3(gx, nqc + nkc), dim3(kThreads), 0, st,
                             a, nqc, heads_per);
  if (e != cudaSuccess || (!a.dwq && !a.dwk)) return e;
  return launch_pdl(norm_rope_dw_kernel, dim3(D / 32, 2), dim3(1024), 0, st, (const float*)a.ws,
                    a.dwq, a.dwk, gx * nqc, gx * nkc, D);
}

}  // namespace

template <typename T>
cudaError_t launch_norm_rope_fwd(const NormRopeArgs<T>& a, int d, cudaStream_t st) {
  return d == 32 ? fwd<T, 32>(a, st) : d == 64 ? fwd<T, 64>(a, st) : fwd<T, 128>(a, st);
}
template <typename T>
cudaError_t launch_norm_rope_bwd(const NormRopeArgs<T>& a, int d, cudaStream_t st) {
  return d == 32 ? bwd<T, 32>(a, st) : d == 64 ? bwd<T, 64>(a, st) : bwd<T, 128>(a, st);
}
template cudaError_t launch_norm_rope_fwd(const NormRopeArgs<float>&, int, cudaStream_t);
template cudaError_t launch_norm_rope_fwd(const NormRopeArgs<__nv_bfloat16>&, int, cudaStream_t);
template cudaError_t launch_norm_rope_bwd(const NormRopeArgs<float>&, int, cudaStream_t);
template cudaError_t launch_norm_rope_bwd(const NormRopeArgs<__nv_bfloat16>&, int, cudaStream_t);

}  // namespace psa
