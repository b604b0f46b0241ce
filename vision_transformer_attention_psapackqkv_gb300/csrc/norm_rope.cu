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
// of table for 2 bytes of bf16 data) are read once for eight heads; few tokens (decoding)
// take one head per group instead, where the latency of one row is the whole time.
// Measured, bf16: 2 x 8192 tokens of 32 + 8 heads of 128 channels, read from a packed
// projection: forward 56.5 us (5.9 TB/s, 0.89 of the copy bandwidth), backward 109 us (4.6 TB/s;
// with 116 registers for two rows in work and two on their way, 16 warps per SM are what
// bounds it); 64 tokens: 2.8 us.
#include <algorithm>

#include "lm.cuh"
#include "ptx.cuh"

namespace psa {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 2;  // heads whose rows a group loads at once, backward

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = LANES / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Pairs of channels: one instruction for two.
__device__ __forceinline__ float2 at2(const float* x) { return make_float2(x[0], x[1]); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ void set2(float* x, float2 v) {
  x[0] = v.x;
  x[1] = v.y;
}
template <int VEC>
__device__ __forceinline__ float dot(const float (&x)[VEC], const float (&y)[VEC]) {
  float2 s = __fmul2_rn(at2(x), at2(y));
#pragma unroll
  for (int e = 2; e < VEC; e += 2) s = __ffma2_rn(at2(x + e), at2(y + e), s);
  return s.x + s.y;
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
                                       float sign) {
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

  // c o x + s o x' of a packed row (every lane of the warp takes part: shuffles); x returns the
  // row itself
  template <typename T>
  __device__ __forceinline__ void apply(bool interleaved, const uint4& raw, float (&x)[VEC],
                                        float (&y)[VEC]) const {
    unpack_vec(raw, x);
    if (interleaved) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[e] = x[e ^ 1];
    } else {
      uint4 other;
      other.x = __shfl_sync(0xffffffffu, raw.x, partner);
      other.y = __shfl_sync(0xffffffffu, raw.y, partner);
      other.z = __shfl_sync(0xffffffffu, raw.z, partner);
      other.w = __shfl_sync(0xffffffffu, raw.w, partner);
      unpack_vec(other, y);
    }
#pragma unroll
    for (int e = 0; e < VEC; e += 2)
      set2(y + e, __ffma2_rn(at2(c + e), at2(x + e), __fmul2_rn(at2(s + e), at2(y + e))));
  }
  // the weights of x and of x' go into c and s
  __device__ __forceinline__ void weigh(bool interleaved, const float (&w)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      c[e] *= w[e];
      s[e] *= interleaved ? w[e ^ 1] : __shfl_sync(0xffffffffu, w[e], partner);
    }
  }
};

// (the weights need only be 4-byte aligned)
template <int VEC>
__device__ __forceinline__ void load_weight(const float* w, int c0, float (&x)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] = 1.f;
  if (w) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = w[c0 + e];
  }
}

// A group takes HEADS heads of its token: blockIdx.y counts the chunks of q's heads (nqc of
// them), then those of k's, so that no chunk holds heads of both.
template <typename T, int D, int HEADS>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_fwd_kernel(const NormRopeArgs<T> a, int nqc) {
  constexpr int VEC = kVec<T>, LANES = D / VEC, GROUPS = kThreads / LANES;
  pdl_launch_dependents();
  pdl_wait();
  const int lr = threadIdx.x % LANES, c0 = lr * VEC;
  const unsigned token = blockIdx.x * GROUPS + threadIdx.x / LANES;
  const bool live = token < (unsigned)(a.B * a.N);
  const int b = live ? token / (unsigned)a.N : 0, n = live ? token - b * a.N : 0;
  const bool is_q = (int)blockIdx.y < nqc;
  const int h0 = (is_q ? blockIdx.y : blockIdx.y - nqc) * HEADS;
  const int heads = (live ? is_q ? a.nh : a.nkv : 0) - h0;  // this group's
  const long long in_sh = is_q ? a.q.sh : a.k.sh, out_sh = is_q ? a.oq.sh : a.ok.sh;
  const T* in = (is_q ? a.q.row(b, h0, n) : a.k.row(b, h0, n)) + c0;
  T* out = (is_q ? a.oq.row(b, h0, n) : a.ok.row(b, h0, n)) + c0;

  uint4 raw[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i)
    raw[i] = i < heads ? *reinterpret_cast<const uint4*>(in + i * in_sh) : make_uint4(0, 0, 0, 0);
  int pos = n;
  if (a.positions && live) pos = a.positions[token];
  const bool valid = live && pos >= 0 && pos < a.max_pos;
  Turn<VEC> turn;
  turn.load(a, valid ? pos : 0, lr, 1.f);
  float w[VEC];
  load_weight(is_q ? a.wq : a.wk, c0, w);
  turn.weigh(a.interleaved, w);
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    // y = r (R (w o x)): the root's factor comes last
    float x[VEC], y[VEC];
    turn.template apply<T>(a.interleaved, raw[i], x, y);
    const float r = rsqrtf(group_sum<LANES>(dot(x, x)) * (1.f / D) + a.eps);
#pragma unroll
    for (int e = 0; e < VEC; e += 2) set2(y + e, __fmul2_rn(at2(y + e), both(r)));
    if (valid && i < heads) *reinterpret_cast<uint4*>(out + i * out_sh) = pack_vec(y);
  }
}

// A CTA goes through tokens blockIdx.x * GROUPS + group, + gridDim.x * GROUPS, ... and a
// chunk of heads of q or of k; its sum of g' o xhat is one row of partial sums.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2)
    norm_rope_bwd_kernel(const NormRopeArgs<T> a, int nqc, int heads_per) {
  constexpr int VEC = kVec<T>, LANES = D / VEC, GROUPS = kThreads / LANES;
  __shared__ float part[GROUPS][D];
  pdl_launch_dependents();
  pdl_wait();
  const int lr = threadIdx.x % LANES, grp = threadIdx.x / LANES, c0 = lr * VEC;
  const unsigned tokens = a.B * a.N;
  const bool is_q = (int)blockIdx.y < nqc;
  const int chunk = is_q ? blockIdx.y : blockIdx.y - nqc;
  const int h0 = chunk * heads_per, heads = min((is_q ? a.nh : a.nkv) - h0, heads_per);
  const View<const T> in = is_q ? a.q : a.k, gin = is_q ? a.gq : a.gk;
  const View<T> out = is_q ? a.oq : a.ok;
  float w[VEC], dw[VEC];
  load_weight(is_q ? a.wq : a.wk, c0, w);
#pragma unroll
  for (int e = 0; e < VEC; ++e) dw[e] = 0.f;

  for (unsigned t0 = blockIdx.x * GROUPS; t0 < tokens; t0 += gridDim.x * GROUPS) {
    const unsigned token = t0 + grp;
    const bool live = token < tokens;
    const int b = live ? token / (unsigned)a.N : 0, n = live ? token - b * a.N : 0;
    int pos = n;
    if (a.positions && live) pos = a.positions[token];
    const bool valid = live && pos >= 0 && pos < a.max_pos;
    const T *x0 = in.row(b, h0, n) + c0, *g0 = gin.row(b, h0, n) + c0;
    T* d0 = out.row(b, h0, n) + c0;
    Turn<VEC> turn;
    turn.load(a, valid ? pos : 0, lr, -1.f);
    // the next kBatch heads' rows are on their way while these are worked on
    uint4 nx[kBatch], ng[kBatch];
    auto load = [&](int h) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        nx[i] = ng[i] = make_uint4(0, 0, 0, 0);
        if (valid && h + i < heads) {
          nx[i] = *reinterpret_cast<const uint4*>(x0 + (h + i) * in.sh);
          ng[i] = *reinterpret_cast<const uint4*>(g0 + (h + i) * gin.sh);
        }
      }
    };
    load(0);
    for (int h = 0; h < heads; h += kBatch) {
      uint4 rx[kBatch], rg[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        rx[i] = nx[i];
        rg[i] = ng[i];
      }
      load(h + kBatch);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        float x[VEC], g[VEC], raw[VEC];
        unpack_vec(rx[i], x);
        turn.template apply<T>(a.interleaved, rg[i], raw, g);
        float gw[VEC];
#pragma unroll
        for (int e = 0; e < VEC; e += 2) set2(gw + e, __fmul2_rn(at2(g + e), at2(w + e)));
        const float ss = group_sum<LANES>(dot(x, x)), gx = group_sum<LANES>(dot(gw, x));
        // rows of padding, and those past the last head, hold zeros here: with r = 0 (without it
        // eps = 0 makes NaN of them) their share is 0 and their dx is 0
        const float r = valid && h + i < heads ? rsqrtf(ss * (1.f / D) + a.eps) : 0.f;
        const float2 r2 = both(r), back = both(-gx * r * r * (1.f / D));
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const float2 xe = at2(x + e);
          set2(dw + e, __ffma2_rn(at2(g + e), __fmul2_rn(xe, r2), at2(dw + e)));
          set2(x + e, __fmul2_rn(r2, __ffma2_rn(xe, back, at2(gw + e))));
        }
        if (live && h + i < heads) *reinterpret_cast<uint4*>(d0 + (h + i) * out.sh) = pack_vec(x);
      }
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
#pragma unroll 8
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
  // eight heads per group, or four, once that still fills the device's threads
  const long long lanes = (long long)a.B * a.N * (a.nh + a.nkv) * (D / kVec<T>), full = 152 * 2048;
  return lanes / 8 >= full ? fwd<T, D, 8>(a, st) : lanes / 4 >= full ? fwd<T, D, 4>(a, st) : fwd<T, D, 1>(a, st);
}

template <typename T, int D>
cudaError_t bwd(const NormRopeArgs<T>& a, cudaStream_t st) {
  constexpr int GROUPS = kThreads / (D / kVec<T>);
  // up to four CTAs per SM between the chunks of heads, each with one partial row: chunks of
  // 8 heads (the angles are loaded once for them) where there are tokens enough, else of 4
  const int blocks = cdiv((long long)a.B * a.N, GROUPS);
  const int chunks8 = cdiv(a.nh, 8) + cdiv(a.nkv, 8);
  int heads_per = (long long)blocks * chunks8 >= kNormRopeParts ? 8 : 4;
  heads_per = std::max(heads_per, cdiv(std::max(a.nh, a.nkv), kNormRopeParts / 2));
  const int nqc = cdiv(a.nh, heads_per), nkc = cdiv(a.nkv, heads_per);
  const int gx = std::max(1, std::min(blocks, kNormRopeParts / (nqc + nkc)));
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
