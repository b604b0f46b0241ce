// lm.cuh -- what the token-sequence kernels share: strided views of rows, which keys a
// query sees, and the launch interfaces behind include/psa.h's section on token
// sequences.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn.cuh"

namespace psa {

// A view [B, heads, N, d] (strides in elements, channels contiguous).
template <typename T>
struct View {
  T* p;
  long long sb, sh, sn;
  __host__ __device__ __forceinline__ T* row(int b, int h, int n) const {
    return p + (b * sb + h * sh + n * sn);
  }
};

// Elements of one 16-byte vector.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

__device__ __forceinline__ void unpack_vec(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack_vec(const uint4& u, float (&x)[4]) {
  x[0] = __uint_as_float(u.x);
  x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z);
  x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack_vec(const float (&x)[8]) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ uint4 pack_vec(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                    __float_as_uint(x[3]));
}

// ---------------------------------------------------------------- norms + rotation
// Positions of several axes: which axis each pair of channels turns with, and where a token
// stands on each.
struct RopeAxes {
  int axes, grid[4];     // grid: extents, the last axis innermost, where positions is null
  uint32_t axis_of[4];   // two bits for each pair of channels
  bool normalize;
};
template <typename T>
struct NormRopeArgs {
  View<const T> q, k;        // inputs
  View<const T> gq, gk;      // backward: gradients of the outputs
  View<T> oq, ok;            // forward: outputs; backward: gradients of the inputs
  const float *wq, *wk;      // [d] or null
  const float *cos, *sin;    // [max_pos, rot / 2]
  const int* positions;      // [B, N] or null; several axes: [axes, B, N]
  float *dwq, *dwk;          // backward: [d] or null
  float* ws;                 // backward: partial sums
  int B, nh, nkv, N, rot, max_pos;
  bool interleaved;
  float eps;
  RopeAxes ax;               // several axes
};
// Most CTAs of the backward, each with a partial sum of one weight's gradient in the
// workspace (four per SM).
constexpr int kNormRopeParts = 608;
template <typename T>
cudaError_t launch_norm_rope_fwd(const NormRopeArgs<T>& a, int d, cudaStream_t st);
template <typename T>
cudaError_t launch_norm_rope_bwd(const NormRopeArgs<T>& a, int d, cudaStream_t st);
// The same over several axes.
template <typename T>
cudaError_t launch_norm_rope_axes_fwd(const NormRopeArgs<T>& a, int d, cudaStream_t st);
template <typename T>
cudaError_t launch_norm_rope_axes_bwd(const NormRopeArgs<T>& a, int d, cudaStream_t st);

// ---------------------------------------------------------------- window attention
// A window problem: query i stands at position i + off (off = n_k - n_q); it sees key j
// iff j <= p + right and (j >= p - left or j < sinks), 0 <= p < len, j < len.  No limit
// on a side is a window of n_k there, so that no arithmetic has a special case.
struct Window {
  int B, nh, nkv, nq, nk;
  int left, right, sinks;  // left, right in 0 .. n_k, sinks in 0 .. n_k
  const int* lens;         // or null
  __device__ __forceinline__ int len(int b) const {
    return lens ? max(0, min(lens[b], nk)) : nk;
  }
};

// The key tiles of BN keys that queries at positions p0 .. p1 (not empty, within 0 ..
// len - 1) see between them: the sinks' tiles in front of the window, then the window's.
template <int BN>
struct KeyTiles {
  int sink, first, count;  // sink tiles 0 .. sink - 1, then first .. ; count in all
  KeyTiles() = default;
  __device__ __forceinline__ KeyTiles(const Window& w, int len, int p0, int p1) {
    if (p0 > p1) {
      sink = first = count = 0;
      return;
    }
    const int hi = min(len - 1, p1 + w.right), lo = max(0, p0 - w.left);
    first = lo / BN;
    sink = w.sinks > 0 ? min(first, (min(w.sinks, hi + 1) + BN - 1) / BN) : 0;
    count = sink + hi / BN - first + 1;
  }
  __device__ __forceinline__ int tile(int t) const { return t < sink ? t : first + t - sink; }
};

// Whether position p sees one key only: its probability is 1 whatever the score, so that no
// gradient passes through it (dP - delta would leave a rounding error instead of 0).  These are
// position 0, or the last one, or all of them, as the window is.
__device__ __forceinline__ bool sees_one(const Window& w, int len, int p) {
  if (p == 0) return w.right == 0 || len == 1;
  return w.left == 0 && w.sinks == 0 && (w.right == 0 || p == len - 1);
}

// The query rows (first, count) that see a key among k0 .. k1, clipped to n_q rows.
__host__ __device__ __forceinline__ void query_range(const Window& w, int len, int k0, int k1,
                                                     int& i0, int& n) {
  const int off = w.nk - w.nq, from = k0 - w.right;
  if (k1 > len - 1) k1 = len - 1;
  int p0 = off > 0 ? off : 0;
  if (p0 < from) p0 = from;
  int p1 = len - 1;
  if (k0 >= w.sinks && k1 + w.left < p1) p1 = k1 + w.left;
  i0 = p0 - off;
  n = k0 <= k1 && p1 >= p0 ? p1 - p0 + 1 : 0;
}

template <typename T>
struct WindowArgs {
  Window w;
  View<const T> q, k, v, o, dO;
  View<T> out, dq, dk, dv;
  float* lse;          // [B, nh, n_q]; forward: written (or null), backward: read
  float* delta;        // the backward's workspace; CUDA cores: rowsum(dO o O), [B, nh, n_q]
  float scale;
};
// Tensor cores (window_fwd.cu, window_bwd.cu); delta points at the backward's workspace.
cudaError_t launch_window_fwd_tc(const WindowArgs<__nv_bfloat16>& a, int d, cudaStream_t st);
// The rows that see something in fp32, [B, nh, n_q, d], and lse alone.
cudaError_t launch_window_fwd_raw(const WindowArgs<__nv_bfloat16>& a, float* raw, int d, cudaStream_t st);
cudaError_t launch_window_bwd_tc(const WindowArgs<__nv_bfloat16>& a, int d, cudaStream_t st);
size_t window_bwd_tc_ws_bytes(const Window& w, int d);
// CUDA cores (window_simt.cu).
cudaError_t launch_window_fwd_simt(const WindowArgs<float>& a, int d, cudaStream_t st);
cudaError_t launch_window_bwd_simt(const WindowArgs<float>& a, int d, cudaStream_t st);

// Sums of the probabilities for each key (window_weights.cu).
size_t window_weights_ws_bytes(const Window& w);
cudaError_t launch_window_weights(const Window& w, View<const __nv_bfloat16> q, View<const __nv_bfloat16> k,
                                  const float* lse, float* weights, float* ws, float scale, int d,
                                  cudaStream_t st);

// ---------------------------------------------------------------- caches
struct CacheArgs {
  int B, nkv, N, max_len;
  const int *starts, *counts;
};
template <typename T>
cudaError_t launch_kv_append(const CacheArgs& c, View<const T> k, View<const T> v, View<T> kc,
                             View<T> vc, int d, cudaStream_t st);
template <typename T>
cudaError_t launch_kv4_append(const CacheArgs& c, View<const T> k, View<const T> v, void* kcodes,
                              void* kscales, void* vcodes, void* vscales, int d, cudaStream_t st);
template <typename T>
cudaError_t launch_kv4_read(const CacheArgs& c, const void* kcodes, const void* kscales,
                            const void* vcodes, const void* vscales, View<T> k, View<T> v, int d,
                            cudaStream_t st);

// ---------------------------------------------------------------- eviction from a cache
struct EvictArgs {
  int B, nkv, max_len, keep, sinks, recent;
  const float* weights;    // [B, nkv, max_len]
  const int* positions;    // [B, nkv, max_len]
  const int* lens;         // [B]
  View<uint4> k, v;        // strides in 16 bytes
  float* weights_out;
  int *positions_out, *lens_out;
  int *counts, *moves;     // workspace: moves of each list, then their sources and targets,
  uint32_t* words;         // then two bits for each row of lists that shared memory does not hold
};
size_t evict_ws_bytes(int lists, int keep, int max_len);
cudaError_t launch_kv_evict(EvictArgs a, int row16, void* ws, cudaStream_t st);

// ---------------------------------------------------------------- one token over a cache
struct DecodeArgs {
  Window w;  // nq = 1; lens set
  View<const __nv_bfloat16> q, k, v;
  View<__nv_bfloat16> o;
  const void *kcodes, *kscales, *vcodes, *vscales;  // 4-bit cache
  float* ws;
  float scale;
  // partial results: blocks of 16 keys of a run, runs that there is room for in ws
  int run, parts;
  // along with weights for each key: [B, nkv, n_k], the scores' place in the workspace, and how many
  // keys of a list have one
  float *weights, *scores;
  long long slots;
};
// Parts that a sequence's keys are cut into, by the problem's sizes alone.
int decode_splits(const Window& w);
size_t decode_ws_bytes(const Window& w, int d);
cudaError_t launch_window_decode(const DecodeArgs& a, int d, bool kv4, cudaStream_t st);
size_t decode_weights_ws_bytes(const Window& w, int d);
cudaError_t launch_window_decode_weights(const DecodeArgs& a, int d, cudaStream_t st);
// Partial results of runs of blocks of 16 keys alone, [B, nh, parts][d + 4]: outputs relative to the
// maximum (log2 units), the maximum, the sum.  A sequence has as many as it has runs.
struct DecodeRuns {
  int run, parts;
};
DecodeRuns decode_runs(const Window& w);
size_t decode_parts_ws_bytes(const Window& w, int d);
cudaError_t launch_window_decode_parts(DecodeArgs a, int d, cudaStream_t st);

// ---------------------------------------------------------------- behind a shared prefix
struct PrefixShape {
  int B, nh, nkv, nq, P, nk;
};
struct PrefixArgs {
  PrefixShape s;
  View<const __nv_bfloat16> q, kp, vp, k, v;
  View<__nv_bfloat16> o;
  const int* lens;
  float* lse;  // prompts; or null
  void* ws;
  float scale;
};
// Runs of the kernel over the prefix, at most: one for each SM.  On a part with fewer of them what is left
// over makes a second wave; the cuts, and the results' bits, stay the same.
constexpr int kPrefixCtas = 152;
size_t prefix_ws_bytes(const PrefixShape& s, int d);
cudaError_t launch_prefix_attn(const PrefixArgs& a, int d, bool decode, cudaStream_t st);

}  // namespace psa
