// lm_api.cu -- host side of the token-sequence entry points of include/psa.h: validation of
// views and problems, dispatch by type.  Nothing here allocates or synchronises, and every
// argument is checked before the first CUDA call.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/psa.h"
#include "lm.cuh"

namespace {

using psa::View;

psa_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? PSA_OK : PSA_ERR_CUDA; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int elem_bytes(psa_dtype_t t) { return t == PSA_DTYPE_F32 ? 4 : 2; }

constexpr long long kMaxRows = 1LL << 28;        // rows of one sequence
constexpr long long kMaxStride = 1LL << 38;      // elements (tensor maps hold 2^40 bytes)

// A view [B, heads, N, d]: strides of single entries are put in order, the others checked.
psa_status_t check_view(psa_rows_t& v, int B, int heads, int N, int d, psa_dtype_t t) {
  if (!v.ptr) return PSA_ERR_INVALID_ARG;
  const int e = elem_bytes(t);
  long long* stride[3] = {&v.stride_n, &v.stride_h, &v.stride_b};
  const int extent[3] = {N, heads, B};
  int order[3], n = 0;
  for (int i = 0; i < 3; ++i)
    if (extent[i] > 1) order[n++] = i;
  std::sort(order, order + n, [&](int x, int y) { return *stride[x] < *stride[y]; });
  long long least = d;
  for (int i = 0; i < n; ++i) {
    const long long s = *stride[order[i]];
    if (s < least || s > kMaxStride) return PSA_ERR_INVALID_ARG;
    least = s * extent[order[i]];
    if (least > (1LL << 45)) return PSA_ERR_UNSUPPORTED;
  }
  for (int i = 0; i < 3; ++i)
    if (extent[i] <= 1) *stride[i] = d;
  if (!aligned(v.ptr, 16)) return PSA_ERR_ALIGNMENT;
  for (int i = 0; i < 3; ++i)
    if (*stride[i] * e % 16 != 0) return PSA_ERR_ALIGNMENT;
  return PSA_OK;
}

template <typename T>
View<T> view(const psa_rows_t& v) {
  return View<T>{static_cast<T*>(v.ptr), v.stride_b, v.stride_h, v.stride_n};
}

bool known(psa_dtype_t t) { return t == PSA_DTYPE_F32 || t == PSA_DTYPE_BF16; }

#define PSA_TRY(x)                        \
  do {                                    \
    const psa_status_t e_ = (x);          \
    if (e_ != PSA_OK) return e_;          \
  } while (0)

// ---------------------------------------------------------------- norms + rotation
psa_status_t check_norm_rope(const psa_norm_rope_t& p) {
  if (p.B <= 0 || p.num_heads <= 0 || p.num_kv_heads <= 0 || p.N <= 0 || p.head_dim <= 0 ||
      !known(p.dtype) || p.rotary_dim < 0 || p.max_pos <= 0 ||
      (p.interleaved != 0 && p.interleaved != 1) || !isfinite(p.eps) || p.eps < 0.f)
    return PSA_ERR_INVALID_ARG;
  if (p.head_dim != 32 && p.head_dim != 64 && p.head_dim != 128) return PSA_ERR_UNSUPPORTED;
  if (p.rotary_dim > p.head_dim || p.rotary_dim % 16 != 0) return PSA_ERR_INVALID_ARG;
  if (p.num_heads > 32767 || p.num_kv_heads > 32767 || (long long)p.B * p.N > (1LL << 30))
    return PSA_ERR_UNSUPPORTED;
  return PSA_OK;
}

psa_status_t check_tables(const float* qw, const float* kw, const float* cos, const float* sin,
                          const int* positions, const psa_norm_rope_t& p) {
  if (p.rotary_dim > 0 && (!cos || !sin)) return PSA_ERR_INVALID_ARG;
  if (!positions && p.N > p.max_pos) return PSA_ERR_INVALID_ARG;
  if (!aligned(qw, 4) || !aligned(kw, 4) || !aligned(cos, 16) || !aligned(sin, 16) ||
      !aligned(positions, 4))
    return PSA_ERR_ALIGNMENT;
  return PSA_OK;
}

template <typename T>
psa::NormRopeArgs<T> norm_rope_args(psa_rows_t q, psa_rows_t k, const float* qw, const float* kw,
                                    const float* cos, const float* sin, const int* positions,
                                    psa_rows_t oq, psa_rows_t ok, const psa_norm_rope_t& p) {
  psa::NormRopeArgs<T> a{};
  a.q = view<const T>(q);
  a.k = view<const T>(k);
  a.oq = view<T>(oq);
  a.ok = view<T>(ok);
  a.wq = qw;
  a.wk = kw;
  a.cos = cos;
  a.sin = sin;
  a.positions = positions;
  a.B = p.B;
  a.nh = p.num_heads;
  a.nkv = p.num_kv_heads;
  a.N = p.N;
  a.rot = p.rotary_dim;
  a.max_pos = p.max_pos;
  a.interleaved = p.interleaved != 0;
  a.eps = p.eps;
  return a;
}

template <typename T>
psa_status_t run_norm_rope_bwd(psa::NormRopeArgs<T> a, psa_rows_t gq, psa_rows_t gk, float* dwq,
                               float* dwk, void* ws, int d, cudaStream_t st) {
  a.gq = view<const T>(gq);
  a.gk = view<const T>(gk);
  a.dwq = dwq;
  a.dwk = dwk;
  a.ws = static_cast<float*>(ws);
  return from_cuda(psa::launch_norm_rope_bwd(a, d, st));
}

// ---------------------------------------------------------------- window attention
psa_status_t check_window(const psa_window_t& p) {
  if (p.B <= 0 || p.num_heads <= 0 || p.num_kv_heads <= 0 || p.n_q <= 0 || p.n_k <= 0 ||
      p.head_dim <= 0 || p.sinks < 0 || !known(p.dtype) || p.num_heads % p.num_kv_heads != 0)
    return PSA_ERR_INVALID_ARG;
  if (p.head_dim != 64 && p.head_dim != 128) return PSA_ERR_UNSUPPORTED;
  if ((long long)p.B * p.num_heads > 65535 || p.n_q > kMaxRows || p.n_k > kMaxRows)
    return PSA_ERR_UNSUPPORTED;
  // rows in all, so that the kernels' tile counts are ints
  if ((long long)p.B * p.num_heads * std::max(p.n_q, p.n_k) > (1LL << 36)) return PSA_ERR_UNSUPPORTED;
  return PSA_OK;
}

psa_status_t check_scale(float scale) {
  return isfinite(scale) && scale > 0.f ? PSA_OK : PSA_ERR_INVALID_ARG;
}

psa::Window window(const psa_window_t& p, const int* lens) {
  auto limit = [&](int w) { return w < 0 || w > p.n_k ? p.n_k : w; };
  return psa::Window{p.B,   p.num_heads, p.num_kv_heads, p.n_q, p.n_k, limit(p.window_left),
                     limit(p.window_right), std::min(p.sinks, p.n_k), lens};
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

template <typename T>
psa::WindowArgs<T> window_args(const psa_window_t& p, const int* lens, psa_rows_t q, psa_rows_t k,
                               psa_rows_t v, float scale) {
  psa::WindowArgs<T> a{};
  a.w = window(p, lens);
  a.q = view<const T>(q);
  a.k = view<const T>(k);
  a.v = view<const T>(v);
  a.scale = scale;
  return a;
}

template <typename T>
psa_status_t run_window_fwd(psa::WindowArgs<T> a, psa_rows_t o, float* lse, int d, cudaStream_t st) {
  a.out = view<T>(o);
  a.lse = lse;
  if constexpr (sizeof(T) == 2)
    return from_cuda(psa::launch_window_fwd_tc(a, d, st));
  else
    return from_cuda(psa::launch_window_fwd_simt(a, d, st));
}

template <typename T>
psa_status_t run_window_bwd(psa::WindowArgs<T> a, psa_rows_t o, psa_rows_t dO, const float* lse,
                            psa_rows_t dq, psa_rows_t dk, psa_rows_t dv, void* ws, int d,
                            cudaStream_t st) {
  a.o = view<const T>(o);
  a.dO = view<const T>(dO);
  a.lse = const_cast<float*>(lse);
  a.delta = static_cast<float*>(ws);
  a.dq = view<T>(dq);
  a.dk = view<T>(dk);
  a.dv = view<T>(dv);
  if constexpr (sizeof(T) == 2)
    return from_cuda(psa::launch_window_bwd_tc(a, d, st));
  else
    return from_cuda(psa::launch_window_bwd_simt(a, d, st));
}

// ---------------------------------------------------------------- caches
psa_status_t check_cache(const psa_cache_t& p) {
  if (p.B <= 0 || p.num_kv_heads <= 0 || p.N <= 0 || p.max_len <= 0 || p.head_dim <= 0 ||
      !known(p.dtype))
    return PSA_ERR_INVALID_ARG;
  if (p.head_dim != 64 && p.head_dim != 128) return PSA_ERR_UNSUPPORTED;
  if ((long long)p.B * p.num_kv_heads > 65535 || p.N > kMaxRows || p.max_len > kMaxRows)
    return PSA_ERR_UNSUPPORTED;
  return PSA_OK;
}

psa_status_t check_kv4(const void* kc, const void* ks, const void* vc, const void* vs) {
  if (!kc || !ks || !vc || !vs) return PSA_ERR_INVALID_ARG;
  return aligned(kc, 16) && aligned(ks, 16) && aligned(vc, 16) && aligned(vs, 16)
             ? PSA_OK
             : PSA_ERR_ALIGNMENT;
}

psa::CacheArgs cache_args(const psa_cache_t& p, const int* starts, const int* counts) {
  return psa::CacheArgs{p.B, p.num_kv_heads, p.N, p.max_len, starts, counts};
}

// What both single-token entry points ask of the problem, q, o and the workspace.
psa_status_t check_decode(const psa_window_t& p, psa_rows_t& q, psa_rows_t& o, const int* lens,
                          const void* ws, size_t ws_bytes, float scale) {
  PSA_TRY(check_window(p));
  PSA_TRY(check_scale(scale));
  if (p.n_q != 1 || !lens || !ws) return PSA_ERR_INVALID_ARG;
  if (p.dtype != PSA_DTYPE_BF16) return PSA_ERR_UNSUPPORTED;
  PSA_TRY(check_view(q, p.B, p.num_heads, 1, p.head_dim, p.dtype));
  PSA_TRY(check_view(o, p.B, p.num_heads, 1, p.head_dim, p.dtype));
  if (!aligned(ws, 16) || !aligned(lens, 4)) return PSA_ERR_ALIGNMENT;
  return ws_bytes >= psa_window_attn_decode_workspace_size(p) ? PSA_OK : PSA_ERR_INVALID_ARG;
}

psa::DecodeArgs decode_args(const psa_window_t& p, const int* lens, psa_rows_t q, psa_rows_t o,
                            void* ws, float scale) {
  psa::DecodeArgs a{};
  a.w = window(p, lens);
  a.q = view<const __nv_bfloat16>(q);
  a.o = view<__nv_bfloat16>(o);
  a.ws = static_cast<float*>(ws);
  a.scale = scale;
  return a;
}

}  // namespace

extern "C" {

psa_status_t psa_qk_norm_rope_fwd(psa_rows_t q, psa_rows_t k, const float* q_weight,
                                  const float* k_weight, const float* cos, const float* sin,
                                  const int* positions, psa_rows_t q_out, psa_rows_t k_out,
                                  psa_norm_rope_t p, cudaStream_t st) {
  PSA_TRY(check_norm_rope(p));
  PSA_TRY(check_view(q, p.B, p.num_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_view(k, p.B, p.num_kv_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_view(q_out, p.B, p.num_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_view(k_out, p.B, p.num_kv_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_tables(q_weight, k_weight, cos, sin, positions, p));
  if (p.dtype == PSA_DTYPE_F32)
    return from_cuda(psa::launch_norm_rope_fwd(
        norm_rope_args<float>(q, k, q_weight, k_weight, cos, sin, positions, q_out, k_out, p),
        p.head_dim, st));
  return from_cuda(psa::launch_norm_rope_fwd(
      norm_rope_args<__nv_bfloat16>(q, k, q_weight, k_weight, cos, sin, positions, q_out, k_out, p),
      p.head_dim, st));
}

size_t psa_qk_norm_rope_bwd_workspace_size(psa_norm_rope_t p) {
  return check_norm_rope(p) == PSA_OK ? (size_t)2 * psa::kNormRopeParts * p.head_dim * 4 : 0;
}

psa_status_t psa_qk_norm_rope_bwd(psa_rows_t q, psa_rows_t k, const float* q_weight,
                                  const float* k_weight, const float* cos, const float* sin,
                                  const int* positions, psa_rows_t dq_out, psa_rows_t dk_out,
                                  psa_rows_t dq, psa_rows_t dk, float* dq_weight, float* dk_weight,
                                  void* ws, size_t ws_bytes, psa_norm_rope_t p, cudaStream_t st) {
  PSA_TRY(check_norm_rope(p));
  PSA_TRY(check_view(q, p.B, p.num_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_view(k, p.B, p.num_kv_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_view(dq_out, p.B, p.num_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_view(dk_out, p.B, p.num_kv_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_view(dq, p.B, p.num_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_view(dk, p.B, p.num_kv_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_tables(q_weight, k_weight, cos, sin, positions, p));
  if (!ws) return PSA_ERR_INVALID_ARG;
  if (!aligned(ws, 16) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return PSA_ERR_ALIGNMENT;
  if (ws_bytes < psa_qk_norm_rope_bwd_workspace_size(p)) return PSA_ERR_INVALID_ARG;
  if (p.dtype == PSA_DTYPE_F32)
    return run_norm_rope_bwd(
        norm_rope_args<float>(q, k, q_weight, k_weight, cos, sin, positions, dq, dk, p), dq_out,
        dk_out, dq_weight, dk_weight, ws, p.head_dim, st);
  return run_norm_rope_bwd(
      norm_rope_args<__nv_bfloat16>(q, k, q_weight, k_weight, cos, sin, positions, dq, dk, p),
      dq_out, dk_out, dq_weight, dk_weight, ws, p.head_dim, st);
}

psa_status_t psa_window_attn_fwd(psa_rows_t q, psa_rows_t k, psa_rows_t v, const int* lens,
                                 psa_rows_t o, float* lse, psa_window_t p, float scale,
                                 cudaStream_t st) {
  PSA_TRY(check_window(p));
  PSA_TRY(check_scale(scale));
  PSA_TRY(check_view(q, p.B, p.num_heads, p.n_q, p.head_dim, p.dtype));
  PSA_TRY(check_view(k, p.B, p.num_kv_heads, p.n_k, p.head_dim, p.dtype));
  PSA_TRY(check_view(v, p.B, p.num_kv_heads, p.n_k, p.head_dim, p.dtype));
  PSA_TRY(check_view(o, p.B, p.num_heads, p.n_q, p.head_dim, p.dtype));
  if (!aligned(lens, 4) || !aligned(lse, 4)) return PSA_ERR_ALIGNMENT;
  if (p.dtype == PSA_DTYPE_F32)
    return run_window_fwd(window_args<float>(p, lens, q, k, v, scale), o, lse, p.head_dim, st);
  return run_window_fwd(window_args<__nv_bfloat16>(p, lens, q, k, v, scale), o, lse, p.head_dim, st);
}

size_t psa_window_attn_bwd_workspace_size(psa_window_t p) {
  if (check_window(p) != PSA_OK) return 0;
  return round256(p.dtype == PSA_DTYPE_BF16 ? psa::window_bwd_tc_ws_bytes(window(p, nullptr), p.head_dim)
                                            : (size_t)p.B * p.num_heads * p.n_q * 4);
}

psa_status_t psa_window_attn_bwd(psa_rows_t q, psa_rows_t k, psa_rows_t v, psa_rows_t o,
                                 psa_rows_t do_, const float* lse, const int* lens, psa_rows_t dq,
                                 psa_rows_t dk, psa_rows_t dv, void* ws, size_t ws_bytes,
                                 psa_window_t p, float scale, cudaStream_t st) {
  PSA_TRY(check_window(p));
  PSA_TRY(check_scale(scale));
  PSA_TRY(check_view(q, p.B, p.num_heads, p.n_q, p.head_dim, p.dtype));
  PSA_TRY(check_view(k, p.B, p.num_kv_heads, p.n_k, p.head_dim, p.dtype));
  PSA_TRY(check_view(v, p.B, p.num_kv_heads, p.n_k, p.head_dim, p.dtype));
  PSA_TRY(check_view(o, p.B, p.num_heads, p.n_q, p.head_dim, p.dtype));
  PSA_TRY(check_view(do_, p.B, p.num_heads, p.n_q, p.head_dim, p.dtype));
  PSA_TRY(check_view(dq, p.B, p.num_heads, p.n_q, p.head_dim, p.dtype));
  PSA_TRY(check_view(dk, p.B, p.num_kv_heads, p.n_k, p.head_dim, p.dtype));
  PSA_TRY(check_view(dv, p.B, p.num_kv_heads, p.n_k, p.head_dim, p.dtype));
  if (!lse || !ws) return PSA_ERR_INVALID_ARG;
  if (!aligned(lens, 4) || !aligned(lse, 4) || !aligned(ws, 16)) return PSA_ERR_ALIGNMENT;
  if (ws_bytes < psa_window_attn_bwd_workspace_size(p)) return PSA_ERR_INVALID_ARG;
  if (p.dtype == PSA_DTYPE_F32)
    return run_window_bwd(window_args<float>(p, lens, q, k, v, scale), o, do_, lse, dq, dk, dv, ws,
                          p.head_dim, st);
  return run_window_bwd(window_args<__nv_bfloat16>(p, lens, q, k, v, scale), o, do_, lse, dq, dk,
                        dv, ws, p.head_dim, st);
}

size_t psa_window_attn_decode_workspace_size(psa_window_t p) {
  if (check_window(p) != PSA_OK || p.n_q != 1) return 0;
  return psa::decode_ws_bytes(window(p, nullptr), p.head_dim);
}

psa_status_t psa_window_attn_decode(psa_rows_t q, psa_rows_t k_cache, psa_rows_t v_cache,
                                    const int* lens, psa_rows_t o, void* ws, size_t ws_bytes,
                                    psa_window_t p, float scale, cudaStream_t st) {
  PSA_TRY(check_decode(p, q, o, lens, ws, ws_bytes, scale));
  PSA_TRY(check_view(k_cache, p.B, p.num_kv_heads, p.n_k, p.head_dim, p.dtype));
  PSA_TRY(check_view(v_cache, p.B, p.num_kv_heads, p.n_k, p.head_dim, p.dtype));
  psa::DecodeArgs a = decode_args(p, lens, q, o, ws, scale);
  a.k = view<const __nv_bfloat16>(k_cache);
  a.v = view<const __nv_bfloat16>(v_cache);
  return from_cuda(psa::launch_window_decode(a, p.head_dim, false, st));
}

psa_status_t psa_window_attn_decode_kv4(psa_rows_t q, const void* k_codes, const void* k_scales,
                                        const void* v_codes, const void* v_scales, const int* lens,
                                        psa_rows_t o, void* ws, size_t ws_bytes, psa_window_t p,
                                        float scale, cudaStream_t st) {
  PSA_TRY(check_decode(p, q, o, lens, ws, ws_bytes, scale));
  PSA_TRY(check_kv4(k_codes, k_scales, v_codes, v_scales));
  psa::DecodeArgs a = decode_args(p, lens, q, o, ws, scale);
  a.kcodes = k_codes;
  a.kscales = k_scales;
  a.vcodes = v_codes;
  a.vscales = v_scales;
  return from_cuda(psa::launch_window_decode(a, p.head_dim, true, st));
}

psa_status_t psa_kv_append(psa_rows_t k, psa_rows_t v, const int* starts, const int* counts,
                           psa_rows_t k_cache, psa_rows_t v_cache, psa_cache_t p, cudaStream_t st) {
  PSA_TRY(check_cache(p));
  if (!starts) return PSA_ERR_INVALID_ARG;
  PSA_TRY(check_view(k, p.B, p.num_kv_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_view(v, p.B, p.num_kv_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_view(k_cache, p.B, p.num_kv_heads, p.max_len, p.head_dim, p.dtype));
  PSA_TRY(check_view(v_cache, p.B, p.num_kv_heads, p.max_len, p.head_dim, p.dtype));
  if (!aligned(starts, 4) || !aligned(counts, 4)) return PSA_ERR_ALIGNMENT;
  const psa::CacheArgs c = cache_args(p, starts, counts);
  if (p.dtype == PSA_DTYPE_F32)
    return from_cuda(psa::launch_kv_append<float>(c, view<const float>(k), view<const float>(v),
                                                  view<float>(k_cache), view<float>(v_cache),
                                                  p.head_dim, st));
  using T = __nv_bfloat16;
  return from_cuda(psa::launch_kv_append<T>(c, view<const T>(k), view<const T>(v), view<T>(k_cache),
                                            view<T>(v_cache), p.head_dim, st));
}

psa_status_t psa_kv4_append(psa_rows_t k, psa_rows_t v, const int* starts, const int* counts,
                            void* k_codes, void* k_scales, void* v_codes, void* v_scales,
                            psa_cache_t p, cudaStream_t st) {
  PSA_TRY(check_cache(p));
  if (!starts) return PSA_ERR_INVALID_ARG;
  PSA_TRY(check_view(k, p.B, p.num_kv_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_view(v, p.B, p.num_kv_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_kv4(k_codes, k_scales, v_codes, v_scales));
  if (!aligned(starts, 4) || !aligned(counts, 4)) return PSA_ERR_ALIGNMENT;
  const psa::CacheArgs c = cache_args(p, starts, counts);
  if (p.dtype == PSA_DTYPE_F32)
    return from_cuda(psa::launch_kv4_append<float>(c, view<const float>(k), view<const float>(v),
                                                   k_codes, k_scales, v_codes, v_scales, p.head_dim,
                                                   st));
  using T = __nv_bfloat16;
  return from_cuda(psa::launch_kv4_append<T>(c, view<const T>(k), view<const T>(v), k_codes,
                                             k_scales, v_codes, v_scales, p.head_dim, st));
}

psa_status_t psa_kv4_read(const void* k_codes, const void* k_scales, const void* v_codes,
                          const void* v_scales, psa_rows_t k, psa_rows_t v, psa_cache_t p,
                          cudaStream_t st) {
  PSA_TRY(check_cache(p));
  if (p.N > p.max_len) return PSA_ERR_INVALID_ARG;
  PSA_TRY(check_kv4(k_codes, k_scales, v_codes, v_scales));
  PSA_TRY(check_view(k, p.B, p.num_kv_heads, p.N, p.head_dim, p.dtype));
  PSA_TRY(check_view(v, p.B, p.num_kv_heads, p.N, p.head_dim, p.dtype));
  const psa::CacheArgs c = cache_args(p, nullptr, nullptr);
  if (p.dtype == PSA_DTYPE_F32)
    return from_cuda(psa::launch_kv4_read<float>(c, k_codes, k_scales, v_codes, v_scales,
                                                 view<float>(k), view<float>(v), p.head_dim, st));
  using T = __nv_bfloat16;
  return from_cuda(psa::launch_kv4_read<T>(c, k_codes, k_scales, v_codes, v_scales, view<T>(k),
                                           view<T>(v), p.head_dim, st));
}

}  // extern "C"
