/*
 * psa.h -- C ABI of the GB300 (sm_103a) Position-Sensitive Attention library
 * (libpsa_gb300.so).
 *
 * The operations are those of the vision-rs book, page "Custom Kernels":
 *   section "Flash Attention 2"  -- softmax attention over [BATCH*N_HEADS, N_CTX,
 *     HEAD_DIM] tensors with an online softmax (the N x N matrix is never stored);
 *     the forward, the dQ backward and the dK/dV backward are separate kernels.
 *   section "Position-Sensitive Attention (PSA)" -- PsaPackQkv, PsaExtractV and
 *     PsaMergeAttn around Flash Attention 2, which PSA runs once per V half
 *     (V_lo, V_hi) with HEAD_DIM = KEY_DIM.
 *
 * Notation: KD = key_dim, nh = num_heads, N = H*W, BH = B*nh, qkv_h = nh*4*KD,
 * c = nh*2*KD.  Spatial index n = h*W + w; head-batch index bh = b*nh + head.
 * Per head, QKV channels are [Q | K | V_lo | V_hi], each KD wide: channel
 * head*4*KD + s*KD + d holds element d of plane s (0=Q, 1=K, 2=V_lo, 3=V_hi).
 * The merged output channel head*2*KD + t*KD + d holds element d of half t.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers to dense, contiguous buffers owned
 *     by the caller; the library never allocates, frees or synchronises, and
 *     every call is ordered on the given stream.  Pointers must be 16-byte
 *     aligned (PSA_ERR_ALIGNMENT otherwise).
 *   - Arguments come in the order inputs, outputs, workspace, sizes, stream.
 *   - Validation is host-side and happens before any launch: a NULL required
 *     pointer or a non-positive size gives PSA_ERR_INVALID_ARG; a size the
 *     kernels do not implement gives PSA_ERR_UNSUPPORTED; a failed launch gives
 *     PSA_ERR_CUDA.  Nothing is printed and nothing exits.
 *   - Element types: bf16 (PSA_DTYPE_BF16; fp32 accumulation, softmax
 *     probabilities rounded to bf16 before the P.V product, outputs rounded to
 *     nearest-even) or fp32 (PSA_DTYPE_F32; forward only, fp32 arithmetic).
 *     Log-sum-exp and delta arrays are always fp32.
 *   - Kernels that wait on on-chip barriers give up after a bounded time and
 *     record PSA_ERR_TIMEOUT in a device-side error word that
 *     psa_get_last_device_error() reads and clears.
 *   - The attention kernels are launched with programmatic stream
 *     serialization: their CTAs may start their set-up while the previous
 *     kernel of the stream is finishing, but they read and write no global
 *     memory before that kernel has completed, so results are exactly those of
 *     plain stream order.  (Between the kernels of one call: those that share
 *     nothing may run beside one another.)
 */
#ifndef PSA_GB300_H
#define PSA_GB300_H

#include <stddef.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PSA_OK = 0,
    PSA_ERR_INVALID_ARG = 1,
    PSA_ERR_UNSUPPORTED = 2,
    PSA_ERR_ALIGNMENT = 3,
    PSA_ERR_CUDA = 4,
    PSA_ERR_TIMEOUT = 5
} psa_status_t;

typedef enum { PSA_DTYPE_F32 = 0, PSA_DTYPE_BF16 = 1 } psa_dtype_t;

/* One PSA problem: QKV conv output [B, nh*4*KD, H, W] of the given element type. */
typedef struct {
    int B, num_heads, key_dim, H, W;
    psa_dtype_t dtype;
} psa_shape_t;

/* ---- QKV convolution ---------------------------------------------------------- */

/* The QKV 1x1 convolution whose NCHW output PsaPackQkv and the fused PSA forward
 * read ("Custom Kernels", section "Position-Sensitive Attention (PSA)": PsaPackQkv
 * takes a QKV conv's NCHW output): qkv[b, o, n] = bias[o] + sum_c w[o, c] x[b, c, n]
 * for x_nchw [B, cin, H, W], weight [cout, cin] (row-major), bias [cout] fp32
 * (NULL: none) and qkv_nchw [B, cout, H, W]; bf16 storage, fp32 accumulation,
 * outputs rounded once.  On the tensor cores when cin and H*W are multiples of 8,
 * on CUDA cores otherwise.  Pointers 16-byte aligned (bias 4-byte);
 * PSA_ERR_INVALID_ARG for a NULL required pointer or a non-positive size. */
psa_status_t psa_qkv_conv(const void *x_nchw, const void *weight, const float *bias,
                          void *qkv_nchw, int B, int cin, int cout, int H, int W,
                          cudaStream_t stream);

/* ---- layout kernels (bit-exact element copies) ------------------------------ */

/* PsaPackQkv ("Custom Kernels", section "Position-Sensitive Attention (PSA)"):
 * qkv_nchw [B, qkv_h, H, W] -> packed [4, BH, N, KD] (planes Q, K, V_lo, V_hi).
 * Both dtypes; key_dim up to 128 for all layout kernels. */
psa_status_t psa_pack_qkv(const void *qkv_nchw, void *packed, psa_shape_t shape,
                          cudaStream_t stream);

/* Inverse permutation of psa_pack_qkv (the adjoint the backward needs):
 * packed [4, BH, N, KD] -> qkv_nchw [B, qkv_h, H, W]. */
psa_status_t psa_unpack_qkv(const void *packed, void *qkv_nchw, psa_shape_t shape,
                            cudaStream_t stream);

/* PsaExtractV (same section): the V section [V_lo | V_hi] of every head, as NCHW
 * v_nchw [B, c, H, W] (v_nchw[b, head*2KD + j, n] = qkv[b, head*4KD + 2KD + j, n]). */
psa_status_t psa_extract_v(const void *qkv_nchw, void *v_nchw, psa_shape_t shape,
                           cudaStream_t stream);

/* PsaMergeAttn (same section): o_lo, o_hi [BH, N, KD] -> out_nchw [B, c, H, W]. */
psa_status_t psa_merge_attn(const void *o_lo, const void *o_hi, void *out_nchw,
                            psa_shape_t shape, cudaStream_t stream);

/* Inverse of psa_merge_attn (the adjoint the backward needs):
 * dout_nchw [B, c, H, W] -> do_lo, do_hi [BH, N, KD]. */
psa_status_t psa_unmerge_attn(const void *dout_nchw, void *do_lo, void *do_hi,
                              psa_shape_t shape, cudaStream_t stream);

/* ---- Flash Attention 2 on [BH, N, HEAD_DIM] ("Flash Attention 2" section) ---- */

/* Forward: o = softmax(scale * q k^T) v, lse = log-sum-exp of each score row
 * (natural log, fp32 [BH, n_ctx]; lse may be NULL).  q, k, v, o are
 * [BH, n_ctx, head_dim] of dtype; head_dim in {32, 64} (PSA_ERR_UNSUPPORTED
 * otherwise).  Non-causal, no mask. */
psa_status_t flash_attn2_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
                             int BH, int n_ctx, int head_dim, float scale, psa_dtype_t dtype,
                             cudaStream_t stream);

/* dQ backward: writes delta[bh, i] = sum_c do[bh, i, c] * o[bh, i, c] (fp32
 * [BH, n_ctx], caller-owned) and dq = scale * dS k with dS = P o (dP - delta),
 * P = exp(scale q k^T - lse), dP = do v^T.  lse is the forward's.  bf16 only.
 * Must run before flash_attn2_bwd_dkdv, which reads delta. */
psa_status_t flash_attn2_bwd_dq(const void *q, const void *k, const void *v, const void *o,
                                const void *do_, const float *lse, float *delta, void *dq,
                                int BH, int n_ctx, int head_dim, float scale, psa_dtype_t dtype,
                                cudaStream_t stream);

/* dK/dV backward: dv = P^T do, dk = scale * dS^T q, with delta from
 * flash_attn2_bwd_dq.  bf16 only.  dk, dv are overwritten. */
psa_status_t flash_attn2_bwd_dkdv(const void *q, const void *k, const void *v, const void *do_,
                                  const float *lse, const float *delta, void *dk, void *dv,
                                  int BH, int n_ctx, int head_dim, float scale,
                                  psa_dtype_t dtype, cudaStream_t stream);

/* ---- fused PSA reading and writing NCHW directly ----------------------------- */

/* Forward of the whole PSA attention step: pack, attention over both V halves
 * with one shared softmax (identical to two HEAD_DIM = KD runs), merge; writes
 * out_nchw [B, c, H, W], lse [BH, N] fp32 (nullable) and, when v_nchw is not
 * NULL, the PsaExtractV output [B, c, H, W].  key_dim in {32, 64};
 * N*sizeof(dtype) must be a multiple of 16 (PSA_ERR_ALIGNMENT otherwise);
 * bf16, or fp32 (computed in fp32). */
psa_status_t psa_attention_fwd(const void *qkv_nchw, void *out_nchw, float *lse, void *v_nchw,
                               psa_shape_t shape, float scale, cudaStream_t stream);

/* The same forward with the residual path fused into its epilogue
 * ("Custom Kernels", section "Position-Sensitive Attention (PSA)": PsaExtractV
 * pulls the V section out in NCHW for the residual path, which adds it to the
 * merged attention output): writes out_res [B, c, H, W] = Out + V, each element
 * rounded once, where V is the PsaExtractV output; also writes the plain attention
 * output out and lse [BH, N] when they are not NULL.  The backward of out_res is
 * psa_attention_bwd with dvres_nchw = dout_nchw (the residual adds the upstream
 * gradient into the V channels); it needs out, so callers that train pass out here.
 * Same sizes, dtypes and errors as psa_attention_fwd (out_res is required). */
psa_status_t psa_attention_fwd_residual(const void *qkv_nchw, void *out_res_nchw, void *out_nchw,
                                        float *lse, psa_shape_t shape, float scale,
                                        cudaStream_t stream);

/* Backward of psa_attention_fwd: given qkv, the forward's out and lse, the
 * upstream gradient dout [B, c, H, W] and optionally the gradient dvres of the
 * extracted V (nullable), writes dqkv_nchw [B, qkv_h, H, W] (overwritten, V
 * channels include dvres).  workspace is device memory, 16-byte aligned, of
 * ws_bytes >= psa_attention_bwd_workspace_size(shape) bytes.  Which kernels run:
 *   - key_dim 32, bf16, N <= 512: one kernel per head computes delta on chip and
 *     forms every P and dS once; the workspace is not touched;
 *   - key_dim 32, bf16, 512 < N <= 2048, with the full workspace: the same kernel,
 *     with the dQ accumulator in the workspace;
 *   - otherwise (key_dim 64, longer N, or a workspace of only B*num_heads*N*4
 *     bytes rounded up to 256, the least accepted): the dQ and dK/dV kernels of
 *     the two-kernel form, with delta in the workspace;
 *   - fp32, or rows that are not 16-byte multiples: CUDA-core dQ and dK/dV.
 * key_dim 32 or 64; bf16 or fp32. */
psa_status_t psa_attention_bwd(const void *qkv_nchw, const void *out_nchw, const void *dout_nchw,
                               const float *lse, const void *dvres_nchw, void *dqkv_nchw,
                               void *workspace, size_t ws_bytes, psa_shape_t shape, float scale,
                               cudaStream_t stream);

/* The two kernels psa_attention_bwd runs, for callers that schedule them
 * separately ("Flash Attention 2" section: the dQ and dK/dV backward are separate
 * kernels with their own grids).  psa_attention_bwd_dq writes the Q channels of
 * dqkv_nchw and delta [BH, N] fp32 (rowsum of dOut o Out per head and position);
 * psa_attention_bwd_dkdv then reads delta and writes the K and V channels (V
 * channels include dvres when it is not NULL).  It must run after
 * psa_attention_bwd_dq on the same stream.  Same sizes and errors as
 * psa_attention_bwd. */
psa_status_t psa_attention_bwd_dq(const void *qkv_nchw, const void *out_nchw,
                                  const void *dout_nchw, const float *lse, float *delta,
                                  void *dqkv_nchw, psa_shape_t shape, float scale,
                                  cudaStream_t stream);
psa_status_t psa_attention_bwd_dkdv(const void *qkv_nchw, const void *dout_nchw,
                                    const float *lse, const float *delta,
                                    const void *dvres_nchw, void *dqkv_nchw, psa_shape_t shape,
                                    float scale, cudaStream_t stream);

/* psa_attention_bwd for callers that cannot allocate device memory when they run
 * the backward (for example a plugin whose host framework owns all device
 * allocations, or a latency-critical loop where cudaMalloc / cudaFree would
 * synchronise the device).  The pages have no counterpart: this is a
 * convenience of this library.  Same arguments and results as
 * psa_attention_bwd, minus the workspace.  The delta scratch lives in a fixed
 * 4 MiB array inside the library's device memory, which every GPU that loads the
 * library keeps until the process exits; B * num_heads * H * W may not exceed
 * 1048576.  Errors are checked in this order: a NULL required pointer or an
 * invalid shape (PSA_ERR_INVALID_ARG), then that limit (PSA_ERR_UNSUPPORTED),
 * then every other check of psa_attention_bwd.  The first call on each device,
 * made with that device current, looks up the array's address; make that first
 * call before any stream capture.  The array serves as the workspace of
 * psa_attention_bwd: it holds delta for the two-kernel form (key_dim 64, fp32,
 * rows that are not 16-byte multiples, or N > 2048), or the dQ accumulator of the
 * one-kernel form for key_dim 32 and 512 < N <= 2048 when B * num_heads * N * 32
 * floats fit in it (the two-kernel form otherwise); the one-kernel form for
 * N <= 512 keeps everything on chip and leaves it untouched.  All calls that use
 * the array share it: such calls whose kernels overlap on the GPU (other
 * streams, other threads) race on it, so serialise them.  Nothing in the array
 * needs clearing between calls (each call writes every value it reads before it
 * reads it).  No allocation of any kind is made. */
psa_status_t psa_attention_bwd_noalloc(const void *qkv_nchw, const void *out_nchw,
                                       const void *dout_nchw, const float *lse,
                                       const void *dvres_nchw, void *dqkv_nchw, psa_shape_t shape,
                                       float scale, cudaStream_t stream);

/* Bytes of device workspace for psa_attention_bwd to take its fastest form (0 for
 * an invalid shape): B*num_heads*N*4 rounded up to 256 (delta), or, for key_dim 32
 * and 512 < N <= 2048, B*num_heads*N*32*4 rounded up to 256 (a dQ accumulator). */
size_t psa_attention_bwd_workspace_size(psa_shape_t shape);

/* ---- token sequences: positions, windows, caches -------------------------------- */

/* The entry points of this section work on views: a view [B, heads, N, d] is a base
 * pointer and the strides, in elements, of its first three dimensions; the d channels
 * of a row are contiguous.  A projection's output [B, N, heads, d], a part of its
 * heads, or the first rows of a longer cache are views; nothing has to be copied into
 * a dense tensor first.  Rules (for each view): the pointer and, where a dimension
 * has more than one entry, its stride are multiples of 16 bytes (PSA_ERR_ALIGNMENT);
 * strides are positive and rows do not overlap: with the dimensions in order of
 * stride, each stride is at least the extent times the stride of the one before, d
 * for the first (PSA_ERR_INVALID_ARG).  The stride of a dimension of one entry is not
 * read.  Outputs must not overlap inputs or one another, except where an entry point
 * says so.  int and float arrays are dense and 4-byte aligned (cos and sin 16-byte).
 *
 * A workspace belongs to one call at a time: two calls, or two captured graphs, that
 * may run at the same moment need one each.  Nothing in it has to be cleared, and
 * nothing in it is kept from call to call. */
typedef struct {
    void *ptr;
    long long stride_b, stride_h, stride_n;
} psa_rows_t;

/* Norms of queries and keys with the position rotation. */
typedef struct {
    int B, num_heads, num_kv_heads, N, head_dim;
    psa_dtype_t dtype;
    int rotary_dim;  /* leading channels that are rotated: a multiple of 16, 0 .. head_dim */
    int interleaved; /* 0: channel i turns with i + rotary_dim / 2; 1: channel 2i with 2i + 1 */
    int max_pos;     /* rows of the cos and sin tables */
    float eps;
} psa_norm_rope_t;

/* For each head's row x of q [B, num_heads, N, d] and k [B, num_kv_heads, N, d]:
 *   y = R(pos) (w o x / sqrt(mean(x^2) + eps)),
 * where R turns the pair (a, b) of index i into (a cos - b sin, a sin + b cos) with
 * the entries [pos, i] of the fp32 tables cos, sin [max_pos, rotary_dim / 2], and
 * channels from rotary_dim on are not turned.  Statistics and products are fp32, the
 * result is rounded once.  q_weight, k_weight: fp32 [d] (NULL: ones).  positions:
 * int32 [B, N] on the device (NULL: row n is at position n, N <= max_pos); a token
 * whose position lies outside 0 .. max_pos - 1 is padding: its rows of q_out and
 * k_out are left as they were.  q_out may be the same view as q, k_out as k.
 * head_dim 32, 64 or 128 (PSA_ERR_UNSUPPORTED otherwise); bf16 or fp32.  cos and sin
 * may be NULL only when rotary_dim is 0. */
psa_status_t psa_qk_norm_rope_fwd(psa_rows_t q, psa_rows_t k, const float *q_weight,
                                  const float *k_weight, const float *cos, const float *sin,
                                  const int *positions, psa_rows_t q_out, psa_rows_t k_out,
                                  psa_norm_rope_t p, cudaStream_t stream);

/* Its backward: from the forward's inputs and the gradients dq_out, dk_out of its
 * outputs, writes the gradients dq, dk of q and k (overwritten; zeros in the rows of
 * padding tokens, whose dq_out and dk_out are not used) and of the weights,
 * dq_weight and dk_weight, fp32 [d] (overwritten; either may be NULL: not wanted).
 * The weights' gradients are summed in fp32 in a fixed order: reruns are bitwise
 * identical.  dq may be the same view as dq_out, dk as dk_out.  workspace: 16-byte
 * aligned, at least psa_qk_norm_rope_bwd_workspace_size(p) bytes
 * (PSA_ERR_INVALID_ARG if smaller). */
psa_status_t psa_qk_norm_rope_bwd(psa_rows_t q, psa_rows_t k, const float *q_weight,
                                  const float *k_weight, const float *cos, const float *sin,
                                  const int *positions, psa_rows_t dq_out, psa_rows_t dk_out,
                                  psa_rows_t dq, psa_rows_t dk, float *dq_weight,
                                  float *dk_weight, void *workspace, size_t ws_bytes,
                                  psa_norm_rope_t p, cudaStream_t stream);

/* Bytes of device workspace for psa_qk_norm_rope_bwd (0 for an invalid problem). */
size_t psa_qk_norm_rope_bwd_workspace_size(psa_norm_rope_t p);

/* The same with positions of several axes (time, height and width of video, two axes of a
 * feature map, text next to images): pair i of a token's channels turns with the entry
 * [its position on axis axis_of_pair[i], i] of the tables. */
typedef struct {
    psa_norm_rope_t rope; /* max_pos: rows of the tables, which all axes index */
    int axes;             /* 1 .. 4 */
    int grid[4];          /* extents of the axes where positions is NULL, the last one innermost */
    int normalize;        /* 1: norms as above; 0: y = R(pos) (w o x), eps plays no part (finite, not negative) */
    unsigned char axis_of_pair[64]; /* below axes, for each of rope.rotary_dim / 2 pairs */
} psa_rope_axes_t;

/* positions: int32 [axes, B, N] on the device; a token with any position outside 0 ..
 * max_pos - 1 is padding.  NULL: token n of every sequence is cell n of a grid in raster
 * order (grid[0 .. axes - 1], each 1 .. max_pos, their product N).  Everything else as in
 * psa_qk_norm_rope_fwd; with one axis and normalize 1 the results are the same bits. */
psa_status_t psa_qk_norm_rope_axes_fwd(psa_rows_t q, psa_rows_t k, const float *q_weight,
                                       const float *k_weight, const float *cos, const float *sin,
                                       const int *positions, psa_rows_t q_out, psa_rows_t k_out,
                                       psa_rope_axes_t p, cudaStream_t stream);

/* Its backward, as psa_qk_norm_rope_bwd, with a workspace of at least
 * psa_qk_norm_rope_bwd_workspace_size(p.rope) bytes.  With normalize 0, q and k are read for
 * the weights' gradients alone. */
psa_status_t psa_qk_norm_rope_axes_bwd(psa_rows_t q, psa_rows_t k, const float *q_weight,
                                       const float *k_weight, const float *cos, const float *sin,
                                       const int *positions, psa_rows_t dq_out, psa_rows_t dk_out,
                                       psa_rows_t dq, psa_rows_t dk, float *dq_weight,
                                       float *dk_weight, void *workspace, size_t ws_bytes,
                                       psa_rope_axes_t p, cudaStream_t stream);

/* Attention with a sliding window and first tokens that stay visible: q
 * [B, num_heads, n_q, d], k and v [B, num_kv_heads, n_k, d]; query head h reads
 * key/value head h / (num_heads / num_kv_heads).  Query row i stands at position
 * p = i + n_k - n_q, key row j at position j; the query sees the key if
 *   j <= p + window_right  and  (j >= p - window_left  or  j < sinks),
 * where a negative window means no limit on that side: window_right = 0 is causal,
 * window_left = 255, window_right = 0 a window of 256 positions.  With per-sequence
 * lengths (lens, int32 [B] on the device; NULL: n_k), positions from lens[b] on are
 * padding: they are seen by none and see none.  So are the first n_q - n_k query rows
 * where n_q > n_k: they stand in front of position 0 and see nothing, whatever the
 * window.  A query that sees nothing has output 0 and log-sum-exp -infinity, and gets
 * and gives no gradient.  What rows of padding hold does not matter (NaN included);
 * values inside the lengths must be finite. */
typedef struct {
    int B, num_heads, num_kv_heads, n_q, n_k, head_dim;
    psa_dtype_t dtype;
    int window_left, window_right, sinks;
} psa_window_t;

/* Forward: o = softmax(scale q k^T) v over the visible keys (every row of o is
 * written) and lse, the natural-log log-sum-exp of each row, fp32 [B, num_heads,
 * n_q] (NULL: not wanted).  head_dim 64 or 128 (PSA_ERR_UNSUPPORTED otherwise); bf16
 * (tensor cores; softmax and sums in fp32, probabilities rounded to bf16 before the
 * product with v) or fp32 (CUDA cores, fp32 throughout).  B * num_heads up to 65535. */
psa_status_t psa_window_attn_fwd(psa_rows_t q, psa_rows_t k, psa_rows_t v, const int *lens,
                                 psa_rows_t o, float *lse, psa_window_t p, float scale,
                                 cudaStream_t stream);

/* Backward: from the forward's inputs, its o and lse and the gradient do_ of o, writes
 * dq, dk, dv (every row, overwritten; a key/value head's gradient sums those of its
 * query heads in a fixed order: reruns are bitwise identical).  workspace: 16-byte
 * aligned, at least psa_window_attn_bwd_workspace_size(p) bytes (PSA_ERR_INVALID_ARG
 * if smaller).  Sizes and types as in the forward; bf16: P and dS are rounded to bf16
 * before their products, and delta, the row sums of do_ o o, has the rounding of the o
 * given; rows that see at most eight keys take it from P, do_ and v in fp32 instead. */
psa_status_t psa_window_attn_bwd(psa_rows_t q, psa_rows_t k, psa_rows_t v, psa_rows_t o,
                                 psa_rows_t do_, const float *lse, const int *lens, psa_rows_t dq,
                                 psa_rows_t dk, psa_rows_t dv, void *workspace, size_t ws_bytes,
                                 psa_window_t p, float scale, cudaStream_t stream);

/* Bytes of device workspace for psa_window_attn_bwd (0 for an invalid problem). */
size_t psa_window_attn_bwd_workspace_size(psa_window_t p);

/* Single-token form over a cache: n_q is 1, k_cache and v_cache are views [B,
 * num_kv_heads, n_k, d] of which sequence b has filled the first lens[b] rows (int32 on
 * the device, required; values above n_k count as n_k), its query's own key included:
 * the query stands at position lens[b] - 1 and window_right plays no part.  Rows that
 * are not visible may hold anything (NaN included), and only blocks of 16 or 32 rows
 * with a visible one are read.  A sequence of length 0 or less gets output 0.  bf16,
 * rounded as in the forward (fp32: PSA_ERR_UNSUPPORTED), head_dim 64 or 128, any
 * num_heads / num_kv_heads.  workspace: 16-byte aligned, at least
 * psa_window_attn_decode_workspace_size(p) bytes. */
psa_status_t psa_window_attn_decode(psa_rows_t q, psa_rows_t k_cache, psa_rows_t v_cache,
                                    const int *lens, psa_rows_t o, void *workspace,
                                    size_t ws_bytes, psa_window_t p, float scale,
                                    cudaStream_t stream);

/* Bytes of device workspace for psa_window_attn_decode and psa_window_attn_decode_kv4 (0
 * for an invalid problem); they depend on the problem's sizes, not on the lengths. */
size_t psa_window_attn_decode_workspace_size(psa_window_t p);

/* Attention of a batch whose sequences all begin with the same prefix, which is held and read
 * once: k_prefix, v_prefix [1, num_kv_heads, n_prefix, d].  Behind it each sequence has keys of its
 * own, k and v [B, num_kv_heads, n_k, d]; query head h reads key/value head h / (num_heads /
 * num_kv_heads).  Every query sees the whole prefix.  bf16 (fp32: PSA_ERR_UNSUPPORTED), rounded as
 * in psa_window_attn_fwd, head_dim 64 or 128, n_q <= n_k, B * num_heads up to 65535 and B *
 * num_heads * n_q up to 2^28.  Rows of bf16 alone: a cache in 4 bits is neither read here nor, below,
 * accounted for or cut. */
typedef struct {
    int B, num_heads, num_kv_heads, n_q, n_prefix, n_k, head_dim;
    psa_dtype_t dtype;
} psa_prefix_t;

/* Prompts behind the prefix: q [B, num_heads, n_q, d] are the last n_q of each sequence's n_k own
 * tokens, and query row i also sees the own keys j <= i + n_k - n_q.  lens, int32 [B] on the
 * device (NULL: n_k): own tokens from lens[b] on are padding, whose queries get output 0 and
 * log-sum-exp -infinity, and which are seen by none, whatever they hold.  Every row of o is
 * written, and lse, fp32 [B, num_heads, n_q] (NULL: not wanted).  How the work over the prefix is cut
 * goes by the sizes and the lengths: a row's last bits may differ between batches of other lengths;
 * lengths that are all n_k give the bits of a call without them.  workspace: 16-byte aligned, at least
 * psa_prefix_attn_workspace_size(p) bytes, which hold sums in fp32 (8 to 9 * head_dim bytes for each of
 * many rows of q, and up to 20 MB besides). */
psa_status_t psa_prefix_attn_fwd(psa_rows_t q, psa_rows_t k_prefix, psa_rows_t v_prefix,
                                 psa_rows_t k, psa_rows_t v, const int *lens, psa_rows_t o,
                                 float *lse, void *workspace, size_t ws_bytes, psa_prefix_t p,
                                 float scale, cudaStream_t stream);

/* Single tokens (n_q 1) over caches, of which sequence b has filled the first lens[b] rows (int32
 * on the device, required; values above n_k count as n_k), its query's own key included; a
 * sequence of length 0 sees the prefix alone, one of negative length is not there and gets output
 * 0.  Rows behind the sequences may hold anything. */
psa_status_t psa_prefix_attn_decode(psa_rows_t q, psa_rows_t k_prefix, psa_rows_t v_prefix,
                                    psa_rows_t k_cache, psa_rows_t v_cache, const int *lens,
                                    psa_rows_t o, void *workspace, size_t ws_bytes, psa_prefix_t p,
                                    float scale, cudaStream_t stream);

/* Bytes of device workspace for both (0 for an invalid problem). */
size_t psa_prefix_attn_workspace_size(psa_prefix_t p);

/* Rows for a cache: row n of sequence b (n < counts[b], int32 [B] on the device; NULL:
 * all N) goes to cache row starts[b] + n (int32 [B] on the device).  Rows that fall
 * outside the cache's max_len rows are dropped; all other cache rows stay as they
 * were. */
typedef struct {
    int B, num_kv_heads, N, max_len, head_dim;
    psa_dtype_t dtype; /* of the rows */
} psa_cache_t;

/* Copies k, v [B, num_kv_heads, N, d] into caches of the same type, views [B,
 * num_kv_heads, max_len, d].  head_dim 64 or 128; bf16 or fp32. */
psa_status_t psa_kv_append(psa_rows_t k, psa_rows_t v, const int *starts, const int *counts,
                           psa_rows_t k_cache, psa_rows_t v_cache, psa_cache_t p,
                           cudaStream_t stream);

/* A cache held in 4 bits: codes uint8 [B, num_kv_heads, max_len, d / 2] and scales bf16
 * [B, num_kv_heads, max_len, d / 32], dense and 16-byte aligned.  Each group of 32
 * channels of a row has one scale, its largest magnitude times 1/7 (an fp32 product)
 * rounded to bf16; a code is the nearest multiple of it (an fp32 quotient, ties to even,
 * clamped to -7 .. 7; 0 where the scale is 0) plus 8, and stands for (code - 8) * scale.
 * The code of channel 32 g + 4 a + i is the nibble (a * (d / 32) + g) * 4 + i of its row,
 * low nibble of a byte first.  This quantises and stores the rows of k and v; head_dim 64
 * or 128, rows bf16 or fp32. */
psa_status_t psa_kv4_append(psa_rows_t k, psa_rows_t v, const int *starts, const int *counts,
                            void *k_codes, void *k_scales, void *v_codes, void *v_scales,
                            psa_cache_t p, cudaStream_t stream);

/* The values that rows 0 .. N - 1 of every sequence's 4-bit cache stand for, into the
 * views k and v [B, num_kv_heads, N, d], N <= max_len, rounded once to their type. */
psa_status_t psa_kv4_read(const void *k_codes, const void *k_scales, const void *v_codes,
                          const void *v_scales, psa_rows_t k, psa_rows_t v, psa_cache_t p,
                          cudaStream_t stream);

/* psa_window_attn_decode over a cache held in 4 bits (p.n_k rows, p.dtype that of q and
 * o: bf16).  The codes' values enter the products exactly; scales multiply fp32 sums
 * (keys) and probabilities (values; rounded to bf16 after it).  For the products with keys
 * each group of 32 channels of q is held in fp16 relative to its largest one: a channel
 * loses at most 2^-25 of that, nothing down to 2^-17 of it. */
psa_status_t psa_window_attn_decode_kv4(psa_rows_t q, const void *k_codes, const void *k_scales,
                                        const void *v_codes, const void *v_scales,
                                        const int *lens, psa_rows_t o, void *workspace,
                                        size_t ws_bytes, psa_window_t p, float scale,
                                        cudaStream_t stream);

/* Attention weights summed for each key of a cache, and the eviction of the keys that have
 * least.  weights: fp32 [B, num_kv_heads, n_k], dense: a key/value head's row j holds the sum,
 * over the query heads that share it and all queries so far, of the softmax probability that key
 * j had.  Rows behind a sequence's length are kept at 0 by the caller, or by psa_kv_evict.
 *
 * Adds to weights what the keys of a prompt (k, [B, num_kv_heads, n_k, d]) got from its queries q,
 * or from its last n_q ones: lse, fp32 [B, num_heads, n_q], is psa_window_attn_fwd's of the same
 * problem, which says what a query sees.  Scores and sums are fp32, in a fixed order; entries from a
 * sequence's length on are left as they are.  bf16 (fp32: PSA_ERR_UNSUPPORTED), head_dim 64 or
 * 128.  workspace: at least psa_window_attn_weights_workspace_size(p) bytes. */
psa_status_t psa_window_attn_weights(psa_rows_t q, psa_rows_t k, const int *lens, const float *lse,
                                     float *weights, void *workspace, size_t ws_bytes,
                                     psa_window_t p, float scale, cudaStream_t stream);

/* Bytes of device workspace for psa_window_attn_weights (0 for an invalid problem). */
size_t psa_window_attn_weights_workspace_size(psa_window_t p);

/* psa_window_attn_decode that also adds the probabilities of its step's visible keys to weights
 * (fp32, from the scores before any rounding; heads are added in order: reruns are bitwise
 * identical; entries of keys that are not visible are left as they are).  The same partial sums,
 * joined in another order, make the output.  Same sizes and errors, with up to 4096 query heads
 * for each key/value head (PSA_ERR_UNSUPPORTED); workspace: at least
 * psa_window_attn_decode_weights_workspace_size(p) bytes, which hold the step's scores. */
psa_status_t psa_window_attn_decode_weights(psa_rows_t q, psa_rows_t k_cache, psa_rows_t v_cache,
                                            const int *lens, psa_rows_t o, float *weights,
                                            void *workspace, size_t ws_bytes, psa_window_t p,
                                            float scale, cudaStream_t stream);

/* Bytes of device workspace for psa_window_attn_decode_weights (0 for an invalid problem). */
size_t psa_window_attn_decode_weights_workspace_size(psa_window_t p);

/* Eviction: every sequence that has more than keep rows (lens, int32 [B] on the device) is cut to
 * keep rows in each key/value head.  Those with the largest weights stay; of equal weights those
 * of the lower rows (0 and -0 are equal; NaN is above infinity); before all others those at
 * positions below sinks and at the last `recent` positions: positions, int32 [B, num_kv_heads,
 * max_len], dense, says for each row which token of its sequence it holds, and the last one is the
 * largest among a head's rows.  What stays lies in rows 0 .. keep - 1 afterwards: a row that stays
 * and lies there already is not touched, and those that stay from behind fill the gaps, in the
 * order of their rows.  (The order of a cache's rows plays no part in attention over all of
 * them.)  The caches are changed in place, rows from keep on left as they are.
 *
 * weights_out, positions_out: the same for the rows that stay; in front of the old length and
 * behind them weights_out is set to 0, so that rows appended later start from nothing, and
 * positions_out is left as it was.  They may be the same arrays as weights and positions.  lens_out
 * [B]: min(lens, max_len, keep) (0 for a negative one), not the same array as lens; lens above max_len
 * count as max_len.  All outputs are written for the sequences that have no more than keep rows too.
 * max_len up to 2^24, B * num_kv_heads up to 65535 (PSA_ERR_UNSUPPORTED); head_dim 64 or 128; bf16 or
 * fp32. */
typedef struct {
    int B, num_kv_heads, max_len, head_dim;
    psa_dtype_t dtype;
    int keep, sinks, recent; /* sinks + recent <= keep */
} psa_evict_t;

psa_status_t psa_kv_evict(const float *weights, const int *positions, const int *lens,
                          psa_rows_t k_cache, psa_rows_t v_cache, float *weights_out,
                          int *positions_out, int *lens_out, void *workspace, size_t ws_bytes,
                          psa_evict_t p, cudaStream_t stream);

/* Bytes of device workspace for psa_kv_evict (0 for an invalid problem). */
size_t psa_kv_evict_workspace_size(psa_evict_t p);

/* ---- status ------------------------------------------------------------------- */

/* Static description of a status code. */
const char *psa_status_string(psa_status_t status);

/* Synchronises the stream, then reads and clears the device-side error word
 * (PSA_ERR_TIMEOUT after a bounded on-chip wait gave up; PSA_OK otherwise). */
psa_status_t psa_get_last_device_error(cudaStream_t stream);

/* Diagnostic of the failure path (no counterpart on the pages): launches one warp
 * that waits, through the same bounded on-chip wait as the attention kernels but
 * with a limit of limit_ns nanoseconds (1 .. 100,000,000), on a barrier that
 * nothing arrives at.  The wait gives up, records PSA_ERR_TIMEOUT in the device
 * error word (read it with psa_get_last_device_error) and the kernel returns; the
 * context stays usable.  PSA_ERR_INVALID_ARG for a limit outside that range. */
psa_status_t psa_debug_wait_timeout(unsigned long long limit_ns, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PSA_GB300_H */
