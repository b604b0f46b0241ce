// window_bwd.cu -- attention with a sliding window and first tokens that stay visible:
// backward on tensor cores (tcgen05, bf16), a kernel for dQ and one for dK and dV.
//
//   P = 2^(scale log2(e) S - lse log2(e)), S = Q K^T over the visible keys,
//   dP = dO V^T, dS = P o (dP - delta), delta = rowsum(dO o O),
//   dQ = scale dS K;  dV = P^T dO, dK = scale dS^T Q.
//
// Bound by the tensor cores: 3 products per tile pair for dQ and 4 for dK and dV, where five
// would do if dQ were added up across the CTAs that own the keys.  That sum would need atomics,
// whose order changes results, or a partial dQ per key tile; two kernels need neither, and
// each gradient is summed by one CTA in a fixed order, over the query heads that share a
// key/value head too.
//
// Both kernels: a persistent CTA per SM, 256 row threads (two per row of tensor memory, each
// 64 of the 128 columns), a TMA producer, a warp that issues the products, and one that
// zeroes the rows of padding where they are an operand (0 times NaN is NaN).  bf16 operands
// made by the row threads stay in tensor memory: each thread writes them over the columns
// that it read.  All products come from one warp and complete in the order they are issued
// (observed, as in window_fwd.cu: PTX promises it for products of one shape into the same
// sums, not for S next to dQ):
//   dQ kernel     the next tile's S as soon as this one's is in registers, its dP (two buffers),
//                 then this tile's dQ += dS K (dS in dP's columns), so the row threads find
//                 both operands when they come to the next tile
//   dK/dV kernel  S^T = K Q^T and dP^T = V dO^T have keys as rows: dV += P^T dO and the next
//                 S^T behind it, while the row threads make dS^T; dK += dS^T Q and the next
//                 dP^T, while they make P^T.
// delta and lse come from a small kernel in front: for each tile of 128 rows (the last one
// padded) 128 values of -lse log2(e), then 128 of -delta, so that a tile's 1024 bytes are one
// bulk copy and two neighbouring columns' values one operand of a paired instruction.  delta is
// rowsum(dO o O), or for rows that see few keys the sum of P dP.
// Measured: 2 x 4096 tokens, 16 heads of 128 on 4, a window of 1024 and 4 sinks: 238 us (dK/dV 127
// with the pipe busy 61 % of the time, dQ 93 with 49 %, statistics and parts 10 each; 0.63 PFLOP/s
// counting five products); 16384 tokens causal, 16 heads on 2: 2.65 ms (1.04 PFLOP/s; dK/dV 75 %,
// dQ 67 %).
#include <math.h>

#include <algorithm>

#include "window_tc.cuh"

namespace psa {
namespace {

constexpr int kThreads = 384;
constexpr int kProducer = 8, kIssuer = 9, kFixer = 11;  // warp 10 idles

// How the dK/dV kernel's work is cut.  A key tile's steps are the query tiles that see it,
// for each query head of its group: from a window's few to every query there is (sinks, or no
// window).  Tiles with more than `steps` of them are cut into parts of that many, whose
// fp32 results a small kernel adds in order; part p has the first tiles[p] key tiles.
constexpr int kMaxParts = 32;
struct Cut {
  int parts, steps;
  int tiles[kMaxParts];
  int units;  // over all parts, batch items and key/value heads
  // partial results in front of part p's (part 0: of the key tiles that have a part 1)
  __host__ __device__ __forceinline__ int slot0(int p) const {
    int n = 0;
    for (int i = 1; i <= p; ++i) n += tiles[i == 1 ? 1 : i - 1];
    return n;
  }
};

struct BwdParams {
  Window w;
  View<__nv_bfloat16> dq, dk, dv;
  const float* stat;   // [B, nh, row_tiles, 2, 128]: -lse log2(e), -delta
  float* partial;      // [slots, B * nkv, 2 (dV, dK), 128, D]
  float scale, sl2;
  int units, row_tiles;
  Cut cut;
};

// Unit of this CTA in its round i (from long to short: CTA order, then reverse order).
__device__ __forceinline__ int unit_of(int i) {
  return i * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// -lse log2(e) and -delta of every row; rows that see nothing, and those behind n_q, get 0:
// their scores are masked.  D / 8 lanes share a row, 16 bytes of dO and of O in each, and take
// four rows, all on their way at once.
//
// Rows that see few keys have a delta of their own: there dP - delta may be small next to delta,
// and o, rounded to bf16, leaves delta a rounding error of its own size (dQ and dK of two keys 3.5 to
// 5e-3 off in the 2-norm, where the roundings of dS and the output alone give 2.4e-3).  It is
// sum P dP in fp32, S and dP by tensor instructions, 16 rows and 8 keys a warp.  The error falls
// with the root of the number of keys: from nine on it is under 0.7 of the rounding of dS, and o as
// given does.  (3 x 1000 rows, 8 heads: 33.6 -> 34.3 us a backward; 8192 rows, 32 heads on 8, all with
// eight keys: 188 -> 247.)  The grid's first `again` blocks are for these rows, next to the others rather than
// behind them.
constexpr int kStatRows = 4, kFewKeys = 8;
template <int D>
constexpr int kStatBlock = 256 / (D / 8) * kStatRows;  // rows of a block
constexpr int kFewBlock = 8 * 16;                      // of one for rows that see few keys

// The keys that row i sees: 0 .. front - 1 and lo .. hi, if they are few (and some).
struct FewKeys {
  int front, lo, hi;
  bool any;
  __device__ __forceinline__ FewKeys(const Window& w, int len, int i) {
    const int p = i + w.nk - w.nq;
    lo = max(0, p - w.left);
    hi = min(len - 1, p + w.right);
    front = min(w.sinks, lo);
    any = i < w.nq && p >= 0 && p < len && front + hi - lo + 1 <= kFewKeys;
  }
};
// Whether one of the rows i0 .. i1 may be such: false if the first and the last one are far enough
// from the sequence's ends and the window is wide enough.
__device__ __forceinline__ bool may_see_few(const Window& w, int len, int i0, int i1) {
  const int off = w.nk - w.nq;
  return min(min(max(0, i0 + off) + w.right + 1, len), w.left + min(w.right + 1, len - off - i1)) <= kFewKeys;
}

// -delta of those among a warp's 16 rows from i0 on.  kTiles: of 8 keys, that they see between them
// (16 rows of 8 keys see 23, and the sinks; positions 0 .. 7 behind a wider window see keys 0 .. 7).
template <int D, int kTiles>
__device__ __forceinline__ void few_keys_delta(const WindowArgs<__nv_bfloat16>& a, float* stat, int b, int h, int len,
                                               int i0) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, hk = h / (a.w.nh / a.w.nkv);
  const FewKeys f[2] = {FewKeys(a.w, len, i0 + g), FewKeys(a.w, len, i0 + g + 8)};
  if (!__any_sync(0xffffffffu, f[0].any || f[1].any)) return;
  int first = a.w.nk, last = -1, front = 0;  // of all rows
  float nlse[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    nlse[r] = f[r].any ? -a.lse[((long long)b * a.w.nh + h) * a.w.nq + i0 + g + 8 * r] * kLog2 : 0.f;
    if (!f[r].any) continue;
    first = min(first, f[r].lo);
    last = max(last, f[r].hi);
    front = max(front, f[r].front);
  }
  first = __reduce_min_sync(0xffffffffu, first);
  last = __reduce_max_sync(0xffffffffu, last);
  front = __reduce_max_sync(0xffffffffu, front);
  const int sink = front > 0;  // the sinks' tile, then the windows'
  auto from = [&](int tile) { return tile < sink ? 0 : first + 8 * (tile - sink); };
  auto end = [&](int tile) { return tile < sink ? front : last + 1; };
  float x[kTiles][4], y[kTiles][4];
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[n][e] = y[n][e] = 0.f;
  // (the order of the channels is free: each lane takes 16 neighbouring bytes)
  auto load = [&](const View<const __nv_bfloat16>& v, int head, int row, int c, bool on) {
    return on ? *reinterpret_cast<const uint4*>(v.row(b, head, row) + 32 * c + 8 * t) : make_uint4(0, 0, 0, 0);
  };
#pragma unroll(kTiles == 1 ? D / 32 : 2)
  for (int c = 0; c < D / 32; ++c) {
    const uint4 q0 = load(a.q, h, i0 + g, c, f[0].any), q1 = load(a.q, h, i0 + g + 8, c, f[1].any);
    const uint4 d0 = load(a.dO, h, i0 + g, c, f[0].any), d1 = load(a.dO, h, i0 + g + 8, c, f[1].any);
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      if (from(n) > last) continue;
      const int j = from(n) + g;
      const uint4 k = load(a.k, hk, j, c, j < end(n)), v = load(a.v, hk, j, c, j < end(n));
      mma16816(x[n], q0.x, q1.x, q0.y, q1.y, k.x, k.y);
      mma16816(x[n], q0.z, q1.z, q0.w, q1.w, k.z, k.w);
      mma16816(y[n], d0.x, d1.x, d0.y, d1.y, v.x, v.y);
      mma16816(y[n], d0.z, d1.z, d0.w, d1.w, v.z, v.w);
    }
  }
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const FewKeys& m = f[e / 2];
      const int j = from(n) + 2 * t + e % 2;
      if (m.any && (n < sink ? j < m.front : j >= m.lo && j <= m.hi))
        s[e / 2] += fast_exp2(x[n][e] * (a.scale * kLog2) + nlse[e / 2]) * y[n][e];
    }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    s[r] += __shfl_xor_sync(0xffffffffu, s[r], 1);
    s[r] += __shfl_xor_sync(0xffffffffu, s[r], 2);
    const int i = i0 + g + 8 * r;
    if (t == 0 && f[r].any) stat[i / kTile * (2 * kTile) + kTile + i % kTile] = -s[r];
  }
}

template <int D, bool kNarrow>
__global__ void __launch_bounds__(256, kNarrow ? 2 : 4)
    window_stat_kernel(const WindowArgs<__nv_bfloat16> a, float* stat, int padded, int blocks, int again) {
  constexpr int LANES = D / 8, GROUPS = 256 / LANES;
  pdl_launch_dependents();
  pdl_wait();
  const int off = a.w.nk - a.w.nq;
  if ((int)blockIdx.x < again) {
    const int warp = threadIdx.x / 32;
    int head, i;
    if constexpr (kNarrow) {  // any row of a head
      const int n = (a.w.nq + kFewBlock - 1) / kFewBlock;
      head = blockIdx.x / n;
      i = blockIdx.x % n * kFewBlock + 16 * warp;
    } else {  // the first rows of one head for each warp
      head = 8 * blockIdx.x + warp;
      i = max(0, -off);
      if (head >= a.w.B * a.w.nh) return;
    }
    const int len = a.w.len(head / a.w.nh);
    if (may_see_few(a.w, len, i, i + 15))
      few_keys_delta<D, kNarrow ? 4 : 1>(a, stat + 2 * (long long)head * padded, head / a.w.nh, head % a.w.nh, len, i);
    return;
  }
  const int head = (blockIdx.x - again) / blocks, start = (blockIdx.x - again) % blocks * kStatBlock<D>;
  const int b = head / a.w.nh, h = head % a.w.nh, len = a.w.len(b);
  const int from = max(0, -off), to = min(a.w.nq, len - off);  // rows that see something
  stat += 2 * (long long)head * padded;
  const int lr = threadIdx.x % LANES, i0 = start + threadIdx.x / LANES;
  const bool few = may_see_few(a.w, len, start, start + kStatBlock<D> - 1);
  const __nv_bfloat16 *g = a.dO.row(b, h, i0) + 8 * lr, *o = a.o.row(b, h, i0) + 8 * lr;
  const float* lse = a.lse + (long long)head * a.w.nq;
  uint4 rg[kStatRows], ro[kStatRows];
  float l[kStatRows];
#pragma unroll
  for (int k = 0; k < kStatRows; ++k) {
    const int i = i0 + GROUPS * k;
    rg[k] = ro[k] = make_uint4(0, 0, 0, 0);
    l[k] = 0.f;
    if (i >= from && i < to) {
      l[k] = lse[i];
      if (kNarrow && few && FewKeys(a.w, len, i).any) continue;  // its delta is not made here
      rg[k] = *reinterpret_cast<const uint4*>(g + GROUPS * k * a.dO.sn);
      ro[k] = *reinterpret_cast<const uint4*>(o + GROUPS * k * a.o.sn);
    }
  }
#pragma unroll
  for (int k = 0; k < kStatRows; ++k) {
    const int i = i0 + GROUPS * k;
    float x[8], y[8], s = 0.f;
    unpack_vec(rg[k], x);
    unpack_vec(ro[k], y);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[e] * y[e];
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (lr == 0 && i < padded) {
      float* at = stat + i / kTile * (2 * kTile) + i % kTile;
      at[0] = -l[k] * kLog2;
      if (!few || !FewKeys(a.w, len, i).any) at[kTile] = -s;
    }
  }
}

__device__ __forceinline__ float2 pair(const uint32_t* x) {
  return make_float2(__uint_as_float(x[0]), __uint_as_float(x[1]));
}
// A masked pair's dP may be NaN (padding); its P is 0, and so must its dS be.
__device__ __forceinline__ void drop_masked(const uint32_t (&p)[64], uint32_t (&dp)[64]) {
#pragma unroll
  for (int c = 0; c < 64; ++c)
    if (p[c] == 0u) dp[c] = 0u;
}

// ---------------------------------------------------------------- dQ
template <int D>
struct DqCfg {
  static constexpr uint32_t TILE = kTileBytes<D>;
  static constexpr int KST = D == 128 ? 3 : 4, VST = D == 128 ? 2 : 4;
  static constexpr uint32_t OFF_DO = TILE, OFF_K = 2 * TILE, OFF_V = OFF_K + KST * TILE;
  static constexpr uint32_t OFF_BAR = OFF_V + VST * TILE, SMEM = OFF_BAR + 512 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DQ = 384;  // dP: two buffers
};
struct DqBars {
  uint64_t q_full, q_empty, do_full, do_empty, k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t k_fixed[4], s_full, s_free, dp_full[2], ds_full[2], dq_full, done;
};

// A unit of the dQ kernel: 128 query rows of a head.
struct DqUnit {
  int b, h, hk, row0, len, edge, end;  // end: keys from here on are seen by no row
  KeyTiles<kTile> tiles;
  int p0, p1;
  __device__ __forceinline__ DqUnit(const BwdParams& a, int u) {
    const Window& w = a.w;
    const int heads = w.B * w.nh, x = u % heads;
    b = x / w.nh;
    h = x % w.nh;
    hk = h / (w.nh / w.nkv);
    row0 = (a.row_tiles - 1 - u / heads) * kTile;
    len = w.len(b);
    const int off = w.nk - w.nq;
    p0 = max(0, row0 + off);
    p1 = min(len, min(row0 + kTile, w.nq) + off) - 1;
    tiles = KeyTiles<kTile>(w, len, p0, p1);
    end = min(len, p1 + w.right + 1);
    // the key tile with rows of padding, always the last one if it is visited
    edge = len % kTile != 0 && len < w.nk ? len / kTile : -1;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_dq_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                        const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const BwdParams a) {
  using C = DqCfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = align1024(smem_raw);
  const uint32_t sbase = smem_addr(smem);
  DqBars& bar = *reinterpret_cast<DqBars*>(smem + C::OFF_BAR);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(&bar + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_at + 1);
  static_assert(sizeof(DqBars) + 16 <= 512, "barriers");
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bar.q_full, 1);
    mbar_init(&bar.q_empty, 1);
    mbar_init(&bar.do_full, 1);
    mbar_init(&bar.do_empty, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.k_fixed[i], 1);
      mbar_init(&bar.v_full[i], 1);
      mbar_init(&bar.v_empty[i], 1);
    }
    mbar_init(&bar.s_full, 1);
    mbar_init(&bar.s_free, 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.dp_full[i], 1);
      mbar_init(&bar.ds_full[i], 256);  // by dP buffer: a thread may be a tile ahead of another
    }
    mbar_init(&bar.dq_full, 1);
    mbar_init(&bar.done, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == kFixer) {
    tmem_alloc(tmem_at, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == kProducer) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      bool ok = true;
      int uc = 0, kc = 0;  // units with tiles, tiles
      for (int i = 0; ok && unit_of(i) < a.units; ++i) {
        const DqUnit u(a, unit_of(i));
        for (int t = 0; ok && t < u.tiles.count; ++t, ++kc) {
          const int j0 = u.tiles.tile(t) * kTile, ks = kc % C::KST, vs = kc % C::VST;
          if (kc >= C::KST && !mbar_wait(&bar.k_empty[ks], (kc / C::KST - 1) & 1, abort)) ok = false;
          if (!ok) break;
          if (t == 0) {
            if (uc >= 1 && !mbar_wait(&bar.q_empty, (uc - 1) & 1, abort)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&bar.q_full, C::TILE);
            load_tile<D>(smem, &tmQ, &bar.q_full, u.row0, u.h, u.b);
          }
          mbar_arrive_expect_tx(&bar.k_full[ks], C::TILE);
          load_tile<D>(smem + C::OFF_K + ks * C::TILE, &tmK, &bar.k_full[ks], j0, u.hk, u.b);
          if (t == 0) {
            if (uc >= 1 && !mbar_wait(&bar.do_empty, (uc - 1) & 1, abort)) {
              ++kc;
              ++uc;
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&bar.do_full, C::TILE);
            load_tile<D>(smem + C::OFF_DO, &tmDO, &bar.do_full, u.row0, u.h, u.b);
            ++uc;
          }
          if (kc >= C::VST && !mbar_wait(&bar.v_empty[vs], (kc / C::VST - 1) & 1, abort)) {
            ++kc;
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bar.v_full[vs], C::TILE);
          load_tile<D>(smem + C::OFF_V + vs * C::TILE, &tmV, &bar.v_full[vs], j0, u.hk, u.b);
        }
      }
      if (*abort) {
        // let the copies in flight land before the CTA exits (a wait for one that was not
        // issued any more runs into its time limit)
        if (uc > 0) {
          drain_wait(&bar.q_full, (uc - 1) & 1);
          drain_wait(&bar.do_full, (uc - 1) & 1);
        }
        for (int n = max(0, kc - C::KST); n < kc; ++n) drain_wait(&bar.k_full[n % C::KST], (n / C::KST) & 1);
        for (int n = max(0, kc - C::VST); n < kc; ++n) drain_wait(&bar.v_full[n % C::VST], (n / C::VST) & 1);
      }
    }
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ issuer (converged warp)
    const uint64_t dQ = desc_rows_by_channels(sbase), dDO = desc_rows_by_channels(sbase + C::OFF_DO);
    const uint64_t dK = desc_rows_by_channels(sbase + C::OFF_K), dV = desc_rows_by_channels(sbase + C::OFF_V);
    const uint64_t dKb = desc_channels_by_rows(sbase + C::OFF_K);
    const uint32_t idQ = idesc_bf16_f32(128, D, false, true);
    bool ok = true;
    int kc = 0, uc = 0;
    for (int i = 0; ok && unit_of(i) < a.units; ++i) {
      const DqUnit u(a, unit_of(i));
      const int n = u.tiles.count;
      if (n == 0) continue;
      // tiles of which few columns are seen (sinks, the last one) work on those only
      auto cols_of = [&](int t) { return used_columns(u.tiles.tile(t), u.tiles.first, u.end, a.w.sinks); };
      auto scores = [&](uint32_t tX, uint64_t dA, uint64_t dB, int cols) {
        auto go = [&](uint32_t id) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_warp(tX, dA + kstep_channels(kk), dB + kstep_channels(kk), id, kk > 0 ? 1u : 0u);
        };
        if (cols == kTile) go(idesc_bf16_f32(128, kTile, false, false));
        else go(idesc_bf16_f32(128, cols, false, false));
      };
      // S and dP of tile t
      auto issue_s = [&](int t) -> bool {
        const int c = kc + t, st = c % C::KST;
        if (!mbar_wait(&bar.k_full[st], (c / C::KST) & 1, abort) ||
            (c >= 1 && !mbar_wait(&bar.s_free, (c - 1) & 1, abort)))
          return false;
        tc_fence_after();
        scores(tmem + C::TM_S, dQ, dK + (uint64_t)(st * C::TILE >> 4), cols_of(t));
        mma_commit_warp(&bar.s_full);
        if (t == n - 1) mma_commit_warp(&bar.q_empty);
        return true;
      };
      auto issue_dp = [&](int t) -> bool {
        const int c = kc + t, st = c % C::VST;
        if (!mbar_wait(&bar.v_full[st], (c / C::VST) & 1, abort)) return false;
        tc_fence_after();
        scores(tmem + C::TM_DP + 128 * (c & 1), dDO, dV + (uint64_t)(st * C::TILE >> 4), cols_of(t));
        mma_commit_warp(&bar.dp_full[c & 1]);
        mma_commit_warp(&bar.v_empty[st]);
        if (t == n - 1) mma_commit_warp(&bar.do_empty);
        return true;
      };
      ok = mbar_wait(&bar.q_full, uc & 1, abort) && issue_s(0) && mbar_wait(&bar.do_full, uc & 1, abort) &&
           issue_dp(0);
      for (int t = 0; ok && t < n; ++t) {
        const int c = kc + t, st = c % C::KST;
        if (t + 1 < n && !(issue_s(t + 1) && issue_dp(t + 1))) ok = false;
        if (!ok || !mbar_wait(&bar.ds_full[c & 1], (c / 2) & 1, abort) ||
            !mbar_wait(&bar.k_fixed[st], (c / C::KST) & 1, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t d = dKb + (uint64_t)(st * C::TILE >> 4);
        const uint32_t tDS = tmem + C::TM_DP + 128 * (c & 1);
        const int cols = cols_of(t);
        // 16 keys' dS are 8 columns; those of keys 64 .. 127 start at column 64
        if (cols == kTile) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts_warp(tmem + C::TM_DQ, tDS + 64 * (kk / 4) + 8 * (kk % 4), d + kk * kKstepRows, idQ,
                             t > 0 || kk > 0 ? 1u : 0u);
        } else {
#pragma unroll 1
          for (int kk = 0; 16 * kk < cols; ++kk)
            mma_bf16_ts_warp(tmem + C::TM_DQ, tDS + 64 * (kk / 4) + 8 * (kk % 4), d + kk * kKstepRows, idQ,
                             t > 0 || kk > 0 ? 1u : 0u);
        }
        mma_commit_warp(&bar.k_empty[st]);
        if (t == n - 1) mma_commit_warp(&bar.dq_full);
      }
      kc += n;
      ++uc;
    }
    mma_commit_warp(&bar.done);
    drain_wait(&bar.done, 0);
  } else if (warp == kFixer) {
    // ------------------------------------------------------------ rows of padding in K
    // Every tile passes through this warp, so that k_fixed's phases keep step with the ring.
    int kc = 0;
    bool ok = true;
    for (int i = 0; ok && unit_of(i) < a.units; ++i) {
      const DqUnit u(a, unit_of(i));
      for (int t = 0; t < u.tiles.count; ++t, ++kc) {
        const int st = kc % C::KST;
        if (!mbar_wait(&bar.k_full[st], (kc / C::KST) & 1, abort)) {
          ok = false;
          break;
        }
        if (u.tiles.tile(t) == u.edge) zero_rows<D>(smem + C::OFF_K + st * C::TILE, u.len % kTile, kTile, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.k_fixed[st]);
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ row threads
    const int half = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + C::TM_S + 64 * half + lanes, tP = tmem + C::TM_DP + 64 * half + lanes;
    const uint32_t tQ = tmem + C::TM_DQ + lanes;
    const int off = a.w.nk - a.w.nq;
    int kc = 0, uc = 0;
    bool ok = true;
    for (int i = 0; ok && unit_of(i) < a.units; ++i) {
      const DqUnit u(a, unit_of(i));
      const int q = u.row0 + r, p = q + off;
      // (a row that sees one key has dS = 0: nothing else is made of P here)
      const int jhi = p >= 0 && p < u.len && q < a.w.nq && !sees_one(a.w, u.len, p) ? min(u.len - 1, p + a.w.right) : -1;
      const int jlo = p - a.w.left;
      // rows that do not exist or are padding get anything here and 0 at the end
      const int whole_lo = u.p1 - a.w.left, whole_hi = min(u.len, u.p0 + a.w.right + 1);
      const float* stat = a.stat + 2 * ((long long)(u.b * a.w.nh + u.h) * a.row_tiles * kTile + u.row0) + r;
      const float2 nlse = make_float2(stat[0], stat[0]), ndelta = make_float2(stat[kTile], stat[kTile]);
      const float2 sl = make_float2(a.sl2, a.sl2);
      for (int t = 0; t < u.tiles.count; ++t, ++kc) {
        const int tile0 = u.tiles.tile(t) * kTile, j0 = tile0 + 64 * half;
        const uint32_t tDP = tP + 128 * (kc & 1);
        if (!mbar_wait(&bar.s_full, kc & 1, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t x[64];
        load_cols64(tS, x);
        tc_fence_before();
        mbar_arrive(&bar.s_free);
        const bool whole = tile0 + kTile <= whole_hi && (tile0 >= whole_lo || tile0 + kTile <= a.w.sinks);
        if (!whole) {
          // -inf: P = 0 (columns that were not worked on among them)
          const int hi = jhi - j0, lo = jlo - j0, sk = a.w.sinks - j0;
          hide(x, visible32(lo, hi, sk));
          hide(x + 32, visible32(lo - 32, hi - 32, sk - 32));
        }
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 e = __ffma2_rn(pair(x + c), sl, nlse);
          x[c] = __float_as_uint(fast_exp2(e.x));
          x[c + 1] = __float_as_uint(fast_exp2(e.y));
        }
        if (!mbar_wait(&bar.dp_full[kc & 1], (kc / 2) & 1, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t y[64];
        load_cols64(tDP, y);
        if (!whole) drop_masked(x, y);
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 d = __fmul2_rn(pair(x + c), __fadd2_rn(pair(y + c), ndelta));
          y[c / 2] = pack2(d.x, d.y);
        }
        tmem_store16_async(tDP, y);
        tmem_store16_async(tDP + 16, y + 16);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar.ds_full[kc & 1]);
      }
      if (!ok) break;
      // ---- dQ of this row: half of its channels per thread
      const bool some = u.tiles.count > 0;
      if (some) {
        if (!mbar_wait(&bar.dq_full, uc & 1, abort)) break;
        ++uc;
        tc_fence_after();
      }
      const bool in = q < a.w.nq;
      __nv_bfloat16* dst = a.dq.row(u.b, u.h, in ? q : 0) + half * (D / 2);
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 32) {
        float o[32];
        if (some) {
          tmem_load32(tQ + half * (D / 2) + c, o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        if (in) {
          const bool valid = q + off >= 0 && q + off < u.len;
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            const uint4 v = make_uint4(pack2(o[k] * a.scale, o[k + 1] * a.scale), pack2(o[k + 2] * a.scale, o[k + 3] * a.scale),
                                       pack2(o[k + 4] * a.scale, o[k + 5] * a.scale),
                                       pack2(o[k + 6] * a.scale, o[k + 7] * a.scale));
            *reinterpret_cast<uint4*>(dst + c + k) = valid ? v : make_uint4(0, 0, 0, 0);
          }
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kFixer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- dK and dV
template <int D>
struct DkvCfg {
  static constexpr uint32_t TILE = kTileBytes<D>;
  static constexpr int ST = D == 128 ? 2 : 4;
  static constexpr uint32_t OFF_V = TILE, OFF_Q = 2 * TILE, OFF_DO = OFF_Q + ST * TILE;
  static constexpr uint32_t OFF_STAT = OFF_DO + ST * TILE, STAT = kTile * 8;
  static constexpr uint32_t OFF_BAR = OFF_STAT + ST * STAT, SMEM = OFF_BAR + 512 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 384;
};
struct DkvBars {
  uint64_t kv_full, kv_empty, q_full[4], q_empty[4], do_full[4], do_empty[4];
  uint64_t q_fixed[4], do_fixed[4], s_full, p_full, dp_full, ds_full, acc_full, done;
};

// A key tile of a key/value head, and the steps of one part of it.
struct DkvUnit {
  int b, hk, k0, len, group, part;
  int i0, i1;        // query rows that see a key of the tile
  int tile0, tiles;  // the tiles of 128 they lie in
  int from, steps;   // this part's
  int slot;          // its partial result's place, -1: the tile has one part
  __device__ __forceinline__ void find(const BwdParams& a, int x, int kt) {
    const Window& w = a.w;
    b = x / w.nkv;
    hk = x % w.nkv;
    group = w.nh / w.nkv;
    k0 = kt * kTile;
    len = w.len(b);
    int n;
    query_range(w, len, k0, min(k0 + kTile, w.nk) - 1, i0, n);
    i1 = i0 + n;
    tile0 = i0 / kTile;
    tiles = n > 0 ? (i1 - 1) / kTile - tile0 + 1 : 0;
  }
  __device__ __forceinline__ DkvUnit(const BwdParams& a, int u) {
    const int heads = a.w.B * a.w.nkv;
    // the last parts first, the last key tiles (which the fewest see) of part 0 at the end
    part = a.cut.parts - 1;
    int t = u / heads;
    while (part > 0 && t >= a.cut.tiles[part]) t -= a.cut.tiles[part--];
    find(a, u % heads, t);
    from = part * a.cut.steps;
    steps = max(0, min(group * tiles - from, a.cut.steps));
    slot = group * tiles > a.cut.steps ? (a.cut.slot0(part) + t) * heads + u % heads : -1;
  }
  // a tile that holds rows that see nothing: rows of padding, or in front of position 0
  __device__ __forceinline__ void valid(const Window& w, int row0, int& lo, int& hi) const {
    const int off = w.nk - w.nq;
    lo = max(0, -off - row0);
    hi = min(kTile, len - off - row0);
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_dkdv_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                          const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const BwdParams a) {
  using C = DkvCfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = align1024(smem_raw);
  const uint32_t sbase = smem_addr(smem);
  DkvBars& bar = *reinterpret_cast<DkvBars*>(smem + C::OFF_BAR);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(&bar + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_at + 1);
  static_assert(sizeof(DkvBars) + 16 <= 512, "barriers");
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bar.kv_full, 1);
    mbar_init(&bar.kv_empty, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.q_full[i], 1);
      mbar_init(&bar.q_empty[i], 1);
      mbar_init(&bar.do_full[i], 1);
      mbar_init(&bar.do_empty[i], 1);
      mbar_init(&bar.q_fixed[i], 1);
      mbar_init(&bar.do_fixed[i], 1);
    }
    mbar_init(&bar.s_full, 1);
    mbar_init(&bar.p_full, 256);
    mbar_init(&bar.dp_full, 1);
    mbar_init(&bar.ds_full, 256);
    mbar_init(&bar.acc_full, 1);
    mbar_init(&bar.done, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == kFixer) {
    tmem_alloc(tmem_at, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == kProducer) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      bool ok = true;
      int uc = 0, qc = 0;
      for (int i = 0; ok && unit_of(i) < a.units; ++i) {
        const DkvUnit u(a, unit_of(i));
        const int n = u.steps;
        if (n == 0) continue;
        if (uc >= 1 && !mbar_wait(&bar.kv_empty, (uc - 1) & 1, abort)) break;
        mbar_arrive_expect_tx(&bar.kv_full, 2 * C::TILE);
        load_tile<D>(smem, &tmK, &bar.kv_full, u.k0, u.hk, u.b);
        load_tile<D>(smem + C::OFF_V, &tmV, &bar.kv_full, u.k0, u.hk, u.b);
        ++uc;
        int h = u.hk * u.group + u.from / u.tiles, tile = u.tile0 + u.from % u.tiles;
        for (int t = 0; t < n; ++t, ++qc) {
          const int st = qc % C::ST, par = (qc / C::ST - 1) & 1;
          if (qc >= C::ST && (!mbar_wait(&bar.q_empty[st], par, abort) || !mbar_wait(&bar.do_empty[st], par, abort))) {
            ok = false;
            break;
          }
          // lse and delta travel with Q: S^T is the first to need them
          mbar_arrive_expect_tx(&bar.q_full[st], C::TILE + C::STAT);
          load_tile<D>(smem + C::OFF_Q + st * C::TILE, &tmQ, &bar.q_full[st], tile * kTile, h, u.b);
          bulk_load(smem + C::OFF_STAT + st * C::STAT,
                    a.stat + ((long long)(u.b * a.w.nh + h) * a.row_tiles + tile) * (2 * kTile), C::STAT, &bar.q_full[st]);
          mbar_arrive_expect_tx(&bar.do_full[st], C::TILE);
          load_tile<D>(smem + C::OFF_DO + st * C::TILE, &tmDO, &bar.do_full[st], tile * kTile, h, u.b);
          if (++tile == u.tile0 + u.tiles) {
            tile = u.tile0;
            ++h;
          }
        }
      }
      if (*abort) {
        if (uc > 0) drain_wait(&bar.kv_full, (uc - 1) & 1);
        for (int n = max(0, qc - C::ST); n < qc; ++n) {
          drain_wait(&bar.q_full[n % C::ST], (n / C::ST) & 1);
          drain_wait(&bar.do_full[n % C::ST], (n / C::ST) & 1);
        }
      }
    }
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ issuer (converged warp)
    const uint64_t dK = desc_rows_by_channels(sbase), dV = desc_rows_by_channels(sbase + C::OFF_V);
    const uint64_t dQ = desc_rows_by_channels(sbase + C::OFF_Q), dDO = desc_rows_by_channels(sbase + C::OFF_DO);
    const uint64_t dQb = desc_channels_by_rows(sbase + C::OFF_Q), dDOb = desc_channels_by_rows(sbase + C::OFF_DO);
    const uint32_t idS = idesc_bf16_f32(128, 128, false, false), idG = idesc_bf16_f32(128, D, false, true);
    // rows of the unit (dA) by those of a stage's tile (d0) into tX
    auto scores = [&](uint32_t tX, uint64_t dA, uint64_t d0, int st) {
      const uint64_t d = d0 + (uint64_t)(st * C::TILE >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_bf16_warp(tX, dA + kstep_channels(kk), d + kstep_channels(kk), idS, kk > 0 ? 1u : 0u);
    };
    // tG += tX (bf16, 8 columns for 16 queries; those of queries 64 .. 127 from column 64 on)
    // by a stage's tile
    auto gradient = [&](uint32_t tG, uint32_t tX, uint64_t d0, int st, bool first) {
      const uint64_t d = d0 + (uint64_t)(st * C::TILE >> 4);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_bf16_ts_warp(tG, tX + 64 * (kk / 4) + 8 * (kk % 4), d + kk * kKstepRows, idG, !first || kk > 0 ? 1u : 0u);
    };
    bool ok = true;
    int qc = 0, uc = 0;
    for (int i = 0; ok && unit_of(i) < a.units; ++i) {
      const DkvUnit u(a, unit_of(i));
      const int n = u.steps;
      if (n == 0) continue;
      auto issue_s = [&](int t) -> bool {
        const int c = qc + t, st = c % C::ST;
        if (!mbar_wait(&bar.q_full[st], (c / C::ST) & 1, abort)) return false;
        tc_fence_after();
        scores(tmem + C::TM_S, dK, dQ, st);
        mma_commit_warp(&bar.s_full);
        return true;
      };
      auto issue_dp = [&](int t) -> bool {
        const int c = qc + t, st = c % C::ST;
        if (!mbar_wait(&bar.do_full[st], (c / C::ST) & 1, abort)) return false;
        tc_fence_after();
        scores(tmem + C::TM_DP, dV, dDO, st);
        mma_commit_warp(&bar.dp_full);
        if (t == n - 1) mma_commit_warp(&bar.kv_empty);
        return true;
      };
      ok = mbar_wait(&bar.kv_full, uc & 1, abort) && issue_s(0) && issue_dp(0);
      for (int t = 0; ok && t < n; ++t) {
        const int c = qc + t, st = c % C::ST, par = (c / C::ST) & 1;
        if (!mbar_wait(&bar.p_full, c & 1, abort) || !mbar_wait(&bar.do_fixed[st], par, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        gradient(tmem + C::TM_DV, tmem + C::TM_S, dDOb, st, t == 0);
        mma_commit_warp(&bar.do_empty[st]);
        if (t + 1 < n && !issue_s(t + 1)) ok = false;
        if (!ok || !mbar_wait(&bar.ds_full, c & 1, abort) || !mbar_wait(&bar.q_fixed[st], par, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        gradient(tmem + C::TM_DK, tmem + C::TM_DP, dQb, st, t == 0);
        mma_commit_warp(&bar.q_empty[st]);
        if (t + 1 < n) ok = issue_dp(t + 1);
        else mma_commit_warp(&bar.acc_full);
      }
      qc += n;
      ++uc;
    }
    mma_commit_warp(&bar.done);
    drain_wait(&bar.done, 0);
  } else if (warp == kFixer) {
    // ------------------------------------------------------------ rows that see nothing
    // Every tile passes through this warp, so that the barriers' phases keep step with the
    // ring's.
    int qc = 0;
    bool ok = true;
    for (int i = 0; ok && unit_of(i) < a.units; ++i) {
      const DkvUnit u(a, unit_of(i));
      const int n = u.steps;
      int tile = n > 0 ? u.tile0 + u.from % u.tiles : 0;
      for (int t = 0; t < n; ++t, ++qc) {
        const int st = qc % C::ST, par = (qc / C::ST) & 1;
        int lo, hi;
        u.valid(a.w, tile * kTile, lo, hi);
        unsigned char *dO = smem + C::OFF_DO + st * C::TILE, *Q = smem + C::OFF_Q + st * C::TILE;
        if (!mbar_wait(&bar.do_full[st], par, abort)) {
          ok = false;
          break;
        }
        zero_rows<D>(dO, 0, lo, lane);
        zero_rows<D>(dO, hi, kTile, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.do_fixed[st]);
        if (!mbar_wait(&bar.q_full[st], par, abort)) {
          ok = false;
          break;
        }
        zero_rows<D>(Q, 0, lo, lane);
        zero_rows<D>(Q, hi, kTile, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.q_fixed[st]);
        if (++tile == u.tile0 + u.tiles) tile = u.tile0;
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ row threads
    const int half = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + C::TM_S + 64 * half + lanes, tP = tmem + C::TM_DP + 64 * half + lanes;
    const uint32_t tG = tmem + (half ? C::TM_DK : C::TM_DV) + lanes;
    const float2 sl = make_float2(a.sl2, a.sl2);
    const int off = a.w.nk - a.w.nq;
    int qc = 0, uc = 0;
    bool ok = true;
    for (int i = 0; ok && unit_of(i) < a.units; ++i) {
      const DkvUnit u(a, unit_of(i));
      const int n = u.steps, j = u.k0 + r;
      // the queries (row numbers) that see this key: i0 <= q < i1, from the diagonal on, and
      // within the window unless the key is a sink
      const int qlo = max(u.i0, j - a.w.right - off);
      const int qhi = j >= u.len ? -1 : min(u.i1 - 1, j < a.w.sinks ? u.i1 - 1 : j + a.w.left - off);
      // tiles between these see every key of the unit
      const int whole_lo = u.k0 + kTile <= u.len ? max(u.i0, u.k0 + kTile - 1 - a.w.right - off) : 1 << 30;
      const int whole_hi = min(u.i1 - 1, u.k0 + kTile <= a.w.sinks ? u.i1 - 1 : u.k0 + a.w.left - off);
      const bool first_one = sees_one(a.w, u.len, 0), last_one = sees_one(a.w, u.len, u.len - 1);
      const bool all_one = last_one && a.w.right == 0 && a.w.left == 0 && a.w.sinks == 0;
      int tile = n > 0 ? u.tile0 + u.from % u.tiles : 0;
      for (int t = 0; t < n; ++t, ++qc) {
        const int st = qc % C::ST, q0 = tile * kTile;
        const float4* stat = reinterpret_cast<const float4*>(smem + C::OFF_STAT + st * C::STAT) + 16 * half;
        // (lse, delta) came with Q, which S^T has read: visible to who waits for Q's barrier
        if (!mbar_wait(&bar.q_full[st], (qc / C::ST) & 1, abort) || !mbar_wait(&bar.s_full, qc & 1, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t x[64];
        load_cols64(tS, x);
        const bool whole = q0 >= whole_lo && q0 + kTile - 1 <= whole_hi;
        if (!whole) {
          const int lo = qlo - q0 - 64 * half, hi = qhi - q0 - 64 * half;  // -inf: P = 0
          hide(x, visible32(lo, hi, 0));
          hide(x + 32, visible32(lo - 32, hi - 32, 0));
        }
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          const float4 nlse = stat[c / 4];
          const float2 e0 = __ffma2_rn(pair(x + c), sl, make_float2(nlse.x, nlse.y));
          const float2 e1 = __ffma2_rn(pair(x + c + 2), sl, make_float2(nlse.z, nlse.w));
          const float p0 = fast_exp2(e0.x), p1 = fast_exp2(e0.y), p2 = fast_exp2(e1.x), p3 = fast_exp2(e1.y);
          x[c] = __float_as_uint(p0);
          x[c + 1] = __float_as_uint(p1);
          x[c + 2] = __float_as_uint(p2);
          x[c + 3] = __float_as_uint(p3);
          pk[c / 2] = pack2(p0, p1);
          pk[c / 2 + 1] = pack2(p2, p3);
        }
        tmem_store16_async(tS, pk);
        tmem_store16_async(tS + 16, pk + 16);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar.p_full);
        if (!mbar_wait(&bar.dp_full, qc & 1, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t y[64];
        load_cols64(tP, y);
        if (!whole) {
          // queries that see one key have dS = 0 (a tile that holds one is never seen whole): the
          // columns of position 0 and of the last one, or all of them
          const int at0 = -(q0 + 64 * half + off), at1 = at0 + u.len - 1;
          const bool one0 = first_one && at0 >= 0 && at0 < 64, one1 = last_one && at1 >= 0 && at1 < 64;
          if (all_one || one0 || one1) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (all_one || (one0 && c == at0) || (one1 && c == at1)) x[c] = 0u;
          }
          drop_masked(x, y);
        }
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          const float4 nd = stat[32 + c / 4];
          const float2 d0 = __fmul2_rn(pair(x + c), __fadd2_rn(pair(y + c), make_float2(nd.x, nd.y)));
          const float2 d1 = __fmul2_rn(pair(x + c + 2), __fadd2_rn(pair(y + c + 2), make_float2(nd.z, nd.w)));
          y[c / 2] = pack2(d0.x, d0.y);
          y[c / 2 + 1] = pack2(d1.x, d1.y);
        }
        tmem_store16_async(tP, y);
        tmem_store16_async(tP + 16, y + 16);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar.ds_full);
        if (++tile == u.tile0 + u.tiles) tile = u.tile0;
      }
      if (!ok) break;
      // ---- the first 128 threads write dV's rows, the others dK's
      if (n > 0) {
        if (!mbar_wait(&bar.acc_full, uc & 1, abort)) break;
        ++uc;
        tc_fence_after();
      }
      if (u.slot >= 0) {
        // a part of a tile's sums (parts behind the sequence's last have none)
        if (n == 0) continue;
        float4* dst = reinterpret_cast<float4*>(a.partial + ((long long)(2 * u.slot + half) * kTile + r) * D);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_load32(tG + c, o);
#pragma unroll
          for (int k = 0; k < 32; k += 4) dst[(c + k) / 4] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
        tc_fence_before();
        continue;
      }
      if (u.part > 0) continue;
      const bool in = j < a.w.nk;
      const View<__nv_bfloat16>& out = half ? a.dk : a.dv;
      __nv_bfloat16* dst = out.row(u.b, u.hk, in ? j : 0);
      const float f = half ? a.scale : 1.f;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        if (n > 0) {
          tmem_load32(tG + c, o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        if (in) {
#pragma unroll
          for (int k = 0; k < 32; k += 8)
            *reinterpret_cast<uint4*>(dst + c + k) =
                make_uint4(pack2(o[k] * f, o[k + 1] * f), pack2(o[k + 2] * f, o[k + 3] * f),
                           pack2(o[k + 4] * f, o[k + 5] * f), pack2(o[k + 6] * f, o[k + 7] * f));
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kFixer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds the parts of one key tile, in order: 8 channels of dV or dK per thread.
template <int D>
__global__ void __launch_bounds__(256) window_parts_kernel(const BwdParams a) {
  pdl_launch_dependents();
  pdl_wait();
  const int heads = a.w.B * a.w.nkv, x = blockIdx.x % heads, kt = blockIdx.x / heads;
  DkvUnit u(a, (a.cut.units / heads - a.cut.tiles[0] + kt) * heads + x);  // the tile's part 0
  if (u.slot < 0) return;
  const int parts = (u.group * u.tiles + a.cut.steps - 1) / a.cut.steps;
  const bool is_k = blockIdx.z;
  const int row = blockIdx.y * (256 / (D / 8)) + threadIdx.x / (D / 8), c = threadIdx.x % (D / 8) * 8;
  if (u.k0 + row >= a.w.nk) return;
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < parts; ++p) {
    const long long slot = (long long)(a.cut.slot0(p) + kt) * heads + x;
    const float4* src = reinterpret_cast<const float4*>(a.partial + ((2 * slot + is_k) * kTile + row) * D + c);
    const float4 v = src[0], w = src[1];
    o[0] += v.x; o[1] += v.y; o[2] += v.z; o[3] += v.w;
    o[4] += w.x; o[5] += w.y; o[6] += w.z; o[7] += w.w;
  }
  const float f = is_k ? a.scale : 1.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] *= f;
  const View<__nv_bfloat16>& out = is_k ? a.dk : a.dv;
  *reinterpret_cast<uint4*>(out.row(u.b, u.hk, u.k0 + row) + c) = pack_vec(o);
}

int padded_rows(const Window& w) { return (w.nq + kTile - 1) / kTile * kTile; }
size_t stat_bytes(const Window& w) { return (size_t)w.B * w.nh * padded_rows(w) * sizeof(float2); }

// By the sizes alone (full lengths, 152 SMs).  A tile is cut only where one of them would
// take much longer than an SM's share of all: sinks behind a window (4096 positions, a window
// of 1024, groups of 4: the sinks' tile has 128 steps, the others 36, and 32 down to 4 at the
// end), or a long causal triangle of few heads.  Parts are half an SM's share, but no smaller
// than what a tile of the window has anyway: each costs a tile of fp32 sums written and read.
Cut cut_of(const Window& w) {
  constexpr int kSms = 152;
  const int key_tiles = (w.nk + kTile - 1) / kTile, group = w.nh / w.nkv;
  auto steps = [&](int kt) -> long long {
    int i0, n;
    query_range(w, w.nk, kt * kTile, std::min((kt + 1) * kTile, w.nk) - 1, i0, n);
    return n > 0 ? (long long)group * ((i0 + n - 1) / kTile - i0 / kTile + 1) : 0;
  };
  long long total = 0, most = 0, plain = 0;  // plain: of the tiles without sinks
  for (int kt = 0; kt < key_tiles; ++kt) {
    const long long s = steps(kt);
    total += s;
    most = std::max(most, s);
    if (kt * kTile >= w.sinks) plain = std::max(plain, s);
  }
  const long long share = (total * w.B * w.nkv + kSms - 1) / kSms;
  Cut c{};
  c.parts = 1;
  c.steps = (int)std::max(most, 1LL);
  c.tiles[0] = key_tiles;
  if (most > share + share / 4) {
    long long part = std::max<long long>((share + 1) / 2, 8);
    if (plain <= share) part = std::max(part, plain);
    c.steps = (int)std::max(part, (most + kMaxParts - 1) / kMaxParts);
    c.parts = (int)((most + c.steps - 1) / c.steps);
    for (int p = 1; p < c.parts; ++p) {
      int n = c.tiles[p - 1];
      while (n > 0 && steps(n - 1) <= (long long)p * c.steps) --n;
      c.tiles[p] = n;
    }
  }
  int units = 0;
  for (int p = 0; p < c.parts; ++p) units += c.tiles[p];
  c.units = units * w.B * w.nkv;
  return c;
}

int cut_slots(const Cut& c, const Window& w) {
  return c.parts == 1 ? 0 : (c.slot0(c.parts - 1) + c.tiles[c.parts - 1]) * w.B * w.nkv;
}

template <int D>
cudaError_t bwd(const WindowArgs<__nv_bfloat16>& x, cudaStream_t st) {
  const Window& w = x.w;
  CUtensorMap mq, mdo, mk, mv;
  if (!map_view(&mq, x.q.p, x.q.sb, x.q.sh, x.q.sn, w.B, w.nh, w.nq, D) ||
      !map_view(&mdo, x.dO.p, x.dO.sb, x.dO.sh, x.dO.sn, w.B, w.nh, w.nq, D) ||
      !map_view(&mk, x.k.p, x.k.sb, x.k.sh, x.k.sn, w.B, w.nkv, w.nk, D) ||
      !map_view(&mv, x.v.p, x.v.sb, x.v.sh, x.v.sn, w.B, w.nkv, w.nk, D))
    return cudaErrorInvalidValue;
  BwdParams a{};
  a.w = w;
  a.dq = x.dq;
  a.dk = x.dk;
  a.dv = x.dv;
  float* stat = x.delta;
  a.stat = stat;
  a.scale = x.scale;
  a.sl2 = x.scale * kLog2;
  a.row_tiles = (w.nq + kTile - 1) / kTile;
  auto dq = window_dq_tc_kernel<D>;
  auto dkdv = window_dkdv_tc_kernel<D>;
  cudaError_t e = set_max_dynamic_smem((const void*)dq, DqCfg<D>::SMEM);
  if (e == cudaSuccess) e = set_max_dynamic_smem((const void*)dkdv, DkvCfg<D>::SMEM);
  // with a window this wide to the left, only positions 0 .. kFewKeys - 1 can see few keys
  const bool narrow = w.left < kFewKeys;
  const int heads = w.B * w.nh, padded = padded_rows(w), blocks = (padded + kStatBlock<D> - 1) / kStatBlock<D>;
  const int again = narrow ? (w.nq + kFewBlock - 1) / kFewBlock * heads : (heads + 7) / 8;
  if (e == cudaSuccess)
    e = launch_pdl(narrow ? window_stat_kernel<D, true> : window_stat_kernel<D, false>, dim3(blocks * heads + again),
                   dim3(256), 0, st, x, stat, padded, blocks, again);
  a.cut = cut_of(w);
  a.partial = reinterpret_cast<float*>(reinterpret_cast<char*>(x.delta) + stat_bytes(w));
  if (e == cudaSuccess) {
    a.units = a.cut.units;
    e = launch_pdl(dkdv, dim3(std::min(a.units, device_sm_count())), dim3(kThreads), DkvCfg<D>::SMEM, st, mq, mdo, mk,
                   mv, a);
  }
  if (e == cudaSuccess && a.cut.parts > 1)
    e = launch_pdl(window_parts_kernel<D>, dim3(a.cut.tiles[1] * w.B * w.nkv, kTile / (256 / (D / 8)), 2), dim3(256),
                   0, st, a);
  if (e == cudaSuccess) {
    a.units = w.B * w.nh * a.row_tiles;
    e = launch_pdl(dq, dim3(std::min(a.units, device_sm_count())), dim3(kThreads), DqCfg<D>::SMEM, st, mq, mdo, mk, mv,
                   a);
  }
  return e;
}

}  // namespace

size_t window_bwd_tc_ws_bytes(const Window& w, int d) {
  return stat_bytes(w) + (size_t)cut_slots(cut_of(w), w) * 2 * kTile * d * sizeof(float);
}

cudaError_t launch_window_bwd_tc(const WindowArgs<__nv_bfloat16>& a, int d, cudaStream_t st) {
  return d == 64 ? bwd<64>(a, st) : bwd<128>(a, st);
}

}  // namespace psa
