// window_fwd.cu -- attention with a sliding window and first tokens that stay visible:
// forward on tensor cores (tcgen05, bf16).
//
//   S = Q K^T, P = 2^(scale log2(e) S - m), O = sum P V / sum P over the visible keys, with
//   the running maximum m and sum of an online softmax; lse = ln(sum P) + m ln 2.
//
// Bound by the tensor cores at head dim 128: of a 128 x 128 tile's 2 x 512 cycles there, the
// exponentials take 512 of the multi-function units.  So the kernel is built to keep that
// pipe fed: a persistent CTA per SM with two slots of 128 query rows, whose softmax steps
// run while the other slot's products do.  The two slots share the key/value tiles: two query
// heads of one key/value head at the same rows where their number is even (equal tile
// lists), two neighbouring row tiles of one head otherwise.
//   warps 0-3, 4-7   softmax of slot 0, 1: one thread per row (TMEM lane), 128 columns
//   warp 8           TMA producer: Q of both slots, a ring of K tiles and one of V tiles
//   warp 9           issuer of both slots in turn: per key tile O += P V, then the next tile's
//                    S = Q K^T right behind it: P lies in S's own columns of tensor memory,
//                    and products complete in order, so neither waits for the other in
//                    software, and s_full says that both are done.  PTX promises that order
//                    for products of one shape into the same sums only; that the pipe keeps
//                    it for all of a warp's is observed (no run's bits ever differed: a
//                    test repeats 16384 causal positions 40 times).  The warp runs converged
//                    (descriptors in uniform registers); two issuing threads, one per slot,
//                    interleave on the pipe and make both chains longer (1050 against 732 us
//                    at 16384 causal)
//   warp 10          TMA stores of finished rows, which the softmax threads leave in a
//                    staging tile (stores of their own would hit 32 rows at a time, half a
//                    sector each, and hold up their next arrival until acknowledged)
//   warp 11          zeroes the rows of padding of V tiles (0 times NaN is NaN)
// Only tiles that some row of the pair sees are visited: the sinks' tiles, then the
// window's; masks are applied where a tile is not wholly visible.  O is rescaled only when a
// row's maximum grows by more than 2^8 (O and the sum share the stale maximum, so the result
// is the same).  P is rounded to bf16 for the product with V, as its operand; the sum is of
// the unrounded values.
// Measured: 16384 tokens causal, 16 heads of 128 on 2: 735 us (1.5 PFLOP/s of visible pairs,
// 0.78 of cuBLAS's bf16 rate, the pipe busy 65 % of the time); 8192 tokens, 32 heads on 8, a
// window of 1024 and 4 sinks: 147 us (0.88 PFLOP/s: of ten tiles a row tile visits, two are half
// empty and one holds the sinks, and each unit starts its chain anew); head dim 64: 648 us at
// 16384 causal (0.85 PFLOP/s: the chain S, softmax, P V of a slot is longer than the other
// slot's products, 2.7k cycles a step).
#include <math.h>

#include <algorithm>

#include "window_tc.cuh"

namespace psa {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;

template <int D>
struct Cfg {
  static constexpr int kThreads = 384;
  static constexpr int kProducer = 8, kIssuer = 9, kStore = 10, kFixer = 11;
  // shared memory that a CTA can have, less barriers and alignment, cut into tiles
  static constexpr int KST = D == 128 ? 2 : 5, VST = D == 128 ? 2 : 5;
  static constexpr uint32_t TILE = kTileBytes<D>;
  static constexpr uint32_t OFF_OUT = 2 * TILE, OFF_K = 3 * TILE, OFF_V = OFF_K + KST * TILE;
  static constexpr uint32_t OFF_BAR = OFF_V + VST * TILE;
  static constexpr uint32_t SMEM = OFF_BAR + 512 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  // tensor memory: S of both slots (P in its first half), O of both slots
  static constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;
};

struct Bars {
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], done, staged, stored[2];
  uint64_t k_full[5], k_empty[5], v_full[5], v_fixed[5], v_empty[5];
};

struct FwdParams {
  Window w;
  float* lse;
  float sl2;       // scale * log2(e)
  int units, row_tiles;
  bool head_pairs;  // the slots are two heads (else two row tiles of one head)
};

// Where a slot's rows are and what they see.
struct Slot {
  int h, row0, p0, p1;  // positions of its rows, clipped to the visible ones (empty: p0 > p1)
};

struct Unit {
  int b, hk, len;
  Slot s[2];
  __device__ __forceinline__ Unit(const FwdParams& a, int u) {
    const Window& w = a.w;
    const int group = w.nh / w.nkv;
    // the last row tiles see the most keys in a causal problem: they go first
    int tile, h;
    if (a.head_pairs) {
      const int pairs = w.B * w.nh / 2;
      tile = a.row_tiles - 1 - u / pairs;
      const int x = u % pairs;
      b = x / (w.nh / 2);
      h = 2 * (x % (w.nh / 2));
    } else {
      const int heads = w.B * w.nh;
      tile = 2 * ((a.row_tiles + 1) / 2 - 1 - u / heads);
      const int x = u % heads;
      b = x / w.nh;
      h = x % w.nh;
    }
    hk = h / group;
    len = w.len(b);
    const int off = w.nk - w.nq;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s[i].h = a.head_pairs ? h + i : h;
      s[i].row0 = (a.head_pairs ? tile : tile + i) * kTile;
      s[i].p0 = max(0, s[i].row0 + off);
      s[i].p1 = min(len, min(s[i].row0 + kTile, w.nq) + off) - 1;
    }
  }
};

// The tiles a unit visits (those of both slots), and which of them a slot takes part in.
struct Walk {
  KeyTiles<kTile> all;
  int sink[2], first[2], last[2], end[2];  // end: keys from here on are seen by no row
  int sinks;
  static __device__ __forceinline__ int lo(const Unit& u) {
    return u.s[0].p0 > u.s[0].p1 ? u.s[1].p0 : u.s[1].p0 > u.s[1].p1 ? u.s[0].p0 : min(u.s[0].p0, u.s[1].p0);
  }
  static __device__ __forceinline__ int hi(const Unit& u) {
    return u.s[0].p0 > u.s[0].p1 ? u.s[1].p1 : u.s[1].p0 > u.s[1].p1 ? u.s[0].p1 : max(u.s[0].p1, u.s[1].p1);
  }
  __device__ __forceinline__ Walk(const Window& w, const Unit& u) : all(w, u.len, lo(u), hi(u)) {
    sinks = w.sinks;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool some = u.s[i].p0 <= u.s[i].p1;
      const int top = min(u.len - 1, u.s[i].p1 + w.right);
      first[i] = max(0, u.s[i].p0 - w.left) / kTile;
      last[i] = some ? top / kTile : -1;
      end[i] = top + 1;
      sink[i] = some && w.sinks > 0 ? (min(w.sinks, top + 1) + kTile - 1) / kTile : 0;
    }
  }
  __device__ __forceinline__ bool takes(int slot, int tile) const {
    return tile < sink[slot] || (tile >= first[slot] && tile <= last[slot]);
  }
  // columns that a slot works on in a tile that it takes
  __device__ __forceinline__ int cols(int slot, int tile) const {
    return used_columns(tile, first[slot], end[slot], sinks);
  }
};

// Unit of CTA c in its round i: CTA order in even rounds, reverse order in odd ones, so that
// with units from long to short no CTA collects the long ones.
__device__ __forceinline__ int unit_of(int i) {
  return i * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// The running maximum m (log2 units) takes in a tile's, mx; O (at tO) and the sum l are rescaled
// if it grew by more than 2^8 in a row of the warp.
template <int D>
__device__ __forceinline__ void new_maximum(uint32_t tO, float mx, bool first, float& m, float& l) {
  float alpha = 1.f;
  if (mx > m + 8.f || first) {
    // -inf - -inf: a row that has seen nothing yet has nothing to rescale
    alpha = m == -INFINITY ? 0.f : fast_exp2(m - mx);
    m = mx;
  }
  if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
    l *= alpha;
    // s_full says that every product issued before this S is done, O's among them
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float o[32];
      tmem_load32(tO + c, o);
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] *= alpha;
      tmem_store32(tO + c, o);
    }
  }
}

__device__ __forceinline__ float max32(const uint32_t* x, float mx) {
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    m0 = fmax3(m0, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
    m1 = fmax3(m1, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
  }
  return fmax3(mx, m0, m1);
}

// 2^(x sl - base) of 32 scores, packed into the first half of `to`, and their sum.
__device__ __forceinline__ void exp32(const uint32_t* x, uint32_t* to, float2 sl, float2 nm, float2& l01,
                                      float2& l23) {
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    const float2 x01 = __ffma2_rn(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), sl, nm);
    const float2 x23 = __ffma2_rn(make_float2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3])), sl, nm);
    const float2 p01 = make_float2(fast_exp2(x01.x), fast_exp2(x01.y));
    const float2 p23 = make_float2(fast_exp2(x23.x), fast_exp2(x23.y));
    l01 = __fadd2_rn(l01, p01);
    l23 = __fadd2_rn(l23, p23);
    to[k / 2] = pack2(p01.x, p01.y);
    to[k / 2 + 1] = pack2(p23.x, p23.y);
  }
}

// One tile's step of the online softmax, for one row per thread: scores from tensor memory at tS,
// probabilities in bf16 back over the first half of their columns.  Tiles that every row sees
// whole keep all 128 scores in registers.
template <int D>
__device__ __forceinline__ void whole_step(uint32_t tS, uint32_t tO, float sl2, bool first, float& m, float& l) {
  using Chunk = uint32_t[32];
  uint32_t x[128];
#pragma unroll
  for (int c = 0; c < 128; c += 32) tmem_load32_async(tS + c, *reinterpret_cast<Chunk*>(x + c));
  tmem_wait_ld();
#pragma unroll
  for (int c = 0; c < 128; c += 32) tmem_pin(*reinterpret_cast<Chunk*>(x + c));
  float mx = -INFINITY;
#pragma unroll
  for (int c = 0; c < 128; c += 32) mx = max32(x + c, mx);
  new_maximum<D>(tO, mx * sl2, first, m, l);
  const float2 sl = make_float2(sl2, sl2), nm = make_float2(-m, -m);
  float2 l01 = make_float2(0.f, 0.f), l23 = l01;
#pragma unroll
  for (int c = 0; c < 128; c += 32) exp32(x + c, x + c / 2, sl, nm, l01, l23);
  l += (l01.x + l01.y) + (l23.x + l23.y);
#pragma unroll
  for (int c = 0; c < 64; c += 16) tmem_store16_async(tS + c, x + c);
}

// The others: the columns in use, 32 at a time, once for the maximum and once for the
// exponentials (holding them all costs the step above its registers: 732 -> 969 us at 16384
// causal).  lo, hi, sk: the row's limits relative to the tile (visible32).
template <int D>
__device__ __forceinline__ void masked_step(uint32_t tS, uint32_t tO, int cols, int lo, int hi, int sk, float sl2,
                                            bool first, float& m, float& l) {
  uint32_t x[32];
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < cols; c += 32) {
    tmem_load32_async(tS + c, x);
    tmem_wait_ld();
    tmem_pin(x);
    hide(x, visible32(lo - c, hi - c, sk - c));
    mx = max32(x, mx);
  }
  new_maximum<D>(tO, mx * sl2, first, m, l);
  const float base = m == -INFINITY ? 0.f : m;
  const float2 sl = make_float2(sl2, sl2), nm = make_float2(-base, -base);
  float2 l01 = make_float2(0.f, 0.f), l23 = l01;
#pragma unroll 1
  for (int c = 0; c < cols; c += 32) {
    tmem_load32_async(tS + c, x);
    tmem_wait_ld();
    tmem_pin(x);
    hide(x, visible32(lo - c, hi - c, sk - c));
    exp32(x, x, sl, nm, l01, l23);
    tmem_store16_async(tS + c / 2, x);  // over columns that have been read
  }
  l += (l01.x + l01.y) + (l23.x + l23.y);
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    window_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ CUtensorMap tmO, const FwdParams a) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = align1024(smem_raw);
  const uint32_t sbase = smem_addr(smem);
  Bars& bar = *reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(&bar + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_at + 1);
  static_assert(sizeof(Bars) + 16 <= 512, "barriers");
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 1);
      mbar_init(&bar.q_empty[i], 1);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], kTile);
      mbar_init(&bar.o_full[i], 1);
    }
    mbar_init(&bar.done, 1);
    mbar_init(&bar.staged, kTile);
    mbar_init(&bar.stored[0], 1);
    mbar_init(&bar.stored[1], 1);
    for (int i = 0; i < 5; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 2);  // one arrival per slot
      mbar_init(&bar.v_full[i], 1);
      mbar_init(&bar.v_fixed[i], 1);
      mbar_init(&bar.v_empty[i], 2);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == C::kFixer) {
    tmem_alloc(tmem_at, C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  pdl_launch_dependents();
  pdl_wait();

  if (warp >= 8) {
    if (warp == C::kProducer) {
      // ------------------------------------------------------------ TMA producer
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        bool ok = true;
        int q_count[2] = {0, 0}, kv = 0;
        for (int i = 0; ok && unit_of(i) < a.units; ++i) {
          const Unit u(a, unit_of(i));
          const Walk walk(a.w, u);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (walk.last[s] < 0 || !ok) continue;
            const int n = q_count[s];
            if (n >= 1 && !mbar_wait(&bar.q_empty[s], (n - 1) & 1, abort)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&bar.q_full[s], C::TILE);
            load_tile<D>(smem + s * C::TILE, &tmQ, &bar.q_full[s], u.s[s].row0, u.s[s].h, u.b);
            q_count[s] = n + 1;
          }
          for (int t = 0; ok && t < walk.all.count; ++t, ++kv) {
            const int ks = kv % C::KST, vs = kv % C::VST, row = walk.all.tile(t) * kTile;
            if (kv >= C::KST && !mbar_wait(&bar.k_empty[ks], (kv / C::KST - 1) & 1, abort)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&bar.k_full[ks], C::TILE);
            load_tile<D>(smem + C::OFF_K + ks * C::TILE, &tmK, &bar.k_full[ks], row, u.hk, u.b);
            if (kv >= C::VST && !mbar_wait(&bar.v_empty[vs], (kv / C::VST - 1) & 1, abort)) {
              ++kv;
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&bar.v_full[vs], C::TILE);
            load_tile<D>(smem + C::OFF_V + vs * C::TILE, &tmV, &bar.v_full[vs], row, u.hk, u.b);
          }
        }
        if (*abort) {
          // let the copies in flight land before the CTA exits (a wait for one that was not
          // issued any more runs into its time limit)
          for (int s = 0; s < 2; ++s)
            if (q_count[s] > 0) drain_wait(&bar.q_full[s], (q_count[s] - 1) & 1);
          for (int n = max(0, kv - C::KST); n < kv; ++n) drain_wait(&bar.k_full[n % C::KST], (n / C::KST) & 1);
          for (int n = max(0, kv - C::VST); n < kv; ++n) drain_wait(&bar.v_full[n % C::VST], (n / C::VST) & 1);
        }
      }
    } else if (warp == C::kIssuer) {
      // ------------------------------------------------------------ issuer (converged warp)
      const uint64_t dQ0 = desc_rows_by_channels(sbase);
      const uint64_t dK0 = desc_rows_by_channels(sbase + C::OFF_K);
      const uint64_t dV0 = desc_channels_by_rows(sbase + C::OFF_V);
      const uint32_t idO = idesc_bf16_f32(128, D, false, true);
      bool ok = true;
      int kv0 = 0, q_count[2] = {0, 0}, steps[2] = {0, 0};  // kv0: ring index of the unit's first tile
      for (int i = 0; ok && unit_of(i) < a.units; ++i) {
        const Unit u(a, unit_of(i));
        const Walk walk(a.w, u);
        const int n = walk.all.count;
        bool first[2] = {true, true};
        // S of slot s and the unit's entry e, or the tile's release
        auto issue_s = [&](int s, int e) -> bool {
          const int kn = kv0 + e, st = kn % C::KST, tile = walk.all.tile(e);
          if (!mbar_wait(&bar.k_full[st], (kn / C::KST) & 1, abort)) return false;
          if (!walk.takes(s, tile)) {
            if (lane == 0) mbar_arrive(&bar.k_empty[st]);
            __syncwarp();
            return true;
          }
          tc_fence_after();
          const uint64_t dQ = dQ0 + (uint64_t)(s * C::TILE >> 4), dK = dK0 + (uint64_t)(st * C::TILE >> 4);
          const int cols = walk.cols(s, tile);
          // constant descriptors for the common case: a branch per product costs the pipe its feed
          auto scores = [&](uint32_t id) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_warp(tmem + C::TM_S + 128 * s, dQ + kstep_channels(kk), dK + kstep_channels(kk), id,
                            kk > 0 ? 1u : 0u);
          };
          if (cols == kTile) scores(idesc_bf16_f32(128, kTile, false, false));
          else scores(idesc_bf16_f32(128, cols, false, false));
          mma_commit_warp(&bar.s_full[s]);
          mma_commit_warp(&bar.k_empty[st]);
          if (tile == walk.last[s]) mma_commit_warp(&bar.q_empty[s]);  // the next unit's Q may come
          return true;
        };
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (ok && walk.last[s] >= 0) ok = mbar_wait(&bar.q_full[s], q_count[s] & 1, abort);
          if (ok && n > 0) ok = issue_s(s, 0);
        }
        for (int e = 0; ok && e < n; ++e) {
          const int vn = kv0 + e, st = vn % C::VST, par = (vn / C::VST) & 1;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (!ok) break;
            const bool mine = walk.takes(s, walk.all.tile(e));
            if ((mine && !mbar_wait(&bar.p_full[s], steps[s] & 1, abort)) ||
                !mbar_wait(&bar.v_fixed[st], par, abort)) {
              ok = false;
              break;
            }
            if (mine) {
              ++steps[s];
              tc_fence_after();
              const uint64_t dV = dV0 + (uint64_t)(st * C::TILE >> 4);
              const int cols = walk.cols(s, walk.all.tile(e));
              const uint32_t tO = tmem + C::TM_O + D * s, tP = tmem + C::TM_S + 128 * s;
              if (cols == kTile) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                  mma_bf16_ts_warp(tO, tP + 8 * kk, dV + kk * kKstepRows, idO, !first[s] || kk > 0 ? 1u : 0u);
              } else {
#pragma unroll 1
                for (int kk = 0; 16 * kk < cols; ++kk)
                  mma_bf16_ts_warp(tO, tP + 8 * kk, dV + kk * kKstepRows, idO, !first[s] || kk > 0 ? 1u : 0u);
              }
              first[s] = false;
              mma_commit_warp(&bar.v_empty[st]);
            } else {
              if (lane == 0) mbar_arrive(&bar.v_empty[st]);
              __syncwarp();
            }
            if (e + 1 < n) ok = issue_s(s, e + 1);
            else if (walk.last[s] >= 0) mma_commit_warp(&bar.o_full[s]);
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) q_count[s] += walk.last[s] >= 0;
        kv0 += n;
      }
      mma_commit_warp(&bar.done);
      drain_wait(&bar.done, 0);
    } else if (warp == C::kStore) {
      // ------------------------------------------------------------ finished rows to memory
      if (lane == 0) {
        int n = 0;
        bool ok = true;
        for (int i = 0; ok && unit_of(i) < a.units; ++i) {
          const Unit u(a, unit_of(i));
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (!ok || u.s[s].row0 >= a.w.nq) continue;
            if (!mbar_wait(&bar.staged, n & 1, abort)) {
              ok = false;
              break;
            }
            ++n;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_store_4d(&tmO, smem + C::OFF_OUT + c * kBoxBytes, 64 * c, u.s[s].row0, u.s[s].h, u.b);
            bulk_commit();
            bulk_wait_read_all();
            // whose turn it is: slot 1's after slot 0 (unless it has no rows), else slot 0's
            mbar_arrive(&bar.stored[s == 0 && u.s[1].row0 < a.w.nq ? 1 : 0]);
          }
        }
        bulk_wait_all();
      }
    } else if (warp == C::kFixer) {
      // ------------------------------------------------------------ rows of padding in V
      // Every tile passes through this warp, so that v_fixed's phases keep step with the ring.
      int kv = 0;
      bool ok = true;
      for (int i = 0; ok && unit_of(i) < a.units; ++i) {
        const Unit u(a, unit_of(i));
        const Walk walk(a.w, u);
        // the tile that sequence b ends in (rows past n_k are zero already: TMA's fill)
        const int edge = u.len % kTile != 0 && u.len < a.w.nk ? u.len / kTile : -1;
        for (int t = 0; t < walk.all.count; ++t, ++kv) {
          const int st = kv % C::VST;
          if (!mbar_wait(&bar.v_full[st], (kv / C::VST) & 1, abort)) {
            ok = false;
            break;
          }
          if (walk.all.tile(t) == edge) zero_rows<D>(smem + C::OFF_V + st * C::TILE, u.len % kTile, kTile, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.v_fixed[st]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax of a slot
    const int s = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + C::TM_S + 128 * s + lanes, tO = tmem + C::TM_O + D * s + lanes;
    const int off = a.w.nk - a.w.nq;
    int steps = 0, outs = 0, uses = 0;
    bool ok = true;
    for (int i = 0; ok && unit_of(i) < a.units; ++i) {
      int b, h, q, len, jhi, jlo;  // this row, and the keys it sees: none if jhi < 0
      int whole_lo, whole_hi;      // tiles between these are seen whole by every valid row
      int end;
      KeyTiles<kTile> tiles;
      {
        const Unit u(a, unit_of(i));
        const Slot me = s ? u.s[1] : u.s[0];
        b = u.b;
        h = me.h;
        len = u.len;
        q = me.row0 + r;
        const int p = q + off;
        jhi = p >= 0 && p < len && q < a.w.nq ? min(len - 1, p + a.w.right) : -1;
        jlo = p - a.w.left;
        tiles = KeyTiles<kTile>(a.w, len, me.p0, me.p1);
        // rows that do not exist or are padding get anything here and 0 at the end
        whole_lo = me.p1 - a.w.left;
        whole_hi = min(len, me.p0 + a.w.right + 1);
        end = min(len, me.p1 + a.w.right + 1);
      }
      float m = -INFINITY, l = 0.f;
      for (int t = 0; t < tiles.count; ++t) {
        const int tile = tiles.tile(t), j0 = tile * kTile;
        const int cols = used_columns(tile, tiles.first, end, a.w.sinks);
        if (!mbar_wait(&bar.s_full[s], steps & 1, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (j0 + kTile <= whole_hi && (j0 >= whole_lo || j0 + kTile <= a.w.sinks))
          whole_step<D>(tS, tO, a.sl2, t == 0, m, l);
        else
          masked_step<D>(tS, tO, cols, jlo - j0, jhi - j0, a.w.sinks - j0, a.sl2, t == 0, m, l);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar.p_full[s]);
        ++steps;
      }
      if (!ok) break;
      // ---- the rows' results, through the staging tile
      const bool some = tiles.count > 0;
      if (some) {
        if (!mbar_wait(&bar.o_full[s], outs & 1, abort)) break;
        ++outs;
        tc_fence_after();
      }
      if (q - r >= a.w.nq) continue;
      const bool sees = jhi >= 0;
      const float inv = 1.f / l;
      // the staging tile is this slot's once the use before it has been read
      if (s || uses > 0) {
        if (!mbar_wait(&bar.stored[s], (s ? uses : uses - 1) & 1, abort)) break;
      }
      ++uses;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        if (some) {
          tmem_load32(tO + c, o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = sees ? o[k] * inv : 0.f;
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        const uint32_t box = sbase + C::OFF_OUT + (c / 64) * kBoxBytes;
#pragma unroll
        for (int k = 0; k < 32; k += 8)
          st_shared_v4(box + swizzled_offset(r, (c % 64 + k) / 8, 128), pack2(o[k], o[k + 1]), pack2(o[k + 2], o[k + 3]),
                       pack2(o[k + 4], o[k + 5]), pack2(o[k + 6], o[k + 7]));
      }
      tc_fence_before();
      fence_proxy_async_smem();
      mbar_arrive(&bar.staged);
      if (q < a.w.nq && a.lse)
        a.lse[((long long)b * a.w.nh + h) * a.w.nq + q] = sees ? m * kLn2 + logf(l) : -INFINITY;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kFixer) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

template <int D>
cudaError_t fwd(const WindowArgs<__nv_bfloat16>& x, cudaStream_t st) {
  using C = Cfg<D>;
  const Window& w = x.w;
  CUtensorMap mq, mk, mv, mo;
  if (!map_view(&mo, x.out.p, x.out.sb, x.out.sh, x.out.sn, w.B, w.nh, w.nq, D) ||
      !map_view(&mq, x.q.p, x.q.sb, x.q.sh, x.q.sn, w.B, w.nh, w.nq, D) ||
      !map_view(&mk, x.k.p, x.k.sb, x.k.sh, x.k.sn, w.B, w.nkv, w.nk, D) ||
      !map_view(&mv, x.v.p, x.v.sb, x.v.sh, x.v.sn, w.B, w.nkv, w.nk, D))
    return cudaErrorInvalidValue;
  FwdParams a{};
  a.w = w;
  a.lse = x.lse;
  a.sl2 = x.scale * kLog2;
  a.row_tiles = (w.nq + kTile - 1) / kTile;
  a.head_pairs = (w.nh / w.nkv) % 2 == 0;
  a.units = a.head_pairs ? w.B * w.nh / 2 * a.row_tiles : w.B * w.nh * ((a.row_tiles + 1) / 2);
  auto kern = window_fwd_tc_kernel<D>;
  const cudaError_t e = set_max_dynamic_smem((const void*)kern, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(std::min(a.units, device_sm_count())), dim3(C::kThreads), C::SMEM, st,
                    mq, mk, mv, mo, a);
}

}  // namespace

cudaError_t launch_window_fwd_tc(const WindowArgs<__nv_bfloat16>& a, int d, cudaStream_t st) {
  return d == 64 ? fwd<64>(a, st) : fwd<128>(a, st);
}

}  // namespace psa
