// prefix_attn.cu -- attention of a batch whose sequences share a long prefix (bf16, tcgen05):
//
//   o = softmax over [prefix keys | own keys that the query sees] of scale q k^T, times v
//
// The prefix is read once for all sequences: the queries of one key/value head, of all sequences
// and of the heads that share it, are the rows of one product with its keys.  A tile of 128 rows
// is a box of tq queries, tg heads and tb sequences, those extents that need the fewest tiles.
// The prefix part is an online softmax without masks (but for the last tile's columns), as the
// window attention's forward: two slots of 128 rows whose softmax steps run while the other
// slot's products do, P in S's columns of tensor memory, products issued in order by one
// converged warp.  The slots share the key/value tiles; a row tile without a partner takes both
// slots and alternates between them.
//   warps 0-3, 4-7   softmax of slot 0, 1: one thread per row
//   warp 8           TMA producer: Q of both slots, a ring of K tiles and one of V tiles
//   warp 9           issuer of the products, tensor memory
// The prefix is cut into parts, so that all SMs are busy when rows are few, and every part leaves
// its rows' sums (fp32, relative to the part's maximum) in the workspace.  They lie with a row's
// neighbours in the tile side by side, four channels each: what 32 lanes write, and read again, is
// contiguous.
// Own keys: the single-token kernel's partial sums (decoding), or the window kernel's output and
// log-sum-exp (prompts; that output is rounded to bf16 once more than the result has to be, 2^-9 of
// its own share).  A last kernel joins all of a row's sums.
#include <algorithm>

#include "softmax_tc.cuh"

namespace psa {
namespace {

template <int D>
struct Cfg {
  static constexpr int kThreads = 320, kProducer = 8, kIssuer = 9;
  static constexpr int KST = D == 128 ? 3 : 5, VST = D == 128 ? 2 : 5;
  static constexpr uint32_t TILE = kTileBytes<D>;
  static constexpr uint32_t OFF_K = 2 * TILE, OFF_V = OFF_K + KST * TILE;
  static constexpr uint32_t OFF_BAR = OFF_V + VST * TILE, SMEM = OFF_BAR + 512 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;
};

struct Bars {
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], done;
  uint64_t k_full[5], k_empty[5], v_full[5], v_empty[5];
};

// The rows' tiles and the prefix' parts.
struct Plan {
  int B, nh, nkv, group, nq, P;
  int tq, tg, tb;              // a row tile's box
  int q_tiles, g_tiles, row_tiles;
  int key_tiles, parts;
  int slots() const { return row_tiles % 2 ? 2 * parts : parts; }  // places for a row's sums
};

struct Params {
  Plan p;
  float4* sums;   // [nkv * row_tiles][slots][D / 4][128]
  float2* stats;  // [nkv * row_tiles][slots][128]: maximum (log2 units), sum
  float sl2;      // scale * log2(e)
  int units, slots;
};

struct Unit {
  int hk, part, t0, n;  // key tiles t0 .. t0 + n - 1
  int rt;               // slot 0's row tile
  bool alone;           // slot 1 has the same one, and every second key tile
  __device__ __forceinline__ Unit(const Params& a, int u) {
    const int pairs = (a.p.row_tiles + 1) / 2;
    rt = 2 * (u % pairs);
    u /= pairs;
    part = u % a.p.parts;
    hk = u / a.p.parts;
    t0 = (int)((long long)a.p.key_tiles * part / a.p.parts);
    n = (int)((long long)a.p.key_tiles * (part + 1) / a.p.parts) - t0;
    alone = rt + 1 >= a.p.row_tiles;
  }
  __device__ __forceinline__ bool takes(int slot, int e) const { return !alone || (e & 1) == slot; }
  __device__ __forceinline__ int first(int slot) const { return alone ? slot : 0; }
  // one past a slot's last entry; first if it has none
  __device__ __forceinline__ bool some(int slot) const { return first(slot) < n; }
  __device__ __forceinline__ int last(int slot) const { return alone ? n - 1 - ((n - 1 - slot) & 1) : n - 1; }
  __device__ __forceinline__ int row_tile(int slot) const { return alone ? rt : rt + slot; }
};

__device__ __forceinline__ int unit_of(int i) {
  return i * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// Where a row tile's box begins.
struct Box {
  int q, g, b;
  __host__ __device__ __forceinline__ Box(const Plan& p, int rt) {
    q = rt % p.q_tiles * p.tq;
    rt /= p.q_tiles;
    g = rt % p.g_tiles * p.tg;
    b = rt / p.g_tiles * p.tb;
  }
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const Params a) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = align1024(smem_raw);
  const uint32_t sbase = smem_addr(smem);
  Bars& bar = *reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(&bar + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_at + 1);
  static_assert(sizeof(Bars) + 16 <= 512, "barriers");
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const Plan& p = a.p;
  const int rows = p.tq * p.tg * p.tb;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 1);
      mbar_init(&bar.q_empty[i], 1);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], kTile);
      mbar_init(&bar.o_full[i], 1);
    }
    mbar_init(&bar.done, 1);
    for (int i = 0; i < 5; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 2);  // one arrival per slot
      mbar_init(&bar.v_full[i], 1);
      mbar_init(&bar.v_empty[i], 2);
    }
    *abort = 0;
    fence_mbar_init();
  }
  // rows that no box fills are zeros (their scores must not move a warp's maxima)
  if (warp < 2) zero_rows<D>(smem + warp * C::TILE, rows, kTile, lane);
  if (warp == C::kIssuer) {
    tmem_alloc(tmem_at, C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  pdl_launch_dependents();
  pdl_wait();

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
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!ok || !u.some(s)) continue;
          const int n = q_count[s];
          if (n >= 1 && !mbar_wait(&bar.q_empty[s], (n - 1) & 1, abort)) {
            ok = false;
            continue;
          }
          mbar_arrive_expect_tx(&bar.q_full[s], (uint32_t)(rows * D * 2));
          const Box box(p, u.row_tile(s));
          load_tile<D>(smem + s * C::TILE, &tmQ, &bar.q_full[s], box.q, u.hk * p.group + box.g, box.b);
          q_count[s] = n + 1;
        }
        for (int e = 0; ok && e < u.n; ++e) {
          const int ks = kv % C::KST, vs = kv % C::VST, row = (u.t0 + e) * kTile;
          if (kv >= C::KST && !mbar_wait(&bar.k_empty[ks], (kv / C::KST - 1) & 1, abort)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bar.k_full[ks], C::TILE);
          load_tile<D>(smem + C::OFF_K + ks * C::TILE, &tmK, &bar.k_full[ks], row, u.hk, 0);
          ++kv;
          if (kv > C::VST && !mbar_wait(&bar.v_empty[vs], ((kv - 1) / C::VST - 1) & 1, abort)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bar.v_full[vs], C::TILE);
          load_tile<D>(smem + C::OFF_V + vs * C::TILE, &tmV, &bar.v_full[vs], row, u.hk, 0);
        }
      }
      if (*abort) {
        // let the copies in flight land before the CTA exits (a wait for one that was not issued
        // any more runs into its time limit)
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
      auto cols = [&](int e) { return min(kTile, (p.P - (u.t0 + e) * kTile + 15) & ~15); };
      bool first[2] = {true, true};
      // S of slot s and entry e, or the tile's release
      auto issue_s = [&](int s, int e) -> bool {
        const int kn = kv0 + e, st = kn % C::KST;
        if (!mbar_wait(&bar.k_full[st], (kn / C::KST) & 1, abort)) return false;
        if (!u.takes(s, e)) {
          if (lane == 0) mbar_arrive(&bar.k_empty[st]);
          __syncwarp();
          return true;
        }
        tc_fence_after();
        const uint64_t dQ = dQ0 + (uint64_t)(s * C::TILE >> 4), dK = dK0 + (uint64_t)(st * C::TILE >> 4);
        auto scores = [&](uint32_t id) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_warp(tmem + C::TM_S + 128 * s, dQ + kstep_channels(kk), dK + kstep_channels(kk), id,
                          kk > 0 ? 1u : 0u);
        };
        const int c = cols(e);
        if (c == kTile) scores(idesc_bf16_f32(128, kTile, false, false));
        else scores(idesc_bf16_f32(128, c, false, false));
        mma_commit_warp(&bar.s_full[s]);
        mma_commit_warp(&bar.k_empty[st]);
        if (e == u.last(s)) mma_commit_warp(&bar.q_empty[s]);  // the next unit's Q may come
        return true;
      };
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (ok && u.some(s)) ok = mbar_wait(&bar.q_full[s], q_count[s] & 1, abort);
        if (ok) ok = issue_s(s, 0);
      }
      // a slot that alternates has its first scores under way before its first entry
      for (int e = 0; ok && e < u.n; ++e) {
        const int vn = kv0 + e, st = vn % C::VST;
        if (!mbar_wait(&bar.v_full[st], (vn / C::VST) & 1, abort)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!ok) break;
          if (u.takes(s, e)) {
            if (!mbar_wait(&bar.p_full[s], steps[s] & 1, abort)) {
              ok = false;
              break;
            }
            ++steps[s];
            tc_fence_after();
            const uint64_t dV = dV0 + (uint64_t)(st * C::TILE >> 4);
            const uint32_t tO = tmem + C::TM_O + D * s, tP = tmem + C::TM_S + 128 * s;
            const int c = cols(e);
            if (c == kTile) {
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                mma_bf16_ts_warp(tO, tP + 8 * kk, dV + kk * kKstepRows, idO, !first[s] || kk > 0 ? 1u : 0u);
            } else {
#pragma unroll 1
              for (int kk = 0; 16 * kk < c; ++kk)
                mma_bf16_ts_warp(tO, tP + 8 * kk, dV + kk * kKstepRows, idO, !first[s] || kk > 0 ? 1u : 0u);
            }
            first[s] = false;
            mma_commit_warp(&bar.v_empty[st]);
            if (e == u.last(s)) mma_commit_warp(&bar.o_full[s]);
          } else {
            if (lane == 0) mbar_arrive(&bar.v_empty[st]);
            __syncwarp();
          }
          if (e + 1 < u.n) ok = issue_s(s, e + 1);
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) q_count[s] += u.some(s);
      kv0 += u.n;
    }
    mma_commit_warp(&bar.done);
    drain_wait(&bar.done, 0);
  } else {
    // ------------------------------------------------------------ softmax of a slot
    const int s = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + C::TM_S + 128 * s + lanes, tO = tmem + C::TM_O + D * s + lanes;
    int steps = 0, outs = 0;
    bool ok = true;
    for (int i = 0; ok && unit_of(i) < a.units; ++i) {
      const Unit u(a, unit_of(i));
      float m = -INFINITY, l = 0.f;
      for (int e = u.first(s); e < u.n; e += u.alone ? 2 : 1) {
        const int valid = p.P - (u.t0 + e) * kTile;  // columns of the prefix' last tile
        if (!mbar_wait(&bar.s_full[s], steps & 1, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool first = e == u.first(s);
        if (valid >= kTile) whole_step<D>(tS, tO, a.sl2, first, m, l);
        else masked_step<D>(tS, tO, (valid + 15) & ~15, 0, valid - 1, 0, a.sl2, first, m, l);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar.p_full[s]);
        ++steps;
      }
      if (!ok) break;
      // ---- the rows' sums
      const long long at = ((long long)u.hk * p.row_tiles + u.row_tile(s)) * a.slots + (u.alone ? 2 * u.part + s : u.part);
      if (u.some(s)) {
        if (!mbar_wait(&bar.o_full[s], outs & 1, abort)) break;
        ++outs;
        tc_fence_after();
        float4* dst = a.sums + at * (D / 4) * kTile + r;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_load32(tO + c, o);
          if (r < rows) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              dst[(c + k) / 4 * kTile] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
        tc_fence_before();
      }
      if (r < rows) a.stats[at * kTile + r] = make_float2(m, l);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// ---------------------------------------------------------------- a row's sums, joined
constexpr int kJoinRows = 32, kJoinChannels = 32, kJoinThreads = 256;

struct JoinArgs {
  Plan p;
  const float4* sums;
  const float2* stats;
  int slots;
  View<__nv_bfloat16> o;
  const int* lens;
  int nk;
  // own keys, decoding: partial sums [B, nh, splits][D + 2]; prompts: log-sum-exp [B, nh, nq] (with
  // the output in o), and where the whole rows' goes to
  const float* own;
  int splits;
  const float* own_lse;
  float* lse;
};

// 32 rows of a tile, 32 channels: lanes are rows while the prefix' sums are added (each warp
// four channels), then channels.
template <int D, bool kDecode>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const JoinArgs a) {
  __shared__ float sum[kJoinRows][kJoinChannels + 4];
  __shared__ float top[kJoinRows], total[kJoinRows];
  pdl_launch_dependents();
  pdl_wait();
  const Plan& p = a.p;
  const int groups = kTile / kJoinRows;
  const int tile = blockIdx.x / groups, rt = tile % p.row_tiles, hk = tile / p.row_tiles;
  const int r0 = blockIdx.x % groups * kJoinRows, c0 = blockIdx.y * kJoinChannels;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = p.tq * p.tg * p.tb;
  if (r0 >= rows) return;
  const Box box(p, rt);
  // row r of the tile
  struct Row {
    int b, h, q;
    bool valid;
  };
  auto row_of = [&](int r) {
    Row x;
    const int i = r % p.tq, g = r / p.tq % p.tg, bb = r / (p.tq * p.tg);
    x.b = box.b + bb;
    x.h = hk * p.group + box.g + g;
    x.q = box.q + i;
    x.valid = r < rows && x.b < p.B && box.g + g < p.group && x.q < p.nq;
    return x;
  };
  const int mine = rt == p.row_tiles - 1 && p.row_tiles % 2 ? 2 * p.parts : p.parts;  // sums of a row
  const long long at = ((long long)hk * p.row_tiles + rt) * a.slots;
  const float2* stats = a.stats + at * kTile + r0 + lane;
  const Row me = row_of(r0 + lane);
  // ---- maximum over the parts and the own keys (every warp for itself)
  float m = -INFINITY, l = 0.f;
  float2 own = make_float2(-INFINITY, 0.f);
  if (me.valid) {
#pragma unroll 4
    for (int s = 0; s < mine; ++s) m = fmaxf(m, stats[s * kTile].x);
    if constexpr (kDecode) {
      const float* src = a.own + ((long long)me.b * p.nh + me.h) * a.splits * (D + 2) + D;
      for (int s = 0; s < a.splits; ++s) own.x = fmaxf(own.x, src[s * (D + 2)]);
      for (int s = 0; s < a.splits; ++s) {
        const float x = src[s * (D + 2)];
        own.y += src[s * (D + 2) + 1] * (x == -INFINITY ? 0.f : fast_exp2(x - own.x));
      }
    } else {
      own = make_float2(kLog2 * a.own_lse[((long long)me.b * p.nh + me.h) * p.nq + me.q], 1.f);
      if (own.x == -INFINITY) own.y = 0.f;
    }
    m = fmaxf(m, own.x);
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (me.valid) {
    const float4* src = a.sums + (at * (D / 4) + c0 / 4 + warp) * kTile + r0 + lane;
#pragma unroll 4
    for (int s = 0; s < mine; ++s) {
      const float2 x = stats[s * kTile];
      const float f = x.x == -INFINITY ? 0.f : fast_exp2(x.x - m);
      l += x.y * f;
      if (x.y != 0.f) {  // (a part that had no tile has left nothing)
        const float4 v = src[(long long)s * (D / 4) * kTile];
        acc.x += v.x * f;
        acc.y += v.y * f;
        acc.z += v.z * f;
        acc.w += v.w * f;
      }
    }
    l += own.y * (own.x == -INFINITY ? (own.y != own.y ? own.y : 0.f) : fast_exp2(own.x - m));
  }
  *reinterpret_cast<float4*>(&sum[lane][4 * warp]) = acc;
  if (warp == 0) {
    top[lane] = m;
    total[lane] = l;
  }
  __syncthreads();
  for (int i = warp; i < kJoinRows; i += kJoinThreads / 32) {
    const Row x = row_of(r0 + i);
    if (!x.valid) continue;
    // padding: a slot of the batch that is not in use, or a row behind its sequence
    const int n = a.lens ? a.lens[x.b] : a.nk;
    const bool pad = kDecode ? n < 0 : x.q + a.nk - p.nq >= min(n, a.nk);
    const float mm = top[i];
    float v = sum[i][lane];
    __nv_bfloat16* o = a.o.row(x.b, x.h, x.q) + c0 + lane;
    if constexpr (kDecode) {
      const float* src = a.own + ((long long)x.b * p.nh + x.h) * a.splits * (D + 2);
      for (int s = 0; s < a.splits; ++s) {
        const float y = src[s * (D + 2) + D];
        if (y != -INFINITY) v += src[s * (D + 2) + c0 + lane] * fast_exp2(y - mm);
      }
    } else {
      const long long row = ((long long)x.b * p.nh + x.h) * p.nq + x.q;
      const float y = kLog2 * a.own_lse[row];
      if (y != -INFINITY) v += __bfloat162float(*o) * fast_exp2(y - mm);
      if (a.lse && blockIdx.y == 0 && lane == 0) a.lse[row] = pad ? -INFINITY : mm * kLn2 + logf(total[i]);
    }
    *o = __float2bfloat16_rn(pad ? 0.f : v / total[i]);
  }
}

// The box of a row tile that needs the fewest tiles, and of those the one with most queries.
Plan make_plan(const PrefixShape& x) {
  Plan p{};
  p.B = x.B;
  p.nh = x.nh;
  p.nkv = x.nkv;
  p.group = x.nh / x.nkv;
  p.nq = x.nq;
  p.P = x.P;
  auto cdiv = [](int a, int b) { return (a + b - 1) / b; };
  for (int tq = 1; tq <= std::min(p.nq, kTile); ++tq) {
    const int tg = std::min(p.group, kTile / tq), tb = std::min(p.B, kTile / (tq * tg));
    const int tiles = cdiv(p.nq, tq) * cdiv(p.group, tg) * cdiv(p.B, tb);
    if (tq == 1 || tiles <= p.row_tiles) {
      p.tq = tq;
      p.tg = tg;
      p.tb = tb;
      p.row_tiles = tiles;
    }
  }
  p.q_tiles = cdiv(p.nq, p.tq);
  p.g_tiles = cdiv(p.group, p.tg);
  p.key_tiles = cdiv(p.P, kTile);
  // Parts: the fewest rounds over the SMs, counted in key tiles; a unit's beginning and end and the
  // joining of its sums take about as long as three more (measured: 64 sequences, 32 heads on 8,
  // 16384 keys).
  const long long pairs = (long long)p.nkv * cdiv(p.row_tiles, 2);
  long long best = -1;
  for (int parts = 1; parts <= std::min(p.key_tiles, kMaxPrefixParts); ++parts) {
    const long long time = ((pairs * parts + 151) / 152) * (cdiv(p.key_tiles, parts) + 3);
    if (best < 0 || time < best) {
      best = time;
      p.parts = parts;
    }
  }
  return p;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t sums_bytes(const Plan& p, int d) { return (size_t)p.nkv * p.row_tiles * p.slots() * kTile * d * 4; }
size_t stats_bytes(const Plan& p) { return (size_t)p.nkv * p.row_tiles * p.slots() * kTile * 8; }

template <int D>
cudaError_t prefix_part(const PrefixArgs& x, const Plan& p, cudaStream_t st) {
  using C = Cfg<D>;
  Params a{};
  a.p = p;
  a.sums = static_cast<float4*>(x.ws);
  a.stats = reinterpret_cast<float2*>(static_cast<char*>(x.ws) + sums_bytes(p, D));
  a.sl2 = x.scale * kLog2;
  a.units = p.nkv * ((p.row_tiles + 1) / 2) * p.parts;
  a.slots = p.slots();
  CUtensorMap mq, mk, mv;
  if (!map_view_box(&mq, x.q.p, x.q.sb, x.q.sh, x.q.sn, p.B, p.nh, p.nq, D, p.tq, p.tg, p.tb) ||
      !map_view(&mk, x.kp.p, x.kp.sb, x.kp.sh, x.kp.sn, 1, p.nkv, p.P, D) ||
      !map_view(&mv, x.vp.p, x.vp.sb, x.vp.sh, x.vp.sn, 1, p.nkv, p.P, D))
    return cudaErrorInvalidValue;
  auto kern = prefix_tc_kernel<D>;
  const cudaError_t e = set_max_dynamic_smem((const void*)kern, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(std::min(a.units, device_sm_count())), dim3(C::kThreads), C::SMEM, st, mq, mk, mv, a);
}

template <int D>
cudaError_t run(const PrefixArgs& x, bool decode, cudaStream_t st) {
  const Plan p = make_plan(x.s);
  char* ws = static_cast<char*>(x.ws);
  float* own = reinterpret_cast<float*>(ws + sums_bytes(p, D) + stats_bytes(p));
  cudaError_t e = prefix_part<D>(x, p, st);
  if (e != cudaSuccess) return e;
  JoinArgs j{};
  j.p = p;
  j.sums = reinterpret_cast<const float4*>(ws);
  j.stats = reinterpret_cast<const float2*>(ws + sums_bytes(p, D));
  j.slots = p.slots();
  j.o = x.o;
  j.lens = x.lens;
  j.nk = x.s.nk;
  const Window w{p.B, p.nh, p.nkv, p.nq, x.s.nk, x.s.nk, 0, 0, x.lens};
  if (decode) {
    DecodeArgs d{};
    d.w = w;
    d.q = x.q;
    d.k = x.k;
    d.v = x.v;
    d.ws = own;
    d.scale = x.scale;
    e = launch_window_decode_parts(d, D, st);
    j.own = own;
    j.splits = decode_splits(w);
  } else {
    WindowArgs<__nv_bfloat16> f{};
    f.w = w;
    f.q = x.q;
    f.k = x.k;
    f.v = x.v;
    f.out = x.o;
    f.lse = own;
    f.scale = x.scale;
    e = launch_window_fwd_tc(f, D, st);
    j.own_lse = own;
    j.lse = x.lse;
  }
  if (e != cudaSuccess) return e;
  const dim3 grid(p.nkv * p.row_tiles * (kTile / kJoinRows), D / kJoinChannels);
  return launch_pdl(decode ? prefix_join_kernel<D, true> : prefix_join_kernel<D, false>, grid, dim3(kJoinThreads), 0, st, j);
}

}  // namespace

size_t prefix_ws_bytes(const PrefixShape& x, int d) {
  const Plan p = make_plan(x);
  const Window w{x.B, x.nh, x.nkv, x.nq, x.nk, x.nk, 0, 0, nullptr};
  const size_t own = x.nq == 1 ? decode_parts_ws_bytes(w, d) : 0;
  return round256(sums_bytes(p, d) + stats_bytes(p) + std::max(own, (size_t)x.B * x.nh * x.nq * 4));
}

cudaError_t launch_prefix_attn(const PrefixArgs& a, int d, bool decode, cudaStream_t st) {
  return d == 64 ? run<64>(a, decode, st) : run<128>(a, decode, st);
}

}  // namespace psa
