// prefix_attn.cu -- attention of a batch whose sequences share a long prefix (bf16, tcgen05):
//
//   o = softmax over [prefix keys | own keys that the query sees] of scale q k^T, times v
//
// The prefix is read once for all sequences: the queries of one key/value head, of all sequences
// and of the heads that share it, are the rows of one product with its keys.  A tile of 128 rows
// is a box of tq queries, tg heads and tb sequences, those extents that need the fewest tiles (with
// lengths: one of two boxes, chosen on the device).
// The prefix part is an online softmax without masks (but for the last tile's columns), as the
// window attention's forward: two slots of 128 rows whose softmax steps run while the other
// slot's products do, P in S's columns of tensor memory, products issued in order by one
// converged warp.  The slots share the key/value tiles; a row tile without a partner takes both
// slots and alternates between them.
//   warps 0-3, 4-7   softmax of slot 0, 1: one thread per row
//   warp 8           TMA producer: Q of both slots, a ring of K tiles and one of V tiles
//   warp 9           issuer of the products, tensor memory
// Row tiles of padding alone are left out (counted on the device).  All SMs get an equal run of steps, a
// step being a key tile of a pair of row tiles, or of one that has no partner (half the products, so that
// of few row tiles an odd one costs what two would).  Where a run ends
// inside the prefix a row's sums come in pieces (fp32, relative to the piece's maximum).  They lie in the
// workspace with a row's neighbours in the tile side by side, four channels each: what 32 lanes write,
// and read again, is contiguous.
// Own keys: the single-token kernel's partial sums (decoding), or the window kernel's output in fp32
// and log-sum-exp (prompts).  A last kernel joins all of a row's sums and rounds once.
//
// Measured, 32 heads of 128 on 8, on the device.  64 tokens behind 16384 shared and up to 1024 own
// keys: 78 us (prefix 24, own keys 34: 5.1 TB/s, joining 14; 242 MB in all, 36 us at the copy
// bandwidth).  16 prompts of 20 to 77 tokens behind 8192 keys: 143 us (prefix 105: a third of its
// rows hold no query; own keys 20, joining 26).  A step of two row tiles takes 1.6 us where its
// products take 1.07 (tensor pipe busy 56 % of the time, no other unit above a third): two warps a
// scheduler for the softmax, as in the window attention.
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

constexpr int kStagedLens = 256;  // lengths that are read once, into shared memory

struct Bars {
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], done;
  uint64_t k_full[5], k_empty[5], v_full[5], v_empty[5];
};

// How the rows are cut into tiles: the box of one, and how many there are.
struct Boxes {
  int tq, tg, tb;  // queries, heads of a group, sequences
  int q_tiles, g_tiles, row_tiles;
  __host__ __device__ __forceinline__ int rows() const { return tq * tg * tb; }
};
// With lengths there are two ways to cut (Plan's `ways`), and the device takes the one that needs
// fewer tiles.
struct Plan {
  int B, nh, nkv, group, nq, P, nk;
  int ways;
  Boxes way[2];
  int key_tiles;
  // (not indexed: it lies with the kernel's parameters)
  __host__ __device__ __forceinline__ Boxes boxes(int i) const { return i ? way[1] : way[0]; }
  __host__ __device__ __forceinline__ int most_tiles() const {
    return ways > 1 && way[1].row_tiles > way[0].row_tiles ? way[1].row_tiles : way[0].row_tiles;
  }
};

// How the work is dealt: units (a key/value head's pair of the row tiles in use) of key_tiles
// steps lie one behind another, and CTA c of `ctas` takes an equal run of all steps.  What it
// leaves of a unit is a piece, and lies at place unit + c: of neighbouring pieces one of the two is
// larger.
struct Deal {
  int tiles, pairs, key_tiles, ctas;
  long long steps;
  __host__ __device__ __forceinline__ Deal(const Plan& p, int tiles_in_use) {
    tiles = tiles_in_use;
    pairs = (tiles + 1) / 2;
    key_tiles = p.key_tiles;
    steps = (long long)p.nkv * pairs * key_tiles;
    // a CTA for each SM, but not for less than two key tiles
    const long long c = (steps + 1) / 2;
    ctas = c < kPrefixCtas ? (int)c : kPrefixCtas;
  }
  __host__ __device__ __forceinline__ long long from(int cta) const { return cta < ctas ? steps * cta / ctas : steps; }
  __host__ __device__ __forceinline__ int cta_of(long long step) const { return (int)(((step + 1) * ctas - 1) / steps); }
  __host__ __device__ __forceinline__ int first_cta(int unit) const { return cta_of((long long)unit * key_tiles); }
  __host__ __device__ __forceinline__ int last_cta(int unit) const { return cta_of((long long)(unit + 1) * key_tiles - 1); }
};

struct Params {
  Plan p;
  float4* sums;   // [units + ctas][2 slots][D / 4][128]
  float2* stats;  // [units + ctas][2 slots][128]: maximum (log2 units), sum
  // Prompts with lengths: row tiles of padding alone are left out.  tile_of [most_tiles]: those in
  // use; place [most_tiles + 2]: their number, which way the rows are cut, then each tile's index among
  // them or -1.
  const int* lens;
  int *tile_of, *place;
  float sl2;      // scale * log2(e)
};

// What a CTA does of a unit: it begins at step `pos` of all.
struct Piece {
  int hk, t0, n;   // key tiles t0 .. t0 + n - 1
  int unit, tile;  // slot 0's row tile, counted among those in use
  bool alone;      // slot 1 has the same one, and every second key tile
  __device__ __forceinline__ Piece(const Deal& d, long long pos, long long end) {
    unit = (int)(pos / d.key_tiles);
    t0 = (int)(pos - (long long)unit * d.key_tiles);
    n = (int)min((long long)(d.key_tiles - t0), end - pos);
    hk = unit / d.pairs;
    tile = 2 * (unit - hk * d.pairs);
    alone = tile + 1 >= d.tiles;
  }
  __device__ __forceinline__ bool takes(int slot, int e) const { return !alone || (e & 1) == slot; }
  __device__ __forceinline__ int first(int slot) const { return alone ? slot : 0; }
  __device__ __forceinline__ bool some(int slot) const { return first(slot) < n; }
  __device__ __forceinline__ int last(int slot) const { return alone ? n - 1 - ((n - 1 - slot) & 1) : n - 1; }
};

// Where a row tile's box begins.
struct Box {
  int q, g, b;
  __device__ __forceinline__ Box(const Boxes& x, int rt) {
    q = rt % x.q_tiles * x.tq;
    rt /= x.q_tiles;
    g = rt % x.g_tiles * x.tg;
    b = rt / x.g_tiles * x.tb;
  }
  // whether some row is not padding (asked before pdl_wait: the lengths come from L2, the first of them
  // by way of shared memory).  No way out of the loop: its reads do not wait for one another.
  __device__ __forceinline__ bool in_use(const Plan& p, int tb, const int* lens, const int* staged) const {
    const int end = min(b + tb, p.B);
    int longest = 0;
#pragma unroll 4
    for (int i = b; i < min(end, kStagedLens); ++i) longest = max(longest, staged[i]);
#pragma unroll 4
    for (int i = max(b, kStagedLens); i < end; ++i) longest = max(longest, ld_global_l2(lens + i));
    return q + p.nk - p.nq < min(longest, p.nk);
  }
};

// kLengths: a.lens is there (a kernel of its own: decoding and prompts without lengths are 1 % faster
// without what counts the tiles).
template <int D, bool kLengths>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tmQ0, const __grid_constant__ CUtensorMap tmQ1,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const Params a) {
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
  __shared__ int2 before[C::kThreads / 32];
  __shared__ int staged[kStagedLens], chosen_rows;

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
  if (warp == C::kIssuer) {
    tmem_alloc(tmem_at, C::TM_COLS);
    tmem_relinquish();
  }
  // The row tiles in use, each thread a run of them: passes 0 and 1 count them for the two ways to cut
  // the rows, pass 2 writes the list of the one that needs fewer.  Every CTA writes the same list, of
  // which it reads its own entries after the barrier below.  (One loop: these instructions run once, and
  // fetching them is most of what they cost.)
  int tiles = p.way[0].row_tiles, which = 0;
  if constexpr (kLengths) {
    for (int i = threadIdx.x; i < min(p.B, kStagedLens); i += C::kThreads) staged[i] = ld_global_l2(a.lens + i);
    __syncthreads();
    int mine[2] = {0, 0}, at = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const Boxes x = p.boxes(pass < 2 ? pass : which);
      const int per = pass < p.ways || pass == 2 ? (x.row_tiles + C::kThreads - 1) / C::kThreads : 0;
      const int from = min(x.row_tiles, (int)threadIdx.x * per), to = min(x.row_tiles, from + per);
      int n = 0;
#pragma unroll 1
      for (int rt = from; rt < to; ++rt) {
        const bool used = Box(x, rt).in_use(p, x.tb, a.lens, staged);
        if (pass == 2) {
          if (used) a.tile_of[at + n] = rt;
          if (blockIdx.x == 0) a.place[2 + rt] = used ? at + n : -1;
        }
        n += used;
      }
      if (pass == 0) mine[0] = n;
      if (pass != 1) continue;
      mine[1] = n;
      const int all0 = __reduce_add_sync(0xffffffffu, mine[0]), all1 = __reduce_add_sync(0xffffffffu, mine[1]);
      if (lane == 0) before[warp] = make_int2(all0, all1);
      __syncthreads();
      const int2 others = lane < C::kThreads / 32 ? before[lane] : make_int2(0, 0);
      const int2 all = make_int2(__reduce_add_sync(0xffffffffu, others.x), __reduce_add_sync(0xffffffffu, others.y));
      which = p.ways > 1 && all.y < all.x;
      tiles = which ? all.y : all.x;
      const int upto = which ? mine[1] : mine[0];
      at = __reduce_add_sync(0xffffffffu, lane >= warp ? 0 : which ? others.y : others.x) - upto;
      int sum = upto;
#pragma unroll 1
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += y;
      }
      at += sum;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      a.place[0] = tiles;
      a.place[1] = which;
    }
  }
  // rows that no box fills are zeros (their scores must not move a warp's maxima)
  if (warp < 2) zero_rows<D>(smem + warp * C::TILE, p.boxes(which).rows(), kTile, lane);
  if (kLengths && threadIdx.x == 0) chosen_rows = p.boxes(which).rows();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  const Deal deal(p, tiles);
  // The kernel before this one is the own keys', which shares nothing with it and lets it start only
  // once all that came before has completed: this one runs beside its end, and waits for it before
  // its own, so that the joining kernel finds both done.
  pdl_launch_dependents();
  const long long begin = deal.from(blockIdx.x), end = deal.from(blockIdx.x + 1);

  if (warp == C::kProducer) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const Boxes cut = p.boxes(which);
      const CUtensorMap* tmQ = which ? &tmQ1 : &tmQ0;
      tma_prefetch_desc(tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      bool ok = true;
      int q_count[2] = {0, 0}, kv = 0;
      for (long long pos = begin; ok && pos < end;) {
        const Piece u(deal, pos, end);
        pos += u.n;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!ok || !u.some(s)) continue;
          const int n = q_count[s];
          if (n >= 1 && !mbar_wait(&bar.q_empty[s], (n - 1) & 1, abort)) {
            ok = false;
            continue;
          }
          mbar_arrive_expect_tx(&bar.q_full[s], (uint32_t)(cut.rows() * D * 2));
          const int tile = u.alone ? u.tile : u.tile + s;
          const Box box(cut, kLengths ? a.tile_of[tile] : tile);
          load_tile<D>(smem + s * C::TILE, tmQ, &bar.q_full[s], box.q, u.hk * p.group + box.g, box.b);
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
    for (long long pos = begin; ok && pos < end;) {
      const Piece u(deal, pos, end);
      pos += u.n;
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
    for (long long pos = begin; ok && pos < end;) {
      int n, e0, step, valid;  // what the loop needs (the piece again behind it: registers)
      {
        const Piece u(deal, pos, end);
        n = u.n;
        e0 = u.first(s);
        step = u.alone ? 2 : 1;
        valid = p.P - (u.t0 + e0) * kTile;  // columns from the entry's tile on
      }
      float m = -INFINITY, l = 0.f;
      for (int e = e0; e < n; e += step, valid -= step * kTile) {
        if (!mbar_wait(&bar.s_full[s], steps & 1, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool first = e == e0;
        if (valid >= kTile) whole_step<D>(tS, tO, a.sl2, first, m, l);
        else masked_step<D>(tS, tO, (valid + 15) & ~15, 0, valid - 1, 0, a.sl2, first, m, l);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar.p_full[s]);
        ++steps;
      }
      if (!ok) break;
      // ---- the rows' sums
      const Piece u(deal, pos, end);
      pos += n;
      const bool valid_row = r < (kLengths ? *(volatile int*)&chosen_rows : p.way[0].rows());
      const long long at = 2LL * (u.unit + blockIdx.x) + s;
      if (u.some(s)) {
        if (!mbar_wait(&bar.o_full[s], outs & 1, abort)) break;
        ++outs;
        tc_fence_after();
        float4* dst = a.sums + at * (D / 4) * kTile + r;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_load32(tO + c, o);
          if (valid_row) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              dst[(c + k) / 4 * kTile] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
        tc_fence_before();
      }
      if (valid_row) a.stats[at * kTile + r] = make_float2(m, l);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
  pdl_wait();
}

// ---------------------------------------------------------------- a row's sums, joined
constexpr int kJoinRows = 32, kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

struct JoinArgs {
  Plan p;
  const float4* sums;
  const float2* stats;
  const int* place;  // or null: cut the first way, all row tiles in use
  View<__nv_bfloat16> o;
  const int* lens;
  int nk;
  // own keys, decoding: partial sums [B, nh, parts][D + 4] of runs of blocks of 16 keys; prompts:
  // outputs [B, nh, nq, D] and log-sum-exp [B, nh, nq], and where the whole rows' goes to
  const float* own;
  int run, parts;
  const float* own_lse;
  float* lse;
};

// 32 rows of a tile, CH channels.  Lanes are rows while the prefix' sums are added (each warp some
// of the channels), then channels.
template <int D, int CH, bool kDecode>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const JoinArgs a) {
  constexpr int Q = CH / 4 / kJoinWarps;  // fours of channels that a warp adds
  extern __shared__ float2 stats[];       // [sums of a row][32]
  __shared__ __align__(16) float sum[kJoinRows][CH + 4];
  __shared__ float own_m[kJoinRows], own_l[kJoinRows], top[kJoinRows], total[kJoinRows];
  pdl_launch_dependents();
  pdl_wait();
  const Plan& p = a.p;
  constexpr int groups = kTile / kJoinRows;
  const int hk = blockIdx.z, rt = blockIdx.x / groups;
  const int tiles = a.place ? a.place[0] : p.way[0].row_tiles, at_use = a.place ? a.place[2 + rt] : rt;
  const Boxes cut = p.boxes(a.place ? a.place[1] : 0);
  const int r0 = blockIdx.x % groups * kJoinRows, c0 = blockIdx.y * CH;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = cut.rows();
  if (rt >= cut.row_tiles || r0 >= rows) return;  // (there are CTAs for the way that has more tiles)
  const Box box(cut, rt);
  struct Row {
    int b, h, q;
    bool valid;
  };
  auto row_of = [&](int r) {
    Row x;
    const int g = r / cut.tq, bb = g / cut.tg;
    x.b = box.b + bb;
    x.h = box.g + g - bb * cut.tg;
    x.q = box.q + r - g * cut.tq;
    x.valid = r < rows && x.b < p.B && x.h < p.group && x.q < p.nq;
    x.h += hk * p.group;
    return x;
  };
  // this tile's sums: `mine` of them, `step` places apart
  const Deal d(p, tiles);
  const int unit = hk * d.pairs + at_use / 2;
  const bool alone = at_use + 1 == d.tiles && d.tiles % 2;
  const int step = alone ? 1 : 2;
  int mine = 0;
  long long at = 0;
  if (at_use >= 0) {
    const int c = d.first_cta(unit);
    mine = (d.last_cta(unit) - c + 1) * (alone ? 2 : 1);
    at = 2LL * (unit + c) + (alone ? 0 : at_use & 1);
  }
  for (int s = warp; s < mine; s += kJoinWarps) stats[s * 32 + lane] = a.stats[(at + s * step) * kTile + r0 + lane];
  auto own_parts = [&](int b) { return ((max(0, min(a.lens[b], a.nk)) + 15) / 16 + a.run - 1) / a.run; };
  // the own keys' maximum and sum
  if constexpr (kDecode) {
    // (eight lanes for each of a warp's four rows: one latency for all of them)
    const int i = warp * 4 + lane / 8;
    const Row x = row_of(r0 + i);
    float m = -INFINITY, l = 0.f;
    if (x.valid) {
      const float* src = a.own + ((long long)x.b * p.nh + x.h) * a.parts * (D + 4) + D;
      const int own = own_parts(x.b);
      for (int s = lane % 8; s < own; s += 8) {
        const float2 y = *reinterpret_cast<const float2*>(src + s * (D + 4));
        const float n = fmaxf(m, y.x);
        l = l * (m == -INFINITY ? 0.f : fast_exp2(m - n)) + y.y * (y.x == -INFINITY ? 0.f : fast_exp2(y.x - n));
        m = n;
      }
    }
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, d), l2 = __shfl_xor_sync(0xffffffffu, l, d), n = fmaxf(m, m2);
      l = l * (m == -INFINITY ? 0.f : fast_exp2(m - n)) + l2 * (m2 == -INFINITY ? 0.f : fast_exp2(m2 - n));
      m = n;
    }
    if (lane % 8 == 0) {
      own_m[i] = m;
      own_l[i] = l;
    }
  } else if (warp == 0) {
    const Row x = row_of(r0 + lane);
    const float m = x.valid ? kLog2 * a.own_lse[((long long)x.b * p.nh + x.h) * p.nq + x.q] : -INFINITY;
    own_m[lane] = m;
    own_l[lane] = m == -INFINITY ? 0.f : 1.f;
  }
  __syncthreads();
  float m = own_m[lane], l = 0.f;
  for (int s = 0; s < mine; ++s) m = fmaxf(m, stats[s * 32 + lane].x);
  float4 acc[Q];
#pragma unroll
  for (int c = 0; c < Q; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r0 + lane < rows) {
    const float4* src = a.sums + (at * (D / 4) + c0 / 4 + warp * Q) * kTile + r0 + lane;
    constexpr int U = Q > 2 ? 2 : 8;  // pieces on their way at a time
    for (int s0 = 0; s0 < mine; s0 += U) {
      float4 v[U][Q];
      float f[U];
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const float2 st = s0 + x < mine ? stats[(s0 + x) * 32 + lane] : make_float2(-INFINITY, 0.f);
        f[x] = st.x == -INFINITY ? 0.f : fast_exp2(st.x - m);
        l += st.y * f[x];
#pragma unroll
        for (int c = 0; c < Q; ++c)  // (a piece that had no tile for the slot has left nothing)
          v[x][c] = st.y != 0.f ? src[((long long)(s0 + x) * step * (D / 4) + c) * kTile] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int x = 0; x < U; ++x)
#pragma unroll
        for (int c = 0; c < Q; ++c) {
          acc[c].x += v[x][c].x * f[x];
          acc[c].y += v[x][c].y * f[x];
          acc[c].z += v[x][c].z * f[x];
          acc[c].w += v[x][c].w * f[x];
        }
    }
  }
#pragma unroll
  for (int c = 0; c < Q; ++c) *reinterpret_cast<float4*>(&sum[lane][4 * (warp * Q + c)]) = acc[c];
  if (warp == 0) {
    // (a NaN among the own keys' scores stays one: their sum is NaN then)
    const float f = own_m[lane] == -INFINITY ? 0.f : fast_exp2(own_m[lane] - m);
    top[lane] = m;
    total[lane] = l + own_l[lane] * f;
  }
  __syncthreads();
  // lanes are fours of channels now, and rows (CH 32) or parts of the own keys side by side
  constexpr int F = CH / 4, R = 32 / F;
  const int c4 = lane % F, sub = lane / F;
#pragma unroll 2
  for (int i0 = warp * R; i0 < kJoinRows; i0 += kJoinWarps * R) {
    const int i = i0 + sub;
    const Row x = row_of(r0 + i);
    if (!x.valid) continue;
    // padding: a slot of the batch that is not in use, or a row behind its sequence
    const int n = a.lens ? a.lens[x.b] : a.nk;
    const bool pad = kDecode ? n < 0 : x.q + a.nk - p.nq >= min(n, a.nk);
    const float mm = top[i], inv = 1.f / total[i];
    float4 v = *reinterpret_cast<const float4*>(&sum[i][4 * c4]);
    auto add = [&](const float4& y, float f) {
      v.x += y.x * f;
      v.y += y.y * f;
      v.z += y.z * f;
      v.w += y.w * f;
    };
    uint2* o = reinterpret_cast<uint2*>(a.o.row(x.b, x.h, x.q) + c0 + 4 * c4);
    if constexpr (kDecode) {
      const float* src = a.own + ((long long)x.b * p.nh + x.h) * a.parts * (D + 4);
      const int own = own_parts(x.b);
#pragma unroll 8
      for (int s = 0; s < own; ++s) {
        const float y = src[s * (D + 4) + D], f = y == -INFINITY ? 0.f : fast_exp2(y - mm);
        add(*reinterpret_cast<const float4*>(src + s * (D + 4) + c0 + 4 * c4), f);
      }
    } else if (own_m[i] != -INFINITY) {
      const long long row = ((long long)x.b * p.nh + x.h) * p.nq + x.q;
      add(*reinterpret_cast<const float4*>(a.own + row * D + c0 + 4 * c4), fast_exp2(own_m[i] - mm));
    }
    *o = pad ? make_uint2(0, 0) : make_uint2(pack2(v.x * inv, v.y * inv), pack2(v.z * inv, v.w * inv));
    if (!kDecode && a.lse && c4 == 0 && blockIdx.y == 0)
      a.lse[((long long)x.b * p.nh + x.h) * p.nq + x.q] = pad ? -INFINITY : mm * kLn2 + logf(total[i]);
  }
}

// The box of a row tile that needs the fewest tiles, and of those the one with most queries.  With
// lengths, tiles of padding alone cost nothing, and a tile of several sequences is in use up to the
// longest of them: for lengths anywhere below n_q (`spread`) that is tb / (tb + 1) of their tiles, and half
// a tile.
Boxes best_boxes(const Plan& p, bool spread) {
  auto cdiv = [](int a, int b) { return (a + b - 1) / b; };
  Boxes x{};
  double least = 0;
  for (int tq = 1; tq <= std::min(p.nq, kTile); ++tq) {
    const int tg = std::min(p.group, kTile / tq), tb = std::min(p.B, kTile / (tq * tg));
    const double across = (double)cdiv(p.group, tg) * cdiv(p.B, tb);
    const double tiles = across * (spread ? (double)p.nq / tq * tb / (tb + 1) + 0.5 : cdiv(p.nq, tq));
    if (tq == 1 || tiles <= least) {
      least = tiles;
      x.tq = tq;
      x.tg = tg;
      x.tb = tb;
    }
  }
  x.q_tiles = cdiv(p.nq, x.tq);
  x.g_tiles = cdiv(p.group, x.tg);
  x.row_tiles = x.q_tiles * x.g_tiles * cdiv(p.B, x.tb);
  return x;
}

// Two ways where there are lengths, because which of them needs fewer tiles is known on the device only.
// Measured, 16 prompts behind 8192 keys, 32 heads on 8, boxes of 2 queries, 4 heads, 16 sequences against
// 32, 4, 1: lengths of 20 to 77 162 and 143 us, all 77 170 and 196, all 38 107 and 141.  Counting both ways
// costs 0.5 to 4 us of that.
Plan make_plan(const PrefixShape& x, bool lengths) {
  Plan p{};
  p.B = x.B;
  p.nh = x.nh;
  p.nkv = x.nkv;
  p.group = x.nh / x.nkv;
  p.nq = x.nq;
  p.P = x.P;
  p.nk = x.nk;
  p.key_tiles = (p.P + kTile - 1) / kTile;
  p.way[0] = best_boxes(p, false);
  p.way[1] = best_boxes(p, lengths);
  const Boxes &a = p.way[0], &b = p.way[1];
  p.ways = a.tq == b.tq && a.tg == b.tg && a.tb == b.tb ? 1 : 2;
  return p;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t pieces_at_most(const Plan& p) {
  const Deal d(p, p.most_tiles());
  return (size_t)p.nkv * d.pairs + d.ctas;
}
size_t sums_bytes(const Plan& p, int d) { return pieces_at_most(p) * 2 * kTile * d * 4; }
size_t stats_bytes(const Plan& p) { return pieces_at_most(p) * 2 * kTile * 8; }
size_t tiles_bytes(const Plan& p) { return round256((2 * (size_t)p.most_tiles() + 2) * 4); }

// A row's sums at most: the runs that a unit's steps fill, and one that begins or ends in it; with
// row tiles left out there may be one unit for each key/value head, and one tile alone.
int sums_at_most(const Plan& p, bool all_in_use) {
  const int units = p.nkv * (all_in_use ? Deal(p, p.way[0].row_tiles).pairs : 1);
  const int most = std::min(kPrefixCtas, (kPrefixCtas + units - 1) / units + 1);
  return all_in_use && p.way[0].row_tiles % 2 == 0 ? most : 2 * most;
}

template <int D>
cudaError_t prefix_part(const PrefixArgs& x, const Plan& p, bool decode, cudaStream_t st) {
  using C = Cfg<D>;
  Params a{};
  a.p = p;
  a.sums = static_cast<float4*>(x.ws);
  a.stats = reinterpret_cast<float2*>(static_cast<char*>(x.ws) + sums_bytes(p, D));
  a.lens = decode ? nullptr : x.lens;
  a.tile_of = reinterpret_cast<int*>(static_cast<char*>(x.ws) + sums_bytes(p, D) + stats_bytes(p));
  a.place = a.tile_of + p.most_tiles();
  a.sl2 = x.scale * kLog2;
  CUtensorMap mq[2], mk, mv;
  for (int w = 0; w < 2; ++w) {
    const Boxes c = p.boxes(w);
    if (!map_view_box(&mq[w], x.q.p, x.q.sb, x.q.sh, x.q.sn, p.B, p.nh, p.nq, D, c.tq, c.tg, c.tb))
      return cudaErrorInvalidValue;
  }
  if (!map_view(&mk, x.kp.p, x.kp.sb, x.kp.sh, x.kp.sn, 1, p.nkv, p.P, D) ||
      !map_view(&mv, x.vp.p, x.vp.sb, x.vp.sh, x.vp.sn, 1, p.nkv, p.P, D))
    return cudaErrorInvalidValue;
  auto kern = a.lens ? prefix_tc_kernel<D, true> : prefix_tc_kernel<D, false>;
  const cudaError_t e = set_max_dynamic_smem((const void*)kern, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(Deal(p, p.most_tiles()).ctas), dim3(C::kThreads), C::SMEM, st, mq[0], mq[1], mk, mv, a);
}

template <int D>
cudaError_t run(const PrefixArgs& x, bool decode, cudaStream_t st) {
  const Plan p = make_plan(x.s, !decode && x.lens);
  char* ws = static_cast<char*>(x.ws);
  const int* tiles = reinterpret_cast<const int*>(ws + sums_bytes(p, D) + stats_bytes(p));
  float* own = reinterpret_cast<float*>(ws + sums_bytes(p, D) + stats_bytes(p) + tiles_bytes(p));
  cudaError_t e;
  JoinArgs j{};
  j.p = p;
  j.sums = reinterpret_cast<const float4*>(ws);
  j.stats = reinterpret_cast<const float2*>(ws + sums_bytes(p, D));
  j.place = !decode && x.lens ? tiles + p.most_tiles() : nullptr;
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
    const DecodeRuns r = decode_runs(w);
    j.own = own;
    j.run = r.run;
    j.parts = r.parts;
  } else {
    WindowArgs<__nv_bfloat16> f{};
    f.w = w;
    f.q = x.q;
    f.k = x.k;
    f.v = x.v;
    f.lse = own + (size_t)p.B * p.nh * p.nq * D;
    f.scale = x.scale;
    e = launch_window_fwd_raw(f, own, D, st);
    j.own = own;
    j.own_lse = f.lse;
    j.lse = x.lse;
  }
  if (e != cudaSuccess) return e;
  e = prefix_part<D>(x, p, decode, st);
  if (e != cudaSuccess) return e;
  // Rows are few when decoding: their channels go to several CTAs then, each of which reads the
  // statistics (64 tokens behind 16384 keys, own caches of 1024: 91 us in all, 106 with whole rows).  Where
  // rows fill the SMs that costs more than it gives (16 prompts of 39 to 77 tokens behind 8192 keys: 175
  // us instead of 151).
  const int groups = p.nkv * p.most_tiles() * (kTile / kJoinRows), smem = sums_at_most(p, !j.place) * kJoinRows * (int)sizeof(float2);
  auto kern = groups >= 304 ? (decode ? prefix_join_kernel<D, D, true> : prefix_join_kernel<D, D, false>)
                            : (decode ? prefix_join_kernel<D, 32, true> : prefix_join_kernel<D, 32, false>);
  e = set_max_dynamic_smem((const void*)kern, 2 * kPrefixCtas * kJoinRows * (int)sizeof(float2));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(groups / p.nkv, groups >= 304 ? 1 : D / 32, p.nkv), dim3(kJoinThreads), smem, st, j);
}

}  // namespace

size_t prefix_ws_bytes(const PrefixShape& x, int d) {
  const Plan p = make_plan(x, true);  // (its tiles are no fewer than those without lengths)
  const size_t sums = sums_bytes(p, d) + stats_bytes(p) + tiles_bytes(p);
  const Window w{x.B, x.nh, x.nkv, x.nq, x.nk, x.nk, 0, 0, nullptr};
  const size_t own = x.nq == 1 ? decode_parts_ws_bytes(w, d) : 0;
  return round256(sums + std::max(own, (size_t)x.B * x.nh * x.nq * (d + 1) * 4));
}

cudaError_t launch_prefix_attn(const PrefixArgs& a, int d, bool decode, cudaStream_t st) {
  return d == 64 ? run<64>(a, decode, st) : run<128>(a, decode, st);
}

}  // namespace psa
