// window_weights.cu -- what each key of a prompt got of the attention: the column sums of the
// probabilities, on tensor cores (tcgen05, bf16).
//
//   weights[hk, j] += sum over the query heads h of hk and the queries i that see key j of
//                     2^(scale log2(e) q_hi . k_j - log2(e) lse_hi)
//
// The forward has left lse, so one product and one exponential per visible pair remain.  Keys are
// the product's rows (S^T = K Q^T): a thread owns a key, and its sum over the queries stays in a
// register, with no exchange between lanes and no atomics.
//
// Per 128 x 128 tile at head dim 128 the product takes 512 cycles of the tensor pipe, as many of
// shared memory's bandwidth for its operands, and the exponentials 512 of the multi-function
// units; a warp that goes through 128 scores spends most of its time on latencies.  So four key
// tiles, each with four warps and a score tile, share the query tiles that stream by: four warps a
// scheduler fill one another's gaps, and a query tile is read from the L2 once for four products.
// Measured, 2 x 4096 causal, 16 heads of 128 on 4, on the device: 76 us (0.91 PFLOP/s of visible
// pairs, 0.47 of cuBLAS's bf16 rate; tensor pipe and multi-function units busy 46 % each, a step's
// four products and the waits between them are what is left).  Two key tiles with their operand in
// tensor memory and a ring of three score tiles: 86 us with four warps a tile, 79 with eight, and
// more barriers; with barriers that every thread arrives at instead of one lane a warp 85 us.
//   warps 0-15       sums, four warps for each key tile: one thread per key
//   warp 16          TMA producer: key tiles, a ring of query tiles
//   warp 17          issuer of the products (converged), tensor memory
// A unit is four key tiles of a list (sequence and key/value head), its steps the query tiles that
// see one of them.  All units' steps, one behind another, are cut into equal runs, one for each
// CTA (counted on the device: lengths decide); a run's sums of a unit are a piece of their own, and a
// second kernel adds a unit's pieces to the weights in order.
// A tile of queries holds 128 of one head; of fewer queries than that, several heads.
#include <algorithm>

#include "window_tc.cuh"

namespace psa {
namespace {

constexpr int kTiles = 4;  // key tiles of a unit
constexpr int kUnitKeys = kTiles * kTile;
constexpr int kWeightCtas = 152;  // a run for each SM; the same on a part with fewer of them, so that bits are too

template <int D>
struct Cfg {
  static constexpr int kWarps = 4 * kTiles + 2, kThreads = 32 * kWarps, kProducer = 4 * kTiles, kIssuer = kProducer + 1;
  static constexpr int QST = D == 128 ? 2 : 6;
  static constexpr uint32_t TILE = kTileBytes<D>;
  static constexpr uint32_t OFF_K = QST * TILE, OFF_LSE = OFF_K + kTiles * TILE;
  static constexpr uint32_t OFF_BAR = OFF_LSE + 8 * kTiles * kTile * 4, SMEM = OFF_BAR + 512 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};
struct Bars {
  uint64_t k_full[kTiles], k_empty[kTiles], q_full[8], q_empty[8], s_full[kTiles], s_empty[kTiles], done;
};

struct Params {
  Window w;
  const float* lse;
  float* pieces;  // [units + kWeightCtas][kUnitKeys]: piece of unit u and CTA c at u + c
  int2* spans;    // [units]: first and last CTA that has a piece
  float sl2;      // scale * log2(e)
  int tq, tg;     // queries and heads of a query tile
  int q_shift;    // i >> q_shift: the query tile of query i (128 queries, or all of them)
  int group, head_tiles;
  int key_units, units;
};

struct Unit {
  int list, b, hk, k0, len;
  int tile0, tiles, steps;  // query tiles that hold a row that sees a key of the unit, times head tiles
  __device__ __forceinline__ Unit(const Params& a, int u) {
    const Window& w = a.w;
    list = u / a.key_units;
    k0 = (u - list * a.key_units) * kUnitKeys;
    b = list / w.nkv;
    hk = list - b * w.nkv;
    len = w.len(b);
    int last;
    range(a, k0, kUnitKeys, tile0, last);
    tiles = last - tile0 + 1;
    steps = tiles * a.head_tiles;
  }
  // query tiles first .. last hold a row that sees one of n keys (none: 0 .. -1)
  __device__ __forceinline__ void range(const Params& a, int key, int n, int& first, int& last) const {
    int i0, rows;
    query_range(a.w, len, key, min(key + n, a.w.nk) - 1, i0, rows);
    first = rows > 0 ? i0 >> a.q_shift : 0;
    last = rows > 0 ? (i0 + rows - 1) >> a.q_shift : -1;
  }
};

// A CTA's run of steps: piece by piece.
struct Run {
  int unit, s, n;  // steps s .. s + n - 1 of `unit`
  long long left;
  // on to the next piece
  __device__ __forceinline__ bool next(const Params& a) {
    unit += n > 0;
    s = n > 0 ? 0 : s;
    if (left <= 0) return false;
    int steps = 0;
    while (unit < a.units && (steps = Unit(a, unit).steps) == 0) ++unit;
    if (unit >= a.units) return false;  // (lengths that changed since they were counted)
    n = (int)min((long long)(steps - s), left);
    left -= n;
    return true;
  }
};

// A place in a ring of N, and how often it has been there (its parity).
template <int N>
struct Place {
  int at = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      parity ^= 1;
    }
  }
};

// A step of a unit: a tile of heads, a tile of queries.
struct Step {
  int qt, ht;
  __device__ __forceinline__ Step(const Unit& u, int s) {
    ht = s / u.tiles;
    qt = u.tile0 + s - ht * u.tiles;
  }
  __device__ __forceinline__ void next(const Unit& u) {
    if (++qt == u.tile0 + u.tiles) {
      qt = u.tile0;
      ++ht;
    }
  }
};

// The query tiles that see one of a unit's key tiles.
struct KeyTile {
  int first, last;
  __device__ __forceinline__ KeyTile(const Params& a, const Unit& u, int i) {
    u.range(a, u.k0 + i * kTile, kTile, first, last);
  }
  __device__ __forceinline__ bool any() const { return last >= first; }
  __device__ __forceinline__ bool takes(int query_tile) const { return query_tile >= first && query_tile <= last; }
};

// Four neighbouring columns' statistics (a pointer that comes of an aligned base would be read as
// a generic one, with a global load's latency).
__device__ __forceinline__ float4 shared4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}

__device__ __forceinline__ void shared16x4(uint32_t at, float4 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = shared4(at + 16 * i);
}

// Sum of 2^(x sl + l) over 16 scores.
__device__ __forceinline__ void add16(const uint32_t* x, const float4 (&l)[4], float2 sl, float2& s01, float2& s23) {
  float2 y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = __ffma2_rn(make_float2(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1])), sl, make_float2(l[i].x, l[i].y));
    y[2 * i + 1] = __ffma2_rn(make_float2(__uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3])), sl, make_float2(l[i].z, l[i].w));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = make_float2(fast_exp2(y[i].x), fast_exp2(y[i].y));
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    s01 = __fadd2_rn(s01, y[i]);
    s23 = __fadd2_rn(s23, y[i + 1]);
  }
}

// The same over those of 32 scores whose bit in `see` is set (what others and their statistics hold
// does not matter); l: shared address of the columns' statistics.
__device__ __forceinline__ void add_seen(const uint32_t* x, uint32_t l, float2 sl, uint32_t see, float2& s01, float2& s23) {
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    const float4 n = shared4(l + 4 * k);
    const float2 a = __ffma2_rn(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), sl, make_float2(n.x, n.y));
    const float2 c = __ffma2_rn(make_float2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3])), sl, make_float2(n.z, n.w));
    float p[4] = {fast_exp2(a.x), fast_exp2(a.y), fast_exp2(c.x), fast_exp2(c.y)};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (!(see & (1u << (k + e)))) p[e] = 0.f;
    s01 = __fadd2_rn(s01, make_float2(p[0], p[1]));
    s23 = __fadd2_rn(s23, make_float2(p[2], p[3]));
  }
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    window_weights_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                             const Params a) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ long long before[C::kWarps];
  __shared__ int2 start;
  unsigned char* smem = align1024(smem_raw);
  const uint32_t sbase = smem_addr(smem);
  Bars& bar = *reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(&bar + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_at + 1);
  static_assert(sizeof(Bars) + 16 <= 512, "barriers");
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.s_empty[i], 4);  // one arrival per warp
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&bar.q_full[i], 1);
      mbar_init(&bar.q_empty[i], 1);
    }
    mbar_init(&bar.done, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == C::kIssuer) {
    tmem_alloc(tmem_at, 512);
    tmem_relinquish();
  }
  pdl_launch_dependents();
  pdl_wait();
  // ---- where this CTA's run begins: every thread counts a run of units
  Run run;
  {
    const int per = (a.units + C::kThreads - 1) / C::kThreads;
    const int from = min(a.units, (int)threadIdx.x * per), to = min(a.units, from + per);
    long long mine = 0;
    for (int u = from; u < to; ++u) mine += Unit(a, u).steps;
    long long upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += y;
    }
    if (lane == 31) before[warp] = upto;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long all = 0;
#pragma unroll
    for (int i = 0; i < C::kWarps; ++i) {
      upto += i < warp ? before[i] : 0;
      all += before[i];
    }
    // (no CTA in front of the last one with a run has none: a unit's pieces are its span's)
    const long long ctas = min((long long)gridDim.x, all), c = blockIdx.x;
    const long long begin = c < ctas ? all * c / ctas : 0, end = c < ctas ? all * (c + 1) / ctas : 0;
    if (begin < end && upto - mine <= begin && begin < upto) {
      long long at = upto - mine;
      int u = from, n;
      while (at + (n = Unit(a, u).steps) <= begin) {
        at += n;
        ++u;
      }
      start = make_int2(u, (int)(begin - at));
    }
    __syncthreads();
    run = Run{start.x, start.y, 0, end - begin};
  }
  const uint32_t tmem = *tmem_at;

  if (warp == C::kProducer) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      const uint32_t q_bytes = (uint32_t)(a.tq * a.tg * D * 2);
      tma_prefetch_desc(&tmK);
      bool ok = true;
      int qn = 0, kn[kTiles] = {};
      while (ok && run.next(a)) {
        const Unit u(a, run.unit);
        Step t(u, run.s);
        for (int i = 0; ok && i < run.n; ++i, ++qn, t.next(u)) {
          const int qs = qn % C::QST;
          if (qn >= C::QST && !mbar_wait(&bar.q_empty[qs], (qn / C::QST - 1) & 1, abort)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bar.q_full[qs], q_bytes);
          const int h = u.hk * a.group + t.ht * a.tg;
          load_tile<D>(smem + qs * C::TILE, &tmQ, &bar.q_full[qs], t.qt * a.tq, h, u.b);
          if (i > 0) continue;
          // the unit's keys, each as soon as the products with the last one's are done
#pragma unroll
          for (int w = 0; w < kTiles; ++w) {
            if (!ok || !KeyTile(a, u, w).any()) continue;
            if (kn[w] > 0 && !mbar_wait(&bar.k_empty[w], (kn[w] - 1) & 1, abort)) {
              ok = false;
              continue;
            }
            mbar_arrive_expect_tx(&bar.k_full[w], C::TILE);
            load_tile<D>(smem + C::OFF_K + w * C::TILE, &tmK, &bar.k_full[w], u.k0 + w * kTile, u.hk, u.b);
            ++kn[w];
          }
        }
      }
      if (*abort) {
        // let the copies in flight land before the CTA exits
#pragma unroll
        for (int w = 0; w < kTiles; ++w)
          if (kn[w] > 0) drain_wait(&bar.k_full[w], (kn[w] - 1) & 1);
        for (int n = max(0, qn - C::QST); n < qn; ++n) drain_wait(&bar.q_full[n % C::QST], (n / C::QST) & 1);
      }
    }
  } else if (warp == C::kIssuer) {
    // ------------------------------------------------------------ issuer (converged warp)
    const uint64_t dQ0 = desc_rows_by_channels(sbase), dK0 = desc_rows_by_channels(sbase + C::OFF_K);
    const uint32_t id = idesc_bf16_f32(128, (a.tq * a.tg + 15) / 16 * 16, false, false);
    bool ok = true;
    uint32_t k_parity[kTiles] = {}, s_parity[kTiles] = {};
    Place<C::QST> q;
    while (ok && run.next(a)) {
      const Unit u(a, run.unit);
      const KeyTile tile[kTiles] = {KeyTile(a, u, 0), KeyTile(a, u, 1), KeyTile(a, u, 2), KeyTile(a, u, 3)};
      Step t(u, run.s);
      for (int i = 0; ok && i < run.n; ++i, t.next(u)) {
        if (!mbar_wait(&bar.q_full[q.at], q.parity, abort)) {
          ok = false;
          break;
        }
        const uint64_t dQ = dQ0 + (uint64_t)(q.at * C::TILE >> 4);
#pragma unroll
        for (int w = 0; w < kTiles; ++w) {
          if (!ok || !tile[w].any()) continue;
          // (every key tile that was loaded is waited for, whether this piece's steps need it or not)
          if (i == 0 && !mbar_wait(&bar.k_full[w], k_parity[w], abort)) {
            ok = false;
            continue;
          }
          if (!tile[w].takes(t.qt)) continue;
          // (the first use waits for nothing: its barrier's phase before the first is over)
          if (!mbar_wait(&bar.s_empty[w], s_parity[w] ^ 1, abort)) {
            ok = false;
            continue;
          }
          tc_fence_after();
          const uint64_t dK = dK0 + (uint64_t)(w * C::TILE >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_warp(tmem + 128 * w, dK + kstep_channels(kk), dQ + kstep_channels(kk), id, kk > 0 ? 1u : 0u);
          mma_commit_warp(&bar.s_full[w]);
          s_parity[w] ^= 1;
        }
        if (ok) mma_commit_warp(&bar.q_empty[q.at]);
        q.next();
      }
#pragma unroll
      for (int w = 0; w < kTiles; ++w)
        if (ok && tile[w].any()) {
          mma_commit_warp(&bar.k_empty[w]);
          k_parity[w] ^= 1;
        }
    }
    mma_commit_warp(&bar.done);
    drain_wait(&bar.done, 0);
  } else {
    // ------------------------------------------------------------ sums over the queries
    using Chunk = uint32_t[32];
    const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem + 128 * wg + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t stats = sbase + C::OFF_LSE + warp * 2 * kTile * 4;  // this warp's, of two steps
    const Window& w = a.w;
    const int off = w.nk - w.nq, group = a.group, rows = a.tq * a.tg;
    int my_g[4], my_i[4];  // columns lane + 32 x, whose statistics this lane fetches
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      my_g[x] = (lane + 32 * x) / a.tq;
      my_i[x] = lane + 32 * x - my_g[x] * a.tq;
      if (lane + 32 * x >= rows) my_g[x] = 1 << 20;  // none
    }
    const float2 sl = make_float2(a.sl2, a.sl2);
    uint32_t parity = 0, flip = 0;
    bool ok = true;
    while (ok && run.next(a)) {
      const Unit u(a, run.unit);
      const int k0 = u.k0 + wg * kTile, j = k0 + r, k1 = k0 + kTile - 1;
      const KeyTile tile(a, u, wg);
      // queries that see this thread's key
      const int lo = max(max(j - w.right, 0) - off, 0);
      const int hi = min((j < w.sinks ? u.len - 1 : min(u.len - 1, j + w.left)) - off, w.nq - 1);
      // query tiles that every key of the tile sees whole: first_whole .. last_whole
      int first_whole = 1, last_whole = 0;
      if (rows == kTile) {
        const int from = max(max(0, k1 - w.right) - off, 0);
        const int to = min(min(k1 < w.sinks ? u.len - 1 : k0 + w.left, u.len - 1) - off, w.nq - 1);
        first_whole = a.tq < kTile ? from > 0 : (from + kTile - 1) / kTile;
        last_whole = a.tq < kTile ? (to >= w.nq - 1 ? 0 : -1) : ((to + 1) >> 7) - 1;
      }
      // the lane's columns of a step: lse, or (the product below is then -infinity) infinity
      float lse[4] = {0.f, 0.f, 0.f, 0.f};
      const float* list_lse = a.lse + ((long long)u.b * w.nh + u.hk * group) * w.nq;
      auto fetch = [&](const Step& t) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int q = t.qt * a.tq + my_i[x], g = t.ht * a.tg + my_g[x];
          lse[x] = g < group && q < w.nq ? list_lse[(long long)g * w.nq + q] : INFINITY;
        }
      };
      float sum = 0.f;
      Step t(u, run.s);
      int i = 0;
      // on to the next step that this key tile takes part in
      auto seek = [&]() {
        while (i < run.n && !tile.takes(t.qt)) {
          ++i;
          t.next(u);
        }
      };
      seek();
      if (i < run.n) fetch(t);
      while (i < run.n) {
        const uint32_t l = stats + flip;
        flip ^= kTile * 4;
#pragma unroll
        for (int x = 0; x < 4; ++x) st_shared_f32(l + 4 * (lane + 32 * x), -kLog2 * lse[x]);
        __syncwarp();
        const Step now = t;
        const bool whole = t.qt >= first_whole && t.qt <= last_whole && (t.ht + 1) * a.tg <= group;
        ++i;
        t.next(u);
        seek();
        if (i < run.n) fetch(t);  // on its way during this step
        if (!mbar_wait(&bar.s_full[wg], parity, abort)) {
          ok = false;
          break;
        }
        parity ^= 1;
        tc_fence_after();
        float2 s01 = make_float2(0.f, 0.f), s23 = s01;
        if (whole) {
#pragma unroll
          for (int c = 0; c < kTile; c += 32) {
            uint32_t x[32];
            float4 l0[4];
            tmem_load32_async(tS + c, x);
            shared16x4(l + 4 * c, l0);
            tmem_wait_ld();
            tmem_pin(x);
            if (c + 32 == kTile) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar.s_empty[wg]);
            }
            add16(x, l0, sl, s01, s23);
            shared16x4(l + 4 * c + 64, l0);
            add16(x + 16, l0, sl, s01, s23);
          }
        } else {
          const int q0 = now.qt * a.tq, heads = min(a.tg, group - now.ht * a.tg);
          const int from = max(0, lo - q0), to = min(a.tq - 1, hi - q0);
#pragma unroll 1
          for (int c = 0; c < rows; c += 32) {
            uint32_t x[32];
            tmem_load32_async(tS + c, x);
            uint32_t see = 0;
            const int last = min(heads - 1, (c + 31) / a.tq);
            if (from <= to)
              for (int g = c / a.tq; g <= last; ++g) see |= visible32(g * a.tq + from - c, g * a.tq + to - c, 0);
            tmem_wait_ld();
            tmem_pin(x);
            add_seen(x, l + 4 * c, sl, see, s01, s23);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.s_empty[wg]);
        }
        sum += (s01.x + s01.y) + (s23.x + s23.y);
      }
      if (!ok) break;
      a.pieces[((long long)run.unit + blockIdx.x) * kUnitKeys + wg * kTile + r] = sum;
      if (threadIdx.x == 0) {
        if (run.s == 0) a.spans[run.unit].x = blockIdx.x;
        if (run.s + run.n == u.steps) a.spans[run.unit].y = blockIdx.x;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds the pieces of every key inside its sequence, in order.
__global__ void __launch_bounds__(kUnitKeys) window_weights_add_kernel(const Params a, float* weights) {
  pdl_launch_dependents();
  pdl_wait();
  const int unit = blockIdx.x;
  const Unit u(a, unit);
  const int j = u.k0 + threadIdx.x;
  if (u.steps == 0 || j >= u.len) return;
  const int2 span = a.spans[unit];
  float s = 0.f;
  for (int c = span.x; c <= span.y; ++c) s += a.pieces[((long long)unit + c) * kUnitKeys + threadIdx.x];
  weights[(long long)u.list * a.w.nk + j] += s;
}

void query_tile(const Window& w, int& tq, int& tg) {
  tq = std::min(w.nq, kTile);
  tg = std::min(w.nh / w.nkv, kTile / tq);
}

template <int D>
cudaError_t weights(const Window& w, View<const __nv_bfloat16> q, View<const __nv_bfloat16> k, const float* lse,
                    float* out, float* ws, float scale, cudaStream_t st) {
  using C = Cfg<D>;
  Params a{};
  a.w = w;
  a.lse = lse;
  a.sl2 = scale * kLog2;
  query_tile(w, a.tq, a.tg);
  a.q_shift = a.tq == kTile ? 7 : 31;
  a.group = w.nh / w.nkv;
  a.head_tiles = (a.group + a.tg - 1) / a.tg;
  a.key_units = (w.nk + kUnitKeys - 1) / kUnitKeys;
  a.units = w.B * w.nkv * a.key_units;
  a.pieces = ws;
  a.spans = reinterpret_cast<int2*>(ws + ((size_t)a.units + kWeightCtas) * kUnitKeys);
  CUtensorMap mq, mk;
  if (!map_view_box(&mq, q.p, q.sb, q.sh, q.sn, w.B, w.nh, w.nq, D, a.tq, a.tg, 1) ||
      !map_view(&mk, k.p, k.sb, k.sh, k.sn, w.B, w.nkv, w.nk, D))
    return cudaErrorInvalidValue;
  auto kern = window_weights_tc_kernel<D>;
  cudaError_t e = set_max_dynamic_smem((const void*)kern, C::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(kWeightCtas), dim3(C::kThreads), C::SMEM, st, mq, mk, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(window_weights_add_kernel, dim3(a.units), dim3(kUnitKeys), 0, st, a, out);
}

}  // namespace

size_t window_weights_ws_bytes(const Window& w) {
  const size_t units = (size_t)w.B * w.nkv * ((w.nk + kUnitKeys - 1) / kUnitKeys);
  return (units + kWeightCtas) * kUnitKeys * 4 + units * 8;
}

cudaError_t launch_window_weights(const Window& w, View<const __nv_bfloat16> q, View<const __nv_bfloat16> k,
                                  const float* lse, float* weights_out, float* ws, float scale, int d,
                                  cudaStream_t st) {
  return d == 64 ? weights<64>(w, q, k, lse, weights_out, ws, scale, st)
                 : weights<128>(w, q, k, lse, weights_out, ws, scale, st);
}

}  // namespace psa
