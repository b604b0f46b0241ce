// window_weights.cu -- what each key of a prompt got of the attention: the column sums of the
// probabilities, on tensor cores (tcgen05, bf16).
//
//   weights[hk, j] += sum over the query heads h of hk and the queries i that see key j of
//                     2^(scale log2(e) q_hi . k_j - log2(e) lse_hi)
//
// The forward has left lse, so one product and one exponential per visible pair remain.  Keys are
// the product's rows (S^T = K Q^T): a thread owns a key, and its sum over the queries stays in a
// register, with no exchange between lanes and no atomics.  Per 128 x 128 tile at head dim 128
// the product takes 512 cycles of the tensor pipe and the exponentials 512 of the multi-function
// units.  Four key tiles stay in shared memory, each with a score tile in tensor memory and four
// warps, and share the query tiles that stream by.
//   warps 0-15       sums, four warps for each key tile: one thread per key
//   warp 16          TMA producer: key tiles, a ring of query tiles
//   warp 17          issuer of the products (converged), tensor memory
// A unit is four key tiles of a list (sequence and key/value head) and one of `parts` equal parts of
// the query tiles that see it; its sums go to the workspace, and a second kernel adds them to the
// weights in order.  Units go from those with most steps to those with fewest over the CTAs.
// A tile of queries holds 128 of one head; of fewer queries than that, several heads.
#include <algorithm>

#include "window_tc.cuh"

namespace psa {
namespace {

constexpr int kTiles = 4;               // key tiles of a unit
constexpr int kUnitKeys = kTiles * kTile;

template <int D>
struct Cfg {
  static constexpr int kThreads = 32 * (4 * kTiles + 2), kProducer = 4 * kTiles, kIssuer = kProducer + 1;
  static constexpr int QST = D == 128 ? 2 : 6;
  static constexpr uint32_t TILE = kTileBytes<D>;
  static constexpr uint32_t OFF_Q = kTiles * TILE, OFF_LSE = OFF_Q + QST * TILE;
  static constexpr uint32_t OFF_BAR = OFF_LSE + 2 * kTiles * kTile * 4, SMEM = OFF_BAR + 512 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};
struct Bars {
  uint64_t k_full[kTiles], k_empty[kTiles], q_full[8], q_empty[8], s_full[kTiles], s_empty[kTiles];
  uint64_t stats[2 * kTiles], done;
};

struct Params {
  Window w;
  const float* lse;
  float* ws;
  float sl2;        // scale * log2(e)
  int tq, tg;       // queries and heads of a query tile
  int parts, units;
};

struct Unit {
  int list, b, hk, k0, len, part;
  int tile0, tiles;  // query tiles that hold a row that sees a key of the unit
  int from, steps;   // of the unit's part; step s: head tile s / tiles, query tile s % tiles
  __device__ __forceinline__ Unit(const Params& a, int u) {
    const Window& w = a.w;
    const int lists = w.B * w.nkv;
    list = u % lists;
    const int x = u / lists;  // key tiles in order: in a causal problem the first are seen by most
    part = x % a.parts;
    k0 = x / a.parts * kUnitKeys;
    b = list / w.nkv;
    hk = list % w.nkv;
    len = w.len(b);
    int last;
    range(a, k0, kUnitKeys, tile0, last);
    tiles = last - tile0 + 1;
    const int all = tiles * ((w.nh / w.nkv + a.tg - 1) / a.tg);
    from = (int)((long long)all * part / a.parts);
    steps = (int)((long long)all * (part + 1) / a.parts) - from;
  }
  // query tiles first .. last hold a row that sees one of n keys (none: last < first)
  __device__ __forceinline__ void range(const Params& a, int key, int n, int& first, int& last) const {
    int i0, rows;
    query_range(a.w, len, key, min(key + n, a.w.nk) - 1, i0, rows);
    first = rows > 0 ? i0 / a.tq : 0;
    last = rows > 0 ? (i0 + rows - 1) / a.tq : -1;
  }
};

// A step of a unit: a tile of heads, a tile of queries.
struct Step {
  int s, qt, ht;
  __device__ __forceinline__ explicit Step(const Unit& u) : s(0) {
    ht = u.tiles > 0 ? u.from / u.tiles : 0;
    qt = u.tile0 + u.from - ht * u.tiles;
  }
  __device__ __forceinline__ void next(const Unit& u) {
    ++s;
    if (++qt == u.tile0 + u.tiles) {
      qt = u.tile0;
      ++ht;
    }
  }
};

// One of a unit's key tiles: the query tiles that see it, and whether the part has one of them.
struct KeyTile {
  int first, last;
  bool used;
  __device__ __forceinline__ KeyTile(const Params& a, const Unit& u, int i) {
    u.range(a, u.k0 + i * kTile, kTile, first, last);
    used = false;
    if (last < first || u.steps == 0) return;
    // the part's query tiles go round from `at`
    const int at = Step(u).qt, end = at + u.steps - 1, round = u.tiles;
    used = u.steps >= round || (first <= end && last >= at) || (first + round <= end && last + round >= at);
  }
  __device__ __forceinline__ bool takes(int query_tile) const { return query_tile >= first && query_tile <= last; }
};

__device__ __forceinline__ int unit_of(int i) {
  return i * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// Four neighbouring columns' statistics (a pointer that comes of an aligned base would be read as
// a generic one, with a global load's latency).
__device__ __forceinline__ float4 shared4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}

// Sum of 2^(x sl + l) over 32 scores, or those whose bit in `see` is set (what others and their
// statistics hold does not matter); l: shared address of the columns' statistics.
template <bool kMasked>
__device__ __forceinline__ void add32(const uint32_t* x, uint32_t l, float2 sl, float2& s01, float2& s23,
                                      uint32_t see = 0) {
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    const float4 n = shared4(l + 4 * k);
    const float2 a = __ffma2_rn(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), sl, make_float2(n.x, n.y));
    const float2 c = __ffma2_rn(make_float2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3])), sl, make_float2(n.z, n.w));
    float p[4] = {fast_exp2(a.x), fast_exp2(a.y), fast_exp2(c.x), fast_exp2(c.y)};
    if constexpr (kMasked)
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
      mbar_init(&bar.s_empty[i], kTile);
      mbar_init(&bar.stats[2 * i], kTile);
      mbar_init(&bar.stats[2 * i + 1], kTile);
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
      const uint32_t q_bytes = (uint32_t)(a.tq * a.tg * D * 2);
      bool ok = true;
      int kn[kTiles] = {}, qn = 0;
      for (int i = 0; ok && unit_of(i) < a.units; ++i) {
        const Unit u(a, unit_of(i));
        for (Step t(u); ok && t.s < u.steps; t.next(u), ++qn) {
          const int qs = qn % C::QST;
          if (qn >= C::QST && !mbar_wait(&bar.q_empty[qs], (qn / C::QST - 1) & 1, abort)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bar.q_full[qs], q_bytes);
          const int h = u.hk * (a.w.nh / a.w.nkv) + t.ht * a.tg;
          load_tile<D>(smem + C::OFF_Q + qs * C::TILE, &tmQ, &bar.q_full[qs], t.qt * a.tq, h, u.b);
          if (t.s > 0) continue;
          // the unit's keys, each as soon as the last unit's products are done with its place
#pragma unroll
          for (int w = 0; w < kTiles; ++w) {
            if (!ok || !KeyTile(a, u, w).used) continue;
            if (kn[w] > 0 && !mbar_wait(&bar.k_empty[w], (kn[w] - 1) & 1, abort)) {
              ok = false;
              continue;
            }
            mbar_arrive_expect_tx(&bar.k_full[w], C::TILE);
            load_tile<D>(smem + w * C::TILE, &tmK, &bar.k_full[w], u.k0 + w * kTile, u.hk, u.b);
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
    const uint64_t dK0 = desc_rows_by_channels(sbase), dQ0 = desc_rows_by_channels(sbase + C::OFF_Q);
    const uint32_t id = idesc_bf16_f32(128, (a.tq * a.tg + 15) / 16 * 16, false, false);
    bool ok = true;
    int kn[kTiles] = {}, sn[kTiles] = {}, qn = 0;
    for (int i = 0; ok && unit_of(i) < a.units; ++i) {
      const Unit u(a, unit_of(i));
      if (u.steps == 0) continue;
      const KeyTile tile[kTiles] = {KeyTile(a, u, 0), KeyTile(a, u, 1), KeyTile(a, u, 2), KeyTile(a, u, 3)};
      for (Step t(u); ok && t.s < u.steps; t.next(u), ++qn) {
        const int qs = qn % C::QST;
        if (!mbar_wait(&bar.q_full[qs], (qn / C::QST) & 1, abort)) {
          ok = false;
          break;
        }
        const uint64_t dQ = dQ0 + (uint64_t)(qs * C::TILE >> 4);
#pragma unroll
        for (int w = 0; w < kTiles; ++w) {
          if (!ok || !tile[w].takes(t.qt)) continue;
          // (a phase that has completed already costs one test)
          if (!mbar_wait(&bar.k_full[w], kn[w] & 1, abort) ||
              (sn[w] > 0 && !mbar_wait(&bar.s_empty[w], (sn[w] - 1) & 1, abort))) {
            ok = false;
            continue;
          }
          tc_fence_after();
          const uint64_t dK = dK0 + (uint64_t)(w * C::TILE >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_warp(tmem + 128 * w, dK + kstep_channels(kk), dQ + kstep_channels(kk), id, kk > 0 ? 1u : 0u);
          mma_commit_warp(&bar.s_full[w]);
          ++sn[w];
        }
        if (ok) mma_commit_warp(&bar.q_empty[qs]);
      }
      if (!ok) break;
#pragma unroll
      for (int w = 0; w < kTiles; ++w)
        if (tile[w].used) {
          mma_commit_warp(&bar.k_empty[w]);
          ++kn[w];
        }
    }
    mma_commit_warp(&bar.done);
    drain_wait(&bar.done, 0);
  } else {
    // ------------------------------------------------------------ sums over the queries
    const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem + 128 * wg + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t stats = sbase + C::OFF_LSE + wg * 2 * kTile * 4;
    const Window& w = a.w;
    const int off = w.nk - w.nq, group = w.nh / w.nkv, rows = a.tq * a.tg;
    const int my_g = r / a.tq, my_i = r % a.tq;  // the column whose statistics this thread fetches
    const float2 sl = make_float2(a.sl2, a.sl2);
    bool ok = true;
    int used = 0;
    for (int i = 0; ok && unit_of(i) < a.units; ++i) {
      const Unit u(a, unit_of(i));
      const int k0 = u.k0 + wg * kTile, j = k0 + r, k1 = k0 + kTile - 1;
      if (k0 >= w.nk) continue;
      const KeyTile tile(a, u, wg);
      // queries that see this thread's key
      const int lo = max(max(j - w.right, 0) - off, 0);
      const int hi = min((j < w.sinks ? u.len - 1 : min(u.len - 1, j + w.left)) - off, w.nq - 1);
      // on to the part's next step that this key tile takes part in
      auto seek = [&](Step& t) {
        while (t.s < u.steps && !tile.takes(t.qt)) t.next(u);
      };
      // this thread's column of a step: lse, or (the product below is then -infinity) infinity
      auto fetch = [&](const Step& t) {
        const int q = t.qt * a.tq + my_i, g = t.ht * a.tg + my_g;
        if (r >= rows || g >= group || q >= w.nq) return INFINITY;
        return __ldg(a.lse + ((long long)u.b * w.nh + u.hk * group + g) * w.nq + q);
      };
      float sum = 0.f;
      Step t(u);
      if (!tile.used) t.s = u.steps;
      seek(t);
      float lse = t.s < u.steps ? fetch(t) : 0.f;
      while (t.s < u.steps) {
        const uint32_t l = stats + (used & 1) * kTile * 4;
        uint64_t* ready = &bar.stats[2 * wg + (used & 1)];
        st_shared_f32(l + 4 * r, -kLog2 * lse);
        mbar_arrive(ready);
        const Step now = t;
        t.next(u);
        seek(t);
        if (t.s < u.steps) lse = fetch(t);  // on its way during this step
        const int q0 = now.qt * a.tq;
        const int heads = min(a.tg, group - now.ht * a.tg), p0 = q0 + off, p1 = p0 + a.tq - 1;
        const bool whole = rows == kTile && heads == a.tg && q0 + a.tq <= w.nq && p0 >= 0 && p1 < u.len &&
                           p0 >= k1 - w.right && (p1 <= k0 + w.left || k1 < w.sinks);
        if (!mbar_wait(ready, (used >> 1) & 1, abort) || !mbar_wait(&bar.s_full[wg], used & 1, abort)) {
          ok = false;
          break;
        }
        ++used;
        tc_fence_after();
        float2 s01 = make_float2(0.f, 0.f), s23 = s01;
        if (whole) {
          uint32_t x[64];
          load_cols64(tS, x);
          add32<false>(x, l, sl, s01, s23);
          add32<false>(x + 32, l + 128, sl, s01, s23);
          load_cols64(tS + 64, x);
          tc_fence_before();
          mbar_arrive(&bar.s_empty[wg]);
          add32<false>(x, l + 256, sl, s01, s23);
          add32<false>(x + 32, l + 384, sl, s01, s23);
        } else {
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
            add32<true>(x, l + 4 * c, sl, s01, s23, see);
          }
          tc_fence_before();
          mbar_arrive(&bar.s_empty[wg]);
        }
        sum += (s01.x + s01.y) + (s23.x + s23.y);
      }
      if (!ok) break;
      if (j < w.nk) a.ws[((long long)u.part * w.B * w.nkv + u.list) * w.nk + j] = sum;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds the parts' sums of every key inside its sequence, in order.
__global__ void __launch_bounds__(256)
    window_weights_add_kernel(const Window w, const float* ws, float* weights, int sums) {
  pdl_launch_dependents();
  pdl_wait();
  const int list = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
  if (j >= w.len(list / w.nkv)) return;
  const long long at = (long long)list * w.nk + j, step = (long long)w.B * w.nkv * w.nk;
  float s = 0.f;
  for (int i = 0; i < sums; ++i) s += ws[i * step + at];
  weights[at] += s;
}

// Equal parts of a unit's query tiles, so that no unit is longer than half a CTA's share (the CTAs'
// loads then differ by less than that), but not shorter than four steps.
int unit_parts(const Window& w, int tq, int tg) {
  const long long per = (w.nh / w.nkv + tg - 1) / tg;
  long long all = 0, most = 0;
  for (long long k0 = 0; k0 < w.nk; k0 += kUnitKeys) {
    int i0, n;
    query_range(w, w.nk, (int)k0, (int)std::min<long long>(k0 + kUnitKeys, w.nk) - 1, i0, n);
    const long long steps = n > 0 ? ((i0 + n - 1) / tq - i0 / tq + 1) * per : 0;
    all += steps;
    most = std::max(most, steps);
  }
  const long long share = std::max<long long>(1, all * w.B * w.nkv / 152);
  return (int)std::max<long long>(1, std::min<long long>({(2 * most + share - 1) / share, most / 4, 16}));
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
  a.ws = ws;
  a.sl2 = scale * kLog2;
  query_tile(w, a.tq, a.tg);
  a.parts = unit_parts(w, a.tq, a.tg);
  a.units = w.B * w.nkv * ((w.nk + kUnitKeys - 1) / kUnitKeys) * a.parts;
  CUtensorMap mq, mk;
  if (!map_view_box(&mq, q.p, q.sb, q.sh, q.sn, w.B, w.nh, w.nq, D, a.tq, a.tg, 1) ||
      !map_view(&mk, k.p, k.sb, k.sh, k.sn, w.B, w.nkv, w.nk, D))
    return cudaErrorInvalidValue;
  auto kern = window_weights_tc_kernel<D>;
  cudaError_t e = set_max_dynamic_smem((const void*)kern, C::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(std::min(a.units, device_sm_count())), dim3(C::kThreads), C::SMEM, st, mq, mk, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(window_weights_add_kernel, dim3((w.nk + 255) / 256, w.B * w.nkv), dim3(256), 0, st, w,
                    (const float*)ws, out, a.parts);
}

}  // namespace

size_t window_weights_ws_bytes(const Window& w) {
  int tq, tg;
  query_tile(w, tq, tg);
  return (size_t)unit_parts(w, tq, tg) * w.B * w.nkv * w.nk * 4;
}

cudaError_t launch_window_weights(const Window& w, View<const __nv_bfloat16> q, View<const __nv_bfloat16> k,
                                  const float* lse, float* weights_out, float* ws, float scale, int d,
                                  cudaStream_t st) {
  return d == 64 ? weights<64>(w, q, k, lse, weights_out, ws, scale, st)
                 : weights<128>(w, q, k, lse, weights_out, ws, scale, st);
}

}  // namespace psa
