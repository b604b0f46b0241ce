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
// units; tensor memory holds four score tiles, so that both run all the time.
//   warps 0-3, 4-7   sums of the even and of the odd steps: one thread per key
//   warp 8           TMA producer: key tiles, a ring of query tiles
//   warp 9           issuer of the products (converged), tensor memory
// A unit is a key tile of a list (sequence and key/value head) and one of `parts` equal parts of
// the query tiles that see it; its sums go to the workspace, and a second kernel adds them to the
// weights in order.  Units go from those with most steps to those with fewest over the CTAs.
// A tile of queries holds 128 of one head; of fewer queries than that, several heads.
#include <algorithm>

#include "window_tc.cuh"

namespace psa {
namespace {

template <int D>
struct Cfg {
  static constexpr int kThreads = 320, kProducer = 8, kIssuer = 9;
  static constexpr int KST = D == 128 ? 2 : 4, QST = D == 128 ? 4 : 8;
  static constexpr uint32_t TILE = kTileBytes<D>;
  static constexpr uint32_t OFF_Q = KST * TILE, OFF_LSE = OFF_Q + QST * TILE;
  static constexpr uint32_t OFF_BAR = OFF_LSE + 4 * kTile * 4, SMEM = OFF_BAR + 512 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};
struct Bars {
  uint64_t k_full[4], k_empty[4], q_full[8], q_empty[8], s_full[4], s_empty[4], stats[4], done;
};

struct Params {
  Window w;
  const float* lse;
  float* ws;
  float sl2;                // scale * log2(e)
  int tq, tg;               // queries and heads of a query tile
  int key_tiles, parts, units;
};

struct Unit {
  int list, b, hk, k0, len, part;
  int tile0, tiles;  // query tiles that hold a row that sees a key of the tile
  int from, steps;   // of the unit's part; step s: head tile s / tiles, query tile s % tiles
  __device__ __forceinline__ Unit(const Params& a, int u) {
    const Window& w = a.w;
    const int lists = w.B * w.nkv;
    list = u % lists;
    const int x = u / lists;  // key tiles in order: in a causal problem the first are seen by most
    part = x % a.parts;
    k0 = x / a.parts * kTile;
    b = list / w.nkv;
    hk = list % w.nkv;
    len = w.len(b);
    int i0, n;
    query_range(w, len, k0, min(k0 + kTile, w.nk) - 1, i0, n);
    tile0 = i0 / a.tq;
    tiles = n > 0 ? (i0 + n - 1) / a.tq - tile0 + 1 : 0;
    const int all = tiles * ((w.nh / w.nkv + a.tg - 1) / a.tg);
    from = (int)((long long)all * part / a.parts);
    steps = (int)((long long)all * (part + 1) / a.parts) - from;
  }
};

__device__ __forceinline__ int unit_of(int i) {
  return i * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// Sum of 2^(x sl - l) over 32 scores; l: the columns' statistics in shared memory.
__device__ __forceinline__ void add32(const uint32_t* x, const float* l, float2 sl, float2& s01, float2& s23) {
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    const float4 n = *reinterpret_cast<const float4*>(l + k);
    const float2 a = __ffma2_rn(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), sl, make_float2(n.x, n.y));
    const float2 c = __ffma2_rn(make_float2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3])), sl, make_float2(n.z, n.w));
    s01 = __fadd2_rn(s01, make_float2(fast_exp2(a.x), fast_exp2(a.y)));
    s23 = __fadd2_rn(s23, make_float2(fast_exp2(c.x), fast_exp2(c.y)));
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
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.s_empty[i], kTile);
      mbar_init(&bar.stats[i], kTile);
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
      int kn = 0, qn = 0;
      for (int i = 0; ok && unit_of(i) < a.units; ++i) {
        const Unit u(a, unit_of(i));
        if (u.steps == 0) continue;
        const int ks = kn % C::KST;
        if (kn >= C::KST && !mbar_wait(&bar.k_empty[ks], (kn / C::KST - 1) & 1, abort)) break;
        mbar_arrive_expect_tx(&bar.k_full[ks], C::TILE);
        load_tile<D>(smem + ks * C::TILE, &tmK, &bar.k_full[ks], u.k0, u.hk, u.b);
        ++kn;
        for (int s = u.from; s < u.from + u.steps; ++s, ++qn) {
          const int qs = qn % C::QST;
          if (qn >= C::QST && !mbar_wait(&bar.q_empty[qs], (qn / C::QST - 1) & 1, abort)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bar.q_full[qs], q_bytes);
          const int row = (u.tile0 + s % u.tiles) * a.tq, h = u.hk * (a.w.nh / a.w.nkv) + s / u.tiles * a.tg;
          load_tile<D>(smem + C::OFF_Q + qs * C::TILE, &tmQ, &bar.q_full[qs], row, h, u.b);
        }
      }
      if (*abort) {
        // let the copies in flight land before the CTA exits
        for (int n = max(0, kn - C::KST); n < kn; ++n) drain_wait(&bar.k_full[n % C::KST], (n / C::KST) & 1);
        for (int n = max(0, qn - C::QST); n < qn; ++n) drain_wait(&bar.q_full[n % C::QST], (n / C::QST) & 1);
      }
    }
  } else if (warp == C::kIssuer) {
    // ------------------------------------------------------------ issuer (converged warp)
    const uint64_t dK0 = desc_rows_by_channels(sbase), dQ0 = desc_rows_by_channels(sbase + C::OFF_Q);
    const uint32_t id = idesc_bf16_f32(128, (a.tq * a.tg + 15) / 16 * 16, false, false);
    bool ok = true;
    int kn = 0, t = 0;
    for (int i = 0; ok && unit_of(i) < a.units; ++i) {
      const Unit u(a, unit_of(i));
      if (u.steps == 0) continue;
      const int ks = kn % C::KST;
      if (!mbar_wait(&bar.k_full[ks], (kn / C::KST) & 1, abort)) break;
      const uint64_t dK = dK0 + (uint64_t)(ks * C::TILE >> 4);
      for (int s = 0; s < u.steps; ++s, ++t) {
        const int qs = t % C::QST, buf = t & 3;
        if (!mbar_wait(&bar.q_full[qs], (t / C::QST) & 1, abort) ||
            (t >= 4 && !mbar_wait(&bar.s_empty[buf], (t / 4 - 1) & 1, abort))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t dQ = dQ0 + (uint64_t)(qs * C::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_bf16_warp(tmem + 128 * buf, dK + kstep_channels(kk), dQ + kstep_channels(kk), id, kk > 0 ? 1u : 0u);
        mma_commit_warp(&bar.s_full[buf]);
        mma_commit_warp(&bar.q_empty[qs]);
      }
      if (!ok) break;
      mma_commit_warp(&bar.k_empty[ks]);
      ++kn;
    }
    mma_commit_warp(&bar.done);
    drain_wait(&bar.done, 0);
  } else {
    // ------------------------------------------------------------ sums over the queries
    const int wg = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    float* stats = reinterpret_cast<float*>(smem + C::OFF_LSE) + wg * 2 * kTile;
    const Window& w = a.w;
    const int off = w.nk - w.nq, group = w.nh / w.nkv, rows = a.tq * a.tg;
    const int my_g = r / a.tq, my_i = r % a.tq;  // the column whose statistics this thread fetches
    const float2 sl = make_float2(a.sl2, a.sl2);
    bool ok = true;
    int t = 0, used = 0;
    for (int i = 0; ok && unit_of(i) < a.units; ++i) {
      const Unit u(a, unit_of(i));
      const int j = u.k0 + r, k1 = u.k0 + kTile - 1;
      // queries that see this thread's key
      const int lo = max(max(j - w.right, 0) - off, 0);
      const int hi = min((j < w.sinks ? u.len - 1 : min(u.len - 1, j + w.left)) - off, w.nq - 1);
      auto fetch = [&](int s) {
        const int step = u.from + s, ht = step / u.tiles, q = (u.tile0 + step % u.tiles) * a.tq + my_i;
        const int g = ht * a.tg + my_g;
        if (r >= rows || g >= group || q >= w.nq) return -INFINITY;
        return -kLog2 * __ldg(a.lse + ((long long)u.b * w.nh + u.hk * group + g) * w.nq + q);
      };
      float sum = 0.f;
      int s = (t & 1) == wg ? 0 : 1;
      float next = s < u.steps ? fetch(s) : 0.f;
      for (; s < u.steps; s += 2) {
        const int buf = (t + s) & 3;
        float* l = stats + (used & 1) * kTile;
        uint64_t* ready = &bar.stats[2 * wg + (used & 1)];
        l[r] = next;
        mbar_arrive(ready);
        if (s + 2 < u.steps) next = fetch(s + 2);
        const int step = u.from + s, ht = step / u.tiles, q0 = (u.tile0 + step % u.tiles) * a.tq;
        const int heads = min(a.tg, group - ht * a.tg), p0 = q0 + off, p1 = p0 + a.tq - 1;
        const bool whole = rows == kTile && heads == a.tg && q0 + a.tq <= w.nq && p0 >= 0 && p1 < u.len &&
                           p0 >= k1 - w.right && (p1 <= u.k0 + w.left || k1 < w.sinks);
        if (!mbar_wait(ready, (used >> 1) & 1, abort) || !mbar_wait(&bar.s_full[buf], ((t + s) >> 2) & 1, abort)) {
          ok = false;
          break;
        }
        ++used;
        tc_fence_after();
        const uint32_t tS = tmem + 128 * buf + lanes;
        float2 s01 = make_float2(0.f, 0.f), s23 = s01;
        if (whole) {
          uint32_t x[64], y[64];
          load_cols64(tS, x);
          using Chunk = uint32_t[32];
          tmem_load32_async(tS + 64, *reinterpret_cast<Chunk*>(y));
          tmem_load32_async(tS + 96, *reinterpret_cast<Chunk*>(y + 32));
          add32(x, l, sl, s01, s23);
          add32(x + 32, l + 32, sl, s01, s23);
          tmem_wait_ld();
          tmem_pin(*reinterpret_cast<Chunk*>(y));
          tmem_pin(*reinterpret_cast<Chunk*>(y + 32));
          tc_fence_before();
          mbar_arrive(&bar.s_empty[buf]);
          add32(y, l + 64, sl, s01, s23);
          add32(y + 32, l + 96, sl, s01, s23);
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
            // hidden ones have no statistics either
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float e = fast_exp2(fmaf(__uint_as_float(x[k]), a.sl2, l[c + k]));
              s01.x += see & (1u << k) ? e : 0.f;
            }
          }
          tc_fence_before();
          mbar_arrive(&bar.s_empty[buf]);
        }
        sum += (s01.x + s01.y) + (s23.x + s23.y);
      }
      if (!ok) break;
      t += u.steps;
      if (j < w.nk) a.ws[((long long)(2 * u.part + wg) * w.B * w.nkv + u.list) * w.nk + j] = sum;
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

// Equal parts of a key tile's query tiles, so that no unit is longer than a quarter of a CTA's
// share (the CTAs' loads then differ by less than that), but not shorter than four steps.
int unit_parts(const Window& w, int tq, int tg) {
  const long long per = ((w.nh / w.nkv + tg - 1) / tg);
  const long long key_tiles = (w.nk + kTile - 1) / kTile;
  long long all = 0, most = 0;
  for (long long kt = 0; kt < key_tiles; ++kt) {
    int i0, n;
    query_range(w, w.nk, (int)kt * kTile, (int)std::min<long long>((kt + 1) * kTile, w.nk) - 1, i0, n);
    const long long steps = n > 0 ? ((i0 + n - 1) / tq - i0 / tq + 1) * per : 0;
    all += steps;
    most = std::max(most, steps);
  }
  const long long share = std::max<long long>(1, all * w.B * w.nkv / 152);
  return (int)std::max<long long>(1, std::min<long long>({(4 * most + share - 1) / share, most / 4, 16}));
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
  a.key_tiles = (w.nk + kTile - 1) / kTile;
  a.parts = unit_parts(w, a.tq, a.tg);
  a.units = w.B * w.nkv * a.key_tiles * a.parts;
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
                    (const float*)ws, out, 2 * a.parts);
}

}  // namespace

size_t window_weights_ws_bytes(const Window& w) {
  int tq, tg;
  query_tile(w, tq, tg);
  return (size_t)2 * unit_parts(w, tq, tg) * w.B * w.nkv * w.nk * 4;
}

cudaError_t launch_window_weights(const Window& w, View<const __nv_bfloat16> q, View<const __nv_bfloat16> k,
                                  const float* lse, float* weights_out, float* ws, float scale, int d,
                                  cudaStream_t st) {
  return d == 64 ? weights<64>(w, q, k, lse, weights_out, ws, scale, st)
                 : weights<128>(w, q, k, lse, weights_out, ws, scale, st);
}

}  // namespace psa
