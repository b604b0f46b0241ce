// kv_evict.cu -- eviction from a cache: of every sequence's rows of a key/value head the `keep`
// with the largest weight stay, the first `sinks` positions and the last `recent` ones always.
//
// Rows 0 .. keep - 1 hold what stays afterwards.  A row that stays and stands there already is
// not touched; those that stay from behind fill the gaps, in order.  Sources lie at keep or
// behind it and targets in front of it, so the moves are independent of one another and need no
// second cache; a step that evicts one row moves at most one.
//
// The selection is a radix select: a CTA for each list (sequence and key/value head) finds the
// keep-th largest weight as a sortable integer in three passes of 11, 11 and 10 bits over the
// list's keys in shared memory, then walks the list once more for the gaps and the rows that
// fill them.  A warp owns a run of neighbouring rows, so that ranks are ballots inside it and
// one scan over the warps' totals.  The moves are a copy bound by memory: a second kernel over all
// lists, or, where a list can have no more than kFewMoves, the same one.
#include <algorithm>

#include "lm.cuh"
#include "ptx.cuh"

namespace psa {
namespace {

constexpr int kBins = 2048;
constexpr int kKeysInShared = 48 * 1024;  // longer lists are read again in every pass
constexpr int kFewMoves = 32;
constexpr int kMoveThreads = 256, kMoveUnroll = 4;
constexpr uint32_t kSafe = 0xffffffffu;
constexpr uint32_t kAll = 0xffffffffu;

// Larger weights have larger keys; both zeros are alike, NaN is above infinity.
__device__ __forceinline__ uint32_t sortable(float w) {
  if (w != w) return kSafe - 1;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Shared {
  uint32_t hist[kBins];
  uint32_t warp[32];
  uint32_t digit, need;
};

// Sum of x over the warps in front of this one, and over all (x: the same in a warp's lanes).
__device__ __forceinline__ uint32_t over_warps(Shared& sh, uint32_t x, uint32_t& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  __syncthreads();  // of the use before
  if (lane == 0) sh.warp[warp] = x;
  __syncthreads();
  const uint32_t v = lane < warps ? sh.warp[lane] : 0u;
  total = __reduce_add_sync(kAll, v);
  return __reduce_add_sync(kAll, lane < warp ? v : 0u);
}

__global__ void __launch_bounds__(1024)
    evict_select_kernel(const EvictArgs a, const int cap, const int row16, const bool move) {
  extern __shared__ uint32_t keys[];
  __shared__ Shared sh;
  pdl_launch_dependents();
  pdl_wait();
  const int list = blockIdx.x, b = list / a.nkv, h = list % a.nkv;
  const int tid = threadIdx.x, threads = blockDim.x, warp = tid >> 5, lane = tid & 31;
  const int len = max(0, min(a.lens[b], a.max_len)), count = min(len, a.keep);
  const float* w = a.weights + (long long)list * a.max_len;
  const int* pos = a.positions + (long long)list * a.max_len;
  float* w_out = a.weights_out + (long long)list * a.max_len;
  int* pos_out = a.positions_out + (long long)list * a.max_len;
  int* src = a.moves + (long long)list * 2 * cap;
  int* dst = src + cap;
  if (h == 0 && tid == 0) a.lens_out[b] = count;
  if (count == len) {
    if (tid == 0) a.counts[list] = 0;
    for (int r = tid; r < len; r += threads) {
      w_out[r] = w[r];
      pos_out[r] = pos[r];
    }
    return;
  }
  // ---- which rows are kept whatever their weight
  long long safe_from = 1LL << 40;
  if (a.recent > 0) {
    int newest = INT_MIN;
    for (int r = tid; r < len; r += threads) newest = max(newest, pos[r]);
    newest = __reduce_max_sync(kAll, newest);
    if (lane == 0) sh.warp[warp] = (uint32_t)newest;
    __syncthreads();
    newest = __reduce_max_sync(kAll, lane < threads / 32 ? (int)sh.warp[lane] : INT_MIN);
    safe_from = (long long)newest - a.recent + 1;
  }
  const bool cached = len <= kKeysInShared;
  auto make = [&](int r) {
    const int p = pos[r];
    return p < a.sinks || p >= safe_from ? kSafe : sortable(w[r]);
  };
  if (cached)
    for (int r = tid; r < len; r += threads) keys[r] = make(r);
  auto key = [&](int r) { return cached ? keys[r] : make(r); };

  // ---- the count-th largest key, and how many of its equals are kept
  uint32_t top = 0, need = count;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass < 2 ? 11 : 10;
    for (int i = tid; i < kBins; i += threads) sh.hist[i] = 0;
    __syncthreads();
    for (int r0 = warp * 32; r0 < len; r0 += threads) {
      const int r = r0 + lane;
      const uint32_t k = r < len ? key(r) : 0u;
      const bool in = r < len && (pass == 0 || (k >> (shift + bits)) == top);
      const uint32_t who = __ballot_sync(kAll, in);
      if (who == 0) continue;
      const uint32_t digit = (k >> shift) & ((1u << bits) - 1u);
      const int first = __ffs(who) - 1;
      // (equal digits of a whole warp would be added one after another)
      const uint32_t common = __shfl_sync(kAll, digit, first);
      if (__all_sync(kAll, !in || digit == common)) {
        if (lane == first) atomicAdd(&sh.hist[digit], __popc(who));
      } else if (in) {
        atomicAdd(&sh.hist[digit], 1u);
      }
    }
    __syncthreads();
    // bins from the top: thread t sums those of its share
    const int per = kBins / threads, hi = kBins - 1 - tid * per;
    uint32_t mine = 0;
    for (int i = 0; i < per; ++i) mine += sh.hist[hi - i];
    uint32_t upto = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, upto, x);
      if (lane >= x) upto += y;
    }
    uint32_t total;
    upto += over_warps(sh, __shfl_sync(kAll, upto, 31), total);
    uint32_t above = upto - mine;
    if (above < need && need <= upto) {
      int d = hi;
      while (above + sh.hist[d] < need) above += sh.hist[d--];
      sh.digit = d;
      sh.need = need - above;
    }
    __syncthreads();
    top = top << bits | sh.digit;
    need = sh.need;
  }

  // ---- ranks: a run of rows for each warp
  const int run = (len + threads - 1) / threads * 32, from = min(len, warp * run), to = min(len, from + run);
  uint32_t n = 0, total;
  for (int r0 = from; r0 < to; r0 += 32) {
    const int r = r0 + lane;
    n += __popc(__ballot_sync(kAll, r < to && key(r) == top));
  }
  const uint32_t ties = over_warps(sh, n, total);
  const uint32_t below = (1u << lane) - 1u;
  // calls f(row, kept, gap, mover) for this warp's rows, ties in the order of rows
  auto walk = [&](auto f) {
    uint32_t seen = ties;
    for (int r0 = from; r0 < to; r0 += 32) {
      const int r = r0 + lane;
      const uint32_t k = r < to ? key(r) : 0u;
      const uint32_t eq = __ballot_sync(kAll, r < to && k == top);
      const bool kept = r < to && (k > top || (k == top && seen + __popc(eq & below) < need));
      seen += __popc(eq);
      f(r, kept, r < to && r < count && !kept, r >= count && kept);
    }
  };
  uint32_t gaps = 0, movers = 0;
  walk([&](int, bool, bool gap, bool mover) {
    gaps += __popc(__ballot_sync(kAll, gap));
    movers += __popc(__ballot_sync(kAll, mover));
  });
  uint32_t moves;
  uint32_t gap_at = over_warps(sh, gaps, moves), mover_at = over_warps(sh, movers, total);
  const bool apart = w_out != w, apart_pos = pos_out != pos;
  walk([&](int r, bool kept, bool gap, bool mover) {
    const uint32_t g = __ballot_sync(kAll, gap), m = __ballot_sync(kAll, mover);
    if (gap) dst[gap_at + __popc(g & below)] = r;
    if (mover) src[mover_at + __popc(m & below)] = r;
    gap_at += __popc(g);
    mover_at += __popc(m);
    if (kept && r < count) {
      if (apart) w_out[r] = w[r];
      if (apart_pos) pos_out[r] = pos[r];
    }
  });
  if (tid == 0) a.counts[list] = moves;
  __syncthreads();
  for (uint32_t i = tid; i < moves; i += threads) {
    const int s = src[i], d = dst[i];
    const float x = w[s];
    const int p = pos[s];
    w_out[d] = x;
    pos_out[d] = p;
  }
  if (move) {
    const long long n16 = (long long)moves * 2 * row16;
    for (long long i = tid; i < n16; i += threads) {
      const int m = i / (2 * row16), c = i % (2 * row16);
      uint4* base = c < row16 ? a.k.row(b, h, 0) + c : a.v.row(b, h, 0) + c - row16;
      const long long step = c < row16 ? a.k.sn : a.v.sn;
      base[dst[m] * step] = base[src[m] * step];
    }
  }
  __syncthreads();
  // rows that come behind the kept ones later start from nothing
  for (int r = count + tid; r < len; r += threads) w_out[r] = 0.f;
}

// 16 bytes per thread: K's row, then V's, of each move of a list.
template <int ROW16>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, const int cap) {
  pdl_launch_dependents();
  pdl_wait();
  const int list = blockIdx.y, b = list / a.nkv, h = list % a.nkv;
  const int n = a.counts[list] * 2 * ROW16, first = blockIdx.x * kMoveThreads * kMoveUnroll + threadIdx.x;
  const int* src = a.moves + (long long)list * 2 * cap;
  const int* dst = src + cap;
  // (a stride of kMoveThreads is a whole number of rows: a thread's column stays)
  const int c = first % (2 * ROW16);
  uint4* base = c < ROW16 ? a.k.row(b, h, 0) + c : a.v.row(b, h, 0) + c - ROW16;
  const long long step = c < ROW16 ? a.k.sn : a.v.sn;
  uint4 x[kMoveUnroll];
  uint4* to[kMoveUnroll];
#pragma unroll
  for (int i = 0; i < kMoveUnroll; ++i) {
    const int at = first + i * kMoveThreads;
    to[i] = nullptr;
    if (at < n) {
      const int m = at / (2 * ROW16);
      to[i] = base + dst[m] * step;
      x[i] = base[src[m] * step];
    }
  }
#pragma unroll
  for (int i = 0; i < kMoveUnroll; ++i)
    if (to[i]) *to[i] = x[i];
}

int most_moves(int keep, int max_len) { return std::max(0, std::min(keep, max_len - keep)); }

}  // namespace

size_t evict_ws_bytes(int lists, int keep, int max_len) {
  return ((size_t)lists * 4 + 15) / 16 * 16 + (size_t)lists * 2 * most_moves(keep, max_len) * 4;
}

cudaError_t launch_kv_evict(EvictArgs a, int row16, void* ws, cudaStream_t st) {
  const int lists = a.B * a.nkv, cap = most_moves(a.keep, a.max_len);
  a.counts = static_cast<int*>(ws);
  a.moves = reinterpret_cast<int*>(static_cast<char*>(ws) + ((size_t)lists * 4 + 15) / 16 * 16);
  const cudaError_t e = set_max_dynamic_smem((const void*)evict_select_kernel, kKeysInShared * 4);
  if (e != cudaSuccess) return e;
  const bool fused = cap <= kFewMoves;
  const int threads = a.max_len > 4096 ? 1024 : 256;
  const int smem = std::min(a.max_len, kKeysInShared) * 4;
  const cudaError_t s = launch_pdl(evict_select_kernel, dim3(lists), dim3(threads), smem, st, a, cap, row16, fused);
  if (s != cudaSuccess || fused) return s;
  const long long units = (long long)cap * 2 * row16, per = kMoveThreads * kMoveUnroll;
  const dim3 grid((unsigned)((units + per - 1) / per), lists);
  auto kern = row16 == 8 ? evict_move_kernel<8> : row16 == 16 ? evict_move_kernel<16> : evict_move_kernel<32>;
  return launch_pdl(kern, grid, dim3(kMoveThreads), 0, st, a, cap);
}

}  // namespace psa
