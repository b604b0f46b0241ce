// kv_evict.cu -- eviction from a cache: of every sequence's rows of a key/value head the `keep`
// with the largest weight stay, the first `sinks` positions and the last `recent` ones always.
//
// Rows 0 .. keep - 1 hold what stays afterwards.  A row that stays and stands there already is
// not touched; those that stay from behind fill the gaps, in order.  Sources lie at keep or
// behind it and targets in front of it, so the moves are independent of one another and need no
// second cache; a step that evicts one row moves at most one.
//
// The selection is a radix select: a CTA for each list (sequence and key/value head) makes
// sortable integers of the weights in shared memory, counts their first 13 bits (sign, exponent, 4
// bits of the mantissa: fewer would meet in the same counters), gathers those that share the bits
// of the keep-th largest, and compares these with one another.  What stays is then one bit per
// row: ranks, gaps and the rows that fill them are sums over words of 32 rows.  Latencies and
// instructions of the one CTA bound it (the counters' atomics are a third).  The moves are a copy
// bound by memory: a second kernel over all lists, or, where a list can have no more than
// kFewMoves, the same one.
// Measured, 8 sequences of up to 16384 rows of 8 heads of 128 in bf16 cut to 8192: 50 us, of which
// the selection takes 28 and the moves 21 (126 MB read and written at 5.9 TB/s, 0.87 of the copy
// bandwidth); one row of 2049 out of 256 lists: 10 us.  Few long lists leave most SMs idle, and lists
// beyond kKeysInShared are read again from memory: 8 lists of 16384 rows cut to half 30 us, of 40960
// 66, of 65536 161, of 2^20 3.1 ms.
#include <algorithm>

#include "lm.cuh"
#include "ptx.cuh"

namespace psa {
namespace {

constexpr int kBits = 13, kBins = 1 << kBits;  // of a key's first digit: 4 bits of the mantissa
constexpr int kKeysInShared = 40 * 1024;       // longer lists are read again in every pass
constexpr int kGathered = 1024;                // more that share their first digit are counted where they are
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
  uint32_t hist[kBins], some[kGathered];
  unsigned long long warp[32];
  uint32_t digit, need, gathered;
};

// Sum of x over the threads in front of this one; total: over all.
__device__ __forceinline__ unsigned long long in_front(Shared& sh, unsigned long long x, unsigned long long& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  auto scan = [&](unsigned long long v) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned long long y = __shfl_up_sync(kAll, v, d);
      if (lane >= d) v += y;
    }
    return v;
  };
  const unsigned long long upto = scan(x);
  __syncthreads();  // of the use before
  if (lane == 31) sh.warp[warp] = upto;
  __syncthreads();
  const unsigned long long w = scan(lane < warps ? sh.warp[lane] : 0);
  total = __shfl_sync(kAll, w, 31);
  const unsigned long long before = __shfl_sync(kAll, w, max(warp - 1, 0));
  return (warp > 0 ? before : 0) + upto - x;
}

// The bin that holds the need-th largest, from counts that are complete; what is above it is
// taken off need.
__device__ __forceinline__ uint32_t find_bin(Shared& sh, uint32_t& need) {
  const int tid = threadIdx.x, per = kBins / blockDim.x, hi = kBins - 1 - tid * per;
  uint32_t mine = 0;
  for (int i = 0; i < per; i += 4) {
    const uint4 c = *reinterpret_cast<const uint4*>(&sh.hist[hi - i - 3]);
    mine += c.x + c.y + c.z + c.w;
  }
  unsigned long long total;
  uint32_t above = (uint32_t)in_front(sh, mine, total);
  if (above < need && need <= above + mine) {
    int d = hi;
    while (above + sh.hist[d] < need) above += sh.hist[d--];
    sh.digit = d;
    sh.need = need - above;
  }
  __syncthreads();
  need = sh.need;
  return sh.digit;
}

// kCached: the list's keys, and two bits for each, lie in shared memory.
template <bool kCached>
__global__ void __launch_bounds__(1024)
    evict_select_kernel(const EvictArgs a, const int cap, const int row16, const bool move) {
  extern __shared__ uint32_t dynamic[];
  __shared__ __align__(16) Shared sh;
  pdl_launch_dependents();
  const int list = blockIdx.x, b = list / a.nkv, h = list % a.nkv;
  const int tid = threadIdx.x, threads = blockDim.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < kBins / 4; i += threads) reinterpret_cast<uint4*>(sh.hist)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) sh.gathered = 0;
  pdl_wait();
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
  uint32_t* keys = dynamic;  // (positions at first)
  long long safe_from = 1LL << 40;
  if (kCached || a.recent > 0) {
    int newest = INT_MIN;
#pragma unroll 8
    for (int r = tid; r < len; r += threads) {
      const int p = pos[r];
      if (kCached) keys[r] = p;
      newest = max(newest, p);
    }
    newest = __reduce_max_sync(kAll, newest);
    if (lane == 0) sh.warp[warp] = (uint32_t)newest;
    __syncthreads();
    newest = __reduce_max_sync(kAll, lane < threads / 32 ? (int)(uint32_t)sh.warp[lane] : INT_MIN);
    if (a.recent > 0) safe_from = (long long)newest - a.recent + 1;
  }
  // ---- keys, and how many have the same first digit; what stays in its place already
  const bool apart = w_out != w, apart_pos = pos_out != pos;
  auto to_key = [&](float x, int p) { return p < a.sinks || p >= safe_from ? kSafe : sortable(x); };
  __syncthreads();
#pragma unroll 8
  for (int r = tid; r < len; r += threads) {
    const float x = w[r];
    const int p = kCached ? (int)keys[r] : pos[r];
    const uint32_t k = to_key(x, p);
    if (kCached) keys[r] = k;
    atomicAdd(&sh.hist[k >> (32 - kBits)], 1u);
    if (r < count) {  // (gaps are written again below)
      if (apart) w_out[r] = x;
      if (apart_pos) pos_out[r] = p;
    }
  }
  auto key = [&](int r) {
    if constexpr (kCached) return keys[r];
    else return to_key(w[r], pos[r]);
  };
  __syncthreads();
  uint32_t need = count, top = find_bin(sh, need);

  // ---- the count-th largest key, and how many of its equals are kept
  const uint32_t shared_by = sh.hist[top];
  if (shared_by <= kGathered) {
#pragma unroll 4
    for (int r = tid; r < len; r += threads) {
      const uint32_t k = key(r);
      if (k >> (32 - kBits) == top) sh.some[atomicAdd(&sh.gathered, 1u)] = k;
    }
    __syncthreads();
    for (uint32_t i = tid; i < shared_by; i += threads) {
      const uint32_t k = sh.some[i];
      uint32_t above = 0, equal = 0;
#pragma unroll 8
      for (uint32_t x = 0; x < shared_by; ++x) {
        above += sh.some[x] > k;
        equal += sh.some[x] == k;
      }
      if (above < need && need <= above + equal) {  // (its equals say the same)
        sh.digit = k;
        sh.need = need - above;
      }
    }
    __syncthreads();
    top = sh.digit;
    need = sh.need;
  } else {
#pragma unroll 1
    for (int shift = 32 - kBits; shift > 0;) {
      const int bits = min(shift, kBits), at = shift - bits;
      __syncthreads();  // the counts are read
      for (int i = tid; i < kBins; i += threads) sh.hist[i] = 0;
      __syncthreads();
      for (int r = tid; r < len; r += threads) {
        const uint32_t k = key(r);
        if (k >> shift == top) atomicAdd(&sh.hist[(k >> at) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      const uint32_t digit = find_bin(sh, need);
      top = top << bits | digit;
      shift = at;
    }
  }

  // ---- one bit per row: larger than that key, or equal to it
  const int words = (len + 31) / 32;
  uint32_t* larger;
  if constexpr (kCached) larger = keys + (len + 3) / 4 * 4;
  else larger = a.words + (long long)list * 2 * ((a.max_len + 31) / 32);
  uint32_t* equal = larger + words;
#pragma unroll 4
  for (int x = warp; x < words; x += threads / 32) {
    const int r = x * 32 + lane;
    const uint32_t k = r < len ? key(r) : 0u;
    const uint32_t gt = __ballot_sync(kAll, r < len && k > top), eq = __ballot_sync(kAll, r < len && k == top);
    if (lane == 0) {
      larger[x] = gt;
      equal[x] = eq;
    }
  }
  __syncthreads();
  // a thread has a run of words: of equal keys the first `need` rows stay
  const int run = (words + threads - 1) / threads, from = min(words, tid * run), to = min(words, from + run);
  unsigned long long n = 0, total;
  for (int x = from; x < to; ++x) n += __popc(equal[x]);
  uint32_t ties = (uint32_t)in_front(sh, n, total);
  // gaps in the upper half, rows that fill them in the lower one
  auto in_place = [&](int x) {  // the word's rows below count
    const int m = count - x * 32;
    return m >= 32 ? kAll : m <= 0 ? 0u : (1u << m) - 1u;
  };
  n = 0;
  for (int x = from; x < to; ++x) {
    uint32_t eq = equal[x];
    const uint32_t c = __popc(eq);
    for (uint32_t drop = ties + c > need ? min(c, ties + c - need) : 0u; drop > 0; --drop) eq &= ~(0x80000000u >> __clz(eq));
    ties += c;
    const uint32_t kept = larger[x] | eq, here = in_place(x);
    larger[x] = kept;
    n += (unsigned long long)__popc(~kept & here) << 32 | __popc(kept & ~here);
  }
  unsigned long long at = in_front(sh, n, total);
  const uint32_t moves = (uint32_t)total;
  for (int x = from; x < to; ++x) {
    // where the word's gaps are listed, or the rows that fill some (of the word that has both, the
    // latter are the first of their list)
    const uint32_t kept = larger[x], here = in_place(x);
    equal[x] = here ? (uint32_t)(at >> 32) : (uint32_t)at;
    at += (unsigned long long)__popc(~kept & here) << 32 | __popc(kept & ~here);
  }
  if (tid == 0) a.counts[list] = moves;
  __syncthreads();
#pragma unroll 4
  for (int x = warp; x < words; x += threads / 32) {
    const uint32_t kept = larger[x], here = in_place(x), first = equal[x];
    const uint32_t gaps = ~kept & here, movers = kept & ~here, bit = 1u << lane, below = bit - 1u;
    if (gaps & bit) dst[first + __popc(gaps & below)] = x * 32 + lane;
    if (movers & bit) src[(here ? 0u : first) + __popc(movers & below)] = x * 32 + lane;
  }
  __syncthreads();
#pragma unroll 4
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

// 16 bytes per thread: K's row, then V's, of a list's moves, kMoveUnroll at a time; the next ones'
// places are fetched while these rows are on their way.
template <int ROW16>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, const int cap) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int PER = kMoveThreads / (2 * ROW16);  // moves of a CTA's threads
  const int list = blockIdx.y, b = list / a.nkv, h = list % a.nkv;
  const int n = a.counts[list], c = threadIdx.x % (2 * ROW16), stride = gridDim.x * PER * kMoveUnroll;
  const int* src = a.moves + (long long)list * 2 * cap;
  const int* dst = src + cap;
  uint4* base = c < ROW16 ? a.k.row(b, h, 0) + c : a.v.row(b, h, 0) + c - ROW16;
  const long long step = c < ROW16 ? a.k.sn : a.v.sn;
  int from[kMoveUnroll], to[kMoveUnroll];
  auto fetch = [&](int m) {
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i) {
      to[i] = -1;
      if (m + i * PER < n) {
        from[i] = src[m + i * PER];
        to[i] = dst[m + i * PER];
      }
    }
  };
  int m = blockIdx.x * PER * kMoveUnroll + threadIdx.x / (2 * ROW16);
  fetch(m);
  for (; m < n; m += stride) {
    uint4 x[kMoveUnroll];
    uint4* at[kMoveUnroll];
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i) {
      at[i] = nullptr;
      if (to[i] < 0) continue;
      x[i] = base[from[i] * step];
      at[i] = base + to[i] * step;
    }
    fetch(m + stride);
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i)
      if (at[i]) *at[i] = x[i];
  }
}

// Keys, and two bits, of a list.
constexpr int shared_bytes(int rows) { return (rows + 3) / 4 * 16 + (rows + 31) / 32 * 8; }

int most_moves(int keep, int max_len) { return std::max(0, std::min(keep, max_len - keep)); }

}  // namespace

size_t evict_ws_bytes(int lists, int keep, int max_len) {
  const size_t words = max_len > kKeysInShared ? (size_t)lists * 2 * ((max_len + 31) / 32) * 4 : 0;
  return ((size_t)lists * 4 + 15) / 16 * 16 + (size_t)lists * 2 * most_moves(keep, max_len) * 4 + words;
}

cudaError_t launch_kv_evict(EvictArgs a, int row16, void* ws, cudaStream_t st) {
  const int lists = a.B * a.nkv, cap = most_moves(a.keep, a.max_len);
  a.counts = static_cast<int*>(ws);
  a.moves = reinterpret_cast<int*>(static_cast<char*>(ws) + ((size_t)lists * 4 + 15) / 16 * 16);
  a.words = reinterpret_cast<uint32_t*>(a.moves + (size_t)lists * 2 * cap);
  const bool fused = cap <= kFewMoves, cached = a.max_len <= kKeysInShared;
  // (a power of two that divides the bins)
  const int threads = a.max_len > 8192 ? 1024 : a.max_len > 1024 ? 512 : 256;
  const int smem = cached ? shared_bytes(a.max_len) : 0;
  auto select = cached ? evict_select_kernel<true> : evict_select_kernel<false>;
  if (cached) {
    const cudaError_t e = set_max_dynamic_smem((const void*)select, shared_bytes(kKeysInShared));
    if (e != cudaSuccess) return e;
  }
  const cudaError_t s = launch_pdl(select, dim3(lists), dim3(threads), smem, st, a, cap, row16, fused);
  if (s != cudaSuccess || fused) return s;
  // eight CTAs per SM between the lists, if they have that many moves
  const int per = kMoveThreads / (2 * row16) * kMoveUnroll;
  const dim3 grid(std::min((cap + per - 1) / per, std::max(1, 8 * 152 / lists)), lists);
  auto kern = row16 == 8 ? evict_move_kernel<8> : row16 == 16 ? evict_move_kernel<16> : evict_move_kernel<32>;
  return launch_pdl(kern, grid, dim3(kMoveThreads), 0, st, a, cap);
}

}  // namespace psa
