// window_tc.cuh -- what the tensor-core kernels of the window attention share: tile shapes,
// tensor maps over strided rows, loads, and the zeroing of a tile's rows of padding.
#pragma once

#include "lm.cuh"
#include "ptx_tiles4d.cuh"

namespace psa {

constexpr int kTile = 128;  // rows of a tile, queries and keys
constexpr float kLog2 = 1.4426950408889634074f;

// A [128 rows, D] bf16 tile in shared memory as TMA writes it: D / 64 boxes of 128 rows of
// 128 bytes, 128-byte swizzle.
template <int D>
constexpr uint32_t kTileBytes = kTile * D * 2;
constexpr uint32_t kBoxBytes = kTile * 128;

template <int D>
__device__ __forceinline__ void load_tile(unsigned char* dst, const CUtensorMap* map, uint64_t* bar,
                                          int row, int h, int b) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tma_load_4d(dst + c * kBoxBytes, map, bar, 64 * c, row, h, b);
}

// Operand whose rows are the product's M or N and whose channels its K: 16 channels on.
__device__ __forceinline__ constexpr uint64_t kstep_channels(int kk) {
  return (uint64_t)((kk / 4) * (kBoxBytes >> 4) + (kk % 4) * 2);
}
// Operand whose channels are the product's N and whose rows its K: 16 rows on.
constexpr uint64_t kKstepRows = (16 * 128) >> 4;

__device__ __forceinline__ uint64_t desc_rows_by_channels(uint32_t base) {
  return desc_kmajor(SmemTile{base, 128u, kTile}, 0);
}
__device__ __forceinline__ uint64_t desc_channels_by_rows(uint32_t base) {
  return desc_mnmajor(SmemTile{base, 128u, kTile}, 0);
}

// Zeroes rows [r0, r1) of a loaded tile (one warp), for the async proxy to read.
template <int D>
__device__ __forceinline__ void zero_rows(unsigned char* tile, int r0, int r1, int lane) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    uint4* p = reinterpret_cast<uint4*>(tile + c * kBoxBytes);
    for (int i = r0 * 8 + lane; i < r1 * 8; i += 32) p[i] = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
}

// Columns of a key tile that some row sees, in steps of the product's 16: all up to the last
// visible key, or in front of the window the sinks alone.
__device__ __forceinline__ int used_columns(int tile, int first, int end, int sinks) {
  const int to = (tile < first ? min(sinks, end) : end) - tile * kTile;
  return min(kTile, (to + 15) & ~15);
}

// The keys of a 32-column chunk that a row sees, one bit each: columns lo .. hi and those below
// sk, all relative to the chunk's first.
__device__ __forceinline__ uint32_t visible32(int lo, int hi, int sk) {
  const uint32_t upto = hi >= 31 ? 0xffffffffu : hi < 0 ? 0u : (2u << hi) - 1u;
  const uint32_t from = lo <= 0 ? 0xffffffffu : lo > 31 ? 0u : 0xffffffffu << lo;
  const uint32_t sinks = sk <= 0 ? 0u : sk > 31 ? 0xffffffffu : (1u << sk) - 1u;
  return upto & (from | sinks);
}
// Scores whose bit is not set become -infinity.
__device__ __forceinline__ void hide(uint32_t* x, uint32_t mask) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (!(mask & (1u << c))) x[c] = 0xff800000u;
}

// 64 columns of this thread's lane, one wait.
__device__ __forceinline__ void load_cols64(uint32_t t, uint32_t (&r)[64]) {
  using Chunk = uint32_t[32];
  tmem_load32_async(t, *reinterpret_cast<Chunk*>(r));
  tmem_load32_async(t + 32, *reinterpret_cast<Chunk*>(r + 32));
  tmem_wait_ld();
  tmem_pin(*reinterpret_cast<Chunk*>(r));
  tmem_pin(*reinterpret_cast<Chunk*>(r + 32));
}

// Tensor map over a view's rows: 4-D (d, N, heads, B), box {64 channels, 128 rows}.
bool map_view(CUtensorMap* m, const void* base, long long sb, long long sh, long long sn, int B,
              int heads, int N, int d);
// The same with a box of several heads and batches.
bool map_view_box(CUtensorMap* m, const void* base, long long sb, long long sh, long long sn, int B,
                  int heads, int N, int d, int box_rows, int box_heads, int box_batches);

}  // namespace psa
