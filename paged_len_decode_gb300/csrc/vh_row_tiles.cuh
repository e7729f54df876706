// vh_row_tiles.cuh -- the work list of a batch of rows: the 16-token tiles that
// a window and sinks leave of each, and equal shares of the list of all.
#pragma once

#include "vh_common.cuh"

namespace vh {

__device__ __forceinline__ int share_begin(int c, int n, int total) {
  return c * (total / n) + min(c, total % n);
}

__device__ __forceinline__ int share_of(int t, int n, int total) {
  const int q = total / n, r = total % n, big = r * (q + 1);
  return t < big ? t / (q + 1) : r + (t - big) / q;
}

// The tiles of a row: `sink` tiles from tile 0, then tiles from `first` on.
struct RowTiles {
  int sink, first, count;
  __device__ int tile(int k) const { return k < sink ? k : k - sink + first; }
};

__device__ __forceinline__ RowTiles tiles_of(int L, int window, int sinks) {
  RowTiles r;
  r.sink = (min(sinks, L) + kTile - 1) / kTile;
  r.first = max(r.sink, max(0, L - window) / kTile);
  r.count = r.sink + (L + kTile - 1) / kTile - r.first;
  return r;
}

// Bit k: key 16 tile + k is visible.
__device__ __forceinline__ uint32_t visible16(int tile, int L, int window, int sinks) {
  auto below = [](int x) -> uint32_t { return x <= 0 ? 0u : (x >= kTile ? 0xFFFFu : (1u << x) - 1u); };
  const int j0 = tile * kTile;
  return below(L - j0) & (below(sinks - j0) | (~below(L - window - j0) & 0xFFFFu));
}

// In-place inclusive prefix sum of cum[1..n] (cum[0] = 0).
__device__ inline void scan_rows(int* cum, int n, int* tot) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + blockDim.x - 1) / blockDim.x;
  const int lo = min(n, tid * per), hi = min(n, lo + per);
  int sum = 0;
  for (int i = lo; i < hi; ++i) sum += cum[1 + i];
  int x = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) tot[warp] = x;
  __syncthreads();
  int run = x - sum;
  for (int w = 0; w < warp; ++w) run += tot[w];
  for (int i = lo; i < hi; ++i) {
    run += cum[1 + i];
    cum[1 + i] = run;
  }
  __syncthreads();
}

// First row with cum[row + 1] > t, from row lo on.
__device__ __forceinline__ int row_of(const int* cum, int lo, int B, int t) {
  int hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

}  // namespace vh
