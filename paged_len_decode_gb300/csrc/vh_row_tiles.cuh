// vh_row_tiles.cuh -- the work list of a batch of rows: the 16-token tiles that
// a window and sinks leave of each, and equal shares of the list of all.
#pragma once

#include "vh_common.cuh"

namespace vh {

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

// cum[0 .. B]: prefix sums of count_row(b) over the rows, and *most the largest of them (cum[0] and
// *most are 0 and the warp `mine` is synchronised).  Up to kWarpRows rows are counted and summed by
// that warp, which goes on to its first copies while the others wait for the sums; more rows
// by all threads.  (Hardware barrier 2.)
template <int kWarpRows, typename Count>
__device__ __forceinline__ void sum_rows(int B, int* cum, int* most_of, int* tot, bool mine, Count count_row) {
  const int lane = threadIdx.x & 31;
  if (B > kWarpRows) {
    __syncthreads();
    int most = 0;
    for (int b = threadIdx.x; b < B; b += blockDim.x) {
      const int n = count_row(b);
      cum[1 + b] = n;
      most = max(most, n);
    }
    atomicMax(most_of, most);
    __syncthreads();
    scan_rows(cum, B, tot);
  } else if (mine) {
    int n[kWarpRows / 32], run = 0;
#pragma unroll
    for (int x = 0; x < kWarpRows / 32; ++x) n[x] = x * 32 + lane < B ? count_row(x * 32 + lane) : 0;
#pragma unroll
    for (int x = 0; x < kWarpRows / 32; ++x) {
      if (x * 32 >= B) break;
      int v = n[x];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += y;
      }
      v += run;
      if (x * 32 + lane < B) cum[1 + x * 32 + lane] = v;
      run = __shfl_sync(0xffffffffu, v, 31);
    }
    int most = 0;
#pragma unroll
    for (int x = 0; x < kWarpRows / 32; ++x) most = max(most, n[x]);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) *most_of = most;
    __syncwarp();
    asm volatile("bar.arrive 2, %0;" ::"r"(static_cast<int>(blockDim.x)) : "memory");
  } else {
    named_sync(2, blockDim.x);
  }
}

// What CTA c of N takes of the list: tiles t0 .. t1 - 1, from row b0 (or a later one) on.
struct Share {
  int n_eff;       // CTAs that share the tiles; 0: whole rows a CTA
  int t0, t1, b0;
};

// Either T / n tiles each, of which a CTA takes at least q: it reads a tile in some time, and the
// longest row's pieces, R / q of them, are then added at `piece` times that each, so q = sqrt(R
// piece) is the least of both; or whole rows, which need no merge: that takes about as long as 6 tiles.
__device__ __forceinline__ Share share_of_cta(const int* cum, int B, int c, int N, int most, float piece) {
  const int T = cum[B];
  const int q = max(1, static_cast<int>(sqrtf(static_cast<float>(most) * piece) + 0.5f));
  const int rows_each = (B + N - 1) / N;
  const bool by_row = most * rows_each <= max(q, T / N) + 6;
  Share s;
  s.n_eff = by_row ? 0 : min(N, (T + q - 1) / q);
  s.t0 = s.t1 = s.b0 = 0;
  if (by_row) {
    s.b0 = min(c * rows_each, B);
    s.t0 = cum[s.b0];
    s.t1 = cum[min(s.b0 + rows_each, B)];
  } else if (c < s.n_eff) {
    const int each = T / s.n_eff, rest = T - each * s.n_eff;  // the first `rest` CTAs take one tile more
    s.t0 = c * each + min(c, rest);
    s.t1 = s.t0 + each + (c < rest ? 1 : 0);
  }
  return s;
}

}  // namespace vh
