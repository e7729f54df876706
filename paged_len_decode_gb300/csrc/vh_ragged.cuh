// vh_ragged.cuh -- device helpers of ragged batches: the row of a token or of
// a block of tokens, the checks of a row's extent, and weights in merges.
#pragma once

#include "vh_common.cuh"

namespace vh {

// These kernels are always launched as programmatic dependents: their CTAs may
// take their places while the previous kernel on the stream still runs, but
// touch no memory before this wait has returned, when that kernel and all
// before it are complete.  Only then may the next kernel do the same, so one
// that reads ahead of its own wait (VH_FLAG_PDL) meets finished work as it would
// behind an ordinary launch.
__device__ __forceinline__ void pdl_begin() {
  pdl_wait();
  pdl_launch_dependents();
}

// Largest b in [0, B) with key(b) <= x, for a non-decreasing key; -1 if there
// is none.  One warp: every round probes 32 places at once, so 1000 rows take
// two rounds of loads (a thread alone would take ten).
template <typename Key>
__device__ __forceinline__ int warp_last_at_most(int B, int x, int lane, Key key) {
  int lo = 0, n = B;  // key(lo - 1) <= x is known, or lo == 0; the answer lies in [lo - 1, lo + n)
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = lo + (lane + 1) * step - 1;  // last place of this lane's share
    const int i = min(at, lo + n - 1);
    const bool le = lane * step < n && key(i) <= x;
    const int c = __popc(__ballot_sync(0xffffffffu, le));  // shares whose last place is <= x
    const int done = min(n, c * step);
    lo += done;
    n = min(n - done, step - 1 < 0 ? 0 : step - 1);
  }
  return lo - 1;
}

// A piece's weight in a merge: not 0 however small beside the others, so that its
// infinities stay (a NaN stays a NaN).
__device__ __forceinline__ float at_least_tiny(float w) { return w < 1.2e-38f ? 1.2e-38f : w; }

// A row of a ragged batch.
struct RaggedRow {
  int start, end;  // its tokens
  int len;         // its tokens in the cache, the new ones among them
  bool ok;         // active and consistent
};

__device__ __forceinline__ RaggedRow ragged_row(const int32_t* token_start, const int32_t* seq_lens,
                                                const int32_t* active, int b, int T, int max_len,
                                                int32_t* err_flag, bool report) {
  RaggedRow r;
  r.start = token_start ? token_start[b] : b;
  r.end = token_start ? token_start[b + 1] : b + 1;
  r.len = seq_lens[b];
  const bool act = active[b] != 0;
  const bool sane = r.start >= 0 && r.end >= r.start && r.end <= T && r.len >= r.end - r.start && r.len <= max_len;
  r.ok = act && sane;
  if (report && act && !sane && r.end != r.start) flag_error(err_flag, VH_ERR_SEQLEN);
  return r;
}

// The row of token t, by one warp; -1 if it belongs to none.  Up to 32 rows are
// read at once, one a lane, so that a look-up costs one round trip to memory;
// with more rows the row is searched first.
__device__ __forceinline__ int warp_row_of_token(const int32_t* token_start, const int32_t* seq_lens,
                                                 const int32_t* active, int t, int B, int T, int max_len, int lane,
                                                 int32_t* err_flag, bool report, RaggedRow& r) {
  if (token_start && B <= 32) {
    RaggedRow mine{};
    bool here = false;
    if (lane < B) {
      mine = ragged_row(token_start, seq_lens, active, lane, T, max_len, nullptr, false);
      here = mine.start <= t && t < mine.end;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, here);
    if (hit == 0) return -1;
    const int row = 31 - __clz(hit);
    r.start = __shfl_sync(0xffffffffu, mine.start, row);
    r.end = __shfl_sync(0xffffffffu, mine.end, row);
    r.len = __shfl_sync(0xffffffffu, mine.len, row);
    r.ok = __shfl_sync(0xffffffffu, mine.ok ? 1 : 0, row) != 0;
    if (!r.ok && report && active[row]) flag_error(err_flag, VH_ERR_SEQLEN);
    return row;
  }
  const int row = token_start ? warp_last_at_most(B, t, lane, [&](int b) { return __ldg(token_start + b); }) : t;
  if (row < 0) return -1;
  r = ragged_row(token_start, seq_lens, active, row, T, max_len, err_flag, report);
  return r.start <= t && t < r.end ? row : -1;  // (offsets out of order may find a row that starts behind t)
}

}  // namespace vh
