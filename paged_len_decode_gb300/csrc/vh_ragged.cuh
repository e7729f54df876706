// vh_ragged.cuh -- device helpers of ragged batches: the row of a token or of
// a block of tokens, and the checks of a row's extent.
#pragma once

#include "vh_common.cuh"

namespace vh {

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

}  // namespace vh
