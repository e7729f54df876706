// window_decode.cu -- single-token GQA attention over a sliding window and
// sinks of a paged cache, rows split over CTAs and merged in the launch.
//
// Operation: row b, L = seq_lens[b]; V = {j < L: j < S or j >= L - W};
//   o = sum_{j in V} softmax(scale <q_rot, K_j>) V_j,
// with a running max and sum in fp32.
//
// Bound by HBM: 4 G flops for the 4 bytes of a key and value element.
//  * Work list: a row's visible keys touch ns = ceil(min(S, L) / 16) tiles of
//    16 tokens at its head and the tiles from the window's first key to its
//    end; tiles between are not in the list.  The list of all rows is cut into
//    N ranges that differ by at most a tile, one a CTA, so a row is split
//    wherever its tiles straddle CTAs (a CTA has two partial rows at most).
//  * The producer warp describes 32 tiles at a time, one a lane (row, page,
//    visible keys), a batch ahead of its use, and copies each with tiled
//    tensor copies: one box of 16 tokens x all heads of the CTA per 64
//    columns of K and V, or for tiles whose visible keys lie in one half,
//    8-token boxes of that half only.  A page id out of range becomes a page
//    past the tensor, which the copy engine fills with zeros.
//  * A consumer warp per kv head: S^T = K q^T and O^T += V^T P^T on
//    mma.sync m16n8k16, the G heads padded to 8 columns, q and P split into a
//    high part and a residual of the element type so that products keep 16
//    bits of them (22 in fp16).  Keys outside V get -inf before the max, and
//    their rows of V are zeroed in shared memory, so nothing they hold counts.
//    Infinities that are seen make a NaN of a residual's product (0 times infinity,
//    or infinities of both signs) that the definition does not have: a warp whose
//    outputs come out as no numbers computes its share of the row once more, with
//    plain products in fp32.
//  * Merge: partial (o, lse) go to the workspace; a counter per row tells the
//    last CTA to arrive, which adds the pieces in their order in the row, so
//    the result does not depend on who is last.
#include "vh_ragged.cuh"
#include "vh_window.h"

namespace vh {

namespace {

constexpr int kMaxHeads = 8;                 // kv heads (consumer warps) of a CTA
constexpr int kThreadsMax = 32 * (kMaxHeads + 1);
constexpr int kWarpRows = 128;               // rows that the producer warp sums up alone
enum { kMiscTot = 0, kMiscAbort = 32, kMiscLost = 33, kMiscMost = 34, kMiscPart = 36, kMiscInts = 48 };  // part: 4 ints each

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
__device__ void scan_rows(int* cum, int n, int* tot) {
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

// Outputs of row b and kv head h from tiles k0 .. k1 - 1 of the row's list, by one warp and
// without split operands, for rows whose outputs are no numbers: a key has a lane for each
// half of its dimensions, then a lane has its columns of the values.  piece, lse: where the
// partial outputs go, or null: the final ones go to p.out.  About 11 us a tile (4 rows of
// 8000 tokens, 32 / 8 heads of 128: 40 us, with an infinity in each row 185), so the
// producer's wait for a stage would need a share of 90,000 tiles of one row to run out.  Out
// of line, so that the common path keeps its registers.  (More loads at a time, 120 us
// instead of 185, cost 8 q heads of one kv head 2 % of the common path.)
template <int D, int G, typename E>
__device__ __noinline__ void plain_outputs(const WindowDecodeParams& p, int b, int h, int L, int k0, int k1, float* piece, float* lse) {
  constexpr int PER = D / 32;
  constexpr float kDown = 24.f;  // weights of 2^-24 at most: 2^24 values near the type's end do not overflow
  const float NEG_INF = __int_as_float(0xff800000);
  const int lane = threadIdx.x & 31, key = lane & 15, half = lane >> 4;
  const RowTiles rt = tiles_of(L, p.window, p.sinks);
  const long long row = (static_cast<long long>(b) * p.Hq + static_cast<long long>(h) * G) * D;
  float o[G][PER], M[G], sum[G];
#pragma unroll
  for (int n = 0; n < G; ++n) {
    M[n] = NEG_INF;
    sum[n] = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[n][e] = 0.f;
  }
#pragma unroll 1
  for (int k = k0; k < k1; ++k) {
    const int tile = rt.tile(k);
    const uint32_t mask = visible16(tile, L, p.window, p.sinks);
    long long at[2];  // of the tile's halves (one page, but for pages of 8 tokens); -1: a page id out of range, read as zeros
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = tile * kTile + 8 * x;
      at[x] = -1;
      if (!(mask & (0xFFu << (8 * x)))) continue;
      const long long lp = static_cast<long long>(b) * p.max_pages_per_seq + j / p.P;
      const int page = p.page_table ? p.page_table[lp] : static_cast<int>(lp);
      if (page >= 0 && page < p.num_pages)
        at[x] = page * p.memory.page_stride + (j % p.P) * p.memory.token_stride + h * p.memory.head_stride;
    }
    // scores
    float s[G];
#pragma unroll
    for (int n = 0; n < G; ++n) s[n] = 0.f;
    const bool seen = (mask >> key) & 1u;
    const long long mine = (key < 8 ? at[0] : at[1]) + (key & 7) * p.memory.token_stride;
    if (seen && (key < 8 ? at[0] : at[1]) >= 0)
#pragma unroll 1
      for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(p.memory.k + mine + d);
        const float2 x = E::to_float2(w.x), y = E::to_float2(w.y);
#pragma unroll
        for (int n = 0; n < G; ++n) {
          const float4 a = *reinterpret_cast<const float4*>(p.q_rot + row + n * D + d);
          s[n] += a.x * x.x + a.y * x.y + a.z * y.x + a.w * y.y;
        }
      }
#pragma unroll
    for (int n = 0; n < G; ++n) {
      s[n] += __shfl_xor_sync(0xffffffffu, s[n], 16);
      s[n] = seen ? s[n] * p.scale_log2 : NEG_INF;
      float mx = s[n];
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      mx = fmaxf(mx, M[n]);
      const float ms = mx == NEG_INF ? 0.f : mx, by = at_least_tiny(exp2f(M[n] - ms));
      M[n] = mx;
      s[n] = s[n] == NEG_INF ? 0.f : at_least_tiny(exp2f(s[n] - ms - kDown));  // the weight
      float add = s[n];
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) add += __shfl_xor_sync(0xffffffffu, add, off);
      sum[n] = sum[n] * by + add;
#pragma unroll
      for (int e = 0; e < PER; ++e) o[n][e] *= by;
    }
    // values
#pragma unroll 1
    for (int r = 0; r < kTile; ++r) {
      if (!((mask >> r) & 1u)) continue;
      const long long page = r < 8 ? at[0] : at[1];
      float v[PER];
#pragma unroll
      for (int e = 0; e < PER; e += 2) {
        const uint32_t w = page < 0 ? 0u : *reinterpret_cast<const uint32_t*>(p.memory.v + page + (r & 7) * p.memory.token_stride + lane * PER + e);
        const float2 x = E::to_float2(w);
        v[e] = x.x;
        v[e + 1] = x.y;
      }
#pragma unroll
      for (int n = 0; n < G; ++n) {
        const float w = __shfl_sync(0xffffffffu, s[n], r);
#pragma unroll
        for (int e = 0; e < PER; ++e) o[n][e] += w * v[e];
      }
    }
  }
#pragma unroll
  for (int n = 0; n < G; ++n) {
    const float il = piece && sum[n] == 0.f ? 0.f : 1.f / sum[n];
#pragma unroll
    for (int e = 0; e < PER; e += 2) {
      const int d = n * D + lane * PER + e;
      if (piece) *reinterpret_cast<float2*>(piece + d) = make_float2(o[n][e] * il, o[n][e + 1] * il);
      else *reinterpret_cast<uint32_t*>(p.out + row + d) = E::pack2(o[n][e] * il, o[n][e + 1] * il);
    }
    if (piece && lane == 0) lse[n] = M[n] + kDown + log2f(sum[n]);
  }
  __syncwarp();
}

template <int D, int G, typename E>
__global__ void __launch_bounds__(kThreadsMax, 1) window_decode_kernel(const __grid_constant__ WindowDecodeParams p) {
  constexpr int KS = D / 16;      // k-steps of the score product = m-tiles of the value product
  constexpr int HALVES = D / 64;  // 128-byte column blocks of a K or V row
  constexpr int PER = D / 32;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hc = p.Hc, S = p.stages, HG = Hc * G;
  const int c = blockIdx.x, gy = blockIdx.y, h0 = gy * Hc;
  int* cum = reinterpret_cast<int*>(smem + p.cum_off);
  int* lens = reinterpret_cast<int*>(smem + p.len_off);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.bar_off);
  int* misc = reinterpret_cast<int*>(bars + 2 * S + 2 + kMaxHeads);
  volatile int* abort_flag = misc + kMiscAbort;
  const uint32_t full0 = smem_addr(bars), empty0 = smem_addr(bars + S);
  const uint32_t qfull = smem_addr(bars + 2 * S), qempty = smem_addr(bars + 2 * S + 1);
  const uint32_t merged0 = smem_addr(bars + 2 * S + 2);  // pieces have come, by consumer warp
  const int max_len = p.max_pages_per_seq * p.P;
  const bool p8 = p.P == 8;
  const float NEG_INF = __int_as_float(0xff800000);
  if (p.early) pdl_launch_dependents();
  else pdl_begin();

  // ---- work list (with VH_FLAG_PDL, before the wait) -------------------------------
  // Up to kWarpRows rows are counted and summed by the producer warp, which goes
  // on to its first copies while the consumers wait for the sums; more rows by
  // all threads.
  auto count_row = [&](int b) -> int {
    const int act = p.active[b], L = p.seq_lens[b];
    const bool ok = act && L >= 1 && L <= max_len;
    if (act && !ok && c == 0 && gy == 0) flag_error(p.err_flag, VH_ERR_SEQLEN);
    lens[b] = L;
    return ok ? tiles_of(L, p.window, p.sinks).count : 0;
  };
  if (warp == Hc) {
    if (lane == 0) {
      *abort_flag = 0;
      misc[kMiscLost] = 0;
      misc[kMiscMost] = 0;
      for (int s = 0; s < S; ++s) {
        mbar_init(full0 + 8 * s, 1);
        mbar_init(empty0 + 8 * s, Hc);
      }
      mbar_init(qfull, 1);
      mbar_init(qempty, Hc);
      for (int x = 0; x < Hc; ++x) mbar_init(merged0 + 8 * x, 1);
      fence_barrier_init();
      cum[0] = 0;
    }
    __syncwarp();
    if (p.B <= kWarpRows) {
      int n[kWarpRows / 32], run = 0;
#pragma unroll
      for (int x = 0; x < kWarpRows / 32; ++x) n[x] = x * 32 + lane < p.B ? count_row(x * 32 + lane) : 0;
#pragma unroll
      for (int x = 0; x < kWarpRows / 32; ++x) {
        if (x * 32 >= p.B) break;
        int v = n[x];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, v, off);
          if (lane >= off) v += y;
        }
        v += run;
        if (x * 32 + lane < p.B) cum[1 + x * 32 + lane] = v;
        run = __shfl_sync(0xffffffffu, v, 31);
      }
      int most = 0;
#pragma unroll
      for (int x = 0; x < kWarpRows / 32; ++x) most = max(most, n[x]);
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) misc[kMiscMost] = most;
      __syncwarp();
      asm volatile("bar.arrive 2, %0;" ::"r"(static_cast<int>(blockDim.x)) : "memory");
    }
  } else if (p.B <= kWarpRows) {
    named_sync(2, blockDim.x);
  }
  if (p.B > kWarpRows) {
    __syncthreads();
    int most = 0;
    for (int b = tid; b < p.B; b += blockDim.x) {
      const int n = count_row(b);
      cum[1 + b] = n;
      most = max(most, n);
    }
    atomicMax(misc + kMiscMost, most);
    __syncthreads();
    scan_rows(cum, p.B, misc + kMiscTot);
  }
  const int T = cum[p.B];
  // Shares: either T / n tiles each, of which a CTA takes at least q (a share streams
  // in about 0.5 us a tile, and the longest row's pieces, R / q of them, are then added
  // at about G / 40 us each, so q = sqrt(R G / 20) is the least of both; one row of 8000
  // tokens, 8 q heads of one kv head: 179 us with q = 1, 23 us with q = 14), or whole
  // rows, which need no merge: that takes 2.5 us (4.8 us against 7.3 for a few rows of
  // a tile or two), as long as 6 tiles.
  const int most = misc[kMiscMost];
  const int q = max(1, static_cast<int>(sqrtf(static_cast<float>(most) * (0.05f * G)) + 0.5f));
  const int rows_each = (p.B + p.N - 1) / p.N;
  const bool by_row = most * rows_each <= max(q, T / p.N) + 6;
  const int n_eff = by_row ? 0 : min(p.N, (T + q - 1) / q);  // CTAs that share the tiles
  int t0 = 0, t1 = 0, b0 = 0;
  if (by_row) {
    b0 = min(c * rows_each, p.B);
    t0 = cum[b0];
    t1 = cum[min(b0 + rows_each, p.B)];
  } else if (c < n_eff) {
    const int each = T / n_eff, rest = T - each * n_eff;  // the first `rest` CTAs take one tile more
    t0 = c * each + min(c, rest);
    t1 = t0 + each + (c < rest ? 1 : 0);
  }
  const bool works = t1 > t0;
  if (works) b0 = row_of(cum, b0, p.B, t0);
  const int tpp = (p.P + kTile - 1) / kTile;  // tiles of a page
  const int tpp_shift = (tpp & (tpp - 1)) == 0 ? __ffs(tpp) - 1 : -1;

  // ---- padding rows, dealt out to the CTAs, are written as zeros ---------------
  auto zero_rows = [&]() {
    for (int b = c; b < p.B; b += p.N) {
      if (cum[b + 1] != cum[b]) continue;
      uint4* dst = reinterpret_cast<uint4*>(p.out + (static_cast<long long>(b) * p.Hq + gy * HG) * D);
      for (int i = tid; i < HG * D / 8; i += blockDim.x) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  };

  if (warp == Hc) {
    // ======================= producer warp =====================================
    // a tile's description, one lane each
    struct Tile {
      int row, tok, page, page2;  // tok: first token in the page; page2: second page (8-token pages)
      uint32_t mask;
    };
    auto describe = [&](int t) -> Tile {
      Tile d{0, 0, 0, 0, 0u};
      if (t >= t1) return d;
      d.row = row_of(cum, b0, p.B, t);
      const int L = lens[d.row], tk = tiles_of(L, p.window, p.sinks).tile(t - cum[d.row]);
      d.mask = visible16(tk, L, p.window, p.sinks);
      auto page_at = [&](int j) -> int {
        const long long lp = static_cast<long long>(d.row) * p.max_pages_per_seq + j;
        return p.page_table ? p.page_table[lp] : static_cast<int>(lp);
      };
      if (p8) {
        if (d.mask & 0x00FFu) d.page = page_at(2 * tk);
        if (d.mask & 0xFF00u) d.page2 = page_at(2 * tk + 1);
      } else {
        const int j = tpp_shift >= 0 ? tk >> tpp_shift : tk / tpp;
        d.page = page_at(j);
        d.tok = (tk - j * tpp) * kTile;
      }
      return d;
    };
    Tile cur{}, nxt{};
    if (works) {
      cur = describe(t0 + lane);
      if (lane == 0) prefetch_tensormap(&p.tmap_k);
      if (lane == 1) prefetch_tensormap(&p.tmap_v);
    }
    if (p.early) pdl_wait();
    zero_rows();
    if (!works) return;
    // Boxes of this lane.  Whole tiles: lanes 0 .. 2 HALVES - 1 take (K or V,
    // column block).  Else one box per (half, head, column block, K or V).
    const int l_kv = lane & 1, l_hf = (lane >> 1) % HALVES;
    const int l_head = (lane / (2 * HALVES)) % Hc, l_g = lane / (2 * HALVES * Hc);
    const void* map16 = l_kv ? static_cast<const void*>(&p.tmap_v) : static_cast<const void*>(&p.tmap_k);
    const void* map8 = l_kv ? static_cast<const void*>(&p.tmap_v8) : static_cast<const void*>(&p.tmap_k8);
    const uint32_t off16 = static_cast<uint32_t>(l_kv * (p.stage_bytes / 2) + l_hf * Hc * 2048);
    const uint32_t off8 = off16 + static_cast<uint32_t>(l_head * 2048 + l_g * 1024);
    const uint64_t policy = l2_policy_evict_first();  // K and V are read once a launch
    int stage = 0, round = 0, nseg = 0, prev_row = -1, issued = 0;
    bool aborted = false;
    for (int t = t0; t < t1; ++t, ++issued) {
      const int w = (t - t0) & 31;
      if (w == 0 && t > t0) cur = nxt;
      const int row = __shfl_sync(0xffffffffu, cur.row, w), tok = __shfl_sync(0xffffffffu, cur.tok, w);
      const uint32_t mask = __shfl_sync(0xffffffffu, cur.mask, w);
      int page = __shfl_sync(0xffffffffu, cur.page, w), page2 = __shfl_sync(0xffffffffu, cur.page2, w);
      if (page < 0 || page >= p.num_pages || page2 < 0 || page2 >= p.num_pages) {
        if (lane == 0) flag_error(p.err_flag, VH_ERR_PAGE);
        if (page < 0 || page >= p.num_pages) page = p.num_pages;  // past the tensor: read as zeros
        if (page2 < 0 || page2 >= p.num_pages) page2 = p.num_pages;
      }
      if (row != prev_row) {
        // the next row's q, once the consumers have taken the last row's
        if (nseg > 0 && !mbar_wait(qempty, (nseg - 1) & 1)) {
          aborted = true;
          break;
        }
        if (lane == 0) {
          const long long qrow = static_cast<long long>(row) * p.Hq + static_cast<long long>(h0) * G;
          mbar_arrive_expect_tx(qfull, static_cast<uint32_t>(HG * D * 4));
          bulk_g2s(smem_addr(smem + p.q_off), p.q_rot + qrow * D, static_cast<uint32_t>(HG * D * 4), qfull);
        }
        ++nseg;
        prev_row = row;
      }
      if (issued >= S && !mbar_wait(empty0 + 8 * stage, (round - 1) & 1)) {
        aborted = true;
        break;
      }
      if (*abort_flag) {
        aborted = true;
        break;
      }
      const bool lo_half = (mask & 0x00FFu) != 0, hi_half = (mask & 0xFF00u) != 0, both = lo_half && hi_half;
      const uint32_t st = smem_addr(smem) + static_cast<uint32_t>(stage * p.stage_bytes), fb = full0 + 8 * stage;
      if (lane == 0) mbar_arrive_expect_tx(fb, static_cast<uint32_t>(both ? p.stage_bytes : p.stage_bytes / 2));
      __syncwarp();
      if (both && p.full_boxes && !p8) {
        if (lane < 2 * HALVES) tma_load_4d_hint(st + off16, map16, l_hf * 64, tok, h0, page, fb, policy);
      } else if (l_g < 2 && (l_g ? hi_half : lo_half)) {
        const int tk = p8 ? 0 : tok + 8 * l_g;
        const int c1 = p.tm_tok_dim == 1 ? tk : h0 + l_head, c2 = p.tm_tok_dim == 1 ? h0 + l_head : tk;
        tma_load_4d_hint(st + off8, map8, l_hf * 64, c1, c2, (p8 && l_g) ? page2 : page, fb, policy);
      }
      if (++stage == S) {
        stage = 0;
        ++round;
      }
      // the next 32 tiles, well ahead, but not before the first copies are under way
      if (w == 7) nxt = describe(t - w + 32 + lane);
    }
    if (aborted) {
      if (lane == 0) flag_error(p.err_flag, VH_ERR_TIMEOUT);
      *abort_flag = 1;
      // copies in flight land before the shared memory goes away
      for (int k = max(0, issued - S); k < issued; ++k) (void)mbar_wait(full0 + 8 * (k % S), (k / S) & 1);
      if (nseg > 0) (void)mbar_wait(qfull, (nseg - 1) & 1);
    }
    return;
  }

  // ========================= consumer warps ======================================
  if (p.early) pdl_wait();
  zero_rows();
  if (!works) return;
  const int w = warp, h = h0 + w;
  const int g4 = lane >> 2, t4 = lane & 3;
  // ldmatrix rows of this lane; chunk c of row r of a swizzled box lies at c ^ (r & 7)
  const int ka_row = (lane & 7) + 8 * ((lane >> 3) & 1), va_row = (lane & 7) + 8 * (lane >> 4);
  const int ksw = (lane >> 4) ^ (ka_row & 7), vsw = ((lane >> 3) & 1) ^ (va_row & 7);
  const uint32_t block_bytes = static_cast<uint32_t>(Hc) * 2048u;  // one column block of all heads
  auto row_off = [&](int r) -> uint32_t { return static_cast<uint32_t>(w * 2048 + r * 128); };

  uint32_t qh[KS][2], ql[KS][2];
  float acc[KS][4];
  float m0 = NEG_INF, m1 = NEG_INF, l0 = 0.f, l1 = 0.f;
  int b = b0, rt0 = cum[b0], rt1 = cum[b0 + 1];
  RowTiles rt = tiles_of(lens[b], p.window, p.sinks);
  int nseg = 0, stage = 0, round = 0, npart = 0;
  int part_row[2];
  bool lost = false;
  for (int t = t0; t < t1 && !lost; ++t) {
    const bool next_row = t >= rt1;
    if (next_row) {
      do {
        ++b;
        rt0 = rt1;
        rt1 = cum[b + 1];
      } while (t >= rt1);
      rt = tiles_of(lens[b], p.window, p.sinks);
    }
    if (next_row || t == t0) {
      if (!mbar_wait(qfull, nseg & 1)) {
        lost = true;
        break;
      }
      const float* qrow = reinterpret_cast<const float*>(smem + p.q_off) + (w * G + (g4 < G ? g4 : 0)) * D;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        float2 x = make_float2(0.f, 0.f), y = x;
        if (g4 < G) {
          x = *reinterpret_cast<const float2*>(qrow + 16 * k + 2 * t4);
          y = *reinterpret_cast<const float2*>(qrow + 16 * k + 2 * t4 + 8);
        }
        split2<E>(x.x, x.y, qh[k][0], ql[k][0]);
        split2<E>(y.x, y.y, qh[k][1], ql[k][1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(qempty);
      ++nseg;
      m0 = m1 = NEG_INF;
      l0 = l1 = 0.f;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
    }
    const uint32_t mask = visible16(rt.tile(t - rt0), lens[b], p.window, p.sinks);
    if (!mbar_wait(full0 + 8 * stage, round & 1)) {
      lost = true;
      break;
    }
    unsigned char* stg = smem + stage * p.stage_bytes;
    if (mask != 0xFFFFu) {
      // rows of V that are not visible (or were not copied) meet P = 0: make them zeros
      unsigned char* vst = stg + p.stage_bytes / 2;
      constexpr int CH = D / 8;
      for (int r = lane / CH; r < kTile; r += 32 / CH) {
        if ((mask >> r) & 1u) continue;
        const int ch = lane % CH;
        *reinterpret_cast<uint4*>(vst + (ch >> 3) * block_bytes + row_off(r) + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
    }

    // scores: lane holds keys g4 and g4 + 8, heads 2 t4 and 2 t4 + 1
    float sh[4] = {0.f, 0.f, 0.f, 0.f}, sl[4] = {0.f, 0.f, 0.f, 0.f};
    {
      const uint32_t ka = smem_addr(stg) + row_off(ka_row);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4(ka + (k >> 2) * block_bytes + ((((2 * k) & 7) ^ ksw) << 4), a0, a1, a2, a3);
        E::mma(sh, a0, a1, a2, a3, qh[k][0], qh[k][1]);
        E::mma(sl, a0, a1, a2, a3, ql[k][0], ql[k][1]);
      }
    }
    const bool va = (mask >> g4) & 1u, vb = (mask >> (g4 + 8)) & 1u;
    const float s0 = va ? (sh[0] + sl[0]) * p.scale_log2 : NEG_INF;
    const float s1 = va ? (sh[1] + sl[1]) * p.scale_log2 : NEG_INF;
    const float s2 = vb ? (sh[2] + sl[2]) * p.scale_log2 : NEG_INF;
    const float s3 = vb ? (sh[3] + sl[3]) * p.scale_log2 : NEG_INF;
    float mx0 = fmaxf(s0, s2), mx1 = fmaxf(s1, s3);
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
    }
    const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
    // (a max of -inf, from keys that hold infinities, is subtracted as 0)
    const float ms0 = mn0 == NEG_INF ? 0.f : mn0, ms1 = mn1 == NEG_INF ? 0.f : mn1;
    const float al0 = exp2f(m0 - ms0), al1 = exp2f(m1 - ms1);
    const float p0 = exp2f(s0 - ms0), p2 = exp2f(s2 - ms0);
    const float p1 = exp2f(s1 - ms1), p3 = exp2f(s3 - ms1);
    l0 = l0 * al0 + (p0 + p2);
    l1 = l1 * al1 + (p1 + p3);
    m0 = mn0;
    m1 = mn1;
    uint32_t ph01, pl01, ph23, pl23;
    split2<E>(p0, p1, ph01, pl01);
    split2<E>(p2, p3, ph23, pl23);
    const uint32_t bh0 = movm_t(ph01), bh1 = movm_t(ph23), bl0 = movm_t(pl01), bl1 = movm_t(pl23);
    if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        acc[mt][0] *= al0;
        acc[mt][1] *= al1;
        acc[mt][2] *= al0;
        acc[mt][3] *= al1;
      }
    }
    {
      const uint32_t va0 = smem_addr(stg) + static_cast<uint32_t>(p.stage_bytes / 2) + row_off(va_row);
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4_t(va0 + (mt >> 2) * block_bytes + ((((2 * mt) & 7) ^ vsw) << 4), a0, a1, a2, a3);
        E::mma(acc[mt], a0, a1, a2, a3, bh0, bh1);
        E::mma(acc[mt], a0, a1, a2, a3, bl0, bl1);
      }
    }
    if (mask != 0xFFFFu) fence_proxy_async_smem();  // the zeros, before the next copy into this stage
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8 * stage);
    if (++stage == S) {
      stage = 0;
      ++round;
    }

    // ---- end of this CTA's share of a row: finished output, or a partial one ------
    if (t + 1 == t1 || t + 1 == rt1) {
      float L0 = l0, L1 = l1;
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        L0 += __shfl_xor_sync(0xffffffffu, L0, off);
        L1 += __shfl_xor_sync(0xffffffffu, L1, off);
      }
      const int n0 = 2 * t4, n1 = 2 * t4 + 1;
      float probe0 = 0.f, probe1 = 0.f;  // become NaN with an output that is no number
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        probe0 += acc[mt][0] * 0.f + acc[mt][2] * 0.f;
        probe1 += acc[mt][1] * 0.f + acc[mt][3] * 0.f;
      }
      const bool odd = (n0 < G && probe0 != 0.f) || (n1 < G && probe1 != 0.f);
      float *piece = nullptr, *lse = nullptr;
      if (rt0 >= t0 && rt1 <= t1) {
        const float il0 = 1.f / L0, il1 = 1.f / L1;
        uint16_t* o0 = p.out + (static_cast<long long>(b) * p.Hq + static_cast<long long>(h) * G + n0) * D;
        uint16_t* o1 = o0 + D;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          const int d = mt * 16 + g4;
          if (n0 < G) {
            o0[d] = E::bits(acc[mt][0] * il0);
            o0[d + 8] = E::bits(acc[mt][2] * il0);
          }
          if (n1 < G) {
            o1[d] = E::bits(acc[mt][1] * il1);
            o1[d + 8] = E::bits(acc[mt][3] * il1);
          }
        }
      } else {
        // piece slot 0 of a CTA belongs to its first row, slot 1 to a later one
        const float il0 = L0 > 0.f ? 1.f / L0 : (L0 == 0.f ? 0.f : L0), il1 = L1 > 0.f ? 1.f / L1 : (L1 == 0.f ? 0.f : L1);
        const long long base = ((static_cast<long long>(gy) * p.N + c) * 2 + (b == b0 ? 0 : 1)) * HG + w * G;
        piece = p.part_o + base * D;
        lse = p.part_lse + base;
        float* o0 = piece + n0 * D;
        float* o1 = o0 + D;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          const int d = mt * 16 + g4;
          if (n0 < G) {
            o0[d] = acc[mt][0] * il0;
            o0[d + 8] = acc[mt][2] * il0;
          }
          if (n1 < G) {
            o1[d] = acc[mt][1] * il1;
            o1[d + 8] = acc[mt][3] * il1;
          }
        }
        if (g4 == 0) {
          if (n0 < G) p.part_lse[base + n0] = m0 + log2f(L0);
          if (n1 < G) p.part_lse[base + n1] = m1 + log2f(L1);
        }
        part_row[npart++ & 1] = b;
      }
      if (__any_sync(0xffffffffu, odd)) {
        __syncwarp();
        plain_outputs<D, G, E>(p, b, h, lens[b], max(t0, rt0) - rt0, t + 1 - rt0, piece, lse);
        // (the next row sets these anew: nothing of them is kept over the call)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qh[k][0] = qh[k][1] = ql[k][0] = ql[k][1] = 0u;
          acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.f;
        }
        m0 = m1 = l0 = l1 = 0.f;
      }
    }
  }
  if (lost) {
    if (lane == 0) flag_error(p.err_flag, VH_ERR_TIMEOUT);
    *abort_flag = 1;
    *reinterpret_cast<volatile int*>(misc + kMiscLost) = 1;
  }

  // ---- count this CTA's pieces (the consumers agree on which there are) ------------
  named_sync(1, 32 * Hc);
  // (only consumers set this one, before the barrier: they all see the same)
  if (*reinterpret_cast<volatile int*>(misc + kMiscLost) || npart == 0) return;
  if (tid < npart) {  // (a thread a piece: their counters answer at the same time)
    const int rb = tid == 0 ? part_row[0] : part_row[1];
    const int first = share_of(cum[rb], n_eff, T), last = share_of(cum[rb + 1] - 1, n_eff, T);
    // acquire-release at GPU scope: publishes this CTA's pieces (ordered before
    // it by the barrier) and lets the last one see all others
    int* counter = p.counters + static_cast<long long>(gy) * p.B + rb;
    const bool mine = atom_add_acq_rel_gpu(counter, 1) == last - first;
    if (mine) *counter = 0;  // ready for the next call
    int* v = misc + kMiscPart + 4 * tid;
    v[0] = mine ? 1 : 0;
    v[1] = first;
    v[2] = last - first + 1;
    v[3] = share_begin(first, n_eff, T) == cum[rb] ? 0 : 1;  // the first piece's slot
  }
  named_sync(1, 32 * Hc);

  // ---- the last CTA of a row adds its pieces: warp w those of kv head w -------------
  uint32_t merges = 0;
  for (int k = 0; k < npart; ++k) {
    const int* v = misc + kMiscPart + 4 * k;
    if (!v[0]) continue;
    const int first = v[1], np = v[2], slot0 = v[3];
    auto piece = [&](int j) -> long long {
      return ((static_cast<long long>(gy) * p.N + first + j) * 2 + (j == 0 ? slot0 : 0)) * HG + w * G;
    };
    float M[G], sum[G], o[G][PER];
#pragma unroll
    for (int n = 0; n < G; ++n) {
      M[n] = NEG_INF;
      sum[n] = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[n][i] = 0.f;
    }
    // Weights of the pieces j0 .. j0 + nj - 1, lane j that of piece j0 + j, and the
    // sums so far in the new maximum's terms.
    float wt[G];
    auto weigh = [&](int j0, int nj) {
#pragma unroll
      for (int n = 0; n < G; ++n) {
        const float lse = lane < nj ? __ldcg(p.part_lse + piece(j0 + lane) + n) : NEG_INF;
        float mx = lse;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        mx = fmaxf(mx, M[n]);
        const float ms = mx == NEG_INF ? 0.f : mx;
        const float sc = at_least_tiny(exp2f(M[n] - ms));
        M[n] = mx;
        wt[n] = lse == NEG_INF ? 0.f : at_least_tiny(exp2f(lse - ms));
        float add = wt[n];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) add += __shfl_xor_sync(0xffffffffu, add, off);
        sum[n] = sum[n] * sc + add;
#pragma unroll
        for (int i = 0; i < PER; ++i) o[n][i] *= sc;
      }
    };
    constexpr int PIECE = G * D * 4;
    const uint32_t share = static_cast<uint32_t>(S * p.stage_bytes / Hc) & ~127u;
    const int each = min(32, static_cast<int>(share / PIECE));
    if (each * G >= 64) {
      // One or two heads a CTA: the warp's share of the stages (all tiles have been
      // consumed) holds many pieces, so they come by bulk copies, one trip to memory for
      // up to 32 of them (12 rows of 6000 tokens, 4 q heads of one kv head: 27 -> 22 us;
      // with 4 kv heads a CTA it would be 4 or 8, and 24 -> 29 us for G = 8).
      const uint32_t room = smem_addr(smem) + static_cast<uint32_t>(w) * share;
      for (int j0 = 0; j0 < np; j0 += each) {
        const int nj = min(each, np - j0);
        // what was read and written there by loads and stores comes before the copies, and
        // what other CTAs wrote (seen by the counter's acquire) too
        asm volatile("fence.proxy.async;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(merged0 + 8 * w, static_cast<uint32_t>(nj * PIECE));
        __syncwarp();
        if (lane < nj) bulk_g2s(room + lane * PIECE, p.part_o + piece(j0 + lane) * D, PIECE, merged0 + 8 * w);
        weigh(j0, nj);
        const bool came = mbar_wait(merged0 + 8 * w, merges & 1u) || mbar_wait(merged0 + 8 * w, merges & 1u);
        ++merges;
        if (!came) {
          if (lane == 0) flag_error(p.err_flag, VH_ERR_TIMEOUT);
          return;
        }
        for (int j = 0; j < nj; ++j) {
          const uint32_t at = room + static_cast<uint32_t>(j * PIECE + lane * PER * 4);
#pragma unroll
          for (int n = 0; n < G; ++n) {
            const float f = __shfl_sync(0xffffffffu, wt[n], j);
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
              float2 x;
              asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(at + n * D * 4 + i * 4));
              o[n][i] += f * x.x;
              o[n][i + 1] += f * x.y;
            }
          }
        }
        __syncwarp();
      }
    } else {
      for (int j0 = 0; j0 < np; j0 += 32) {
        const int nj = min(32, np - j0);
        weigh(j0, nj);
        constexpr int U = 16 / G;  // pieces loaded at a time: 16 loads in flight
        for (int j = 0; j < nj; j += U) {
          float x[U][G][PER];
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int n = 0; n < G; ++n) {
              const float* src = p.part_o + (piece(j0 + min(j + u, nj - 1)) + n) * D + lane * PER;
              if constexpr (PER == 4) {
                const float4 f = __ldcg(reinterpret_cast<const float4*>(src));
                x[u][n][0] = f.x;
                x[u][n][1] = f.y;
                x[u][n][2] = f.z;
                x[u][n][3] = f.w;
              } else {
                const float2 f = __ldcg(reinterpret_cast<const float2*>(src));
                x[u][n][0] = f.x;
                x[u][n][1] = f.y;
              }
            }
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int n = 0; n < G; ++n) {
              const float f = __shfl_sync(0xffffffffu, wt[n], min(j + u, 31));
              if (j + u < nj) {
#pragma unroll
                for (int i = 0; i < PER; ++i) o[n][i] += f * x[u][n][i];
              }
            }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < G; ++n) {
      const float il = 1.f / sum[n];
      uint16_t* dst = p.out + (static_cast<long long>(part_row[k]) * p.Hq + static_cast<long long>(h) * G + n) * D + lane * PER;
#pragma unroll
      for (int i = 0; i < PER; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = E::pack2(o[n][i] * il, o[n][i + 1] * il);
    }
  }
}

using Kernel = void (*)(WindowDecodeParams);

template <typename E>
Kernel select_t(int D, int G) {
  if (D == 128) {
    switch (G) {
      case 1: return &window_decode_kernel<128, 1, E>;
      case 2: return &window_decode_kernel<128, 2, E>;
      case 4: return &window_decode_kernel<128, 4, E>;
      case 8: return &window_decode_kernel<128, 8, E>;
    }
  } else if (D == 64) {
    switch (G) {
      case 1: return &window_decode_kernel<64, 1, E>;
      case 2: return &window_decode_kernel<64, 2, E>;
      case 4: return &window_decode_kernel<64, 4, E>;
      case 8: return &window_decode_kernel<64, 8, E>;
    }
  }
  return nullptr;
}

Kernel select_kernel(int D, int G, bool f16) { return f16 ? select_t<ElemF16>(D, G) : select_t<ElemBf16>(D, G); }

}  // namespace

cudaError_t prepare_window_decode(int max_smem) {
  for (int D : {64, 128})
    for (int G : {1, 2, 4, 8})
      for (bool f16 : {false, true}) {
        const cudaError_t e =
            cudaFuncSetAttribute(select_kernel(D, G, f16), cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

cudaError_t window_decode_occupancy(const WindowDecodeParams& p, int* blocks_per_sm) {
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, select_kernel(p.D, p.G, p.f16 != 0),
                                                       32 * (p.Hc + 1), p.smem_bytes);
}

cudaError_t launch_window_decode(const WindowDecodeParams& p, cudaStream_t stream) {
  return launch_dependent(select_kernel(p.D, p.G, p.f16 != 0), p, dim3(p.N, p.groups), 32 * (p.Hc + 1),
                          static_cast<size_t>(p.smem_bytes), stream);
}

}  // namespace vh
