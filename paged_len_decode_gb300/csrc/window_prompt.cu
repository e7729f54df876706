// window_prompt.cu -- attention of a ragged batch of new tokens over the paged
// cache, with a sliding window and sinks.
//
// Operation: the token in slot i of its row sees V(i) = {j <= i: i - j < W or
// j < S};  o = sum_{j in V(i)} softmax(scale <q, K_j>) V_j, per q head, with
// kv head h = head / G.
//
// Bound by the tensor cores: 4 D flops a query, head and visible key, on
// tcgen05.mma with fp32 accumulators in tensor memory.
//  * Blocks.  A CTA takes 256 rows, a row being a (token, head of the group):
//    the G q heads that share a kv head fill the rows, so short chunks waste
//    less and K and V are read once for the whole group.  The rows form two
//    tiles of 128, whose products and softmax alternate: while one tile's
//    scores are turned into weights, the tensor cores work for the other.  A
//    block holds tokens of one request.  Where such blocks would be few or
//    mostly empty, they have 128 rows (PAIR): the two tiles are then the same
//    rows, over alternate key tiles, and their accumulators are added at the end.
//  * Keys.  A list of boxes, runs of slots within a page: those that hold sinks,
//    then those from the first query's window to the last query.  128 / box of
//    them make a key tile, so that four sinks cost a box and not a tile.  They are
//    copied through the page table; boxes past the list and bad page ids become a
//    page past the tensor, which the copy engine fills with zeros without reading.
//    A tile that one of the two row tiles does not see is skipped for it.
//  * Warps: two warpgroups for the softmax of a row tile each (a thread owns a
//    row, so its maximum and sum need no exchange), one warp that issues the
//    products, two that copy K and V through a ring of stages, and one that
//    draws the CTA's next block from a counter while this one is computed
//    (requests with the longest contexts first, so that the last blocks are
//    short).  The copies of the next block run while the last products and
//    outputs of this one are under way.
//  * Softmax.  Running maximum and sum in fp32; the accumulator is rescaled
//    only when a row's maximum has grown by more than 2^8 since the last time
//    (weights stay below 2^8, in fp16, scaled, below 2^15: inside each type), so it is rare.
//    Weights go back to tensor memory as 16-bit operands of the value product,
//    over the scores: rounding them costs one half step of the element type
//    relatively, as the output's own rounding does, and saves a second product.
//  * What is not seen: scores get -inf; rows of V that no query of the block
//    sees (page tails, freed pages) are zeroed in shared memory.  A value that
//    some rows of a tile see and others do not meets weight 0 there, which is
//    harmless unless it is infinite or NaN; so does one whose weight is too small
//    for the element type.  A block with an output that is no number, although its
//    row's sum is one, therefore runs once more, by the same pipeline, with such
//    values as zeros (two to three times its usual time: V is filtered between copy
//    and product), and then once for each kind of them (+inf, -inf, NaN) that was met,
//    over the key tiles from the first to the last that hold one, with the values of that
//    kind as ones and the others as zeros and weight 1 for every visible key: outputs
//    that come out above zero are set to what they must be.  That is bounded whatever
//    the cache holds, and the waits remain those of a tile.  In a cluster, where
//    partial outputs lie in memory that the runs need, the kinds are noted beside
//    them and set in a last run.  All of this is kept apart from the common path: a
//    function call, or code for it between the products, costs that 2 to 8 us of 43
//    (24 ragged prompts of up to 800 tokens, head_dim 64), though never executed.
//  * Few blocks (short chunks over long contexts): the key tiles of a block are
//    shared by a cluster of up to 16 CTAs, which leave their partial results in
//    shared memory and add them over distributed shared memory, each a share of
//    the rows.
#include "vh_ragged.cuh"
#include "vh_tcgen05.cuh"
#include "vh_window.h"

namespace vh {

namespace {

constexpr int kRows = 128;       // rows of a row tile
constexpr int kKeys = 128;       // keys of a key tile
constexpr int kThreads = 384;    // two softmax warpgroups, and one whose warps issue products and copies
constexpr int kProductWarp = 8, kCopyWarp = 9, kDrawWarp = 11;  // the copy warp takes K and the queries, the next one V
constexpr int kSlots = 2;        // blocks drawn: this one and the next
constexpr float kGrow = 8.f;     // log2 of the growth that rescales
// log2 of the weight of the row's maximum: fp16 weights stay below 2^15 then, and those down to
// 2^-32 of the largest count (at 2^-24 the type's range would end).  bf16 has fp32's range.
template <typename E>
constexpr float kLift = E::kF16 ? 7.f : 0.f;
// The same where a block runs again for its outputs: bf16 values near the type's end may have
// overflowed in the sum of the products, so the weights are 2^-24 at most, for 2^24 keys.
template <typename E>
constexpr float kLiftAgain = E::kF16 ? 7.f : -32.f;
constexpr uint32_t kTmem = 512;  // columns: scores of both row tiles, then their outputs

// What a block is run for: its outputs; and where some of them are no numbers, its
// outputs with values that are no numbers left out, and then which of them such
// values reach: +inf, -inf, NaN, and infinities under a score of -inf (0 times
// infinity is NaN).  What a run has met is noted in bits of its slot: bit 0, outputs
// that are no numbers; bit m - 1, something for mode m.
enum { kPlain, kWithout, kPlusInf, kMinusInf, kNaN, kNoWeight, kSettle };

// One CTA's work: queries of one request and kv head, and a share of their key tiles.
struct Unit {
  int row, first, ntok;         // request, first token, tokens
  int slot;                     // slot of the first token
  int h, z;                     // kv head, share of the keys
  int sink_boxes, from, boxes;  // boxes 0 .. sink_boxes - 1 of the row, then `from` on; `boxes` in all
  int count;                    // key tiles
  int k0, k1;                   // this CTA's of them; k0 == k1: nothing to do
  int mode;                     // kPlain, or once more
  int settle;                   // the last of a cluster's runs: what was noted is set
  int soft;                     // k1, or k0 where the unit runs once more (or has nothing to do)
  int all0, all1;               // k0 and k1 of the first run
  int more;                     // 0: no unit, the CTA is done
};

// The slots of key tile k: column c holds slot base + c, from column `jump` on base + c + gap.
struct Columns {
  int base, jump, gap;
  __device__ int slot(int c) const { return base + c + (c >= jump ? gap : 0); }
};

__device__ __forceinline__ Columns columns_of(int sink_boxes, int from, int k, int shift_box) {
  const int b = k << (7 - shift_box), gap = from - sink_boxes;  // first box; boxes left out
  Columns x;
  const bool sinks = b < sink_boxes;
  x.base = (sinks ? b : b + gap) << shift_box;
  x.jump = sinks ? (sink_boxes - b) << shift_box : kKeys;
  x.gap = gap << shift_box;
  return x;
}

__device__ __forceinline__ int share_begin(int c, int n, int total) { return c * (total / n) + min(c, total % n); }

// The boxes of `ntok` queries from `slot` on.
__device__ __forceinline__ void list_boxes(const PromptParams& p, int slot, int ntok, int& sink_boxes, int& from, int& boxes) {
  const int last = slot + ntok - 1;
  sink_boxes = (min(p.sinks, last + 1) + p.box - 1) >> p.shift_box;
  from = max(sink_boxes, max(0, slot - p.window + 1) >> p.shift_box);
  boxes = sink_boxes + (last >> p.shift_box) + 1 - from;
}

// The key tiles that row tile m of a block sees: below s_end, and from w_begin to w_end.
struct Tiles {
  int s_end, w_begin, w_end;
  __device__ bool has(int k) const { return k < s_end || (k >= w_begin && k < w_end); }
};
__device__ __forceinline__ Tiles tiles_of(const PromptParams& p, const Unit& u, int m) {
  const int per_tile = kRows >> p.shift_g, last = u.slot + u.ntok - 1, f = u.slot + m * per_tile, e = min(last, f + per_tile - 1);
  const int shift = 7 - p.shift_box, to = u.sink_boxes + (e >> p.shift_box) - u.from;
  Tiles t;
  t.s_end = f > last ? 0 : min((u.sink_boxes + (1 << shift) - 1) >> shift, (e >> 7) + 1);
  t.w_begin = (u.sink_boxes + max(0, (max(0, f - p.window + 1) >> p.shift_box) - u.from)) >> shift;
  t.w_end = f > last || to < u.sink_boxes ? 0 : (to >> shift) + 1;
  return t;
}

// What the drawing warp knows of up to 32 requests, one a lane: with these, a
// block is found without reading memory, and blocks of requests with more key
// tiles come first.  (With more requests, block i belongs to the last row b
// with token_start[b] / tokens + b <= i, a search in memory.)
struct Rows {
  RaggedRow r;
  int blocks, before;  // of this request, and of those that come before it
};

__device__ __forceinline__ Rows rows_of(const PromptParams& p, int lane) {
  Rows x{};
  const int per = 1 << p.shift_block;
  int weight = -1;
  if (lane < p.B) {
    x.r = ragged_row(p.token_start, p.seq_lens, p.active, lane, p.T, p.max_pages_per_seq * p.P, p.err_flag, blockIdx.x == 0);
    const int n = x.r.start >= 0 ? min(x.r.end, p.T) - x.r.start : 0;
    x.blocks = n > 0 ? (n + per - 1) >> p.shift_block : 0;
    if (x.r.ok && n > 0) {
      int a, b;
      list_boxes(p, x.r.len - min(n, per), min(n, per), a, b, weight);
    }
  }
  int rank = 0;
  for (int j = 0; j < p.B; ++j) {
    const int w = __shfl_sync(0xffffffffu, weight, j);
    rank += (w > weight || (w == weight && j < lane)) ? 1 : 0;
  }
  for (int j = 0; j < p.B; ++j) {
    const int k = __shfl_sync(0xffffffffu, rank, j), n = __shfl_sync(0xffffffffu, x.blocks, j);
    x.before += k < rank ? n : 0;
  }
  return x;
}

// Unit u, by one warp.  Tokens of inactive and flagged requests are written as
// zeros here.
__device__ __forceinline__ Unit unit_of(const PromptParams& p, const Rows& rows, int u, int lane) {
  Unit r{};
  r.more = 1;
  const int per = 1 << p.shift_block;
  r.z = u & (p.splits - 1);
  const int v = u >> p.shift_splits;
  const int i = static_cast<int>(__umulhi(static_cast<uint32_t>(v), p.hkv_inverse)) - (p.hkv_inverse == 0 ? -v : 0);  // v / Hkv
  r.h = v - i * p.Hkv;
  RaggedRow g{};
  int n;  // number of the block in its request
  if (p.B <= 32) {
    const uint32_t hit = __ballot_sync(0xffffffffu, lane < p.B && i >= rows.before && i < rows.before + rows.blocks);
    if (hit == 0) return r;
    r.row = __ffs(hit) - 1;
    g.start = __shfl_sync(0xffffffffu, rows.r.start, r.row);
    g.end = __shfl_sync(0xffffffffu, rows.r.end, r.row);
    g.len = __shfl_sync(0xffffffffu, rows.r.len, r.row);
    g.ok = __shfl_sync(0xffffffffu, rows.r.ok ? 1 : 0, r.row) != 0;
    // the last block of a request sees the most
    n = __shfl_sync(0xffffffffu, rows.blocks, r.row) - 1 - (i - __shfl_sync(0xffffffffu, rows.before, r.row));
  } else {
    const int bi = p.blocks - 1 - i;
    r.row = warp_last_at_most(p.B, bi, lane, [&](int b) { return (p.token_start[b] >> p.shift_block) + b; });
    if (r.row < 0) return r;
    g = ragged_row(p.token_start, p.seq_lens, p.active, r.row, p.T, p.max_pages_per_seq * p.P, p.err_flag,
                   lane == 0 && r.h == 0 && r.z == 0);
    n = bi - ((g.start >> p.shift_block) + r.row);
  }
  r.first = g.start + n * per;
  r.ntok = min(per, min(g.end, p.T) - r.first);
  if (g.start < 0 || n < 0 || r.ntok <= 0) return r;
  if (!g.ok) {
    if (r.z == 0)
      for (int t = 0; t < r.ntok; ++t) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + ((r.first + t) * static_cast<long long>(p.Hq) + r.h * p.G) * p.D);
        for (int x = lane; x < p.G * p.D / 8; x += 32) dst[x] = make_uint4(0u, 0u, 0u, 0u);
      }
    return r;
  }
  r.slot = g.len - (g.end - r.first);
  list_boxes(p, r.slot, r.ntok, r.sink_boxes, r.from, r.boxes);
  r.count = (r.boxes + (kKeys >> p.shift_box) - 1) >> (7 - p.shift_box);
  if (p.splits == 1) {
    r.k1 = r.count;
    return r;
  }
  const int splits = min(p.splits, r.count);
  if (r.z < splits) {
    r.k0 = share_begin(r.z, splits, r.count);
    r.k1 = share_begin(r.z + 1, splits, r.count);
  }
  return r;
}

// Keys c of 32 that are visible, as bits: c < above, and c >= low or c < sink.
__device__ __forceinline__ uint32_t below32(int x) { return x <= 0 ? 0u : (x >= 32 ? 0xffffffffu : (1u << x) - 1u); }
__device__ __forceinline__ uint32_t visible32(int above, int low, int sink) {
  return below32(above) & (~below32(low) | below32(sink));
}

// The keys of columns c .. c + 31 that the query in slot i sees.
__device__ __forceinline__ uint32_t visible_of(const Columns& cols, int c, int i, int window, int sinks) {
  const int jc = cols.base + c;
  uint32_t vis = visible32(i + 1 - jc, i - window + 1 - jc, sinks - jc);
  if (cols.jump < kKeys) {
    const int jg = jc + cols.gap;  // the word's first slot behind the jump
    const uint32_t lead = below32(cols.jump - c);
    vis = (vis & lead) | (visible32(i + 1 - jg, i - window + 1 - jg, sinks - jg) & ~lead);
  }
  return vis;
}

// Chunk of 16 bytes `c` of row r of the partial outputs that a CTA of a cluster
// leaves in its shared memory (fp32 [256][D]): chunks turned by the row, so that
// 32 rows written at the same chunk fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t part_off(int r, int c) {
  return static_cast<uint32_t>(r * D * 4 + ((c ^ (r & (D / 4 - 1))) << 4));
}

// The two elements of a word of V, as `mode` takes them; `met`: kinds of values found.
template <typename E>
__device__ __forceinline__ uint32_t filtered(uint32_t w, int mode, uint32_t& met) {
  constexpr uint32_t kInf = E::kF16 ? 0x7C00u : 0x7F80u, kOne = E::kF16 ? 0x3C00u : 0x3F80u;
  uint32_t out = 0u;
#pragma unroll
  for (int x = 0; x < 32; x += 16) {
    const uint32_t h = (w >> x) & 0xFFFFu, size = h & 0x7FFFu;
    const int kind = size < kInf ? kPlain : (size > kInf ? kNaN : (h == kInf ? kPlusInf : kMinusInf));
    if (mode == kWithout) {
      if (kind == kPlain) out |= h << x;
      else met |= 1u << (kind - 1);
    } else if (kind == mode || (mode == kNoWeight && (kind == kPlusInf || kind == kMinusInf))) {
      out |= kOne << x;
    }
  }
  return out;
}

// A stage of V (`bytes` of shared memory, a multiple of 2048), by one warp.
template <typename E>
__device__ __forceinline__ uint32_t filter_values(uint32_t addr, int bytes, int mode, int lane) {
  constexpr uint32_t kInf = E::kF16 ? 0x7C007C00u : 0x7F807F80u, kStep = E::kF16 ? 0x04000400u : 0x00800080u;
  uint32_t met = 0u;
  for (int x = lane * 16; x < bytes; x += 4 * 512) {
    uint32_t odd[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr + x + i * 512));
      // bits 15 and 31: an exponent of all ones
      odd[i] = (((w[0] & kInf) + kStep) | ((w[1] & kInf) + kStep) | ((w[2] & kInf) + kStep) | ((w[3] & kInf) + kStep)) & 0x80008000u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (odd[i] == 0u && mode == kWithout) continue;
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      if (odd[i] != 0u) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr + x + i * 512));
#pragma unroll
        for (int y = 0; y < 4; ++y) w[y] = filtered<E>(w[y], mode, met);
      }
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr + x + i * 512), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
    }
  }
  return met;
}

// An output `old` that a value of mode's kind reaches.
__device__ __forceinline__ float reached(float old, int mode) {
  const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fffffff);
  if (old != old) return old;
  return mode == kPlusInf ? inf : (mode == kMinusInf && old != inf ? -inf : nan);
}

// A softmax warp's part of a run that only asks which keys its rows see: weight 1 for every
// visible one (kNoWeight: for those whose score is -inf); then every output whose
// accumulator is above 0 is set, or in a cluster noted (the warp's words of a bit a
// column for +inf, -inf and NaN, in its part of `staging`).  bars: s_full of both row tiles,
// then p_full, o_full and o_seen.  Returns the key tiles done, or -1 if a wait ran out.
template <typename E, int D, bool PAIR>
__device__ __forceinline__ int look_at_values(const PromptParams& p, const Unit& u, int tiles, int blocks, uint32_t tmem,
                                              uint32_t bars, uint32_t staging) {
  const int m = threadIdx.x >> 7, warp = threadIdx.x >> 5;
  const uint32_t noted = staging + static_cast<uint32_t>(warp) * 4096 + 2048;
  tmem += static_cast<uint32_t>((warp & 3) * 32) << 16;
  constexpr uint32_t kOne = E::kF16 ? 0x3C00u : 0x3F80u;
  const int lane = threadIdx.x & 31, r = threadIdx.x & (kRows - 1), mode = u.mode;
  const int before = tiles, per_tile = kRows >> p.shift_g, mq = PAIR ? 0 : m, token = mq * per_tile + (r >> p.shift_g);
  const int last = u.slot + u.ntok - 1, i = min(u.slot + token, last);
  const uint32_t scores = tmem + static_cast<uint32_t>(m * kKeys);
  const Tiles sees = tiles_of(p, u, mq);
#pragma unroll 1
  for (int k = u.k0; k < u.k1; ++k) {
    if (PAIR ? ((k - u.k0) & 1) != m : !sees.has(k)) continue;
    const Columns cols = columns_of(u.sink_boxes, u.from, k, p.shift_box);
    if (!mbar_wait(bars + 8 * m, tiles & 1)) return -1;
    tc_fence_after();
    uint32_t vis[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      vis[c] = visible_of(cols, 32 * c, i, p.window, p.sinks);
      if (mode == kNoWeight) {
        uint32_t x[32], low = 0u;
        tmem_ld32(scores + 32 * c, x);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 32; ++y) low |= (x[y] == 0xff800000u ? 1u : 0u) << y;
        vis[c] &= low;
      }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t w[32];
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        const uint32_t b = vis[2 * half + (x >> 4)] >> (2 * (x & 15));
        w[x] = ((b & 1u) ? kOne : 0u) | ((b & 2u) ? kOne << 16 : 0u);
      }
      tmem_st32(scores + half * 32, w);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bars + 8 * (2 + 2 * m + half));
    }
    ++tiles;
  }
  if (!mbar_wait(bars + 8 * (6 + m), blocks & 1) || ((PAIR || p.splits > 1) && !mbar_wait(bars + 8 * (6 + (m ^ 1)), blocks & 1))) return -1;
  if (lane == 0) mbar_arrive(bars + 8 * (8 + m));
  tc_fence_after();
  __syncwarp();  // (the outputs of the runs before were stored by other lanes)
  // accumulators that hold this run's sums: the row tile's, and for a pair both where there are two tiles
  const bool first = PAIR || tiles > before, second = PAIR && u.k1 - u.k0 > 1;
  const int c_end = PAIR ? min(D, 64 * m + 64) : D;
  uint32_t bits = 0u;
#pragma unroll 1
  for (int c = PAIR ? 64 * m : 0; c < c_end; c += 8) {
    uint32_t x[8], hit = 0u;
    if (first) {
      tmem_ld8(tmem + static_cast<uint32_t>(2 * kKeys + mq * D + c), x);
      tmem_wait_ld();
#pragma unroll
      for (int y = 0; y < 8; ++y) hit |= (x[y] != 0u ? 1u : 0u) << y;
    }
    if (second) {
      tmem_ld8(tmem + static_cast<uint32_t>(2 * kKeys + D + c), x);
      tmem_wait_ld();
#pragma unroll
      for (int y = 0; y < 8; ++y) hit |= (x[y] != 0u ? 1u : 0u) << y;
    }
    if (p.splits > 1) {
      bits |= hit << (c & 31);
      if ((c & 31) == 24) {
        const uint32_t at = noted + static_cast<uint32_t>((min(mode, static_cast<int>(kNaN)) - kPlusInf) * 4 + c / 32) * 128 + lane * 4;
        uint32_t old;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(old) : "r"(at));
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(old | bits) : "memory");
        bits = 0u;
      }
    } else if (hit != 0u && token < u.ntok) {
      uint16_t* at = p.out + ((u.first + token) * static_cast<long long>(p.Hq) + u.h * p.G + (r & (p.G - 1))) * D + c;
#pragma unroll 1
      for (int y = 0; y < 8; ++y)
        if ((hit >> y) & 1u) at[y] = E::bits(reached(E::to_float(at[y]), mode));
    }
  }
  return tiles - before;
}

// 64 columns from c0 on of this thread's row of a cluster's partial results, just written.
// noted: this thread's words of a bit a column for +inf, -inf and NaN, to be cleared, or
// (settle) what they say is set.
template <int D>
__device__ __forceinline__ void settle_part(uint32_t part, int row, int c0, uint32_t noted, bool settle) {
#pragma unroll 1
  for (int c = c0; c < c0 + 64; ++c) {
    const uint32_t at = part + part_off<D>(row, c / 4) + (c % 4) * 4;
    float y;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(y) : "r"(at));
#pragma unroll 1
    for (int kind = kPlusInf; kind <= kNaN; ++kind) {
      const uint32_t word = noted + static_cast<uint32_t>((kind - kPlusInf) * 4 + c / 32) * 128;
      uint32_t bits;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(bits) : "r"(word));
      if (!settle) asm volatile("st.shared.b32 [%0], %1;" ::"r"(word), "r"(0u) : "memory");
      else if ((bits >> (c & 31)) & 1u) y = reached(y, kind);
    }
    if (settle) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(y) : "memory");
  }
}

__device__ __forceinline__ void note_met(uint32_t met, uint32_t bits) {
  asm volatile("red.shared.or.b32 [%0], %1;" ::"r"(met), "r"(bits) : "memory");
}

// What the warps of a CTA share, beside the dynamic shared memory.
template <int D>
struct Shared {
  static constexpr int ST = kPromptStages<D>, QB = kPromptQueries<D>;
  uint64_t bars[3 * ST + 2 * QB + 11 + 2 * kSlots];
  Unit units[kSlots];
  Unit join;        // the block whose partial results a cluster joins
  int met[kSlots];  // of the unit in the slot (see kPlain)
  int span[kSlots][2];  // its key tiles that hold values that are no numbers: the first, and the one behind the last
  uint32_t tmem;
  int abort;

  __device__ __forceinline__ void release(int n, int lane);
  // All warps meet behind the CTA's last unit; false: one of the units before has to run
  // once more (all of them see the same; the drawing warp waits until they have).
  __device__ __forceinline__ bool all_done() {
    tc_fence_before();
    named_sync(1, kThreads);
    if (*static_cast<volatile int*>(&abort)) return true;
    bool more = false;
#pragma unroll
    for (int x = 0; x < kSlots; ++x) {
      const volatile Unit& u = units[x];
      more = more || (u.more != 0 && (u.mode != kPlain || (*static_cast<volatile int*>(&met[x]) & 1) != 0));
    }
    return !more;
  }
  // Waits for unit number n of this CTA, or the one behind it; false: the CTA is done, or a
  // wait ran out and this warp has still to meet the others.
  __device__ __forceinline__ bool next(int& n, bool& lost, int lane);
};

// Their barriers.
template <int D>
struct Bars {
  static constexpr int ST = kPromptStages<D>, QB = kPromptQueries<D>;
  uint32_t at;
  __device__ uint32_t full(int s) const { return at + 8 * s; }
  __device__ uint32_t empty(int s) const { return at + 8 * (ST + s); }
  __device__ uint32_t q_full(int b) const { return at + 8 * (2 * ST + b); }
  __device__ uint32_t q_empty(int b) const { return at + 8 * (2 * ST + QB + b); }
  __device__ uint32_t s_full(int m) const { return at + 8 * (2 * ST + 2 * QB + m); }
  __device__ uint32_t p_full(int m, int half) const { return at + 8 * (2 * ST + 2 * QB + 2 + 2 * m + half); }
  __device__ uint32_t o_full(int m) const { return at + 8 * (2 * ST + 2 * QB + 6 + m); }
  __device__ uint32_t o_seen(int m) const { return at + 8 * (2 * ST + 2 * QB + 8 + m); }
  __device__ uint32_t met() const { return at + 8 * (2 * ST + 2 * QB + 10); }  // both softmax warpgroups
  __device__ uint32_t u_full(int s) const { return at + 8 * (2 * ST + 2 * QB + 11 + s); }
  __device__ uint32_t u_empty(int s) const { return at + 8 * (2 * ST + 2 * QB + 11 + kSlots + s); }
  __device__ uint32_t landed(int s) const { return at + 8 * (2 * ST + 2 * QB + 11 + 2 * kSlots + s); }  // V, to be filtered
};

template <int D>
__device__ __forceinline__ void Shared<D>::release(int n, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(Bars<D>{smem_addr(bars)}.u_empty(n % kSlots));
}
template <int D>
__device__ __forceinline__ bool Shared<D>::next(int& n, bool& lost, int lane) {
  for (;; ++n) {
    lost = !mbar_wait(Bars<D>{smem_addr(bars)}.u_full(n % kSlots), (n / kSlots) & 1);
    if (lost) return false;
    if (units[n % kSlots].more != 0) return true;
    if (all_done()) return false;
    release(n, lane);
  }
}

// The drawing warp's part of a run that is not the first: the `count` tiles of V, number
// `first` of the CTA on, as they land, filtered and passed on to the products' warp.
// phases: of the stages' barriers, a bit each.  Returns them as they are then, or
// kLostPhase if a wait ran out.
constexpr uint32_t kLostPhase = 0x80000000u;
template <typename E, int D>
__device__ __forceinline__ uint32_t pass_on_values(Shared<D>& sh, uint32_t stages, int first, int count, uint32_t phases, int mode, int slot) {
  constexpr int ST = kPromptStages<D>;
  constexpr uint32_t kStage = kKeys * D * 2;
  const Bars<D> bar{smem_addr(sh.bars)};
  const int lane = threadIdx.x & 31;
  uint32_t met = 0u;
  int begin = 0, end = 0;
  for (int t = 0; t < count; ++t) {
    const int s = (2 * (first + t) + 1) % ST;
    if (!mbar_wait(bar.landed(s), (phases >> s) & 1u) || *static_cast<volatile int*>(&sh.abort)) return kLostPhase;
    phases ^= 1u << s;
    const uint32_t here = filter_values<E>(stages + s * kStage, kStage, mode, lane);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar.full(s));
    met |= here;
    if (__any_sync(0xffffffffu, here != 0u)) {
      if (end == 0) begin = t;
      end = t + 1;
    }
  }
  if (mode == kWithout) {
    if (met) note_met(smem_addr(&sh.met[slot]), met);
    if (lane == 0) {
      sh.span[slot][0] = begin;
      sh.span[slot][1] = end;
    }
  }
  __syncwarp();
  return phases;
}

// How far the drawing warp is: the next unit's number in the CTA, and of all, and the tiles
// of V copied for the units so far; `again`: a unit has to run once more.
struct DrawPlace {
  int n, u, tiles;
  bool again, lost;
};

// The drawing warp's work: the CTA's units one after the other, to the first that has to run
// once more, or (AGAIN) all that follow.  The first unit is the CTA's own number; the
// others come from the counter, which the last draw of all sets back for the next call.  A
// cluster has one unit a CTA.  A unit that has to run once more does so in its slot, before
// the slot is given to another.  In those runs this warp takes V from the copies, and passes it
// on filtered.
template <typename E, int D, bool AGAIN>
__device__ __forceinline__ void draw_units(const PromptParams& p, Shared<D>& sh, uint32_t stages, DrawPlace& at) {
  const Bars<D> bar{smem_addr(sh.bars)};
  const int lane = threadIdx.x & 31;
  Rows rows{};
  if (p.B <= 32) rows = rows_of(p, lane);
  const int units = p.blocks * p.Hkv * p.splits;
  int n = at.n, u = at.u, tiles = at.tiles;
  uint32_t kinds[kSlots] = {};  // modes that the slot's unit has still to run in, as bits
  uint32_t landings = 0u;       // phases of the stages' barriers
  bool lost = false;
  for (;; ++n) {
    Unit& slot = sh.units[n % kSlots];
    int mode = kPlain;
    if (n >= kSlots) {
      lost = !mbar_wait(bar.u_empty(n % kSlots), ((n / kSlots) - 1) & 1);
      if (lost) break;
      __syncwarp();
      const uint32_t met = static_cast<uint32_t>(*static_cast<volatile int*>(&sh.met[n % kSlots]));
      if constexpr (AGAIN) {
        uint32_t todo = n % kSlots ? kinds[1] : kinds[0];
        if (slot.mode == kPlain) {
          if (met & 1u) mode = kWithout;
        } else {
          if (slot.mode == kWithout && !slot.settle) {
            todo = met & 6u ? met : met & 8u;
            if (todo && p.splits > 1) todo |= 1u << (kSettle - 1);
          }
          if (todo) mode = __ffs(todo);
          todo &= todo - 1u;
        }
        if (n % kSlots) kinds[1] = todo;
        else kinds[0] = todo;
        __syncwarp();
        if (lane == 0) sh.met[n % kSlots] = 0;
      } else if (met != 0u) {
        at.again = true;
        break;
      }
    }
    Unit x{};
    if (mode != kPlain) {
      x = slot;
      if (x.mode == kPlain) {
        x.all0 = x.k0;
        x.all1 = x.k1;
      }
      const bool looks = mode > kWithout && mode < kSettle;
      x.mode = mode == kSettle ? kWithout : mode;
      x.settle = mode == kSettle;
      x.k0 = x.all0 + (looks ? sh.span[n % kSlots][0] : 0);
      x.k1 = looks ? x.all0 + sh.span[n % kSlots][1] : x.all1;
      x.soft = x.k0;
    } else if (u < units) {
      x = unit_of(p, rows, u, lane);
      x.soft = x.k1;
    }
    __syncwarp();
    if (lane == 0) {
      slot = x;
      if (n == 0) sh.join = x;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar.u_full(n % kSlots));
    if (!x.more) {
      if (sh.all_done()) break;
      lost = !mbar_wait(bar.u_empty(n % kSlots), (n / kSlots) & 1);
      if (lost) break;
      continue;
    }
    lost = *static_cast<volatile int*>(&sh.abort) != 0;
    if (lost) break;
    if (AGAIN && x.mode != kPlain) {
      landings = pass_on_values<E, D>(sh, stages, tiles, x.k1 - x.k0, landings, x.mode, n % kSlots);
      lost = landings == kLostPhase;
      if (lost) break;
    }
    tiles += x.k1 - x.k0;
    if (mode != kPlain || u >= units) continue;
    if (p.splits > 1) {
      u = units;
    } else {
      if (lane == 0) {
        const int drawn = atomicAdd(p.counter, 1);
        if (drawn == units - 1) *p.counter = 0;
        u = gridDim.x + drawn;
      }
      u = __shfl_sync(0xffffffffu, u, 0);
    }
  }
  at.n = n;
  at.u = u;
  at.tiles = tiles;
  at.lost = lost;
}

// The same from a unit that runs once more on, out of line.
template <typename E, int D>
__device__ __noinline__ bool draw_again(const PromptParams& p, Shared<D>& sh, uint32_t stages, int n, int u, int tiles) {
  DrawPlace at{n, u, tiles, false, false};
  draw_units<E, D, true>(p, sh, stages, at);
  return at.lost;
}

// How far a softmax warp is: its unit, tiles and blocks of its row tile done, meetings of
// both warpgroups; `again`: the unit is one that runs once more.
struct SoftmaxPlace {
  int nu, tiles, blocks;
  uint32_t meets;
  bool again, lost;
};

// The softmax warps' work on units from at.nu on: to the first that runs once more, or
// (AGAIN) all that follow.
template <typename E, int D, bool PAIR, bool AGAIN>
__device__ __forceinline__ void softmax_units(const PromptParams& p, Shared<D>& sh, uint32_t base, SoftmaxPlace& at) {
  constexpr int ST = kPromptStages<D>, QB = kPromptQueries<D>;
  const uint32_t sOut = base + (QB * 2 + ST) * kRows * D * 2, sPart = base, sLse = sOut + 7 * 4096 + 1024;
  const Bars<D> bar{smem_addr(sh.bars)};
  const int shift_g = p.shift_g, per_tile = kRows >> shift_g;
  const long long tok_stride = static_cast<long long>(p.Hq) * D;
  auto t_scores = [](uint32_t tmem, int m) { return tmem + static_cast<uint32_t>(m * kKeys); };
  auto t_out = [](uint32_t tmem, int m) { return tmem + static_cast<uint32_t>(2 * kKeys + m * D); };
  // (read anew: kept from the kernel's beginning they would be spilled here)
  int tid;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
  const int lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t tmem = sh.tmem;
  const int m = warp >> 2;
  const int r = tid & (kRows - 1);  // row of the tile = lane of tensor memory
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const float NEG_INF = __int_as_float(0xff800000);
  int tiles = at.tiles, blocks = at.blocks, nu = at.nu;
  uint32_t meets = at.meets;
  bool lost = false;
  auto meet = [&]() {  // of both warpgroups; sets `lost` if the other does not come
    mbar_arrive(bar.met());
    lost = lost || !mbar_wait(bar.met(), meets & 1);
    ++meets;
  };
  for (; !lost && sh.next(nu, lost, lane); ++nu) {
    const Unit& blk = sh.units[nu % kSlots];  // (not released before the block is done)
    if (blk.k0 == blk.soft) {
      if (!AGAIN && blk.mode != kPlain) {
        at.again = true;
        break;
      }
      if (blk.k0 == blk.k1 || blk.mode > kWithout) {
        if (AGAIN && blk.mode > kWithout) {
          const int done = look_at_values<E, D, PAIR>(p, blk, tiles, blocks, sh.tmem, bar.s_full(0), sOut);
          lost = done < 0;
          tiles += done;
          ++blocks;
          if constexpr (PAIR) meet();  // both have read the accumulators
          if (lost) break;
        } else if (p.splits > 1 && blk.count > 0) {  // (a cluster's CTA without a share has nothing to add)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(sLse + tid * 4), "f"(NEG_INF) : "memory");
        }
        sh.release(nu, lane);
        continue;
      }
    }
    const int mq = PAIR ? 0 : m, token = mq * per_tile + (r >> shift_g);
    const int last = blk.slot + blk.ntok - 1;
    const int i = min(blk.slot + token, last);
    const int f = blk.slot + mq * per_tile;                // first and last query of the tile
    const int e = min(last, f + per_tile - 1);
    const Tiles sees = tiles_of(p, blk, mq);  // (as the products' warp has them)
    float top = NEG_INF;  // the maximum that the weights refer to, times scale_log2
    float2 sum2 = make_float2(0.f, 0.f);
    const float lift = AGAIN && blk.mode == kWithout ? kLiftAgain<E> : kLift<E>;
    int n = 0;
    for (int k = blk.k0; k < blk.k1; ++k) {
      if (PAIR ? ((k - blk.k0) & 1) != m : !sees.has(k)) continue;  // not this row tile's
      // which keys this row sees, found while the scores are on their way
      const Columns cols = columns_of(blk.sink_boxes, blk.from, k, p.shift_box);
      const bool edge = (k << (7 - p.shift_box)) < blk.sink_boxes || cols.base + kKeys - 1 > f || cols.base <= e - p.window;
      uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
      if (edge) {
        // sinks, or an edge of the causal mask or of the window
#pragma unroll
        for (int c = 0; c < 4; ++c) vis[c] = visible_of(cols, c * 32, i, p.window, p.sinks);
      }
      if (!mbar_wait(bar.s_full(m), tiles & 1)) {
        lost = true;
        break;
      }
      tc_fence_after();
      uint32_t sc[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t_scores(tmem, m) + lanes + c * 32, sc[c]);
      tmem_wait_ld();
      if constexpr (AGAIN) {  // a visible score of -inf, whose weight is 0
        bool none = false;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int x = 0; x < 32; ++x) none = none || (sc[c][x] == 0xff800000u && (vis[c] & (1u << x)));
        if (none && blk.mode == kWithout && token < blk.ntok) note_met(smem_addr(&sh.met[nu % kSlots]), 1u << (kNoWeight - 1));
      }
      if (edge) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (__all_sync(0xffffffffu, vis[c] == 0xffffffffu)) continue;
#pragma unroll
          for (int x = 0; x < 32; ++x) sc[c][x] = (vis[c] & (1u << x)) ? sc[c][x] : 0xff800000u;
        }
      }
      float mx[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
      for (int x = 0; x < 32; x += 2)
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = fmax3(mx[c], __uint_as_float(sc[c][x]), __uint_as_float(sc[c][x + 1]));
      const float now = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
      if (n == 0) {
        top = now;
      } else if (__any_sync(0xffffffffu, now > top + kGrow)) {
        // the products of the earlier key tiles are complete (the scores' commit
        // came after theirs), and the next waits for this tile's weights
        const float to = fmaxf(top, now);
        const float by = exp2f(top - (to == NEG_INF ? 0.f : to));
#pragma unroll 1
        for (int c = 0; c < D; c += 8) {
          uint32_t o[8];
          tmem_ld8(t_out(tmem, m) + lanes + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 8; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * by);
          tmem_st8(t_out(tmem, m) + lanes + c, o);
        }
        sum2.x *= by;
        sum2.y *= by;
        top = to;
      }
      const float shift = top == NEG_INF ? 0.f : lift - top;
      const float2 scale2 = make_float2(p.scale_log2, p.scale_log2), shift2 = make_float2(shift, shift);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t w[32];
        float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const int c = 2 * half + (x >> 4), y = 2 * (x & 15);
          const float2 a = ffma2(make_float2(__uint_as_float(sc[c][y]), __uint_as_float(sc[c][y + 1])), scale2, shift2);
          const float2 v = make_float2(exp2f(a.x), exp2f(a.y));
          add[x & 1] = fadd2(add[x & 1], v);
          w[x] = E::pack2(v.x, v.y);
        }
        sum2 = fadd2(sum2, fadd2(add[0], add[1]));
        tmem_st32(t_scores(tmem, m) + lanes + half * 32, w);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar.p_full(m, half));
      }
      ++n;
      ++tiles;
    }
    float sum = sum2.x + sum2.y;
    if (lost || !mbar_wait(bar.o_full(m), blocks & 1) || ((PAIR || p.splits > 1) && !mbar_wait(bar.o_full(m ^ 1), blocks & 1))) {
      lost = true;
      break;
    }
    if (lane == 0) mbar_arrive(bar.o_seen(m));
    ++blocks;
    tc_fence_after();
    // The row's output is w0 O_0 + w1 O_1 (the accumulators of both warpgroups, who
    // tell each other their sums) for a pair, which shares the columns between the
    // warpgroups, and O_m / sum otherwise.  A warpgroup that saw no key of a row
    // has sum 0, and what its accumulator holds does not count.
    const uint32_t stage = sOut + static_cast<uint32_t>(warp) * 4096;
    // A live row without weight, whose visible scores are all -inf, is NaN; a share of
    // its keys without weight adds nothing.
    const float none = p.splits == 1 && token < blk.ntok ? __int_as_float(0x7fffffff) : 0.f;
    float w0 = sum == 0.f ? none : 1.f / sum, w1 = 0.f;
    float lse = sum > 0.f ? top - lift + log2f(sum) : (sum == 0.f ? NEG_INF : sum);
    if constexpr (PAIR) {
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(stage + lane * 8), "f"(top), "f"(sum) : "memory");
      meet();
      float top1, sum1;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(top1), "=f"(sum1) : "r"(sOut + static_cast<uint32_t>(warp ^ 4) * 4096 + lane * 8));
      meet();  // the staging space is used again below
      if (lost) break;
      if (m == 1) {  // in the same order on both sides
        const float t = top, u = sum;
        top = top1;
        sum = sum1;
        top1 = t;
        sum1 = u;
      }
      const float both = fmaxf(top, top1), shift = both == NEG_INF ? 0.f : both;
      const float a = sum == 0.f ? 0.f : exp2f(top - shift), b = sum1 == 0.f ? 0.f : exp2f(top1 - shift);
      const float all = a * sum + b * sum1;
      lse = all > 0.f ? both - lift + log2f(all) : (all == 0.f ? NEG_INF : all);
      w0 = all == 0.f ? none : (sum == 0.f ? 0.f : at_least_tiny(a / all));
      w1 = sum1 == 0.f ? 0.f : at_least_tiny(b / all);
    }
    // 64 columns at a time: c0 is the first
    float2 probe = make_float2(0.f, 0.f);  // becomes NaN with any output that is NaN or infinite
    auto load = [&](int c0, uint32_t (&o)[64]) {
      const uint32_t src = t_out(tmem, mq);
      uint32_t x[32], y[32];
      tmem_ld32(src + lanes + c0, x);
      tmem_ld32(src + lanes + c0 + 32, y);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        const uint32_t v = i < 32 ? x[i] : y[i - 32];
        o[i] = w0 == 0.f ? 0u : __float_as_uint(__uint_as_float(v) * w0);
      }
      if constexpr (PAIR) {
        tmem_ld32(t_out(tmem, 1) + lanes + c0, x);
        tmem_ld32(t_out(tmem, 1) + lanes + c0 + 32, y);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          const uint32_t v = i < 32 ? x[i] : y[i - 32];
          o[i] = w1 == 0.f ? o[i] : __float_as_uint(fmaf(__uint_as_float(v), w1, __uint_as_float(o[i])));
        }
      }
#pragma unroll
      for (int i = 0; i < 64; i += 2)
        probe = ffma2(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), make_float2(0.f, 0.f), probe);
    };
    const int c_begin = PAIR ? 64 * m : 0, c_end = PAIR ? min(D, 64 * m + 64) : D;
    const int part_row = mq * kRows + r;
    // The warp's 32 rows leave through 4 KB of shared memory, 128 bytes of each at
    // a time: a thread holds a row, and stores of 16 bytes a row would touch 32
    // lines each.  (Those of a cluster stay in shared memory, in fp32.)
    uint16_t* dst = p.out + (blk.first + mq * per_tile) * tok_stride + static_cast<long long>(blk.h) * p.G * D + (lane & 7) * 8;
    const int row0 = (warp & 3) * 32 + (lane >> 3);  // this lane's rows: row0 + 4 x
    dst += (row0 >> shift_g) * tok_stride + (row0 & (p.G - 1)) * D;
    const int left = ((blk.ntok - mq * per_tile) << shift_g) - row0;
    for (int c0 = c_begin; c0 < c_end; c0 += 64) {
      uint32_t o[64];
      load(c0, o);
      if (p.splits > 1) {
#pragma unroll
        for (int x = 0; x < 16; ++x)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sPart + part_off<D>(part_row, c0 / 4 + x)),
                       "r"(o[4 * x]), "r"(o[4 * x + 1]), "r"(o[4 * x + 2]), "r"(o[4 * x + 3])
                       : "memory");
        if (AGAIN && blk.mode != kPlain) settle_part<D>(sPart, part_row, c0, stage + 2048 + lane * 4, blk.settle != 0);
      } else {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          uint32_t w[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            w[y] = E::pack2(__uint_as_float(o[8 * x + 2 * y]), __uint_as_float(o[8 * x + 2 * y + 1]));
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + swz128(lane, x)), "r"(w[0]), "r"(w[1]),
                       "r"(w[2]), "r"(w[3])
                       : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(stage + swz128(4 * x + (lane >> 3), lane & 7)));
          // (row0 has no bits that 4 x has: the two offsets add up)
          if (4 * x < left)
            *reinterpret_cast<uint4*>(dst + ((4 * x) >> shift_g) * tok_stride + ((4 * x) & (p.G - 1)) * D + c0) = v;
        }
        __syncwarp();
      }
    }
    if (p.splits > 1 && (!PAIR || m == 0)) asm volatile("st.shared.f32 [%0], %1;" ::"r"(sLse + part_row * 4), "f"(lse) : "memory");
    // an output that is no number, in a row whose sum is one: it may come from a value that the row does not see
    if (probe.x + probe.y != 0.f && lse > NEG_INF && token < blk.ntok && (!AGAIN || blk.mode == kPlain))
      note_met(smem_addr(&sh.met[nu % kSlots]), 1u);
    if (p.splits > 1) fence_proxy_async_smem();  // (what was left, before the copies of a run that follows)
    if constexpr (PAIR) {
      meet();  // both have read the accumulators
      if (lost) break;
    }
    sh.release(nu, lane);
  }
  at.nu = nu;
  at.tiles = tiles;
  at.blocks = blocks;
  at.meets = meets;
  at.lost = lost;
}

// The same from a unit that runs once more on, out of line.
template <typename E, int D, bool PAIR>
__device__ __noinline__ bool softmax_again(const PromptParams& p, Shared<D>& sh, uint32_t base, int nu, int tiles, int blocks,
                                           uint32_t meets) {
  SoftmaxPlace at{nu, tiles, blocks, meets, false, false};
  softmax_units<E, D, PAIR, true>(p, sh, base, at);
  return at.lost;
}

template <typename E, int D, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) window_prompt_kernel(const __grid_constant__ PromptParams p) {
  constexpr int HALVES = D / 64;
  constexpr int KS = D / 16;                   // k-steps of the score product
  constexpr uint32_t kQTile = kRows * D * 2;   // bytes of a row tile's queries: [D/64][128 rows][128 B]
  constexpr uint32_t kStage = kKeys * D * 2;   // bytes of K or V of a key tile, likewise
  constexpr uint32_t kBlockBytes = kKeys * 128;  // one 64-element column block
  constexpr int ST = kPromptStages<D>, QB = kPromptQueries<D>;
  constexpr uint32_t kScores = tc_kind_f16(kRows, kKeys, !E::kF16, false);
  constexpr uint32_t kValues = tc_kind_f16(kRows, D, !E::kF16, true);
  extern __shared__ __align__(128) unsigned char smem_raw[];
  __shared__ Shared<D> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int shift_g = p.shift_g, per_tile = kRows >> shift_g;  // tokens of a row tile
  const long long tok_stride = static_cast<long long>(p.Hq) * D;

  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base, sKV = base + QB * 2 * kQTile, sOut = sKV + ST * kStage;
  // partial results of a CTA in a cluster, over the queries and stages, and beside them
  const uint32_t sPart = base, sLse = sOut + 7 * 4096 + 1024;  // (behind what the last warp stages)
  const Bars<D> bar{smem_addr(sh.bars)};
  auto full = [&](int s) { return bar.full(s); };
  auto empty = [&](int s) { return bar.empty(s); };
  auto q_full = [&](int b) { return bar.q_full(b); };
  auto q_empty = [&](int b) { return bar.q_empty(b); };
  auto s_full = [&](int m) { return bar.s_full(m); };
  auto p_full = [&](int m, int half) { return bar.p_full(m, half); };
  auto o_full = [&](int m) { return bar.o_full(m); };
  auto o_seen = [&](int m) { return bar.o_seen(m); };
  auto u_full = [&](int s) { return bar.u_full(s); };
  auto u_empty = [&](int s) { return bar.u_empty(s); };
  volatile int* abort_flag = &sh.abort;
  if (tid == 0) {
    sh.abort = 0;
    for (int x = 0; x < kSlots; ++x) {
      sh.units[x].more = 0;
      sh.met[x] = 0;
    }
    for (int s = 0; s < ST; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
      mbar_init(bar.landed(s), 1);
    }
    for (int b = 0; b < QB; ++b) {
      mbar_init(q_full(b), 1);
      mbar_init(q_empty(b), 1);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(s_full(m), 1);
      mbar_init(p_full(m, 0), kRows);
      mbar_init(p_full(m, 1), kRows);
      mbar_init(o_full(m), 1);
      mbar_init(o_seen(m), 4);
    }
    mbar_init(bar.met(), 2 * kRows);
    for (int x = 0; x < kSlots; ++x) {
      mbar_init(u_full(x), 1);
      mbar_init(u_empty(x), 11);  // every warp but the drawing one
    }
    fence_barrier_init();
  }
  if (warp == kProductWarp) tmem_alloc(smem_addr(&sh.tmem), kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_begin();
  auto release_unit = [&](int n) { sh.release(n, lane); };
  auto give_up = [&]() {
    if (lane == 0) flag_error(p.err_flag, VH_ERR_TIMEOUT);
    *abort_flag = 1;
    __syncwarp();
  };

  if (warp >= kProductWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    const bool leader = elect_one();
    if (warp == kDrawWarp) {
      // ======================= the CTA's next unit =====================================
      DrawPlace at{};
      at.u = blockIdx.x;
      draw_units<E, D, false>(p, sh, sKV, at);
      if (at.again) at.lost = draw_again<E, D>(p, sh, sKV, at.n, at.u, at.tiles);
      if (at.lost) {
        give_up();
        named_sync(1, kThreads);
      }
    } else
    if (warp == kCopyWarp || warp == kCopyWarp + 1) {
      // ======================= copies: K and the queries, and V =======================
      // tile number x of all units: K is stage 2 x of the ring, V the next one
      const int kv = warp - kCopyWarp;
      const void* map = kv ? static_cast<const void*>(&p.tmap_v) : static_cast<const void*>(&p.tmap_k);
      if (leader) {
        if (kv == 0) prefetch_tensormap(&p.tmap_q);
        prefetch_tensormap(map);
      }
      const int nbox = kKeys / p.box;
      int issued = kv, nq = 0;  // number in the ring, blocks of queries
      bool lost = false;
      for (int n = 0; !lost && sh.next(n, lost, lane); ++n) {
        const Unit u = sh.units[n % kSlots];
        release_unit(n);
        if (u.k0 == u.k1) continue;
        // (the drawing warp passes on V of a unit that runs once more)
        const uint32_t done0 = kv == 1 && u.mode != kPlain ? bar.landed(0) : full(0);
        for (int k = u.k0; k < u.k1 && !lost; ++k, issued += 2) {
          // page and first token of this lane's box (at most 16 boxes a tile)
          int page = p.num_pages, tok = 0;
          const int box = (k << (7 - p.shift_box)) + lane;
          if (lane < nbox && box < u.boxes) {
            const int j = (box < u.sink_boxes ? box : box - u.sink_boxes + u.from) << p.shift_box;
            const int of_row = p.shift_page >= 0 ? j >> p.shift_page : j / p.P;
            const long long lp = static_cast<long long>(u.row) * p.max_pages_per_seq + of_row;
            page = p.page_table ? p.page_table[lp] : static_cast<int>(lp);
            tok = j - of_row * p.P;
            if (page < 0 || page >= p.num_pages) {
              flag_error(p.err_flag, VH_ERR_PAGE);
              page = p.num_pages;
            }
          }
          const int s = issued % ST;
          if ((issued >= ST && !mbar_wait(empty(s), ((issued / ST) - 1) & 1)) || *abort_flag) {
            lost = true;
            break;
          }
          const uint32_t done = done0 + 8 * s;
          if (leader) mbar_arrive_expect_tx(done, kStage);
          for (int x = 0; x < nbox; ++x) {
            const int pg = __shfl_sync(0xffffffffu, page, x), tk = __shfl_sync(0xffffffffu, tok, x);
            if (leader) {
              const int c1 = p.tm_tok_dim == 1 ? tk : u.h, c2 = p.tm_tok_dim == 1 ? u.h : tk;
              const uint32_t dst = sKV + s * kStage + x * p.box * 128;
#pragma unroll
              for (int hf = 0; hf < HALVES; ++hf) tma_load_4d(dst + hf * kBlockBytes, map, hf * 64, c1, c2, pg, done);
            }
          }
          if (k == u.k0 && kv == 0) {
            // the block's queries, once the products of the block that had
            // their place have read it (its first keys are on their way already)
            const int b = nq % QB, ntile = !PAIR && u.ntok > per_tile ? 2 : 1;
            if (nq >= QB && !mbar_wait(q_empty(b), ((nq / QB) - 1) & 1)) {
              lost = true;
              issued += 2;
              break;
            }
            if (leader) {
              mbar_arrive_expect_tx(q_full(b), static_cast<uint32_t>(ntile) * kQTile);
              for (int m = 0; m < ntile; ++m)
                for (int hf = 0; hf < HALVES; ++hf)
                  tma_load_3d(sQ + (2 * b + m) * kQTile + hf * kBlockBytes, &p.tmap_q, hf * 64, u.h * p.G,
                              u.first + m * per_tile, q_full(b));
            }
            ++nq;
          }
        }
      }
      if (lost) {
        give_up();
        // copies in flight land before the shared memory goes away
        for (int x = max(kv, issued - 2 * ST); x < issued; x += 2)
          if (x + ST >= issued) (void)mbar_wait(full(x % ST), (x / ST) & 1);
        for (int x = max(0, nq - QB); x < nq; ++x) (void)mbar_wait(q_full(x % QB), (x / QB) & 1);
        named_sync(1, kThreads);
      }
    } else if (warp == kProductWarp) {
      // ======================= products =============================================
      // The tensor cores wait whenever this warp does more between two products
      // than they have queued.  So all that a tile needs is known before, and the
      // warp stays together: a wait that ran out is noted and acted on once a tile
      // (what is multiplied until then is garbage in this CTA's own memory).
      const uint32_t issue = leader ? 1u : 0u;
      const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
      uint32_t ki = 0, kp = 0, vi = 1, vp = 0;  // ring place and phase of the next K and V
      auto next = [&](uint32_t& i, uint32_t& ph) {
        i += 2;
        if (i >= ST) {
          i -= ST;
          ph ^= 1u;
        }
      };
      int nq = 0;
      uint32_t weights0 = 0, weights1 = 0;  // phases of the weights' barriers
      bool ran_out = false;
      auto wait = [&](uint32_t bar, uint32_t parity) { ran_out |= !mbar_wait(bar, parity); };
      bool lost = false;
      const uint32_t k_operand = tc_operand(sKV, 16), v_operand = tc_operand(sKV, kBlockBytes);
      int n = 0;
      for (;;) {  // (a second time only where units run once more)
        for (;; ++n) {
          wait(u_full(n % kSlots), (n / kSlots) & 1);
          lost = __any_sync(0xffffffffu, ran_out);
          auto field = [&](const int& x) { return __shfl_sync(0xffffffffu, x, 0); };  // (uniform, and known to be)
          const Unit& from = sh.units[n % kSlots];
          if (lost || field(from.more) == 0) break;
          Unit blk;
          blk.slot = field(from.slot);
          blk.ntok = field(from.ntok);
          blk.sink_boxes = field(from.sink_boxes);
          blk.from = field(from.from);
          blk.count = field(from.count);
          const int k0 = field(from.k0), k1 = field(from.k1);
          release_unit(n);
          if (k0 == k1) continue;
          const int last = blk.slot + blk.ntok - 1, low = max(0, blk.slot - p.window + 1);
          const int qb = nq % QB;
          // the key tiles that row tile m sees: below s_end, and from w_begin to w_end
          int s_end[2], w_begin[2], w_end[2];
          const int shift = 7 - p.shift_box;  // log2 of the boxes of a tile
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int f = blk.slot + m * per_tile, e = min(last, f + per_tile - 1);
            const int to = blk.sink_boxes + (e >> p.shift_box) - blk.from;  // last box, if it is one of the window's
            s_end[m] = f > last ? 0 : min((blk.sink_boxes + (1 << shift) - 1) >> shift, (e >> 7) + 1);
            w_begin[m] = (blk.sink_boxes + max(0, (max(0, f - p.window + 1) >> p.shift_box) - blk.from)) >> shift;
            w_end[m] = f > last || to < blk.sink_boxes ? 0 : (to >> shift) + 1;
          }
          auto sees_k = [&](int m, int k) -> bool { return k < s_end[m] || (k >= w_begin[m] && k < w_end[m]); };
          const uint32_t q_operand = tc_operand(sQ + 2 * qb * kQTile, 16);
          auto scores = [&](int m) {
            const uint32_t qa = q_operand + (PAIR ? 0 : m) * (kQTile >> 4), kb = k_operand + ki * (kStage >> 4);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              const uint32_t off = ((s >> 2) * kBlockBytes + (s & 3) * 32) >> 4;
              tc_mma(issue, tmem + m * kKeys, qa + off, kb + off, kScores, s > 0);
            }
            tc_commit(issue, s_full(m));
          };
          bool add0 = false, add1 = false;
          // the block's last products of row tile m are issued; its softmax has seen the end
          // of the block before (else it could miss this one)
          auto finish = [&](int m) {
            if (nq > 1) wait(o_seen(m), (nq - 2) & 1);
            tc_commit(issue, o_full(m));
          };
          // values of key tile k: slots that nobody sees may hold anything where an end of
          // what the block sees lies inside the tile, so they become zeros
          const int last_sinks = blk.sink_boxes > 0 ? (blk.sink_boxes - 1) >> shift : -1, first_window = blk.sink_boxes >> shift;
          auto clean = [&](int k) {
            if (k + 1 != blk.count && k != last_sinks && k != first_window) return;
            const uint32_t vb = sKV + vi * kStage;
            const Columns cols = columns_of(blk.sink_boxes, blk.from, k, p.shift_box);
            for (int r = lane / 8; r < kKeys; r += 4) {
              const int j = cols.slot(r);
              if (j <= last && (j < p.sinks || j >= low)) continue;
#pragma unroll
              for (int hf = 0; hf < HALVES; ++hf)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + hf * kBlockBytes + r * 128 + (lane & 7) * 16),
                             "r"(0u)
                             : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
          };
          // the weights arrive in two halves of 64 keys
          auto values = [&](int m, uint32_t& weights, bool& add) {
            const uint32_t va = v_operand + vi * (kStage >> 4), scores_at = tmem + m * kKeys, out_at = tmem + 2 * kKeys + m * D;
            wait(p_full(m, 0), weights);
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < 4; ++s)
              tc_mma_ta(issue, out_at, scores_at + s * 8, va + s * (2048 >> 4), kValues, add || s > 0);
            wait(p_full(m, 1), weights);
            tc_fence_after();
#pragma unroll
            for (int s = 4; s < 8; ++s) tc_mma_ta(issue, out_at, scores_at + s * 8, va + s * (2048 >> 4), kValues, true);
            weights ^= 1u;
            add = true;
          };
          wait(q_full(qb), (nq / QB) & 1);
          wait(full(ki), kp);
          ++nq;
          tc_fence_after();
          if constexpr (PAIR) {
            scores(0);
            tc_commit(issue, empty(ki));
            next(ki, kp);
            if (k0 + 1 < k1) {
              wait(full(ki), kp);
              scores(1);
              tc_commit(issue, empty(ki));
              next(ki, kp);
            }
            if (k0 + 2 >= k1) tc_commit(issue, q_empty(qb));
            // key tile k by row tile place m: its values, then the scores of the tile after next
            auto step = [&](int m, int k, uint32_t& weights, bool& add) {
              wait(full(vi), vp);
              clean(k);
              values(m, weights, add);
              tc_commit(issue, empty(vi));
              next(vi, vp);
              if (k + 2 < k1) {
                wait(full(ki), kp);
                scores(m);
                tc_commit(issue, empty(ki));
                if (k + 3 == k1) tc_commit(issue, q_empty(qb));
                next(ki, kp);
              }
            };
            for (int k = k0; k < k1; k += 2) {
              step(0, k, weights0, add0);
              if (k + 1 < k1) step(1, k + 1, weights1, add1);
              if (__any_sync(0xffffffffu, ran_out)) break;
            }
            finish(0);
            finish(1);
          } else {
            bool see0 = sees_k(0, k0), see1 = sees_k(1, k0);
            if (see0) scores(0);
            if (see1) scores(1);
            tc_commit(issue, empty(ki));
            if (k0 + 1 == k1) tc_commit(issue, q_empty(qb));
            next(ki, kp);
            for (int k = k0; k < k1; ++k) {
              const bool more = k + 1 < k1;
              const bool next0 = more && sees_k(0, k + 1), next1 = more && sees_k(1, k + 1);
              wait(full(vi), vp);
              clean(k);
              if (see0) values(0, weights0, add0);
              if (more) wait(full(ki), kp);
              if (next0) scores(0);
              if (!more) finish(0);
              if (see1) values(1, weights1, add1);
              if (next1) scores(1);
              if (!more) finish(1);
              tc_commit(issue, empty(vi));
              if (more) tc_commit(issue, empty(ki));
              if (k + 2 == k1) tc_commit(issue, q_empty(qb));  // the block's last scores are issued
              next(vi, vp);
              if (more) next(ki, kp);
              see0 = next0;
              see1 = next1;
              if (__any_sync(0xffffffffu, ran_out)) break;
            }
          }
        }
        if (lost || sh.all_done()) break;
        release_unit(n);
        ++n;
      }
      if (lost) {
        give_up();
        // products in flight end before the tensor memory is freed (row tile 0's output
        // barrier serves for that; its softmax has given up or will)
        tc_commit(issue, o_full(0));
        for (int x = 0; x < 2; ++x) (void)mbar_wait(o_full(0), x);
        named_sync(1, kThreads);
      }
    }
  } else {
    // ======================= softmax of row tile m =================================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    SoftmaxPlace at{};
    softmax_units<E, D, PAIR, false>(p, sh, base, at);
    if (at.again) at.lost = softmax_again<E, D, PAIR>(p, sh, base, at.nu, at.tiles, at.blocks, at.meets);
    if (at.lost) {
      give_up();
      tc_fence_before();
      named_sync(1, kThreads);
    }
  }
  if (warp == kProductWarp) tmem_free(sh.tmem, kTmem);
  if (p.splits == 1) return;

  // ======================= the cluster's partial results ============================
  // (all CTAs of a cluster work on one block: they agree on whether there is one)
  const Unit& u = sh.join;
  if (u.count == 0) return;
  cluster_sync();
  if (!*abort_flag) {
    const int rows_valid = u.ntok << shift_g;
    for (int r = u.z + p.splits * warp; r < rows_valid; r += p.splits * (kThreads / 32)) {
      // lane s has the weight of CTA s's piece
      const float NEG_INF = __int_as_float(0xff800000);
      const float lse = lane < p.splits ? cluster_ld(cluster_map(sLse + r * 4, lane)) : NEG_INF;
      float top = lse;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float w = lse == NEG_INF ? 0.f : at_least_tiny(exp2f(lse - top));
      float sum = w;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      constexpr int PER = D / 32;
      float o[PER];
#pragma unroll
      for (int x = 0; x < PER; ++x) o[x] = 0.f;
#pragma unroll 4
      for (int s = 0; s < p.splits; ++s) {
        const float f = __shfl_sync(0xffffffffu, w, s);
        const uint32_t at = cluster_map(sPart + part_off<D>(r, lane * PER / 4) + (lane * PER % 4) * 4, s);
        // (a piece without a visible key was not written)
#pragma unroll
        for (int x = 0; x < PER; x += 2) {
          const float2 v = cluster_ld2(at + x * 4);
          o[x] += f == 0.f ? 0.f : f * v.x;
          o[x + 1] += f == 0.f ? 0.f : f * v.y;
        }
      }
      const float inv = 1.f / sum;
      uint16_t* dst = p.out + (u.first + (r >> shift_g)) * tok_stride + (static_cast<long long>(u.h) * p.G + (r & (p.G - 1))) * D + lane * PER;
#pragma unroll
      for (int x = 0; x < PER; x += 2) *reinterpret_cast<uint32_t*>(dst + x) = E::pack2(o[x] * inv, o[x + 1] * inv);
    }
  }
  cluster_sync();  // others may still read this CTA's shared memory
}

template <typename E, int D>
cudaLaunchConfig_t config(const PromptParams& p, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kPromptSmem<D>;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = static_cast<unsigned>(p.splits);
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 1 : 0;
  return cfg;
}

// Attributes of one variant, and how many of its clusters of 2^x CTAs run at a time.
template <typename E, int D, bool PAIR>
cudaError_t prepare_t(int (&clusters)[5]) {
  cudaError_t e = cudaFuncSetAttribute(window_prompt_kernel<E, D, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPromptSmem<D>);
  if (e != cudaSuccess) return e;
  if (cudaFuncSetAttribute(window_prompt_kernel<E, D, PAIR>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    cudaGetLastError();
  for (int x = 1; x <= 4; ++x) {
    PromptParams p{};
    p.splits = p.ctas = 1 << x;
    cudaLaunchAttribute attr{};
    const cudaLaunchConfig_t cfg = config<E, D>(p, &attr);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, window_prompt_kernel<E, D, PAIR>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    clusters[x] = n < clusters[x] ? n : clusters[x];
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t prepare_window_prompt(int (&clusters)[5]) {
  for (int& c : clusters) c = 1 << 20;
  cudaError_t e = prepare_t<ElemBf16, 64, false>(clusters);
  if (e == cudaSuccess) e = prepare_t<ElemBf16, 64, true>(clusters);
  if (e == cudaSuccess) e = prepare_t<ElemBf16, 128, false>(clusters);
  if (e == cudaSuccess) e = prepare_t<ElemBf16, 128, true>(clusters);
  if (e == cudaSuccess) e = prepare_t<ElemF16, 64, false>(clusters);
  if (e == cudaSuccess) e = prepare_t<ElemF16, 64, true>(clusters);
  if (e == cudaSuccess) e = prepare_t<ElemF16, 128, false>(clusters);
  if (e == cudaSuccess) e = prepare_t<ElemF16, 128, true>(clusters);
  return e;
}

cudaError_t launch_window_prompt(const PromptParams& p, cudaStream_t stream) {
  using Kernel = void (*)(PromptParams);
  const Kernel kernels[8] = {window_prompt_kernel<ElemBf16, 64, false>,  window_prompt_kernel<ElemBf16, 64, true>,
                             window_prompt_kernel<ElemF16, 64, false>,   window_prompt_kernel<ElemF16, 64, true>,
                             window_prompt_kernel<ElemBf16, 128, false>, window_prompt_kernel<ElemBf16, 128, true>,
                             window_prompt_kernel<ElemF16, 128, false>,  window_prompt_kernel<ElemF16, 128, true>};
  return launch_dependent(kernels[(p.D == 128 ? 4 : 0) + (p.f16 ? 2 : 0) + (p.pair ? 1 : 0)], p, dim3(p.ctas), kThreads,
                          p.D == 128 ? kPromptSmem<128> : kPromptSmem<64>, stream, p.splits);
}

}  // namespace vh
