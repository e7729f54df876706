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
//    block holds tokens of one request; block i belongs to the last row b with
//    token_start[b] / tokens + b <= i, so the grid needs no work list.
//  * Keys.  Tiles of 128 slots: those that hold sinks, then those from the
//    first query's window to the last query.  Each is copied box by box through
//    the page table; boxes that nobody sees, and bad page ids, become a page
//    past the tensor, which the copy engine fills with zeros without reading.
//    A tile that one of the two row tiles does not see is skipped for it.
//  * Warps: two warpgroups for the softmax of a row tile each (a thread owns a
//    row, so its maximum and sum need no exchange), one warp that issues the
//    products, one that copies K and V through a ring of stages.
//  * Softmax.  Running maximum and sum in fp32; the accumulator is rescaled
//    only when a row's maximum has grown by more than 2^8 since the last time
//    (weights stay below 2^8, far inside fp32, bf16 and fp16), so it is rare.
//    Weights go back to tensor memory as 16-bit operands of the value product,
//    over the scores: rounding them costs one half step of the element type
//    relatively, as the output's own rounding does, and saves a second product.
//  * What is not seen: scores get -inf; rows of V that no query of the block
//    sees (page tails, freed pages) are zeroed in shared memory.  A value that
//    some rows of a tile see and others do not meets weight 0 there, which is
//    harmless unless it is infinite or NaN; a row that ends with a NaN is
//    therefore computed again over its visible keys alone, one warp a row.
//  * Few blocks (short chunks over long contexts): the key tiles of a block are
//    shared by `splits` CTAs, whose partial results a second kernel adds.
#include "vh_ragged.cuh"
#include "vh_tcgen05.cuh"
#include "vh_window.h"

namespace vh {

namespace {

constexpr int kRows = 128;       // rows of a row tile
constexpr int kKeys = 128;       // keys of a key tile
constexpr int kThreads = 320;    // two softmax warpgroups, product warp, copy warp
constexpr float kGrow = 8.f;     // log2 of the growth that rescales
constexpr uint32_t kTmem = 512;  // columns: scores of both row tiles, then their outputs

// A block of queries and the list of its key tiles.
struct Block {
  int row, first, ntok;  // request, first token, tokens (0: none)
  int slot;              // slot of the first token
  int len;
  bool ok;
  int sink_tiles, from, count;  // key tiles: 0 .. sink_tiles - 1, then `from` on; `count` in all
  __device__ int tile(int k) const { return k < sink_tiles ? k : k - sink_tiles + from; }
};

__device__ __forceinline__ Block block_of(const PromptParams& p, int i, int lane, bool report) {
  Block r{};
  const int per = 2 * kRows / p.G;
  r.row = warp_last_at_most(p.B, i, lane, [&](int b) { return p.token_start[b] / per + b; });
  if (r.row < 0) return r;
  const RaggedRow g =
      ragged_row(p.token_start, p.seq_lens, p.active, r.row, p.T, p.max_pages_per_seq * p.P, p.err_flag, report);
  r.first = g.start + (i - (g.start / per + r.row)) * per;
  r.ntok = min(per, min(g.end, p.T) - r.first);
  if (g.start < 0 || r.first < 0) r.ntok = 0;
  r.ok = g.ok;
  r.len = g.len;
  if (r.ntok <= 0 || !g.ok) return r;
  r.slot = g.len - (g.end - r.first);
  const int last = r.slot + r.ntok - 1;
  r.sink_tiles = (min(p.sinks, last + 1) + kKeys - 1) / kKeys;
  r.from = max(r.sink_tiles, max(0, r.slot - p.window + 1) / kKeys);
  r.count = r.sink_tiles + last / kKeys + 1 - r.from;
  return r;
}

__device__ __forceinline__ int share_begin(int c, int n, int total) { return c * (total / n) + min(c, total % n); }

// Keys c of 32 that are visible, as bits: c < above, and c >= low or c < sink.
__device__ __forceinline__ uint32_t visible32(int above, int low, int sink) {
  auto below = [](int x) -> uint32_t { return x <= 0 ? 0u : (x >= 32 ? 0xffffffffu : (1u << x) - 1u); };
  return below(above) & (~below(low) | below(sink));
}

// One query by one warp, over the visible keys of the block's tiles [k0, k1)
// alone: lanes over head_dim, keys one at a time.  For rows that a value they
// do not see has reached (0 times infinity).  o: the lane's D / 32 elements.
template <typename E, int D>
__device__ __noinline__ void attend_alone(const PromptParams& p, const Block& blk, int k0, int k1, int h, int i,
                                          const uint16_t* q, float (&o)[D / 32], float& m, float& l) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31;
  const float NEG_INF = __int_as_float(0xff800000);
  float qf[PER];
#pragma unroll
  for (int e = 0; e < PER; e += 2) {
    const float2 w = E::to_float2(*reinterpret_cast<const uint32_t*>(q + lane * PER + e));
    qf[e] = w.x;
    qf[e + 1] = w.y;
  }
  m = NEG_INF;
  l = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.f;
  for (int k = k0; k < k1; ++k) {
    const int j0 = blk.tile(k) * kKeys;
    for (int j = j0; j < j0 + kKeys && j <= i; ++j) {
      if (j >= p.sinks && i - j >= p.window) continue;
      const long long lp = static_cast<long long>(blk.row) * p.max_pages_per_seq + j / p.P;
      const int page = p.page_table ? p.page_table[lp] : static_cast<int>(lp);
      const bool ok = page >= 0 && page < p.num_pages;
      const long long off = ok ? page * p.page_stride + (j % p.P) * p.token_stride + h * p.head_stride + lane * PER : 0;
      float s = 0.f, v[PER];
#pragma unroll
      for (int e = 0; e < PER; e += 2) {
        const float2 kk = ok ? E::to_float2(*reinterpret_cast<const uint32_t*>(p.k_cache + off + e)) : make_float2(0.f, 0.f);
        const float2 vv = ok ? E::to_float2(*reinterpret_cast<const uint32_t*>(p.v_cache + off + e)) : make_float2(0.f, 0.f);
        s += qf[e] * kk.x + qf[e + 1] * kk.y;
        v[e] = vv.x;
        v[e + 1] = vv.y;
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= p.scale_log2;
      const float mn = fmaxf(m, s), ms = mn == NEG_INF ? 0.f : mn;
      const float al = exp2f(m - ms), w = exp2f(s - ms);
      m = mn;
      l = l * al + w;
#pragma unroll
      for (int e = 0; e < PER; ++e) o[e] = o[e] * al + w * v[e];
    }
  }
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1) window_prompt_kernel(const __grid_constant__ PromptParams p) {
  constexpr int HALVES = D / 64;
  constexpr int KS = D / 16;                   // k-steps of the score product
  constexpr uint32_t kQTile = kRows * D * 2;   // bytes of a row tile's queries: [D/64][128 rows][128 B]
  constexpr uint32_t kStage = kKeys * D * 2;   // bytes of K or V of a key tile, likewise
  constexpr uint32_t kBlockBytes = kKeys * 128;  // one 64-element column block
  constexpr int ST = kPromptStages<D>;
  constexpr uint32_t kScores = tc_kind_f16(kRows, kKeys, !E::kF16, false);
  constexpr uint32_t kValues = tc_kind_f16(kRows, D, !E::kF16, true);
  extern __shared__ __align__(128) unsigned char smem_raw[];
  __shared__ uint64_t s_bars[2 * ST + 7];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y;
  // heavy blocks (long contexts, under a causal mask) first
  const int bi = gridDim.x - 1 - blockIdx.x;
  const Block blk = block_of(p, bi, lane, warp == 0 && lane == 0 && h == 0 && blockIdx.z == 0);
  if (blk.ntok <= 0) return;
  const int per_tile = kRows / p.G;  // tokens of a row tile
  const long long tok_stride = static_cast<long long>(p.Hq) * D;
  if (!blk.ok) {
    if (blockIdx.z == 0)
      for (int t = 0; t < blk.ntok; ++t) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + (blk.first + t) * tok_stride + static_cast<long long>(h) * p.G * D);
        for (int x = tid; x < p.G * D / 8; x += kThreads) dst[x] = make_uint4(0u, 0u, 0u, 0u);
      }
    return;
  }
  const int splits = min(p.splits, blk.count);
  if (static_cast<int>(blockIdx.z) >= splits) return;
  const int k0 = share_begin(blockIdx.z, splits, blk.count), k1 = share_begin(blockIdx.z + 1, splits, blk.count);
  const int last = blk.slot + blk.ntok - 1;      // slot of the last query
  const int low = max(0, blk.slot - p.window + 1);  // first key of the first query's window
  // row tile m sees key tile t?
  auto sees = [&](int m, int t) -> bool {
    const int f = blk.slot + m * per_tile;
    if (f > last) return false;
    const int e = min(last, f + per_tile - 1);
    return t <= e / kKeys && (t < blk.sink_tiles || t >= max(0, f - p.window + 1) / kKeys);
  };
  // some query of the block sees slot j?
  auto seen = [&](int j) -> bool { return j <= last && (j < p.sinks || j >= low); };

  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base, sKV = base + 2 * kQTile;
  const uint32_t bars = smem_addr(s_bars);
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (ST + s); };
  const uint32_t q_full = bars + 8 * (2 * ST);
  auto s_full = [&](int m) { return bars + 8 * (2 * ST + 1 + m); };
  auto p_full = [&](int m) { return bars + 8 * (2 * ST + 3 + m); };
  auto o_full = [&](int m) { return bars + 8 * (2 * ST + 5 + m); };
  volatile int* abort_flag = &s_abort;
  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < ST; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(q_full, 1);
    for (int m = 0; m < 2; ++m) {
      mbar_init(s_full(m), 1);
      mbar_init(p_full(m), kRows);
      mbar_init(o_full(m), 1);
    }
    fence_barrier_init();
  }
  if (warp == 8) tmem_alloc(smem_addr(&s_tmem), kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  auto t_scores = [&](int m) { return tmem + static_cast<uint32_t>(m * kKeys); };
  auto t_out = [&](int m) { return tmem + static_cast<uint32_t>(2 * kKeys + m * D); };
  auto give_up = [&]() {
    if (lane == 0) flag_error(p.err_flag, VH_ERR_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp == 9) {
    // ======================= copies ==============================================
    const int ntile = blk.ntok > per_tile ? 2 : 1;
    if (lane == 0) {
      prefetch_tensormap(&p.tmap_k);
      prefetch_tensormap(&p.tmap_v);
      mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(ntile) * kQTile);
      for (int m = 0; m < ntile; ++m)
        for (int hf = 0; hf < HALVES; ++hf)
          tma_load_3d(sQ + m * kQTile + hf * kBlockBytes, &p.tmap_q, hf * 64, h * p.G, blk.first + m * per_tile, q_full);
    }
    const int nbox = kKeys / p.box;
    int issued = 0;
    bool lost = false;
    for (int k = k0; k < k1 && !lost; ++k) {
      const int j0 = blk.tile(k) * kKeys;
      // page and first token of this lane's box (at most 16 boxes a tile)
      int page = p.num_pages, tok = 0;
      if (lane < nbox) {
        const int j = j0 + lane * p.box;
        if (j <= last && (j < p.sinks || j + p.box > low)) {
          const long long lp = static_cast<long long>(blk.row) * p.max_pages_per_seq + j / p.P;
          page = p.page_table ? p.page_table[lp] : static_cast<int>(lp);
          tok = j % p.P;
          if (page < 0 || page >= p.num_pages) {
            flag_error(p.err_flag, VH_ERR_PAGE);
            page = p.num_pages;
          }
        }
      }
      for (int kv = 0; kv < 2; ++kv, ++issued) {
        const int s = issued % ST;
        if (issued >= ST && !mbar_wait(empty(s), ((issued / ST) - 1) & 1)) {
          give_up();
          lost = true;
          break;
        }
        if (*abort_flag) {
          lost = true;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(full(s), kStage);
        __syncwarp();
        if (lane < nbox) {
          const void* map = kv ? static_cast<const void*>(&p.tmap_v) : static_cast<const void*>(&p.tmap_k);
          const int c1 = p.tm_tok_dim == 1 ? tok : h, c2 = p.tm_tok_dim == 1 ? h : tok;
#pragma unroll
          for (int hf = 0; hf < HALVES; ++hf)
            tma_load_4d(sKV + s * kStage + hf * kBlockBytes + lane * p.box * 128, map, hf * 64, c1, c2, page, full(s));
        }
      }
    }
    if (lost) {
      // copies in flight land before the shared memory goes away
      for (int x = max(0, issued - ST); x < issued; ++x) (void)mbar_wait(full(x % ST), (x / ST) & 1);
      (void)mbar_wait(q_full, 0);
    }
  } else if (warp == 8) {
    // ======================= products =============================================
    // a key tile's K is stage 2 (k - k0) of the ring, its V the next one
    int done_p[2] = {0, 0};
    bool lost = !mbar_wait(q_full, 0) || !mbar_wait(full(0), 0);
    auto scores = [&](int m, int k) {
      if (lane != 0) return;
      const uint32_t kb = sKV + ((2 * (k - k0)) % ST) * kStage, qb = sQ + m * kQTile;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint32_t off = (s >> 2) * kBlockBytes + (s & 3) * 32;
        tc_mma(t_scores(m), tc_operand(qb + off, 16, 1024), tc_operand(kb + off, 16, 1024), kScores, s > 0);
      }
      tc_commit(s_full(m));
    };
    if (!lost) {
      tc_fence_after();
      for (int m = 0; m < 2; ++m)
        if (sees(m, blk.tile(k0))) scores(m, k0);
      if (lane == 0) tc_commit(empty(0));
    }
    for (int k = k0; k < k1 && !lost; ++k) {
      const int vi = 2 * (k - k0) + 1, t = blk.tile(k);
      if (!mbar_wait(full(vi % ST), (vi / ST) & 1)) {
        lost = true;
        break;
      }
      const uint32_t vb = sKV + (vi % ST) * kStage;
      if (!(seen(t * kKeys) && seen(t * kKeys + kKeys - 1) && (t * kKeys >= low || t * kKeys + kKeys <= p.sinks))) {
        // slots that nobody sees may hold anything: their values become zeros
        for (int r = lane / 8; r < kKeys; r += 4) {
          if (seen(t * kKeys + r)) continue;
#pragma unroll
          for (int hf = 0; hf < HALVES; ++hf)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + hf * kBlockBytes + r * 128 + (lane & 7) * 16),
                         "r"(0u)
                         : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      const bool more = k + 1 < k1;
      if (more && !mbar_wait(full((vi + 1) % ST), ((vi + 1) / ST) & 1)) {
        lost = true;
        break;
      }
      for (int m = 0; m < 2 && !lost; ++m) {
        if (sees(m, t)) {
          if (!mbar_wait(p_full(m), done_p[m] & 1)) {
            lost = true;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
#pragma unroll
            for (int s = 0; s < kKeys / 16; ++s)
              tc_mma_ta(t_out(m), t_scores(m) + s * 8, tc_operand(vb + s * 2048, kBlockBytes, 1024), kValues,
                        done_p[m] > 0 || s > 0);
          }
          ++done_p[m];
        }
        if (more && sees(m, blk.tile(k + 1))) scores(m, k + 1);
        if (m == 0 && lane == 0 && !more) tc_commit(o_full(0));
      }
      if (!lost && lane == 0) {
        tc_commit(empty(vi % ST));
        if (more) tc_commit(empty((vi + 1) % ST));
        else tc_commit(o_full(1));
      }
    }
    if (lost) {
      give_up();
      // products in flight end before the tensor memory is freed
      if (lane == 0) tc_commit(o_full(0));
      (void)mbar_wait(o_full(0), 0);
    }
  } else {
    // ======================= softmax of row tile m =================================
    const int m = warp >> 2;
    const int r = tid & (kRows - 1);  // row of the tile = lane of tensor memory
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int token = m * per_tile + r / p.G;
    const bool valid = token < blk.ntok;
    const int i = min(blk.slot + token, last);
    const int f = blk.slot + m * per_tile;                 // first and last query of the tile
    const int e = min(last, f + per_tile - 1);
    const float NEG_INF = __int_as_float(0xff800000);
    float top = NEG_INF;  // the maximum that the weights refer to, times scale_log2
    float sum = 0.f;
    int n = 0;
    bool lost = false;
    for (int k = k0; k < k1; ++k) {
      const int t = blk.tile(k);
      if (!sees(m, t)) continue;
      if (!mbar_wait(s_full(m), n & 1)) {
        lost = true;
        break;
      }
      tc_fence_after();
      uint32_t sc[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t_scores(m) + lanes + c * 32, sc[c]);
      tmem_wait_ld();
      const int j0 = t * kKeys;
      if (j0 + kKeys - 1 > f || (j0 <= e - p.window && j0 + kKeys > p.sinks)) {
        // an edge of the causal mask, of the window or of the sinks
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int jc = j0 + c * 32;
          const uint32_t vis = visible32(i + 1 - jc, i - p.window + 1 - jc, p.sinks - jc);
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (!((vis >> x) & 1u)) sc[c][x] = 0xff800000u;
        }
      }
      float mx[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
      for (int x = 0; x < 32; ++x)
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = fmaxf(mx[c], __uint_as_float(sc[c][x]));
      const float now = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
      if (n == 0) {
        top = now;
      } else if (__any_sync(0xffffffffu, now > top + kGrow)) {
        // the products of the earlier key tiles are complete (the scores' commit
        // came after theirs), and the next waits for this tile's weights
        const float to = fmaxf(top, now);
        const float by = exp2f(top - (to == NEG_INF ? 0.f : to));
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(t_out(m) + lanes + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * by);
          tmem_st32(t_out(m) + lanes + c * 32, o);
        }
        sum *= by;
        top = to;
      }
      const float shift = top == NEG_INF ? 0.f : top;
      float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const float w = exp2f(fmaf(__uint_as_float(sc[c][x]), p.scale_log2, -shift));
          add[x & 3] += w;
          sc[c][x] = __float_as_uint(w);
        }
      sum += (add[0] + add[1]) + (add[2] + add[3]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const int e0 = c * 64 + 2 * x;
          w[x] = E::pack2(__uint_as_float(sc[e0 >> 5][e0 & 31]), __uint_as_float(sc[(e0 + 1) >> 5][(e0 + 1) & 31]));
        }
        tmem_st32(t_scores(m) + lanes + c * 32, w);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_full(m));
      ++n;
    }
    if (lost) give_up();
    if (!lost && !mbar_wait(o_full(m), 0)) {
      lost = true;
      give_up();
    }
    if (!lost) {
      tc_fence_after();
      const long long row_at = (blk.first + token) * tok_stride + (static_cast<long long>(h) * p.G + r % p.G) * D;
      const long long part =
          ((static_cast<long long>(bi) * p.Hkv + h) * p.splits + blockIdx.z) * (2 * kRows) + m * kRows + r;
      const float inv = sum > 0.f ? 1.f / sum : (n == 0 || top == NEG_INF ? 0.f : 1.f / sum);
      bool nan = false;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(t_out(m) + lanes + c * 32, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const float v = n > 0 ? __uint_as_float(o[x]) * inv : 0.f;
          nan |= !(v == v);
          o[x] = __float_as_uint(v);
        }
        if (valid && p.splits > 1) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + part * D + c * 32);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            dst[x] = make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]), __uint_as_float(o[4 * x + 2]),
                                 __uint_as_float(o[4 * x + 3]));
        } else if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + row_at + c * 32);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              w[y] = E::pack2(__uint_as_float(o[8 * x + 2 * y]), __uint_as_float(o[8 * x + 2 * y + 1]));
            dst[x] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
      }
      if (p.splits > 1 && valid) p.part_lse[part] = sum > 0.f ? top + log2f(sum) : (sum == 0.f ? NEG_INF : sum);
      // rows that ended with a NaN, once more over what they see alone
      uint32_t again = __ballot_sync(0xffffffffu, nan && valid);
      while (again) {
        const int src = __ffs(again) - 1;
        again &= again - 1;
        const int rr = (warp & 3) * 32 + src, tok = m * per_tile + rr / p.G;
        const long long at = (blk.first + tok) * tok_stride + (static_cast<long long>(h) * p.G + rr % p.G) * D;
        float o[D / 32], mm, ll;
        attend_alone<E, D>(p, blk, k0, k1, h, blk.slot + tok, p.q + at, o, mm, ll);
        const float il = ll == 0.f ? 0.f : 1.f / ll;
        if (p.splits > 1) {
          const long long pp =
              ((static_cast<long long>(bi) * p.Hkv + h) * p.splits + blockIdx.z) * (2 * kRows) + m * kRows + rr;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) p.part_o[pp * D + lane * (D / 32) + x] = o[x] * il;
          if (lane == 0) p.part_lse[pp] = ll > 0.f ? mm + log2f(ll) : (ll == 0.f ? NEG_INF : ll);
        } else {
#pragma unroll
          for (int x = 0; x < D / 32; x += 2)
            *reinterpret_cast<uint32_t*>(p.out + at + lane * (D / 32) + x) = E::pack2(o[x] * il, o[x + 1] * il);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_free(tmem, kTmem);
}

// Sum of a row's partial results over the CTAs that shared its block's keys:
// one warp a (token, head).
template <typename E, int D>
__global__ void __launch_bounds__(256) prompt_combine_kernel(const __grid_constant__ PromptParams p) {
  constexpr int PER = D / 32;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (unit >= static_cast<long long>(p.T) * p.Hq) return;
  const int t = static_cast<int>(unit / p.Hq), hq = static_cast<int>(unit % p.Hq);
  const int per = 2 * kRows / p.G, b = warp_last_at_most(p.B, t, lane, [&](int x) { return p.token_start[x]; });
  if (b < 0 || t >= p.token_start[b + 1] || p.token_start[b] < 0) return;
  const int local = t - p.token_start[b], bi = p.token_start[b] / per + b + local / per;
  const Block blk = block_of(p, bi, lane, false);
  if (!blk.ok || blk.row != b || blk.ntok <= 0) return;  // zeros are written already
  const int splits = min(p.splits, blk.count);
  const int r = (local % per) * p.G + hq % p.G;
  const long long part = ((static_cast<long long>(bi) * p.Hkv + hq / p.G) * p.splits) * (2 * kRows) + r;
  const float NEG_INF = __int_as_float(0xff800000);
  // (at most 64 splits: two a lane)
  float lse[2], top = NEG_INF;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int s = lane + 32 * x;
    lse[x] = s < splits ? p.part_lse[part + static_cast<long long>(s) * (2 * kRows)] : NEG_INF;
    top = fmaxf(top, lse[x]);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  const float shift = top == NEG_INF ? 0.f : top;
  float w[2] = {exp2f(lse[0] - shift), exp2f(lse[1] - shift)}, sum = w[0] + w[1];
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  float o[PER];
#pragma unroll
  for (int x = 0; x < PER; ++x) o[x] = 0.f;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float f = __shfl_sync(0xffffffffu, s < 32 ? w[0] : w[1], s & 31);
    const float* src = p.part_o + (part + static_cast<long long>(s) * (2 * kRows)) * D + lane * PER;
#pragma unroll
    for (int x = 0; x < PER; x += 2) {
      const float2 v = *reinterpret_cast<const float2*>(src + x);
      o[x] += f * v.x;
      o[x + 1] += f * v.y;
    }
  }
  const float inv = 1.f / sum;
#pragma unroll
  for (int x = 0; x < PER; x += 2)
    *reinterpret_cast<uint32_t*>(p.out + unit * D + lane * PER + x) = E::pack2(o[x] * inv, o[x + 1] * inv);
}

template <typename E, int D>
cudaError_t launch_t(const PromptParams& p, cudaStream_t stream) {
  window_prompt_kernel<E, D><<<dim3(p.blocks, p.Hkv, p.splits), kThreads, kPromptSmem<D>, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(p.T) * p.Hq + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_combine_kernel<E, D>, p);
}

}  // namespace

cudaError_t prepare_window_prompt() {
  const void* k[4] = {reinterpret_cast<const void*>(&window_prompt_kernel<ElemBf16, 64>),
                      reinterpret_cast<const void*>(&window_prompt_kernel<ElemBf16, 128>),
                      reinterpret_cast<const void*>(&window_prompt_kernel<ElemF16, 64>),
                      reinterpret_cast<const void*>(&window_prompt_kernel<ElemF16, 128>)};
  for (int x = 0; x < 4; ++x) {
    const cudaError_t e = cudaFuncSetAttribute(k[x], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               x & 1 ? kPromptSmem<128> : kPromptSmem<64>);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_window_prompt(const PromptParams& p, cudaStream_t stream) {
  if (p.D == 128) return p.f16 ? launch_t<ElemF16, 128>(p, stream) : launch_t<ElemBf16, 128>(p, stream);
  return p.f16 ? launch_t<ElemF16, 64>(p, stream) : launch_t<ElemBf16, 64>(p, stream);
}

}  // namespace vh
