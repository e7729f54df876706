// quant_decode.cu -- single-token GQA attention over a window and sinks of an
// 8-bit paged cache, rows split over CTAs and merged in the launch.
//
// Operation: row b, L = seq_lens[b]; V = {j < L: j < S or j >= L - W};
//   s_j = scale <q_rot, k8_j> ks_j,  o = sum_{j in V} softmax(s)_j vs_j v8_j,
// with k8, v8 the e4m3 values and ks, vs their scales; a running max and sum in fp32.
//
// Bound by HBM: 2 (D + 4) bytes a visible slot and kv head, for 4 G D flops.
//  * Work list, shares and the merge: those of the windowed decode
//    (vh_row_tiles.cuh): 16-token tiles, equal shares of the list of all rows, one a CTA.
//  * The producer warp describes 32 tiles at a time, a batch ahead of its use, and
//    copies each with four tensor copies: values of K and V of all heads of the
//    CTA, and their scales (two halves each where pages have 8 tokens).
//    A page id out of range becomes a page past the tensor, which the copy engine
//    fills with zeros.
//  * A consumer warp per kv head: S^T = K q^T and O^T += V^T P^T on mma.sync
//    m16n8k16 in fp16, which holds every e4m3 value: the bytes become fp16 pairs in
//    registers (cvt, two values an instruction), and each is read once from shared
//    memory.  The products' order of dimensions is free as long as q and K agree,
//    so a lane takes 16 neighbouring bytes of a key and no transposition is needed;
//    V is transposed by ldmatrix in pairs of bytes, and a byte permutation parts the
//    pairs: a lane then has two neighbouring columns of the output.
//  * q, divided by a power of two that brings its largest element into [1, 2), is
//    split into an fp16 high part and residual: 22 bits of that (and so are the weights
//    of an fp16 output).  ks multiplies the score.  The weight w = p_j vs_j c carries the value's
//    scale, and c, a power of two a head, is lowered when a weight would leave fp16 (w above 2^15),
//    to where the largest one lies in [2^13, 2^14): fp16 then holds weights down to 2^-27 of the
//    largest so far with 11 bits, and loses at most 2^-38 of that of smaller ones.  p refers
//    to a maximum that is raised only when a p would grow above 2^8 (no shuffles in most tiles), and c
//    rises with it by the power of two that the weights lost: a large scale early in the row,
//    whose key has no weight in the end, must not leave c too low for those that have it.
//  * Keys outside V get the score -inf and the scale 0, and their rows of V are zeroed in
//    shared memory, so nothing they hold counts.
//  * Two tiles at a time: one set of waits, votes and masks, and two independent chains
//    of conversions and products (256 rows, 1133 MB: 179 -> 176 us).  Two CTAs on an SM
//    with 100 KB of stages each, 8 consumer warps; 12 warps were no faster (three CTAs,
//    112 us against 110 on 676 MB), all heads of a token in one CTA an SM neither (114).
//  * Merge: the last CTA of a row fetches the pieces by bulk copies into the stages,
//    one trip to memory for up to 32 of them and for both its rows, where loads in
//    rounds of four pieces took 110 us instead of 108 (16 rows, 676 MB).
// Measured: 16 rows of 4096-32768 tokens (32 / 8 heads of 128, 676 MB) 108-110 us = 6.2 TB/s,
// 256 rows under a window of 2048 (1133 MB) 172-175 us = 6.5-6.6 TB/s (96-97 % of a copy's rate), 64
// rows of 200-1200 tokens (86 MB) 23.9 us: start 3 us, SMs that end 5 us apart, merge 3 us.
// Without any arithmetic the same copies take 104, 169 and 21.9 us.
#include "vh_e4m3.cuh"
#include "vh_quant.h"
#include "vh_ragged.cuh"
#include "vh_row_tiles.cuh"

namespace vh {

namespace {

template <int D>
constexpr int kHeadsMost = 512 / D;          // kv heads (consumer warps) of a CTA
constexpr int kWarpRows = 128;               // rows that the producer warp sums up alone
enum { kMiscTot = 0, kMiscAbort = 32, kMiscLost = 33, kMiscMost = 34, kMiscPart = 36, kMiscInts = 48 };  // part: 4 ints each
constexpr float kGrow = 8.f;                 // log2 of the weight that raises the maximum
constexpr float kWeightMost = 32768.f;       // the weight that lowers c
constexpr float kFactorMost = 1.2980742e33f; // 2^110: c at first, and at most
constexpr int kFactorExp = 127 + 110;        // its exponent's bits

__device__ __forceinline__ float lds(uint32_t addr) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr));
  return x;
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr));
  return x;
}
// The largest of the lanes with the same t4 (lane % 4).
__device__ __forceinline__ float max_of_keys(float x) {
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}
__device__ __forceinline__ float sum_of_keys(float x) {
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

template <int D, int G, typename E>
__global__ void __launch_bounds__(32 * (kHeadsMost<D> + 1), D == 128 ? 2 : 1) quant_decode_kernel(const __grid_constant__ QuantDecodeParams p) {
  constexpr int KS = D / 16;      // k-steps of the score product = m-tiles of the value product
  constexpr int CH = D / 16;      // 16-byte chunks of a key
  constexpr int PER = D / 32;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hc = p.Hc, S = p.stages, HG = Hc * G;
  const int c = blockIdx.x, gy = blockIdx.y, h0 = gy * Hc;
  int* cum = reinterpret_cast<int*>(smem + p.cum_off);
  int* lens = reinterpret_cast<int*>(smem + p.len_off);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.bar_off);
  int* misc = reinterpret_cast<int*>(bars + 2 * S + 2 + kHeadsMost<D>);
  volatile int* abort_flag = misc + kMiscAbort;
  const uint32_t full0 = smem_addr(bars), empty0 = smem_addr(bars + S);
  const uint32_t qfull = smem_addr(bars + 2 * S), qempty = smem_addr(bars + 2 * S + 1);
  const uint32_t merged0 = smem_addr(bars + 2 * S + 2);  // pieces have come, by consumer warp
  const int max_len = p.max_pages_per_seq * p.P;
  const bool p8 = p.P == 8;
  const float NEG_INF = __int_as_float(0xff800000);
  // a stage: K, V [head][16][D] bytes, then their scales [head][16] floats, each at a multiple
  // of 128 bytes; with 8-token pages the halves of the tokens come first
  const uint32_t tile_bytes = static_cast<uint32_t>(Hc * kTile * D), scale_bytes = static_cast<uint32_t>(p.scale_bytes);
  const uint32_t head_bytes = p8 ? 8 * D : 16 * D, half_bytes = p8 ? tile_bytes / 2 : 8 * D;
  const uint32_t scale_head = p8 ? 32 : 64, scale_half = p8 ? scale_bytes / 2 : 32;
  if (p.early) pdl_launch_dependents();
  else pdl_begin();

  // ---- work list (with VH_FLAG_PDL, before the wait) -------------------------------
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
  }
  sum_rows<kWarpRows>(p.B, cum, misc + kMiscMost, misc + kMiscTot, warp == Hc, count_row);
  const int T = cum[p.B];
  const Share share = share_of_cta(cum, p.B, c, p.N, misc[kMiscMost], kQuantPiece * G);
  const int n_eff = share.n_eff, t0 = share.t0, t1 = share.t1;
  const bool works = t1 > t0;
  const int b0 = works ? row_of(cum, share.b0, p.B, t0) : 0;

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
    const int tpp = (p.P + kTile - 1) / kTile;  // tiles of a page
    const int tpp_shift = (tpp & (tpp - 1)) == 0 ? __ffs(tpp) - 1 : -1;
    struct Tile {
      int row, tok, page, page2;  // tok: first token in the page; page2: second page (8-token pages)
    };
    // (one lane each; a half of 8 tokens without a visible key has no page)
    auto describe = [&](int t) -> Tile {
      Tile d{0, 0, p.num_pages, p.num_pages};
      if (t >= t1) return d;
      d.row = row_of(cum, b0, p.B, t);
      const int L = lens[d.row], tk = tiles_of(L, p.window, p.sinks).tile(t - cum[d.row]);
      auto page_at = [&](int j) -> int {
        const long long lp = static_cast<long long>(d.row) * p.max_pages_per_seq + j;
        const int page = p.page_table ? p.page_table[lp] : static_cast<int>(lp);
        if (page >= 0 && page < p.num_pages) return page;
        flag_error(p.err_flag, VH_ERR_PAGE);
        return p.num_pages;  // past the tensor: read as zeros
      };
      if (p8) {
        const uint32_t mask = visible16(tk, L, p.window, p.sinks);
        if (mask & 0x00FFu) d.page = page_at(2 * tk);
        if (mask & 0xFF00u) d.page2 = page_at(2 * tk + 1);
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
      if (lane < 4) prefetch_tensormap(lane == 0 ? &p.tmap_k : (lane == 1 ? &p.tmap_v : (lane == 2 ? &p.tmap_ks : &p.tmap_vs)));
    }
    if (p.early) pdl_wait();
    zero_rows();
    if (!works) return;
    // this lane's copy: K, V, and their scales; lanes 4 .. 7 the second half of 8-token pages
    const int kind = lane & 3, half = lane >> 2, copies = p8 ? 8 : 4;
    const void* map = kind == 0 ? static_cast<const void*>(&p.tmap_k)
                                : (kind == 1 ? static_cast<const void*>(&p.tmap_v)
                                             : (kind == 2 ? static_cast<const void*>(&p.tmap_ks) : static_cast<const void*>(&p.tmap_vs)));
    const uint32_t off = kind < 2 ? kind * tile_bytes + half * half_bytes : 2 * tile_bytes + (kind - 2) * scale_bytes + half * scale_half;
    const uint64_t policy = l2_policy_evict_first();  // the cache is read once a launch
    int stage = 0, round = 0, nseg = 0, prev_row = -1, issued = 0;
    bool aborted = false;
    for (int t = t0; t < t1; ++t, ++issued) {
      const int w = (t - t0) & 31;
      if (w == 0 && t > t0) cur = nxt;
      const int row = __shfl_sync(0xffffffffu, cur.row, w), tok = __shfl_sync(0xffffffffu, cur.tok, w);
      const int page = __shfl_sync(0xffffffffu, cur.page, w), page2 = __shfl_sync(0xffffffffu, cur.page2, w);
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
      const uint32_t st = smem_addr(smem) + static_cast<uint32_t>(stage * p.stage_bytes), fb = full0 + 8 * stage;
      if (lane == 0) mbar_arrive_expect_tx(fb, 2 * tile_bytes + static_cast<uint32_t>(Hc) * 128u);
      __syncwarp();
      if (lane < copies) {
        const int pg = half ? page2 : page;
        if (kind < 2) tma_load_4d_hint(st + off, map, 0, tok, h0, pg, fb, policy);
        else tma_load_3d_hint(st + off, map, tok, h0, pg, fb, policy);
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
  // chunk x of row r of a box lies at x ^ turn(r): 128-byte rows are swizzled by the row, 64-byte ones by every other
  auto turn = [](int r) { return D == 128 ? r & 7 : (r >> 1) & 3; };
  // K: this lane's 16-byte chunks of the keys g4 and g4 + 8
  const uint32_t k_row = w * head_bytes + g4 * D;
  // V by ldmatrix: lanes 0-7 the rows of tokens 0-7, 8-15 of tokens 8-15, of one chunk; 16-31 of the next
  const uint32_t v_row = tile_bytes + w * head_bytes + ((lane >> 3) & 1) * half_bytes + (lane & 7) * D;
  const int v_turn = turn(lane & 7), v_next = lane >> 4;
  const uint32_t s_row = 2 * tile_bytes + w * scale_head + g4 * 4;

  uint32_t qh[KS][2], ql[KS][2];
  float acc[KS][4];
  float m0 = NEG_INF, m1 = NEG_INF, l0 = 0.f, l1 = 0.f, c0 = 0.f, c1 = 0.f, f0 = 0.f, f1 = 0.f;
  int b = b0, rt0 = cum[b0], rt1 = cum[b0 + 1];
  RowTiles rt = tiles_of(lens[b], p.window, p.sinks);
  int nseg = 0, stage = 0, round = 0, npart = 0;
  int part_row[2];
  bool lost = false;
  auto rescale = [&](float by0, float by1) {
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      acc[mt][0] *= by0;
      acc[mt][1] *= by1;
      acc[mt][2] *= by0;
      acc[mt][3] *= by1;
    }
  };
  for (int t = t0; t < t1 && !lost;) {
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
      // dims t4 D / 4 + 4 k + {0, 1} and {2, 3} of head g4
      const float* qrow = reinterpret_cast<const float*>(smem + p.q_off) + (w * G + (g4 < G ? g4 : 0)) * D + t4 * (D / 4);
      float top = 0.f, probe = 0.f;  // probe: NaN with an element that is no number
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(qrow + 4 * k);
        top = fmaxf(fmaxf(fmaxf(top, fabsf(x.x)), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
        probe += x.x * 0.f + x.y * 0.f + x.z * 0.f + x.w * 0.f;
      }
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        probe += __shfl_xor_sync(0xffffffffu, probe, off);
      }
      const uint32_t two = min(max(__float_as_uint(top) & 0x7f800000u, 0x00800000u), 0x7e800000u);  // the power of two
      const float down = g4 < G ? __uint_as_float(0x7f000000u - two) : 0.f;
      const float f = probe == 0.f ? __uint_as_float(two) * p.scale_log2 : __int_as_float(0x7fffffff);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(qrow + 4 * k);
        split2<ElemF16>(x.x * down, x.y * down, qh[k][0], ql[k][0]);
        split2<ElemF16>(x.z * down, x.w * down, qh[k][1], ql[k][1]);
      }
      f0 = __shfl_sync(0xffffffffu, f, 8 * t4);
      f1 = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
      __syncwarp();
      if (lane == 0) mbar_arrive(qempty);
      ++nseg;
      m0 = m1 = NEG_INF;
      l0 = l1 = 0.f;
      c0 = c1 = kFactorMost;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
    }

    // Two tiles at a time, x = 0 and 1.  Where the share of a row has an odd number, the last
    // one stands in both places, invisible in the second.
    const int k0 = t - rt0;
    const bool two = t + 1 < min(t1, rt1);
    const int stage1 = !two ? stage : (stage + 1 == S ? 0 : stage + 1);
    const uint32_t round1 = two && stage1 == 0 ? round + 1 : round;
    if (!mbar_wait(full0 + 8 * stage, round & 1) || !mbar_wait(full0 + 8 * stage1, round1 & 1)) {
      lost = true;
      break;
    }
    const uint32_t stg[2] = {smem_addr(smem) + static_cast<uint32_t>(stage * p.stage_bytes), smem_addr(smem) + static_cast<uint32_t>(stage1 * p.stage_bytes)};
    // what is seen ends in a row's last tile, in its last tile of sinks or in the one behind them
    uint32_t mask[2] = {0xFFFFu, two ? 0xFFFFu : 0u};
    const bool edge = !two || k0 + 2 >= rt.count || (k0 <= rt.sink && k0 + 2 >= rt.sink);
    if (edge) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x == 1 && !two) continue;
        mask[x] = visible16(rt.tile(k0 + x), lens[b], p.window, p.sinks);
        // rows of V that are not visible meet the weight 0: make them zeros
        for (int y = lane; y < kTile * CH && mask[x] != 0xFFFFu; y += 32) {
          const int r = y / CH;
          if ((mask[x] >> r) & 1u) continue;
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(stg[x] + tile_bytes + w * head_bytes + (r >> 3) * half_bytes + (r & 7) * D + (y % CH) * 16),
                       "r"(0u)
                       : "memory");
        }
      }
      __syncwarp();
    }

    // scores: lane holds keys g4 and g4 + 8 of each tile, heads 2 t4 and 2 t4 + 1
    float s[2][4], va[2], vb[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t ka[KS], kb[KS];
#pragma unroll
      for (int y = 0; y < CH / 4; ++y) {
        const uint32_t at = stg[x] + k_row + (((t4 * (CH / 4) + y) ^ turn(g4)) << 4);
        const uint4 u = lds16(at), v = lds16(at + half_bytes);
        ka[4 * y] = u.x;
        ka[4 * y + 1] = u.y;
        ka[4 * y + 2] = u.z;
        ka[4 * y + 3] = u.w;
        kb[4 * y] = v.x;
        kb[4 * y + 1] = v.y;
        kb[4 * y + 2] = v.z;
        kb[4 * y + 3] = v.w;
      }
      const float ks_a = lds(stg[x] + s_row), ks_b = lds(stg[x] + s_row + scale_half);
      va[x] = lds(stg[x] + s_row + scale_bytes);
      vb[x] = lds(stg[x] + s_row + scale_bytes + scale_half);
      float sh[4] = {0.f, 0.f, 0.f, 0.f}, sl[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint32_t a0 = e4m3x2_to_f16x2(ka[k]), a1 = e4m3x2_to_f16x2(kb[k]);
        const uint32_t a2 = e4m3x2_to_f16x2_hi(ka[k]), a3 = e4m3x2_to_f16x2_hi(kb[k]);
        mma_f16(sh, a0, a1, a2, a3, qh[k][0], qh[k][1]);
        mma_f16(sl, a0, a1, a2, a3, ql[k][0], ql[k][1]);
      }
      s[x][0] = (sh[0] + sl[0]) * (ks_a * f0);
      s[x][1] = (sh[1] + sl[1]) * (ks_a * f1);
      s[x][2] = (sh[2] + sl[2]) * (ks_b * f0);
      s[x][3] = (sh[3] + sl[3]) * (ks_b * f1);
    }
    if (edge) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!((mask[x] >> g4) & 1u)) {
          s[x][0] = s[x][1] = NEG_INF;
          va[x] = 0.f;
        }
        if (!((mask[x] >> (g4 + 8)) & 1u)) {
          s[x][2] = s[x][3] = NEG_INF;
          vb[x] = 0.f;
        }
      }
    }
    const float mx0 = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
    const float mx1 = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
    if (__any_sync(0xffffffffu, mx0 > m0 + kGrow || mx1 > m1 + kGrow)) {
      // All weights so far shrink by 2^d, d = n - m, and c rises by 2^k, k = ceil(d), at most to its
      // first value: what they are in units of c stays, so that c never follows a weight that
      // no longer counts.  (k = 0 while m is -inf: nothing has lowered c.)
      auto raise = [&](float n, float& m, float& l, float& f) -> float {
        const int e = static_cast<int>(__float_as_uint(f) >> 23);
        const int k = min(static_cast<int>(ceilf(fminf(n - m, 256.f))), kFactorExp - e);
        const float by = exp2f(m - (n == NEG_INF ? 0.f : n) + static_cast<float>(k));
        l *= by * __uint_as_float(static_cast<uint32_t>(max(127 - k, 0)) << 23);
        f = __uint_as_float(static_cast<uint32_t>(e + k) << 23);
        m = n;
        return by;
      };
      const float n0 = fmaxf(m0, max_of_keys(mx0)), n1 = fmaxf(m1, max_of_keys(mx1));
      const float by0 = raise(n0, m0, l0, c0), by1 = raise(n1, m1, l1, c1);
      rescale(by0, by1);
    }
    // (a max of -inf, from scores that are, is subtracted as 0)
    const float ms0 = m0 == NEG_INF ? 0.f : m0, ms1 = m1 == NEG_INF ? 0.f : m1;
    float wt[2][4], top = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      s[x][0] = exp2f(s[x][0] - ms0);
      s[x][1] = exp2f(s[x][1] - ms1);
      s[x][2] = exp2f(s[x][2] - ms0);
      s[x][3] = exp2f(s[x][3] - ms1);
      l0 += s[x][0] + s[x][2];
      l1 += s[x][1] + s[x][3];
    }
    auto weigh = [&]() {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        // (in this order: vs c may be infinite where p is 0)
        wt[x][0] = s[x][0] * va[x] * c0;
        wt[x][1] = s[x][1] * va[x] * c1;
        wt[x][2] = s[x][2] * vb[x] * c0;
        wt[x][3] = s[x][3] * vb[x] * c1;
        top = fmaxf(fmaxf(top, fmaxf(wt[x][0], wt[x][1])), fmaxf(wt[x][2], wt[x][3]));
      }
    };
    weigh();
    if (__any_sync(0xffffffffu, top > kWeightMost)) {
      // c so that the largest weight of the tiles lies in [2^13, 2^14), if that is less than before
      constexpr float kSmall = 1.52587890625e-5f;  // 2^-16: p vs stays finite
      auto lower = [&](int n, float c_old) -> float {
        float u = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) u = fmaxf(u, fmaxf(s[x][n] * (va[x] * kSmall), s[x][2 + n] * (vb[x] * kSmall)));
        const uint32_t e = __float_as_uint(max_of_keys(u)) & 0x7f800000u;
        // 2^(13 - 16 - exponent of u), at least 2^-120
        const int bits = static_cast<int>((127u + 127u - 3u) << 23) - static_cast<int>(e);
        return fminf(c_old, __int_as_float(max(bits, 7 << 23)));
      };
      const float d0 = lower(0, c0), d1 = lower(1, c1);
      rescale(d0 / c0, d1 / c1);  // (powers of two)
      c0 = d0;
      c1 = d1;
      weigh();
    }
    // Weights rounded to fp16 add to the error of a bf16 output a tenth of its own rounding; of an
    // fp16 output they would add as much again, so there the residuals are multiplied too.
    uint32_t bw[2][2], bl[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if constexpr (E::kF16) {
          split2<ElemF16>(wt[x][2 * y], wt[x][2 * y + 1], bw[x][y], bl[x][y]);
          bl[x][y] = movm_t(bl[x][y]);
        } else {
          bw[x][y] = pack_f16x2(wt[x][2 * y], wt[x][2 * y + 1]);
        }
        bw[x][y] = movm_t(bw[x][y]);
      }
    }
#pragma unroll
    for (int mt = 0; mt < KS; mt += 2) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t r[4];
        ldsm_x4_t(stg[x] + v_row + (((mt + v_next) ^ v_turn) << 4), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          // (token 2 t4, token 2 t4 + 1) of column 2 g4 in the lower half, of column 2 g4 + 1 in the upper one
          const uint32_t u = __byte_perm(r[2 * y], 0u, 0x3120), v = __byte_perm(r[2 * y + 1], 0u, 0x3120);
          const uint32_t a0 = e4m3x2_to_f16x2(u), a1 = e4m3x2_to_f16x2_hi(u), a2 = e4m3x2_to_f16x2(v), a3 = e4m3x2_to_f16x2_hi(v);
          mma_f16(acc[mt + y], a0, a1, a2, a3, bw[x][0], bw[x][1]);
          if constexpr (E::kF16) mma_f16(acc[mt + y], a0, a1, a2, a3, bl[x][0], bl[x][1]);
        }
      }
    }
    if (edge) fence_proxy_async_smem();  // the zeros, before the next copy into this stage
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(empty0 + 8 * stage);
      if (two) mbar_arrive(empty0 + 8 * stage1);
    }
    t += two ? 2 : 1;
    stage = stage1 + 1;
    round = round1;
    if (stage == S) {
      stage = 0;
      ++round;
    }

    // ---- end of this CTA's share of a row: finished output, or a partial one ------
    if (t == t1 || t == rt1) {
      const float L0 = sum_of_keys(l0), L1 = sum_of_keys(l1);
      const int n0 = 2 * t4, n1 = 2 * t4 + 1;
      const bool whole = rt0 >= t0 && rt1 <= t1;
      // (a whole row without weight is NaN; a piece without weight adds nothing)
      const float il0 = (!whole && L0 == 0.f ? 0.f : 1.f / L0), il1 = (!whole && L1 == 0.f ? 0.f : 1.f / L1);
      const float ic0 = 1.f / c0, ic1 = 1.f / c1;
      if (whole) {
        uint16_t* o0 = p.out + (static_cast<long long>(b) * p.Hq + static_cast<long long>(h) * G + n0) * D + 2 * g4;
        uint16_t* o1 = o0 + D;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          if (n0 < G) *reinterpret_cast<uint32_t*>(o0 + mt * 16) = E::pack2(acc[mt][0] * il0 * ic0, acc[mt][2] * il0 * ic0);
          if (n1 < G) *reinterpret_cast<uint32_t*>(o1 + mt * 16) = E::pack2(acc[mt][1] * il1 * ic1, acc[mt][3] * il1 * ic1);
        }
      } else {
        // piece slot 0 of a CTA belongs to its first row, slot 1 to a later one
        const long long base = ((static_cast<long long>(gy) * p.N + c) * 2 + (b == b0 ? 0 : 1)) * HG + w * G;
        float* o0 = p.part_o + (base + n0) * D + 2 * g4;
        float* o1 = o0 + D;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          if (n0 < G) *reinterpret_cast<float2*>(o0 + mt * 16) = make_float2(acc[mt][0] * il0 * ic0, acc[mt][2] * il0 * ic0);
          if (n1 < G) *reinterpret_cast<float2*>(o1 + mt * 16) = make_float2(acc[mt][1] * il1 * ic1, acc[mt][3] * il1 * ic1);
        }
        if (g4 == 0) {
          if (n0 < G) p.part_lse[base + n0] = m0 + log2f(L0);
          if (n1 < G) p.part_lse[base + n1] = m1 + log2f(L1);
        }
        part_row[npart++ & 1] = b;
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
  // The warp's share of the stages (all tiles have been consumed) takes the pieces by bulk
  // copies, up to 32 a trip to memory; both rows' come in one where there is room.
  constexpr int PIECE = G * D * 4;
  const uint32_t share_bytes = static_cast<uint32_t>(S * p.stage_bytes / Hc) & ~127u;
  const uint32_t room = smem_addr(smem) + static_cast<uint32_t>(w) * share_bytes;
  const int cap = min(32, static_cast<int>(share_bytes / PIECE));
  const int* const part = misc + kMiscPart;
  const int n0 = part[0] ? part[2] : 0, n1 = npart > 1 && part[4] ? part[6] : 0;
  const bool together = n0 + n1 <= cap;
  float lse[G], wt[G], M[G], sum[G], o[G][PER];
  uint32_t trips = 0;
  // pieces j0 .. j0 + n - 1 of row k, each to a lane's slot from lane `lo` on
  auto fetch = [&](int k, int j0, int lo, int n) {
    if (lane < lo || lane >= lo + n) return;
    const int* v = part + 4 * k;
    const int j = j0 + lane - lo;
    const long long at = ((static_cast<long long>(gy) * p.N + v[1] + j) * 2 + (j == 0 ? v[3] : 0)) * HG + w * G;
    bulk_g2s(room + lane * PIECE, p.part_o + at * D, PIECE, merged0 + 8 * w);
#pragma unroll
    for (int x = 0; x < G; ++x) lse[x] = __ldcg(p.part_lse + at + x);
  };
  auto expect = [&](int n) {
    // what was read and written there by loads and stores comes before the copies, and
    // what other CTAs wrote (seen by the counter's acquire) too
    asm volatile("fence.proxy.async;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(merged0 + 8 * w, static_cast<uint32_t>(n * PIECE));
    __syncwarp();
  };
  // adds the pieces of lanes lo .. lo + n - 1
  auto add = [&](int lo, int n) -> bool {
#pragma unroll
    for (int x = 0; x < G; ++x) {
      const float mine = lane >= lo && lane < lo + n ? lse[x] : NEG_INF;
      float mx = mine;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      mx = fmaxf(mx, M[x]);
      const float ms = mx == NEG_INF ? 0.f : mx, sc = exp2f(M[x] - ms);
      M[x] = mx;
      wt[x] = mine == NEG_INF ? 0.f : at_least_tiny(exp2f(mine - ms));
      float all = wt[x];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
      sum[x] = sum[x] * sc + all;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[x][i] *= sc;
    }
    if (!mbar_wait(merged0 + 8 * w, trips & 1u)) return false;
    for (int j = lo; j < lo + n; ++j) {
      const uint32_t at = room + static_cast<uint32_t>(j * PIECE + lane * PER * 4);
#pragma unroll
      for (int x = 0; x < G; ++x) {
        const float f = __shfl_sync(0xffffffffu, wt[x], j);
#pragma unroll
        for (int i = 0; i < PER; i += 2) {
          float2 y;
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(y.x), "=f"(y.y) : "r"(at + x * D * 4 + i * 4));
          o[x][i] += f * y.x;
          o[x][i + 1] += f * y.y;
        }
      }
    }
    return true;
  };
  if (together && n0 + n1 > 0) {
    expect(n0 + n1);
    fetch(0, 0, 0, n0);
    fetch(1, 0, n0, n1);
  }
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int n = k ? n1 : n0;
    if (n == 0) continue;
#pragma unroll
    for (int x = 0; x < G; ++x) {
      M[x] = NEG_INF;
      sum[x] = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[x][i] = 0.f;
    }
    bool came = true;
    if (together) {
      came = add(k ? n0 : 0, n);
    } else {
      for (int j0 = 0; j0 < n && came; j0 += cap) {
        expect(min(cap, n - j0));
        fetch(k, j0, 0, min(cap, n - j0));
        came = add(0, min(cap, n - j0));
        ++trips;
        __syncwarp();
      }
    }
    if (!came) {
      if (lane == 0) flag_error(p.err_flag, VH_ERR_TIMEOUT);
      (void)mbar_wait(merged0 + 8 * w, trips & 1u);  // (no copy outlives the CTA)
      return;
    }
#pragma unroll
    for (int x = 0; x < G; ++x) {
      const float il = 1.f / sum[x];
      uint16_t* dst = p.out + (static_cast<long long>(k ? part_row[1] : part_row[0]) * p.Hq + static_cast<long long>(h) * G + x) * D + lane * PER;
#pragma unroll
      for (int i = 0; i < PER; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = E::pack2(o[x][i] * il, o[x][i + 1] * il);
    }
  }
}

using Kernel = void (*)(QuantDecodeParams);

template <typename E, int D>
Kernel select_g(int G) {
  switch (G) {
    case 1: return &quant_decode_kernel<D, 1, E>;
    case 2: return &quant_decode_kernel<D, 2, E>;
    case 4: return &quant_decode_kernel<D, 4, E>;
    default: return &quant_decode_kernel<D, 8, E>;
  }
}

Kernel select_kernel(int D, int G, bool f16) {
  return D == 128 ? (f16 ? select_g<ElemF16, 128>(G) : select_g<ElemBf16, 128>(G)) : (f16 ? select_g<ElemF16, 64>(G) : select_g<ElemBf16, 64>(G));
}

}  // namespace

cudaError_t prepare_quant_decode(int max_smem) {
  for (int D : {64, 128})
    for (int G : {1, 2, 4, 8})
      for (bool f16 : {false, true}) {
        const cudaError_t e =
            cudaFuncSetAttribute(select_kernel(D, G, f16), cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

cudaError_t quant_decode_occupancy(const QuantDecodeParams& p, int* blocks_per_sm) {
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, select_kernel(p.D, p.G, p.f16 != 0),
                                                       32 * (p.Hc + 1), p.smem_bytes);
}

cudaError_t launch_quant_decode(const QuantDecodeParams& p, cudaStream_t stream) {
  return launch_dependent(select_kernel(p.D, p.G, p.f16 != 0), p, dim3(p.N, p.groups), 32 * (p.Hc + 1),
                          static_cast<size_t>(p.smem_bytes), stream);
}

}  // namespace vh
