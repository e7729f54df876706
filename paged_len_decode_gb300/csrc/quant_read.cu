// quant_read.cu -- slots of an 8-bit cache, read back into a cache of 16 bits.
//
// Operation: row b, L = seq_lens[b], F = first_slot[b]; for its slots j < min(S, L)
// and F <= j < L, every kv head: out[j] = rne(e4m3(byte) * scale), for K and V.
//
// Bound by HBM: a byte in and two out an element, no arithmetic to speak of.
//  * Work list: the 16-token tiles of all rows, as in the windowed decode, cut
//    into equal shares, one a CTA.
//  * A (K or V, slot, head) is D contiguous bytes: D/16 neighbouring lanes take 16
//    bytes each, multiply by the slot's scale and write 32; a thread has eight such
//    loads under way.  The pages of a tile's two halves (8 tokens lie in one page,
//    whatever the page sizes) are looked up once a tile, a lane each.
// Measured: 16 rows of up to 16384 tokens, 8 heads of 128 (993 MB) 160 us = 6.2 TB/s, 92 % of a
// copy's rate; with four loads a thread 169-179, a first form that looked up pages and divided
// for every 16 bytes 266.
#include <algorithm>

#include "vh_e4m3.cuh"
#include "vh_quant.h"
#include "vh_ragged.cuh"
#include "vh_row_tiles.cuh"

namespace vh {

namespace {

constexpr int kWarpRows = 128;  // rows that one warp sums up alone
constexpr int kFlight = 8;      // loads of a thread under way

template <typename E, int D, int kThreads>
__global__ void __launch_bounds__(kThreads, 640 / kThreads) quant_read_kernel(const __grid_constant__ QuantReadParams p) {
  constexpr int LPR = D / 16;          // lanes of a slot's head
  constexpr int RPB = kThreads / LPR;  // (slot, head)s of the CTA at a time
  extern __shared__ int cum[];         // [B + 1], then lengths and first slots [B]
  __shared__ int most, tot[32];
  int *lens = cum + p.B + 1, *firsts = lens + p.B;
  const int tid = threadIdx.x, lane = tid & 31;
  const int max_len = min(p.max_pages_per_seq * p.P, p.out_per_row * p.out_P);
  pdl_begin();
  if (tid == 0) cum[0] = most = 0;
  __syncwarp();
  sum_rows<kWarpRows>(p.B, cum, &most, tot, tid < 32, [&](int b) -> int {
    const int act = p.active[b], L = p.seq_lens[b], first = p.first_slot ? p.first_slot[b] : 0;
    const bool ok = L >= 1 && L <= max_len && first >= 0;
    if (act && !ok && blockIdx.x == 0) flag_error(p.err_flag, VH_ERR_SEQLEN);
    lens[b] = L;
    firsts[b] = min(first, L);
    return act && ok ? tiles_of(L, L - min(first, L), p.sinks).count : 0;
  });
  const int T = cum[p.B], t0 = share_begin(blockIdx.x, gridDim.x, T), t1 = share_begin(blockIdx.x + 1, gridDim.x, T);
  // this thread's place in a (slot, head), and the (slot, head)s of a tile that it takes: r0 + x RPB, heads
  // inner; K's, then V's
  const int c = (tid % LPR) * 16, r0 = tid / LPR, rows = kTile * p.Hkv;
  int b = 0;
  for (int t = t0; t < t1; ++t) {
    if (t == t0 || t >= cum[b + 1]) b = row_of(cum, b, p.B, t);
    const int L = lens[b], window = L - firsts[b], tile = tiles_of(L, window, p.sinks).tile(t - cum[b]);
    const uint32_t seen = visible16(tile, L, window, p.sinks);
    // lanes 0 and 1: where the halves are read from (values, and scales); 2 and 3: where they go.  -1: nowhere
    long long at = -1, scale_at = -1;
    if (lane < 4 && (seen >> (8 * (lane & 1)) & 0xFFu)) {
      const bool out = lane >= 2;
      const int j = tile * kTile + 8 * (lane & 1), P = out ? p.out_P : p.P, of_row = j / P, off = j - of_row * P;
      const long long lp = static_cast<long long>(b) * (out ? p.out_per_row : p.max_pages_per_seq) + of_row;
      const int32_t* table = out ? p.out_table : p.page_table;
      const int page = table ? table[lp] : static_cast<int>(lp);
      if (page < 0 || page >= (out ? p.out_pages : p.num_pages)) {
        flag_error(p.err_flag, VH_ERR_PAGE);
      } else {
        at = out ? page * p.out_page + off * p.out_token : page * p.memory.page_stride + off * p.memory.token_stride;
        scale_at = page * p.memory.scale_page + off;
      }
    }
    const long long from0 = __shfl_sync(0xffffffffu, at, 0), from1 = __shfl_sync(0xffffffffu, at, 1);
    const long long to0 = __shfl_sync(0xffffffffu, at, 2), to1 = __shfl_sync(0xffffffffu, at, 3);
    const long long s0 = __shfl_sync(0xffffffffu, scale_at, 0), s1 = __shfl_sync(0xffffffffu, scale_at, 1);
    for (int rb = r0; rb < 2 * rows; rb += kFlight * RPB) {
      uint4 w[kFlight];
      float scale[kFlight];
      uint16_t* to[kFlight];
#pragma unroll
      for (int x = 0; x < kFlight; ++x) {
        const int r = rb + x * RPB;
        const bool v = r >= rows;
        const int y = v ? r - rows : r;
        const int j = p.hkv_inverse ? static_cast<int>(__umulhi(static_cast<uint32_t>(y), p.hkv_inverse)) : y;  // y / Hkv
        const int h = y - j * p.Hkv, i = j & 7;
        const long long from = j < 8 ? from0 : from1, dst = j < 8 ? to0 : to1;
        to[x] = nullptr;
        w[x] = make_uint4(0u, 0u, 0u, 0u);
        scale[x] = 0.f;
        if (r < 2 * rows && (seen >> j & 1u) && dst >= 0) {
          to[x] = (v ? p.v_out : p.k_out) + dst + i * p.out_token + h * p.out_head + c;
          if (from >= 0) {
            w[x] = __ldcs(reinterpret_cast<const uint4*>((v ? p.memory.v : p.memory.k) + from + i * p.memory.token_stride + h * p.memory.head_stride + c));
            scale[x] = __ldg((v ? p.memory.v_scale : p.memory.k_scale) + (j < 8 ? s0 : s1) + h * p.memory.scale_head + i);
          }
        }
      }
#pragma unroll
      for (int x = 0; x < kFlight; ++x) {
        if (!to[x]) continue;
        const uint32_t in[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 lo = f16x2_to_float2(e4m3x2_to_f16x2(in[i])), hi = f16x2_to_float2(e4m3x2_to_f16x2_hi(in[i]));
          o[2 * i] = E::pack2(lo.x * scale[x], lo.y * scale[x]);
          o[2 * i + 1] = E::pack2(hi.x * scale[x], hi.y * scale[x]);
        }
        __stcs(reinterpret_cast<uint4*>(to[x]), make_uint4(o[0], o[1], o[2], o[3]));
        __stcs(reinterpret_cast<uint4*>(to[x]) + 1, make_uint4(o[4], o[5], o[6], o[7]));
      }
    }
  }
}

using Kernel = void (*)(QuantReadParams);
template <int kThreads>
Kernel select_t(int D, bool f16) {
  return D == 128 ? (f16 ? quant_read_kernel<ElemF16, 128, kThreads> : quant_read_kernel<ElemBf16, 128, kThreads>)
                  : (f16 ? quant_read_kernel<ElemF16, 64, kThreads> : quant_read_kernel<ElemBf16, 64, kThreads>);
}
Kernel select_kernel(int D, bool f16, int threads) { return threads == 256 ? select_t<256>(D, f16) : select_t<128>(D, f16); }

}  // namespace

cudaError_t prepare_quant_read(int max_smem) {
  for (int D : {64, 128})
    for (bool f16 : {false, true})
      for (int threads : {128, 256}) {
        const cudaError_t e = cudaFuncSetAttribute(select_kernel(D, f16, threads), cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

cudaError_t launch_quant_read(const QuantReadParams& p, int sm_count, cudaStream_t stream) {
  // Tiles that the rows can have at most.  Few: CTAs of 256 threads, all there at once, since a tile
  // takes each of them one trip (8 rows, 264 tiles: 5.9 us, and 6.7 to 9.2 with CTAs of 128).  More:
  // small CTAs that come to the SMs as they get free, five at a time of 24 (16 rows, 993 MB: 159 us, and
  // 167 with the large ones; 180 with five, 173 with the large ones 16 an SM).
  const long long most = p.B * ((std::min<long long>(static_cast<long long>(p.max_pages_per_seq) * p.P,
                                                     static_cast<long long>(p.out_per_row) * p.out_P) + kTile - 1) / kTile);
  const int threads = most <= 16LL * sm_count ? 256 : 128;
  const int ctas = static_cast<int>(std::min<long long>(most, (threads == 256 ? 2 : 24) * sm_count));
  return launch_dependent(select_kernel(p.D, p.f16 != 0, threads), p, dim3(ctas), threads, quant_read_smem(p.B), stream);
}

}  // namespace vh
