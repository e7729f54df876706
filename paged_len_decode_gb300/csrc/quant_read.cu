// quant_read.cu -- slots of an 8-bit cache, read back into a cache of 16 bits.
//
// Operation: row b, L = seq_lens[b], F = first_slot[b]; for its slots j < min(S, L)
// and F <= j < L, every kv head: out[j] = rne(e4m3(byte) * scale), for K and V.
//
// Bound by HBM: a byte in and two out an element, no arithmetic to speak of.
//  * Work list: the 16-token tiles of all rows, as in the windowed decode, cut
//    into equal shares, one a CTA.
//  * A (K or V, slot, head) is D contiguous bytes: D/16 neighbouring lanes take 16
//    bytes each, multiply by the slot's scale and write 32.
#include "vh_e4m3.cuh"
#include "vh_quant.h"
#include "vh_ragged.cuh"
#include "vh_row_tiles.cuh"

namespace vh {

namespace {

constexpr int kThreads = 256;

template <typename E, int D>
__global__ void __launch_bounds__(kThreads) quant_read_kernel(const __grid_constant__ QuantReadParams p) {
  constexpr int LPR = D / 16;              // lanes of a slot's head
  constexpr int RPB = kThreads / LPR;      // (slot, head)s of the CTA at a time
  extern __shared__ int cum[];             // [B + 1]
  __shared__ int tot[32];
  const int tid = threadIdx.x;
  const int max_len = min(p.max_pages_per_seq * p.P, p.out_per_row * p.out_P);
  pdl_begin();
  if (tid == 0) cum[0] = 0;
  for (int b = tid; b < p.B; b += kThreads) {
    const int L = p.seq_lens[b], first = p.first_slot ? p.first_slot[b] : 0;
    const bool act = p.active[b] != 0, ok = L >= 1 && L <= max_len && first >= 0;
    if (act && !ok && blockIdx.x == 0) flag_error(p.err_flag, VH_ERR_SEQLEN);
    cum[1 + b] = act && ok ? tiles_of(L, L - min(first, L), p.sinks).count : 0;
  }
  __syncthreads();
  scan_rows(cum, p.B, tot);
  const int T = cum[p.B], t1 = share_begin(blockIdx.x + 1, gridDim.x, T);
  int b = 0;
  for (int t = share_begin(blockIdx.x, gridDim.x, T); t < t1; ++t) {
    if (b == 0 || t >= cum[b + 1]) b = row_of(cum, b, p.B, t);
    const int L = p.seq_lens[b], first = p.first_slot ? p.first_slot[b] : 0;
    const int tile = tiles_of(L, L - min(first, L), p.sinks).tile(t - cum[b]);
    const int rows = 2 * kTile * p.Hkv;
    for (int r = tid / LPR; r < rows; r += RPB) {
      const int kv = r & 1, x = r >> 1, h = x % p.Hkv, j = tile * kTile + x / p.Hkv;
      if (j >= L || (j < first && j >= p.sinks)) continue;
      const int of_row = j / p.P, off = j - of_row * p.P, to_row = j / p.out_P, to_off = j - to_row * p.out_P;
      const long long lp = static_cast<long long>(b) * p.max_pages_per_seq + of_row, lo = static_cast<long long>(b) * p.out_per_row + to_row;
      const int page = p.page_table ? p.page_table[lp] : static_cast<int>(lp), to = p.out_table ? p.out_table[lo] : static_cast<int>(lo);
      const bool page_ok = page >= 0 && page < p.num_pages, to_ok = to >= 0 && to < p.out_pages;
      if (!page_ok || !to_ok) flag_error(p.err_flag, VH_ERR_PAGE);
      if (!to_ok) continue;
      const int c = (tid % LPR) * 16;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      float scale = 0.f;
      if (page_ok) {
        w = __ldg(reinterpret_cast<const uint4*>((kv ? p.memory.v : p.memory.k) + page * p.memory.page_stride + off * p.memory.token_stride +
                                                 h * p.memory.head_stride + c));
        scale = __ldg((kv ? p.memory.v_scale : p.memory.k_scale) + page * p.memory.scale_page + h * p.memory.scale_head + off);
      }
      uint16_t* dst = (kv ? p.v_out : p.k_out) + to * p.out_page + to_off * p.out_token + h * p.out_head + c;
      const uint32_t in[4] = {w.x, w.y, w.z, w.w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(in[i])), c2 = f16x2_to_float2(e4m3x2_to_f16x2_hi(in[i]));
        o[2 * i] = E::pack2(a.x * scale, a.y * scale);
        o[2 * i + 1] = E::pack2(c2.x * scale, c2.y * scale);
      }
      *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(dst + 8) = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

using Kernel = void (*)(QuantReadParams);
Kernel select_kernel(int D, bool f16) {
  return D == 128 ? (f16 ? quant_read_kernel<ElemF16, 128> : quant_read_kernel<ElemBf16, 128>)
                  : (f16 ? quant_read_kernel<ElemF16, 64> : quant_read_kernel<ElemBf16, 64>);
}

}  // namespace

cudaError_t prepare_quant_read(int max_smem) {
  for (int D : {64, 128})
    for (bool f16 : {false, true}) {
      const cudaError_t e = cudaFuncSetAttribute(select_kernel(D, f16), cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

cudaError_t launch_quant_read(const QuantReadParams& p, cudaStream_t stream) {
  return launch_dependent(select_kernel(p.D, p.f16 != 0), p, dim3(p.ctas), kThreads, 4 * (static_cast<size_t>(p.B) + 1), stream);
}

}  // namespace vh
