// quant_decode.cu -- single-token GQA attention over a window and sinks of an
// 8-bit paged cache.
//
// Operation: row b, L = seq_lens[b]; V = {j < L: j < S or j >= L - W};
//   s_j = scale <q_rot, k8_j> ks_j,  o = sum_{j in V} softmax(s)_j vs_j v8_j,
// with k8, v8 the e4m3 values and ks, vs their scales; a running max and sum in fp32.
//
// First form: a CTA a (row, kv head), whose warps take every fourth visible slot; a lane
// has D/32 of the dimensions.
#include "vh_e4m3.cuh"
#include "vh_quant.h"
#include "vh_ragged.cuh"

namespace vh {

namespace {

constexpr int kWarps = 4;

template <typename E, int D, int G>
__global__ void __launch_bounds__(32 * kWarps) quant_decode_kernel(const __grid_constant__ QuantDecodeParams p) {
  constexpr int PER = D / 32;
  __shared__ float part[kWarps][G][D + 2];
  const int b = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float NEG_INF = __int_as_float(0xff800000);
  pdl_begin();
  const int act = p.active[b], L = p.seq_lens[b];
  const bool ok = act && L >= 1 && L <= p.max_pages_per_seq * p.P;
  if (act && !ok && h == 0 && threadIdx.x == 0) flag_error(p.err_flag, VH_ERR_SEQLEN);
  const long long row = (static_cast<long long>(b) * p.Hq + static_cast<long long>(h) * G) * D;
  if (!ok) {
    for (int i = threadIdx.x; i < G * D; i += blockDim.x) p.out[row + i] = 0;
    return;
  }
  float q[G][PER], o[G][PER], M[G], sum[G];
#pragma unroll
  for (int n = 0; n < G; ++n) {
    M[n] = NEG_INF;
    sum[n] = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      q[n][e] = p.q_rot[row + n * D + lane * PER + e];
      o[n][e] = 0.f;
    }
  }
  const int sinks = min(p.sinks, L), low = max(sinks, L - p.window);
  for (int i = warp; i < sinks + L - low; i += kWarps) {
    const int j = i < sinks ? i : i - sinks + low;
    const long long lp = static_cast<long long>(b) * p.max_pages_per_seq + j / p.P;
    const int page = p.page_table ? p.page_table[lp] : static_cast<int>(lp);
    const bool page_ok = page >= 0 && page < p.num_pages;
    if (!page_ok && lane == 0) flag_error(p.err_flag, VH_ERR_PAGE);
    float k[PER], v[PER], ks = 0.f, vs = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) k[e] = v[e] = 0.f;
    if (page_ok) {
      const long long at = page * p.memory.page_stride + (j % p.P) * p.memory.token_stride + h * p.memory.head_stride + lane * PER;
      const long long sc = page * p.memory.scale_page + h * p.memory.scale_head + j % p.P;
      ks = p.memory.k_scale[sc];
      vs = p.memory.v_scale[sc];
#pragma unroll
      for (int e = 0; e < PER; e += 2) {
        const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(p.memory.k + at + e)));
        const float2 c = f16x2_to_float2(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(p.memory.v + at + e)));
        k[e] = a.x;
        k[e + 1] = a.y;
        v[e] = c.x;
        v[e + 1] = c.y;
      }
    }
#pragma unroll
    for (int n = 0; n < G; ++n) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < PER; ++e) s += q[n][e] * k[e];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s = s * ks * p.scale_log2;
      const float mx = fmaxf(M[n], s), ms = mx == NEG_INF ? 0.f : mx;
      const float by = exp2f(M[n] - ms), w = exp2f(s - ms);
      M[n] = mx;
      sum[n] = sum[n] * by + w;
#pragma unroll
      for (int e = 0; e < PER; ++e) o[n][e] = o[n][e] * by + w * (v[e] * vs);
    }
  }
#pragma unroll
  for (int n = 0; n < G; ++n) {
#pragma unroll
    for (int e = 0; e < PER; ++e) part[warp][n][lane * PER + e] = o[n][e];
    part[warp][n][D] = M[n];
    part[warp][n][D + 1] = sum[n];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < G * D; i += blockDim.x) {
    const int n = i / D, d = i % D;
    float mx = NEG_INF;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, part[w][n][D]);
    const float ms = mx == NEG_INF ? 0.f : mx;
    float all = 0.f, out = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float f = part[w][n][D] == NEG_INF && part[w][n][D + 1] == 0.f ? 0.f : exp2f(part[w][n][D] - ms);
      all += f * part[w][n][D + 1];
      out += f * part[w][n][d];
    }
    p.out[row + i] = E::bits(out / all);
  }
}

using Kernel = void (*)(QuantDecodeParams);

template <typename E, int D>
Kernel select_g(int G) {
  switch (G) {
    case 1: return &quant_decode_kernel<E, D, 1>;
    case 2: return &quant_decode_kernel<E, D, 2>;
    case 4: return &quant_decode_kernel<E, D, 4>;
    default: return &quant_decode_kernel<E, D, 8>;
  }
}

}  // namespace

cudaError_t launch_quant_decode(const QuantDecodeParams& p, cudaStream_t stream) {
  const Kernel k = p.D == 128 ? (p.f16 ? select_g<ElemF16, 128>(p.G) : select_g<ElemBf16, 128>(p.G))
                              : (p.f16 ? select_g<ElemF16, 64>(p.G) : select_g<ElemBf16, 64>(p.G));
  return launch_dependent(k, p, dim3(p.B, p.Hkv), 32 * kWarps, 0, stream);
}

}  // namespace vh
