// window_prompt.cu -- attention of a ragged batch of new tokens over the paged
// cache, with a sliding window and sinks.
//
// Operation: the token in slot i of its row sees V(i) = {j <= i: i - j < W or
// j < S};  o = sum_{j in V(i)} softmax(scale <q, K_j>) V_j, per q head, with
// kv head h = head / G.
//
// First form: one warp per (token, q head), lanes over head_dim, a running max
// and sum over the visible keys one at a time.  Right for every shape and the
// yardstick for a tiled kernel; bound by its own latency.
#include "vh_ragged.cuh"
#include "vh_window.h"

namespace vh {

namespace {

// One warp: attention of one query over its visible keys.  q: the lane's D/32
// elements (fp32).  Returns the lane's output elements.
template <typename E, int D>
__device__ __forceinline__ void attend_row(const PromptParams& p, int b, int h, int i, const float (&q)[D / 32],
                                           float (&o)[D / 32], int lane) {
  constexpr int PER = D / 32;
  const int lo = max(0, i - p.window + 1);
  const int ns = min(p.sinks, lo);
  float m = __int_as_float(0xff800000), l = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.f;
  for (int n = 0; n < ns + i + 1 - lo; ++n) {
    const int j = n < ns ? n : lo + n - ns;
    const long long lp = static_cast<long long>(b) * p.max_pages_per_seq + j / p.P;
    const int page = p.page_table ? p.page_table[lp] : static_cast<int>(lp);
    const bool ok = page >= 0 && page < p.num_pages;
    if (!ok && lane == 0) flag_error(p.err_flag, VH_ERR_PAGE);
    const long long off = page * p.page_stride + (j % p.P) * p.token_stride + h * p.head_stride + lane * PER;
    float k[PER], v[PER];
#pragma unroll
    for (int e = 0; e < PER; e += 2) {
      const float2 kk = ok ? E::to_float2(*reinterpret_cast<const uint32_t*>(p.k_cache + off + e)) : make_float2(0.f, 0.f);
      const float2 vv = ok ? E::to_float2(*reinterpret_cast<const uint32_t*>(p.v_cache + off + e)) : make_float2(0.f, 0.f);
      k[e] = kk.x;
      k[e + 1] = kk.y;
      v[e] = vv.x;
      v[e + 1] = vv.y;
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) s += q[e] * k[e];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float ms = mn == __int_as_float(0xff800000) ? 0.f : mn;
    const float al = exp2f(m - ms), w = exp2f(s - ms);
    m = mn;
    l = l * al + w;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = o[e] * al + w * v[e];
  }
  const float il = 1.f / l;
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] *= il;
}

template <typename E, int D>
__global__ void __launch_bounds__(256) window_prompt_kernel(const __grid_constant__ PromptParams p) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (unit >= static_cast<long long>(p.T) * p.Hq) return;
  const int t = static_cast<int>(unit / p.Hq), hq = static_cast<int>(unit % p.Hq);
  const int b = warp_last_at_most(p.B, t, lane, [&](int r) { return p.token_start[r]; });
  if (b < 0) return;
  const RaggedRow r = ragged_row(p.token_start, p.seq_lens, p.active, b, p.T, p.max_pages_per_seq * p.P, p.err_flag,
                                 lane == 0);
  if (t >= r.end) return;
  const long long at = unit * D + lane * PER;
  float q[PER], o[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.f;
  if (r.ok) {
#pragma unroll
    for (int e = 0; e < PER; e += 2) {
      const float2 w = E::to_float2(*reinterpret_cast<const uint32_t*>(p.q + at + e));
      q[e] = w.x;
      q[e + 1] = w.y;
    }
    attend_row<E, D>(p, b, hq / p.G, r.len - (r.end - t), q, o, lane);
  }
#pragma unroll
  for (int e = 0; e < PER; e += 2) *reinterpret_cast<uint32_t*>(p.out + at + e) = E::pack2(o[e], o[e + 1]);
}

}  // namespace

cudaError_t launch_window_prompt(const PromptParams& p, cudaStream_t stream) {
  const long long units = static_cast<long long>(p.T) * p.Hq;
  const unsigned grid = static_cast<unsigned>((units + 7) / 8);
  if (p.D == 128) {
    if (p.f16) window_prompt_kernel<ElemF16, 128><<<grid, 256, 0, stream>>>(p);
    else window_prompt_kernel<ElemBf16, 128><<<grid, 256, 0, stream>>>(p);
  } else {
    if (p.f16) window_prompt_kernel<ElemF16, 64><<<grid, 256, 0, stream>>>(p);
    else window_prompt_kernel<ElemBf16, 64><<<grid, 256, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace vh
