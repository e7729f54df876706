// mrope_append.cu -- RoPE with several axes of positions and KV append for a
// ragged batch of new tokens.
//
// Operation: token t of row b, in slot i = seq_lens[b] - (token_start[b+1] - t),
//   q_rot[t]     = rope(norm_q(q[t]))             (fp32, or rounded to 16 bits)
//   cache slot i = rne(rope(norm_k(k_new[t]))), v_new[t]
// with pair j of D/2 turned by the angle positions[axis(j)][t] * theta^(-2j/D)
// (cos and sin from the fp32 table) and norm_*(x) = w x / sqrt(mean(x^2) + eps).
//
// Bound by HBM for prompts (T D (Hq (2 + out) + 8 Hkv) bytes, 3 flops an
// element) and by latency for a decode step's few tokens.  A CTA takes
// `tokens_per_cta` consecutive tokens: warp w first looks up token w's row,
// slot and page and gathers the token's cos/sin row into shared memory (one
// pair at a time, since neighbouring pairs may belong to different axes), then
// all threads rotate units of 8 pairs (16-byte loads) and copy v.  The first
// unit of a thread is loaded before the barrier, so its latency and the
// look-ups' overlap.
#include "vh_ragged.cuh"
#include "vh_window.h"

namespace vh {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = kThreads / 32;  // tokens of a CTA: one look-up warp each

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

template <typename E, int D>
__global__ void __launch_bounds__(kThreads) mrope_kv_append_kernel(const __grid_constant__ MropeParams p) {
  constexpr int HALF = D / 2;
  constexpr int UPH = HALF / 8;  // units of a head: 8 pairs each
  __shared__ float s_cs[kMaxTok][D];
  __shared__ long long s_slot[kMaxTok];  // offset of the slot in the cache; -1: no append
  __shared__ int s_live[kMaxTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * p.tokens_per_cta;
  const int ntok = min(p.tokens_per_cta, p.T - t0);
  const int heads = p.Hq + p.Hkv;
  const int units = ntok * heads * UPH;
  const bool ilv = p.rope_interleaved != 0;

  // unit u: token, head (q heads first, then the new k heads) and first pair;
  // a: the 8 first elements, b: their 8 partners (interleaved: 16 in a row)
  uint4 a = make_uint4(0, 0, 0, 0), b = a;
  int tk = 0, h = 0, i = 0;
  auto load = [&](int u) {
    const bool valid = u < units;
    const int hu = valid ? u / UPH : 0;
    tk = hu / heads;
    h = hu - tk * heads;
    i = (valid ? u % UPH : 0) * 8;
    if (!valid) return;
    const uint16_t* src = h < p.Hq ? p.q + (t0 + tk) * p.q_stride + h * D
                                   : p.k_new + (t0 + tk) * p.k_stride + (h - p.Hq) * D;
    a = ldg16(src + (ilv ? 2 * i : i));
    b = ldg16(src + (ilv ? 2 * i + 8 : HALF + i));
  };
  load(tid);

  // ---- look-ups: warp w for token t0 + w ------------------------------------
  if (warp < ntok) {
    const int t = t0 + warp;
    const int row = p.token_start
                        ? warp_last_at_most(p.B, t, lane, [&](int r) { return p.token_start[r]; })
                        : t;
    bool live = false;
    long long slot_off = -1;
    int slot = 0;
    if (row >= 0) {
      const RaggedRow r = ragged_row(p.token_start, p.seq_lens, p.active, row, p.T, p.max_pages_per_seq * p.P,
                                     p.err_flag, lane == 0);
      slot = r.len - (r.end - t);
      live = r.ok && t < r.end;
    }
    if (live) {
      int bad = 0;
      int pos[HALF / 32];
#pragma unroll
      for (int j = 0; j < HALF / 32; ++j) {
        const int pair = lane + 32 * j;
        const int ax = static_cast<int>(p.axis[pair >> 5] >> (2 * (pair & 31))) & 3;
        pos[j] = p.positions ? __ldg(p.positions + static_cast<long long>(ax) * p.T + t) : slot;
      }
      // every axis is checked, those that no pair takes too
      if (lane < p.num_axes) {
        const int x = p.positions ? __ldg(p.positions + static_cast<long long>(lane) * p.T + t) : slot;
        bad = x < 0 || x >= p.max_pos;
      }
      if (__any_sync(0xffffffffu, bad)) {
        live = false;
        if (lane == 0) flag_error(p.err_flag, VH_ERR_POS);
      } else {
#pragma unroll
        for (int j = 0; j < HALF / 32; ++j) {
          const int pair = lane + 32 * j;
          const float* cs = p.cos_sin + static_cast<long long>(pos[j]) * D + pair;
          s_cs[warp][pair] = __ldg(cs);
          s_cs[warp][HALF + pair] = __ldg(cs + HALF);
        }
        const long long lp = static_cast<long long>(row) * p.max_pages_per_seq + slot / p.P;
        const int page = p.page_table ? p.page_table[lp] : static_cast<int>(lp);
        if (page >= 0 && page < p.num_pages)
          slot_off = page * p.page_stride + (slot % p.P) * p.token_stride;
        else if (lane == 0)
          flag_error(p.err_flag, VH_ERR_PAGE);
      }
    }
    if (lane == 0) {
      s_live[warp] = live;
      s_slot[warp] = slot_off;
    }
  }
  __syncthreads();

  // ---- rotation (every lane runs each round: the norm's sum shuffles) ---------
  for (int base = 0; base < units; base += kThreads) {
    if (base > 0) load(base + tid);
    const bool valid = base + tid < units;
    const bool is_q = h < p.Hq;
    float x[8], y[8];
    {
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 fa = E::to_float2(aw[k]), fb = E::to_float2(bw[k]);
        if (ilv) {
          x[k] = fa.x;
          y[k] = fa.y;
          x[4 + k] = fb.x;
          y[4 + k] = fb.y;
        } else {
          x[2 * k] = fa.x;
          x[2 * k + 1] = fa.y;
          y[2 * k] = fb.x;
          y[2 * k + 1] = fb.y;
        }
      }
    }
    const float* nw = is_q ? p.q_norm_w : p.k_norm_w;
    if (p.q_norm_w || p.k_norm_w) {
      // the UPH neighbouring lanes of a head hold its D elements; summed in fp32
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss += x[k] * x[k] + y[k] * y[k];
#pragma unroll
      for (int off = 1; off < UPH; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if (nw) {
        const float r = rsqrtf(ss / static_cast<float>(D) + p.norm_eps);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[k] = __ldg(nw + (ilv ? 2 * (i + k) : i + k)) * (x[k] * r);
          y[k] = __ldg(nw + (ilv ? 2 * (i + k) + 1 : HALF + i + k)) * (y[k] * r);
        }
      }
    }
    if (!valid || !s_live[tk]) continue;
    float rx[8], ry[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float c = s_cs[tk][i + k], s = s_cs[tk][HALF + i + k];
      rx[k] = x[k] * c - y[k] * s;
      ry[k] = y[k] * c + x[k] * s;
    }
    // first 8 elements and partners in memory order: two runs of 8
    float o0[8], o1[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      o0[k] = ilv ? ((k & 1) ? ry[k / 2] : rx[k / 2]) : rx[k];
      o1[k] = ilv ? ((k & 1) ? ry[4 + k / 2] : rx[4 + k / 2]) : ry[k];
    }
    const int e0 = ilv ? 2 * i : i, e1 = ilv ? 2 * i + 8 : HALF + i;
    if (is_q && !p.q16) {
      float* dst = static_cast<float*>(p.q_rot) + (static_cast<long long>(t0 + tk) * p.Hq + h) * D;
      *reinterpret_cast<float4*>(dst + e0) = make_float4(o0[0], o0[1], o0[2], o0[3]);
      *reinterpret_cast<float4*>(dst + e0 + 4) = make_float4(o0[4], o0[5], o0[6], o0[7]);
      *reinterpret_cast<float4*>(dst + e1) = make_float4(o1[0], o1[1], o1[2], o1[3]);
      *reinterpret_cast<float4*>(dst + e1 + 4) = make_float4(o1[4], o1[5], o1[6], o1[7]);
    } else {
      uint16_t* dst;
      if (is_q) {
        dst = static_cast<uint16_t*>(p.q_rot) + (static_cast<long long>(t0 + tk) * p.Hq + h) * D;
      } else {
        if (s_slot[tk] < 0) continue;
        dst = p.k_cache + s_slot[tk] + (h - p.Hq) * p.head_stride;
      }
      *reinterpret_cast<uint4*>(dst + e0) =
          make_uint4(E::pack2(o0[0], o0[1]), E::pack2(o0[2], o0[3]), E::pack2(o0[4], o0[5]), E::pack2(o0[6], o0[7]));
      *reinterpret_cast<uint4*>(dst + e1) =
          make_uint4(E::pack2(o1[0], o1[1]), E::pack2(o1[2], o1[3]), E::pack2(o1[4], o1[5]), E::pack2(o1[6], o1[7]));
    }
  }

  // ---- values: 16 bytes a thread, bit for bit ---------------------------------
  const int vec = p.Hkv * (D / 8);
  for (int u = tid; u < ntok * vec; u += kThreads) {
    const int vt = u / vec, r = u - vt * vec;
    if (!s_live[vt] || s_slot[vt] < 0) continue;
    const uint4 w = ldg16(p.v_new + (t0 + vt) * p.v_stride + r * 8);
    *reinterpret_cast<uint4*>(p.v_cache + s_slot[vt] + (r / (D / 8)) * p.head_stride + (r % (D / 8)) * 8) = w;
  }
}

}  // namespace

cudaError_t launch_mrope_kv_append(const MropeParams& pp, cudaStream_t stream) {
  MropeParams p = pp;
  // One token a CTA while the tokens do not fill the GPU (latency counts), more
  // after that: the look-ups are shared by fewer barriers.
  p.tokens_per_cta = p.T <= 2048 ? 1 : 4;
  const int grid = (p.T + p.tokens_per_cta - 1) / p.tokens_per_cta;
  if (p.D == 128) {
    if (p.f16) mrope_kv_append_kernel<ElemF16, 128><<<grid, kThreads, 0, stream>>>(p);
    else mrope_kv_append_kernel<ElemBf16, 128><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (p.f16) mrope_kv_append_kernel<ElemF16, 64><<<grid, kThreads, 0, stream>>>(p);
    else mrope_kv_append_kernel<ElemBf16, 64><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace vh
