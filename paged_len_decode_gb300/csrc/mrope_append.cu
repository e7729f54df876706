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
// element) and by latency for a decode step's few tokens.  `warps` warps share
// a token and never meet: each looks up the token's row, slot and page itself
// and takes a share of its heads.  A lane has the same 8 pairs of every head it
// rotates (the D/16 neighbouring lanes of a head have its D elements), so their
// cos and sin, gathered pair by pair where neighbouring pairs belong to different
// axes, stay in its registers for the whole token; loads are 16 bytes, and the
// first of them and the values are under way before anything is looked up.
// What counts is bytes in flight and the length of the chain of look-ups: 20 warps
// an SM with three heads' loads a lane each measured 64 us on 16384 tokens (32 / 8
// heads, 403 MB: 6.3 TB/s, 92 % of the copy peak) and 9.6 us on 2413 with the norm;
// 24 warps with two 63.6 and 10.1 us.  In an earlier form four heads took 68 us
// where two took 66, and a CTA of 4 tokens with its angles in shared memory
// behind a barrier 82 us.  Angles gathered beside
// the row's look-up instead of after it, and weights by 16 bytes: 12.2 -> 10.1 us.
#include "vh_ragged.cuh"
#include "vh_window.h"

namespace vh {

namespace {

constexpr int kThreads = 64;  // (small CTAs: no two warps need each other)

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 10) mrope_kv_append_kernel(const __grid_constant__ MropeParams p) {
  constexpr int HALF = D / 2;
  constexpr int UPH = HALF / 8;  // lanes of a head
  constexpr int HPW = 32 / UPH;  // heads that a warp rotates at a time
  constexpr int U = 3;           // of those, in flight
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int t = unit / p.warps, part = unit - t * p.warps;
  pdl_begin();
  if (t >= p.T) return;
  const bool ilv = p.rope_interleaved != 0;
  const int i = (lane % UPH) * 8;                   // first pair
  const int e0 = ilv ? 2 * i : i, e1 = ilv ? 2 * i + 8 : HALF + i;  // the lane's two runs of 8 elements
  const int heads = p.Hq + p.Hkv, step = HPW * p.warps;
  const uint16_t* qrow = p.q + t * p.q_stride;
  const uint16_t* krow = p.k_new + t * p.k_stride;

  // q heads first, then the new k heads
  uint4 a[U], b[U];
  auto load = [&](int h0) {
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const int h = h0 + x * step;
      a[x] = b[x] = make_uint4(0u, 0u, 0u, 0u);
      if (h < heads) {
        const uint16_t* src = h < p.Hq ? qrow + h * D : krow + (h - p.Hq) * D;
        a[x] = ldg16(src + e0);
        b[x] = ldg16(src + e1);
      }
    }
  };
  // the values, 16 bytes a lane: four of them travel while the rest is looked up
  constexpr int VU = 4;
  const int nv = p.Hkv * (D / 8), v0 = part * 32 + lane, vstep = 32 * p.warps;
  const uint16_t* vrow = p.v_new + t * p.v_stride;
  uint4 v[VU];
#pragma unroll
  for (int x = 0; x < VU; ++x)
    if (v0 + x * vstep < nv) v[x] = ldg16(vrow + (v0 + x * vstep) * 8);
  const int first = part * HPW + lane / UPH;
  load(first);  // (needs nothing of what is looked up next)

  // ---- the token's angles, row, slot and page ---------------------------------
  // Given positions depend on nothing but t, so the angles are gathered while the
  // row is looked up (a position out of range reads row 0 and is dealt with below).
  float c[8], s[8];
  const uint32_t axes = static_cast<uint32_t>(p.axis[i >> 5] >> (2 * (i & 31))) & 0xFFFFu;  // of the lane's pairs
  auto gather = [&](int pos) {  // pos: lane a's is the position on axis a
    if (__all_sync(0xffffffffu, axes == (axes & 3u) * 0x5555u)) {
      const float* row_cs = p.cos_sin + static_cast<long long>(__shfl_sync(0xffffffffu, pos, axes & 3u)) * D + i;
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(row_cs + k));
        const float4 y = __ldg(reinterpret_cast<const float4*>(row_cs + HALF + k));
        c[k] = x.x; c[k + 1] = x.y; c[k + 2] = x.z; c[k + 3] = x.w;
        s[k] = y.x; s[k + 1] = y.y; s[k + 2] = y.z; s[k + 3] = y.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float* cs = p.cos_sin + static_cast<long long>(__shfl_sync(0xffffffffu, pos, (axes >> (2 * k)) & 3u)) * D + i + k;
        c[k] = __ldg(cs);
        s[k] = __ldg(cs + HALF);
      }
    }
  };
  auto outside = [&](int pos) { return lane < p.num_axes && (pos < 0 || pos >= p.max_pos); };
  bool bad = false;
  if (p.positions) {
    const int pos = lane < p.num_axes ? __ldg(p.positions + static_cast<long long>(lane) * p.T + t) : 0;
    bad = outside(pos);  // (every axis is checked, those that no pair takes too)
    gather(bad ? 0 : pos);
  }
  RaggedRow r;
  const int row = warp_row_of_token(p.token_start, p.seq_lens, p.active, t, p.B, p.T, p.max_pages_per_seq * p.P, lane,
                                    p.err_flag, lane == 0 && part == 0, r);
  if (row < 0 || !r.ok) return;
  const int slot = r.len - (r.end - t);
  if (!p.positions) {
    bad = outside(slot);
    gather(slot < p.max_pos ? slot : 0);
  }
  const long long lp = static_cast<long long>(row) * p.max_pages_per_seq + slot / p.P;
  const int page = p.page_table ? __ldg(p.page_table + lp) : static_cast<int>(lp);
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) flag_error(p.err_flag, VH_ERR_POS);
    return;
  }
  const bool page_ok = page >= 0 && page < p.num_pages;
  if (!page_ok && lane == 0) flag_error(p.err_flag, VH_ERR_PAGE);
  const long long slot_off = static_cast<long long>(page) * p.page_stride + (slot % p.P) * p.token_stride;

  if (page_ok) {
    auto to = [&](int u) {
      return reinterpret_cast<uint4*>(p.v_cache + slot_off + (u / (D / 8)) * p.head_stride + (u % (D / 8)) * 8);
    };
#pragma unroll
    for (int x = 0; x < VU; ++x)
      if (v0 + x * vstep < nv) *to(v0 + x * vstep) = v[x];
    for (int u = v0 + VU * vstep; u < nv; u += vstep) *to(u) = ldg16(vrow + u * 8);
  }

  // ---- rotation (every lane runs each round: the norm's sum shuffles) ---------
  for (int h0 = first; h0 - lane / UPH < heads; h0 += U * step) {
    if (h0 != first) load(h0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * step;
      const bool is_q = h < p.Hq;
      float x[8], y[8];
      const uint32_t aw[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, bw[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
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
      if (p.q_norm_w || p.k_norm_w) {
        // summed in fp32 over the lanes of the head
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) ss += x[k] * x[k] + y[k] * y[k];
#pragma unroll
        for (int off = 1; off < UPH; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float* nw = is_q ? p.q_norm_w : p.k_norm_w;
        if (nw) {
          const float rs = rsqrtf(ss / static_cast<float>(D) + p.norm_eps);
          // the weights of the lane's two runs of 8 elements
          float wt[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 v4 = __ldg(reinterpret_cast<const float4*>(nw + (k < 2 ? e0 + 4 * k : e1 + 4 * k - 8)));
            wt[4 * k] = v4.x; wt[4 * k + 1] = v4.y; wt[4 * k + 2] = v4.z; wt[4 * k + 3] = v4.w;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[k] = (ilv ? wt[2 * k] : wt[k]) * (x[k] * rs);
            y[k] = (ilv ? wt[2 * k + 1] : wt[8 + k]) * (y[k] * rs);
          }
        }
      }
      if (h >= heads || !(is_q || page_ok)) continue;
      float o0[8], o1[8];  // the two runs of 8 elements
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float rx = x[k] * c[k] - y[k] * s[k], ry = y[k] * c[k] + x[k] * s[k];
        if (ilv) {
          if (k < 4) {
            o0[2 * k] = rx;
            o0[2 * k + 1] = ry;
          } else {
            o1[2 * k - 8] = rx;
            o1[2 * k - 7] = ry;
          }
        } else {
          o0[k] = rx;
          o1[k] = ry;
        }
      }
      if (is_q && !p.q16) {
        float* dst = static_cast<float*>(p.q_rot) + (static_cast<long long>(t) * p.Hq + h) * D;
        *reinterpret_cast<float4*>(dst + e0) = make_float4(o0[0], o0[1], o0[2], o0[3]);
        *reinterpret_cast<float4*>(dst + e0 + 4) = make_float4(o0[4], o0[5], o0[6], o0[7]);
        *reinterpret_cast<float4*>(dst + e1) = make_float4(o1[0], o1[1], o1[2], o1[3]);
        *reinterpret_cast<float4*>(dst + e1 + 4) = make_float4(o1[4], o1[5], o1[6], o1[7]);
      } else {
        uint16_t* dst = is_q ? static_cast<uint16_t*>(p.q_rot) + (static_cast<long long>(t) * p.Hq + h) * D
                             : p.k_cache + slot_off + (h - p.Hq) * p.head_stride;
        *reinterpret_cast<uint4*>(dst + e0) =
            make_uint4(E::pack2(o0[0], o0[1]), E::pack2(o0[2], o0[3]), E::pack2(o0[4], o0[5]), E::pack2(o0[6], o0[7]));
        *reinterpret_cast<uint4*>(dst + e1) =
            make_uint4(E::pack2(o1[0], o1[1]), E::pack2(o1[2], o1[3]), E::pack2(o1[4], o1[5]), E::pack2(o1[6], o1[7]));
      }
    }
  }
}

}  // namespace

cudaError_t launch_mrope_kv_append(const MropeParams& pp, cudaStream_t stream) {
  MropeParams p = pp;
  // A token's heads over several warps while the tokens do not fill the GPU.  16 / 8
  // heads of 128 with the norm, 8, 2 and 1 warps a token: 1 token 3.3, 3.7 and 4.9 us,
  // 128 4.0, 3.9 and 5.1, 512 7.0, 4.4 and 5.3, 1216 11.3, 5.6 and 6.4; without it 64
  // tokens 3.1, 3.1 and 3.8, 2000 14.7, 8.0 and 8.0.
  p.warps = p.T <= 128 ? 8 : (p.T <= 1216 ? 2 : 1);
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(p.T) * p.warps + kThreads / 32 - 1) / (kThreads / 32)));
  return launch_dependent(p.D == 128 ? (p.f16 ? mrope_kv_append_kernel<ElemF16, 128> : mrope_kv_append_kernel<ElemBf16, 128>)
                                     : (p.f16 ? mrope_kv_append_kernel<ElemF16, 64> : mrope_kv_append_kernel<ElemBf16, 64>),
                          p, grid, kThreads, 0, stream);
}

}  // namespace vh
