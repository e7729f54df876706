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
// heads, 403 MB: 6.3 TB/s, 92 % of the copy peak) and 9.6 us on 1981 with the norm;
// 24 warps with two 63.6 and 10.1 us.  In an earlier form four heads took 68 us
// where two took 66, and a CTA of 4 tokens with its angles in shared memory
// behind a barrier 82 us.  Angles gathered beside
// the row's look-up instead of after it, and weights by 16 bytes: 12.2 -> 10.1 us.
//
// Into a cache of 8 bits (Q8) go e4m3_rne(x / s) and the scale s = max |x| / 448 of the head
// (at least 2^-126), each from the fp32 values before any other rounding: the lanes of a head
// agree on its largest value, and write 8 bytes a run instead of 16.  That takes more
// instructions than bytes it saves: 16384 tokens (32 / 8 heads, 370 MB) 66.5 us = 5.6 TB/s, an
// instruction issued in 59 % of the cycles; 71 with the q heads' largest values found too and
// 78 with a comparison for every element.
#include "vh_e4m3.cuh"
#include "vh_ragged.cuh"
#include "vh_window.h"

namespace vh {

namespace {

constexpr int kThreads = 64;  // (small CTAs: no two warps need each other)

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// The largest of top, |x| and |y|, NaN if one of them is.
__device__ __forceinline__ float larger(float top, float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(top), "f"(fabsf(x)), "f"(fabsf(y)));
  return r;
}
// The same of pairs of 16-bit elements, by their bits without the sign (a NaN's are above an infinity's).
__device__ __forceinline__ uint32_t larger_bits(uint32_t top, uint32_t w) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(top), "r"(w & 0x7fff7fffu));
  return r;
}
// The scale of a head whose largest value is `top`.  (Divisions that round to nearest: a value
// that another program quantises by the same rule has the same bits.)
__device__ __forceinline__ float scale_of(float top) {
  return top < __int_as_float(0x7f800000) ? fmaxf(__fdiv_rn(top, kE4m3Max), kScaleMin) : __int_as_float(0x7fffffff);
}
__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = pack_e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Form of the kernel: into a cache of 16 bits, or of 8 for few tokens or many.
enum { k16, k8Few, k8Many };

template <typename E, int D, int FORM>
__global__ void __launch_bounds__(kThreads, FORM == k16 ? 10 : (FORM == k8Few ? 8 : 14)) mrope_kv_append_kernel(const __grid_constant__ MropeParams p) {
  constexpr int HALF = D / 2;
  constexpr int UPH = HALF / 8;  // lanes of a head
  constexpr int HPW = 32 / UPH;  // heads that a warp rotates at a time
  constexpr int U = FORM == k8Many ? 2 : 3;  // of those, in flight
  constexpr bool Q8 = FORM != k16;
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

  [[maybe_unused]] const long long scale_at = static_cast<long long>(page) * p.scale_page + slot % p.P;
  if constexpr (Q8) {
    // 8 elements a lane, D / 8 neighbouring lanes a head (every lane runs each round)
    auto put = [&](int u, const uint4& w) {
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
      uint32_t top2 = larger_bits(larger_bits(larger_bits(ws[0] & 0x7fff7fffu, ws[1]), ws[2]), ws[3]);
#pragma unroll
      for (int off = 1; off < D / 8; off <<= 1) top2 = larger_bits(top2, __shfl_xor_sync(0xffffffffu, top2, off));
      const float scale = scale_of(E::to_float(static_cast<uint16_t>(max(top2 & 0xffffu, top2 >> 16))));
      float x[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = E::to_float2(ws[k]);
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
      if (u >= nv || !page_ok) return;
      const int h = u / (D / 8), c = u % (D / 8);
      *reinterpret_cast<uint2*>(p.v8 + slot_off + h * p.head_stride + c * 8) = e4m3x8(x, __frcp_rn(scale));
      if (c == 0) p.v_scale[scale_at + h * p.scale_head] = scale;
    };
#pragma unroll
    for (int x = 0; x < VU; ++x)
      if (part * 32 + x * vstep < nv) put(v0 + x * vstep, v0 + x * vstep < nv ? v[x] : make_uint4(0u, 0u, 0u, 0u));
    for (int u = v0 + VU * vstep; u - lane < nv; u += vstep) put(u, u < nv ? ldg16(vrow + u * 8) : make_uint4(0u, 0u, 0u, 0u));
  } else if (page_ok) {
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
      if (!Q8 && (h >= heads || !(is_q || page_ok))) continue;
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
      if constexpr (Q8) {
        const bool is_k = !is_q && h < heads;
        if (__any_sync(0xffffffffu, is_k)) {  // (a round of q heads alone skips this)
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) top = larger(top, o0[k], o1[k]);
#pragma unroll
          for (int off = 1; off < UPH; off <<= 1) top = larger(top, top, __shfl_xor_sync(0xffffffffu, top, off));
          const float scale = scale_of(top), inv = __frcp_rn(scale);
          if (is_k && page_ok) {
            uint8_t* dst = p.k8 + slot_off + (h - p.Hq) * p.head_stride;
            *reinterpret_cast<uint2*>(dst + e0) = e4m3x8(o0, inv);
            *reinterpret_cast<uint2*>(dst + e1) = e4m3x8(o1, inv);
            if (lane % UPH == 0) p.k_scale[scale_at + (h - p.Hq) * p.scale_head] = scale;
          }
        }
        if (!is_q) continue;
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

cudaError_t launch_mrope_kv_append(const MropeParams& pp, int sm_count, cudaStream_t stream) {
  MropeParams p = pp;
  // A token's heads over several warps while the tokens do not fill the GPU.  16 / 8
  // heads of 128 with the norm, 8, 2 and 1 warps a token: 1 token 3.3, 3.7 and 4.9 us,
  // 128 4.0, 3.9 and 5.1, 512 7.0, 4.4 and 5.3, 1216 11.3, 5.6 and 6.4; without it 64
  // tokens 3.1, 3.1 and 3.8, 2000 14.7, 8.0 and 8.0.
  p.warps = p.T <= 128 ? 8 : (p.T <= 1216 ? 2 : 1);
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(p.T) * p.warps + kThreads / 32 - 1) / (kThreads / 32)));
  // Into a cache of 8 bits: 16 warps an SM with three heads' loads a lane while they hold all tokens,
  // 28 with two otherwise.  Prompts (16 / 8 heads, with the norm), 16 warps and 28: 1981 tokens 9.6 and
  // 10.7 us; four inputs in turn, 1216 6.2 and 10.3, 1981 11.2 and 12.5, 2432 (16 warps on each of 152 SMs)
  // 12.4 and 16.6, 2700 18.1 and 16.8, 4000 20.4 and 18.0; 32 / 8 heads without it 2432 14.5 and 17.8, 2700 20.8
  // and 18.2; 16384 tokens 76.1 and 66.7 (70.5 with 20 warps).
  using Kernel = void (*)(MropeParams);
  const int form = !p.k8 ? k16 : (p.T <= 16 * sm_count ? k8Few : k8Many);
  const Kernel kernels[4][3] = {
      {mrope_kv_append_kernel<ElemBf16, 64, k16>, mrope_kv_append_kernel<ElemBf16, 64, k8Few>, mrope_kv_append_kernel<ElemBf16, 64, k8Many>},
      {mrope_kv_append_kernel<ElemF16, 64, k16>, mrope_kv_append_kernel<ElemF16, 64, k8Few>, mrope_kv_append_kernel<ElemF16, 64, k8Many>},
      {mrope_kv_append_kernel<ElemBf16, 128, k16>, mrope_kv_append_kernel<ElemBf16, 128, k8Few>, mrope_kv_append_kernel<ElemBf16, 128, k8Many>},
      {mrope_kv_append_kernel<ElemF16, 128, k16>, mrope_kv_append_kernel<ElemF16, 128, k8Few>, mrope_kv_append_kernel<ElemF16, 128, k8Many>}};
  return launch_dependent(kernels[(p.D == 128 ? 2 : 0) + (p.f16 ? 1 : 0)][form], p, grid, kThreads, 0, stream);
}

}  // namespace vh
