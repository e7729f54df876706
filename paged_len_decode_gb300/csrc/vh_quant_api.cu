// vh_quant_api.cu -- host side of the attention over an 8-bit cache and of its
// read-back (declared in include/vh.h): checks, launch plans, launches on the
// caller's stream.  Nothing here synchronises, allocates or reads device memory.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <unordered_map>

#include "../../include/vh.h"
#include "vh_plan.h"
#include "vh_quant.h"

namespace {

using vh::DeviceInfo;
using vh::align_up;
using vh::aligned16;
using vh::device_info;
using vh::kMaxDevices;
using vh::valid_cache;

vh::Prepared g_prepared[kMaxDevices];

bool prepared(const DeviceInfo& dev) {
  return g_prepared[dev.index].once([&](vh::Prepared&) {
    return vh::prepare_quant_read(dev.smem_optin - 1024) == cudaSuccess && vh::prepare_quant_decode(dev.smem_optin) == cudaSuccess;
  });
}

constexpr int kMaxHc = 8;
constexpr int kMaxStages = 8;
// Bytes of stages of a CTA, so that two share an SM.  (16 rows of up to 32768 tokens: 133 us with
// 64 KB, 112 with 84, 110 with 100, and 136 with 140, which one CTA an SM leaves room for.)
constexpr int kStageTarget = 102400;

// Shared-memory plan and automatic CTA count of the decode kernel.
struct DecodePlan {
  bool ok;
  int Hc, groups, stages, stage_bytes, scale_bytes, q_off, cum_off, len_off, bar_off, smem_bytes, auto_n;
};

// kv heads per CTA: the largest divisor of Hkv with tiles of 16 KB at most (64 rows of 4000, 40 / 5 heads of
// 128: five a CTA 76 us, one a CTA 67); fewer if two stages do not fit beside the rows.
bool layout_decode(vh::QuantDecodeParams& p, const DeviceInfo& dev) {
  p.G = p.Hq / p.Hkv;
  for (int hc = std::min(p.Hkv, std::min(512 / p.D, kMaxHc)); hc >= 1; --hc) {
    if (p.Hkv % hc != 0) continue;
    p.Hc = hc;
    p.groups = p.Hkv / hc;
    p.scale_bytes = 2 * static_cast<int>(align_up(static_cast<size_t>(hc) * 32, 128));
    p.stage_bytes = static_cast<int>(align_up(2 * 16 * static_cast<size_t>(hc) * p.D + 2 * static_cast<size_t>(p.scale_bytes), 1024));
    const size_t q = static_cast<size_t>(hc) * p.G * p.D * 4;
    const size_t cum = align_up(4 * (static_cast<size_t>(p.B) + 1), 16), len = align_up(4 * static_cast<size_t>(p.B), 16);
    const size_t fixed = 1024 + q + cum + len + 8 * (2 * kMaxStages + 2 + kMaxHc) + 48 * 4 + 128;
    const size_t budget = static_cast<size_t>(dev.smem_optin);
    if (fixed + 2 * static_cast<size_t>(p.stage_bytes) > budget) continue;
    p.stages = static_cast<int>(std::min<size_t>((budget - fixed) / p.stage_bytes,
                                                 std::max(2, std::min(kMaxStages, kStageTarget / p.stage_bytes))));
    size_t off = static_cast<size_t>(p.stages) * p.stage_bytes;
    p.q_off = static_cast<int>(off);
    p.cum_off = static_cast<int>(off += q);
    p.len_off = static_cast<int>(off += cum);
    p.bar_off = static_cast<int>(off += len);
    off += 8 * (2 * static_cast<size_t>(p.stages) + 2 + kMaxHc) + 48 * 4;
    p.smem_bytes = static_cast<int>(align_up(off, 128) + 1024);  // + up to 1024 to align the base
    return true;
  }
  return false;
}

std::mutex g_mu;
std::unordered_map<uint64_t, DecodePlan> g_plans;

// Plan of p's shape, computed once (the occupancy query costs more host time than a launch).
// The CTA count is at most vh_decode_fused's for the same shape, so that one workspace serves
// all attentions of a decode step.
bool plan_decode(vh::QuantDecodeParams& p, const DeviceInfo& dev, int* auto_n) {
  uint64_t key = static_cast<uint64_t>(dev.index);
  key = (key << 16) | static_cast<uint64_t>(p.B);
  key = (key << 17) | static_cast<uint64_t>(p.Hkv);
  key = (key << 4) | static_cast<uint64_t>(p.Hq / p.Hkv);
  key = (key << 2) | static_cast<uint64_t>(p.D / 64);
  key = (key << 11) | static_cast<uint64_t>(p.P);
  key = (key << 1) | (p.f16 ? 1u : 0u);
  DecodePlan c{};
  {
    std::lock_guard<std::mutex> lk(g_mu);
    auto it = g_plans.find(key);
    if (it != g_plans.end()) c = it->second;
  }
  if (c.auto_n == 0) {
    vh::QuantDecodeParams q = p;
    vh::AttnParams f{};
    f.B = p.B;
    f.Hq = p.Hq;
    f.Hkv = p.Hkv;
    f.D = p.D;
    f.P = p.P;
    f.f16 = p.f16;
    int fused_n = 0, per_sm = 0;
    c.ok = layout_decode(q, dev) && vh::plan_attn(f, dev, true, &fused_n);
    c.auto_n = -1;
    if (c.ok) {
      if (vh::quant_decode_occupancy(q, &per_sm) != cudaSuccess || per_sm < 1) {
        cudaGetLastError();
        return false;  // not remembered: the next call asks again
      }
      c = DecodePlan{true,    q.Hc,      q.groups,  q.stages,  q.stage_bytes, q.scale_bytes, q.q_off,
                     q.cum_off, q.len_off, q.bar_off, q.smem_bytes, 0};
      c.auto_n = std::max(1, std::min(fused_n, dev.sm_count * per_sm / q.groups));
    }
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_plans.size() >= 4096) g_plans.clear();
    g_plans[key] = c;
  }
  if (!c.ok) return false;
  p.G = p.Hq / p.Hkv;
  p.Hc = c.Hc;
  p.groups = c.groups;
  p.stages = c.stages;
  p.stage_bytes = c.stage_bytes;
  p.scale_bytes = c.scale_bytes;
  p.q_off = c.q_off;
  p.cum_off = c.cum_off;
  p.len_off = c.len_off;
  p.bar_off = c.bar_off;
  p.smem_bytes = c.smem_bytes;
  *auto_n = c.auto_n;
  return true;
}

// CTAs that the kernel can use at most: with every row as long as the window, the sinks and
// its pages allow, it takes this many (see share_of_cta).
int useful_ctas(const vh::QuantDecodeParams& p) {
  const long long all = (static_cast<long long>(p.max_pages_per_seq) * p.P + 15) / 16;
  const long long row = std::min(all, (p.sinks + 15LL) / 16 + (p.window + 15LL) / 16 + 1);
  const long long q = std::max(1L, static_cast<long>(std::sqrt(static_cast<float>(row) * (vh::kQuantPiece * p.G)) + 0.5f) - 1);
  return static_cast<int>(std::min<long long>(65535, (p.B * row + q - 1) / q));
}

// Tensor maps of the cache and its scales.
bool encode_maps(vh::QuantDecodeParams& p, const vh::QuantMemory& m) {
  auto dim = [](long long x) { return static_cast<cuuint64_t>(x); };
  const cuuint32_t tokens = p.P == 8 ? 8 : 16, heads = static_cast<cuuint32_t>(p.Hc);
  const cuuint64_t dims[4] = {dim(p.D), dim(p.P), dim(p.Hkv), dim(p.num_pages)};
  const cuuint64_t strides[3] = {dim(m.token_stride), dim(m.head_stride), dim(m.page_stride)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(p.D), tokens, heads, 1};
  const CUtensorMapSwizzle turn = p.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  const cuuint64_t s_dims[3] = {dim(p.P), dim(p.Hkv), dim(p.num_pages)};
  const cuuint64_t s_strides[2] = {dim(4 * m.scale_head), dim(4 * m.scale_page)};
  const cuuint32_t s_box[3] = {tokens, heads, 1};
  auto values = [&](CUtensorMap* t, const void* base) {
    return vh::encode_tiled(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 4, dims, strides, box, turn);
  };
  auto scales = [&](CUtensorMap* t, const void* base) {
    return vh::encode_tiled(t, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, base, 3, s_dims, s_strides, s_box, CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  return values(&p.tmap_k, m.k) && values(&p.tmap_v, m.v) && scales(&p.tmap_ks, m.k_scale) && scales(&p.tmap_vs, m.v_scale);
}

int status_of(cudaError_t e) { return e == cudaSuccess ? VH_OK : VH_ECUDA; }

}  // namespace

extern "C" {

int vh_quant_decode_attn(const float* q_rot, const vh_e4m3* k_cache, const vh_e4m3* v_cache, int64_t page_stride,
                         int64_t token_stride, int64_t head_stride, const float* k_scale, const float* v_scale,
                         int64_t scale_page_stride, int64_t scale_head_stride, int num_pages, const int32_t* page_table,
                         int max_pages_per_seq, const int32_t* seq_lens, const int32_t* active, int window, int sinks,
                         vh_e16* out, float sm_scale, int num_ctas, void* workspace, size_t workspace_bytes,
                         int32_t* err_flag, unsigned flags, int B, int Hq, int Hkv, int D, int page_size, void* stream) try {
  if (!q_rot || !k_cache || !v_cache || !k_scale || !v_scale || !seq_lens || !active || !out ||
      (flags & ~(VH_FLAG_FP16 | VH_FLAG_PDL)) != 0 || window < 0 || sinks < 0 || num_ctas < 0 || num_ctas > 65535 ||
      !(sm_scale == sm_scale) || scale_page_stride < 1 || scale_head_stride < 1 ||
      !valid_cache(B, Hq, Hkv, D, page_size, page_stride, token_stride, head_stride, num_pages, page_table,
                   max_pages_per_seq))
    return VH_EINVAL;
  const vh::QuantMemory m = {k_cache, v_cache, page_stride, token_stride, head_stride, k_scale, v_scale, scale_page_stride, scale_head_stride};
  if (!aligned16(q_rot) || !aligned16(out) || !vh::aligned_quant(m)) return VH_EALIGN;
  if (!workspace) return VH_EWORKSPACE;
  if (!aligned16(workspace)) return VH_EALIGN;
  const DeviceInfo* dev = device_info();
  if (!dev || !prepared(*dev)) return VH_ENODEV;
  vh::QuantDecodeParams p{};
  p.f16 = (flags & VH_FLAG_FP16) != 0;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.P = page_size;
  int auto_n = 0;
  if (!plan_decode(p, *dev, &auto_n)) return VH_EINVAL;
  p.num_pages = num_pages;
  p.page_table = page_table;
  p.max_pages_per_seq = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.active = active;
  p.window = window > 0 ? std::min(window, vh::kNoWindow) : vh::kNoWindow;
  p.sinks = std::min(sinks, vh::kNoWindow);
  p.N = num_ctas > 0 ? num_ctas : std::min(auto_n, useful_ctas(p));
  const vh::WsLayout w = vh::ws_layout(B, Hq, Hkv, D, p.N);
  if (workspace_bytes < w.total) return VH_EWORKSPACE;
  if (!encode_maps(p, m)) return VH_EINVAL;
  p.q_rot = q_rot;
  p.out = out;
  const float scale = sm_scale > 0.f ? sm_scale : 1.0f / sqrtf(static_cast<float>(D));
  p.scale_log2 = scale * 1.4426950408889634f;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.counters = reinterpret_cast<int*>(ws + w.counters);
  p.part_lse = reinterpret_cast<float*>(ws + w.lse);
  p.part_o = reinterpret_cast<float*>(ws + w.o);
  p.err_flag = err_flag;
  p.early = (flags & VH_FLAG_PDL) != 0;
  return status_of(vh::launch_quant_decode(p, static_cast<cudaStream_t>(stream)));
} catch (...) {  // (a plan that the host has no memory for; no exception leaves a C function)
  return VH_ECUDA;
}

int vh_quant_kv_read(const vh_e4m3* k_cache, const vh_e4m3* v_cache, int64_t page_stride, int64_t token_stride,
                     int64_t head_stride, const float* k_scale, const float* v_scale, int64_t scale_page_stride,
                     int64_t scale_head_stride, int num_pages, const int32_t* page_table, int max_pages_per_seq,
                     const int32_t* seq_lens, const int32_t* active, const int32_t* first_slot, int sinks, vh_e16* k_out,
                     vh_e16* v_out, int64_t out_page_stride, int64_t out_token_stride, int64_t out_head_stride,
                     int out_num_pages, const int32_t* out_page_table, int out_max_pages_per_seq, int32_t* err_flag,
                     unsigned flags, int B, int Hkv, int D, int page_size, int out_page_size, void* stream) {
  if (!k_cache || !v_cache || !k_scale || !v_scale || !seq_lens || !active || !k_out || !v_out ||
      (flags & ~VH_FLAG_FP16) != 0 || sinks < 0 || scale_page_stride < 1 || scale_head_stride < 1 ||
      !valid_cache(B, Hkv, Hkv, D, page_size, page_stride, token_stride, head_stride, num_pages, page_table, max_pages_per_seq) ||
      !valid_cache(B, Hkv, Hkv, D, out_page_size, out_page_stride, out_token_stride, out_head_stride, out_num_pages,
                   out_page_table, out_max_pages_per_seq))
    return VH_EINVAL;
  vh::QuantReadParams p{};
  p.memory = {k_cache, v_cache, page_stride, token_stride, head_stride, k_scale, v_scale, scale_page_stride, scale_head_stride};
  if (!vh::aligned_quant(p.memory) || !aligned16(k_out) || !aligned16(v_out) || out_page_stride % 8 != 0 ||
      out_token_stride % 8 != 0 || out_head_stride % 8 != 0)
    return VH_EALIGN;
  const DeviceInfo* dev = device_info();
  if (!dev || !prepared(*dev)) return VH_ENODEV;
  if (vh::quant_read_smem(B) > static_cast<size_t>(dev->smem_optin) - 1024) return VH_EINVAL;
  p.num_pages = num_pages;
  p.page_table = page_table;
  p.max_pages_per_seq = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.active = active;
  p.first_slot = first_slot;
  p.sinks = std::min(sinks, vh::kNoWindow);
  p.k_out = k_out;
  p.v_out = v_out;
  p.out_page = out_page_stride;
  p.out_token = out_token_stride;
  p.out_head = out_head_stride;
  p.out_pages = out_num_pages;
  p.out_table = out_page_table;
  p.out_per_row = out_max_pages_per_seq;
  p.err_flag = err_flag;
  p.f16 = (flags & VH_FLAG_FP16) != 0;
  p.B = B;
  p.Hkv = Hkv;
  p.D = D;
  p.P = page_size;
  p.out_P = out_page_size;
  p.hkv_inverse = Hkv == 1 ? 0u : static_cast<uint32_t>(((1ULL << 32) + Hkv - 1) / Hkv);
  return status_of(vh::launch_quant_read(p, dev->sm_count, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
