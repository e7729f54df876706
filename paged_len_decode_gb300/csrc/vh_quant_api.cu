// vh_quant_api.cu -- host side of the attention over an 8-bit cache and of its
// read-back (declared in include/vh.h): checks, launch plans, launches on the
// caller's stream.  Nothing here synchronises, allocates or reads device memory.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/vh.h"
#include "vh_plan.h"
#include "vh_quant.h"

namespace {

using vh::DeviceInfo;
using vh::aligned16;
using vh::device_info;
using vh::kMaxDevices;
using vh::valid_cache;

struct Prepared {
  std::mutex mu;
  std::atomic<bool> ok{false};
};
Prepared g_prepared[kMaxDevices];

// Kernel attributes, set on the first call on a device (a call that could not set them leaves it to the next one).
bool prepared(const DeviceInfo& dev) {
  Prepared& s = g_prepared[dev.index];
  if (s.ok.load(std::memory_order_acquire)) return true;
  std::lock_guard<std::mutex> lk(s.mu);
  if (s.ok.load(std::memory_order_relaxed)) return true;
  if (vh::prepare_quant_read(dev.smem_optin - 1024) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  s.ok.store(true, std::memory_order_release);
  return true;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? VH_OK : VH_ECUDA; }

}  // namespace

extern "C" {

int vh_quant_decode_attn(const float* q_rot, const vh_e4m3* k_cache, const vh_e4m3* v_cache, int64_t page_stride,
                         int64_t token_stride, int64_t head_stride, const float* k_scale, const float* v_scale,
                         int64_t scale_page_stride, int64_t scale_head_stride, int num_pages, const int32_t* page_table,
                         int max_pages_per_seq, const int32_t* seq_lens, const int32_t* active, int window, int sinks,
                         vh_e16* out, float sm_scale, int num_ctas, void* workspace, size_t workspace_bytes,
                         int32_t* err_flag, unsigned flags, int B, int Hq, int Hkv, int D, int page_size, void* stream) {
  if (!q_rot || !k_cache || !v_cache || !k_scale || !v_scale || !seq_lens || !active || !out ||
      (flags & ~(VH_FLAG_FP16 | VH_FLAG_PDL)) != 0 || window < 0 || sinks < 0 || num_ctas < 0 || num_ctas > 65535 ||
      !(sm_scale == sm_scale) || scale_page_stride < 1 || scale_head_stride < 1 ||
      !valid_cache(B, Hq, Hkv, D, page_size, page_stride, token_stride, head_stride, num_pages, page_table,
                   max_pages_per_seq))
    return VH_EINVAL;
  vh::QuantDecodeParams p{};
  p.memory = {k_cache, v_cache, page_stride, token_stride, head_stride, k_scale, v_scale, scale_page_stride, scale_head_stride};
  if (!aligned16(q_rot) || !aligned16(out) || !vh::aligned_quant(p.memory)) return VH_EALIGN;
  if (!workspace) return VH_EWORKSPACE;
  if (!aligned16(workspace)) return VH_EALIGN;
  const DeviceInfo* dev = device_info();
  if (!dev || !prepared(*dev)) return VH_ENODEV;
  (void)workspace_bytes;
  p.q_rot = q_rot;
  p.num_pages = num_pages;
  p.page_table = page_table;
  p.max_pages_per_seq = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.active = active;
  p.window = window > 0 ? std::min(window, vh::kNoWindow) : vh::kNoWindow;
  p.sinks = std::min(sinks, vh::kNoWindow);
  p.out = out;
  const float scale = sm_scale > 0.f ? sm_scale : 1.0f / sqrtf(static_cast<float>(D));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.err_flag = err_flag;
  p.f16 = (flags & VH_FLAG_FP16) != 0;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.G = Hq / Hkv;
  p.P = page_size;
  return status_of(vh::launch_quant_decode(p, static_cast<cudaStream_t>(stream)));
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
  if (4 * (static_cast<size_t>(B) + 1) > static_cast<size_t>(dev->smem_optin) - 1024) return VH_EINVAL;
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
  p.ctas = dev->sm_count * 4;
  return status_of(vh::launch_quant_read(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
