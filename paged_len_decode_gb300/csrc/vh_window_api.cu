// vh_window_api.cu -- host side of the ragged-batch append, the windowed
// decode attention and the prompt attention (declared in include/vh.h): checks
// of scalars and alignment, launch plans, launches on the caller's stream.
// Nothing here synchronises, allocates or reads device memory.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <unordered_map>

#include <cudaTypedefs.h>  // PFN_cuTensorMapEncodeTiled

#include "../../include/vh.h"
#include "vh_plan.h"
#include "vh_window.h"

namespace {

using vh::DeviceInfo;
using vh::aligned16;
using vh::device_info;
using vh::too_many_tiles;
using vh::valid_paging;
using vh::valid_shape;
using vh::valid_table;
using vh::kMaxDevices;

constexpr int kMaxHc = 8;
constexpr int kMaxStages = 8;
constexpr int kStageTarget = 65536;  // bytes in flight of a CTA, two CTAs on an SM

// Kernel attributes of this file's kernels, set on the first call on a device
// (a call that could not set them leaves it to the next one).
struct Prepared {
  std::mutex mu;
  std::atomic<bool> ok{false};
  int clusters[5] = {};  // clusters of 2^x CTAs of the prompt kernel that run at a time
};
Prepared g_prepared[kMaxDevices];

bool prepared(const DeviceInfo& dev) {
  Prepared& s = g_prepared[dev.index];
  if (s.ok.load(std::memory_order_acquire)) return true;
  std::lock_guard<std::mutex> lk(s.mu);
  if (s.ok.load(std::memory_order_relaxed)) return true;
  if (vh::prepare_window_decode(dev.smem_optin) != cudaSuccess || vh::prepare_window_prompt(s.clusters) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  s.ok.store(true, std::memory_order_release);
  return true;
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Shared-memory plan and automatic CTA count of the windowed decode kernel.
struct DecodePlan {
  bool ok;
  int Hc, groups, stages, stage_bytes, q_off, cum_off, len_off, bar_off, smem_bytes, auto_n;
};

bool layout_decode(vh::WindowDecodeParams& p, const DeviceInfo& dev) {
  p.G = p.Hq / p.Hkv;
  // kv heads per CTA: the largest divisor of Hkv with tiles of at most 32 KB
  // (and at most 8 one-head boxes a half tile, the producer warp's lanes), so
  // that two CTAs share an SM; fewer if two stages do not fit beside the rows
  int hc = std::min(p.Hkv, std::min(512 / p.D, kMaxHc));
  for (;; --hc) {
    if (hc < 1) return false;
    if (p.Hkv % hc != 0) continue;
    p.Hc = hc;
    p.groups = p.Hkv / hc;
    p.stage_bytes = 2 * 16 * hc * p.D * 2;
    const size_t rows = align_up(4 * (static_cast<size_t>(p.B) + 1), 16) + align_up(4 * static_cast<size_t>(p.B), 16);
    const size_t fixed = 1024 + static_cast<size_t>(hc) * p.G * p.D * 4 + rows + 8 * (2 * kMaxStages + 2 + kMaxHc) + 48 * 4 + 128;
    const size_t budget = static_cast<size_t>(dev.smem_optin);
    if (fixed + 2 * static_cast<size_t>(p.stage_bytes) > budget) continue;
    p.stages = static_cast<int>(std::min<size_t>((budget - fixed) / p.stage_bytes,
                                                 std::max(2, std::min(kMaxStages, kStageTarget / p.stage_bytes))));
    size_t off = static_cast<size_t>(p.stages) * p.stage_bytes;
    p.q_off = static_cast<int>(off);
    off += static_cast<size_t>(hc) * p.G * p.D * 4;
    p.cum_off = static_cast<int>(off);
    off += align_up(4 * (static_cast<size_t>(p.B) + 1), 16);
    p.len_off = static_cast<int>(off);
    off += align_up(4 * static_cast<size_t>(p.B), 16);
    p.bar_off = static_cast<int>(off);
    off += 8 * (2 * static_cast<size_t>(p.stages) + 2 + kMaxHc) + 48 * 4;
    p.smem_bytes = static_cast<int>(align_up(off, 128) + 1024);  // + up to 1024 to align the base
    return true;
  }
}

std::mutex g_mu;
std::unordered_map<uint64_t, DecodePlan> g_decode_plans;

// Plan of p's shape, computed once (the occupancy query costs more host time
// than a launch).  The CTA count is at most vh_decode_fused's for the same
// shape, so that one workspace serves both.
bool plan_decode(vh::WindowDecodeParams& p, const DeviceInfo& dev, int* auto_n) {
  uint64_t key = static_cast<uint64_t>(dev.index);
  key = (key << 16) | static_cast<uint64_t>(p.B);
  key = (key << 11) | static_cast<uint64_t>(p.Hkv);
  key = (key << 4) | static_cast<uint64_t>(p.Hq / p.Hkv);
  key = (key << 2) | static_cast<uint64_t>(p.D / 64);
  key = (key << 11) | static_cast<uint64_t>(p.P);
  key = (key << 1) | (p.f16 ? 1u : 0u);
  DecodePlan c{};
  {
    std::lock_guard<std::mutex> lk(g_mu);
    auto it = g_decode_plans.find(key);
    if (it != g_decode_plans.end()) c = it->second;
  }
  if (c.auto_n == 0 && !c.ok) {
    vh::WindowDecodeParams q = p;
    vh::AttnParams f{};
    f.B = p.B;
    f.Hq = p.Hq;
    f.Hkv = p.Hkv;
    f.D = p.D;
    f.P = p.P;
    f.f16 = p.f16;
    int fused_n = 0, per_sm = 0;
    c.ok = layout_decode(q, dev) && vh::plan_attn(f, dev, true, &fused_n);
    if (c.ok) {
      if (vh::window_decode_occupancy(q, &per_sm) != cudaSuccess || per_sm < 1) {
        cudaGetLastError();
        return false;  // not remembered: the next call asks again
      }
      c = DecodePlan{true,      q.Hc,      q.groups,  q.stages,   q.stage_bytes, q.q_off,
                     q.cum_off, q.len_off, q.bar_off, q.smem_bytes, 0};
      c.auto_n = std::max(1, std::min(fused_n, dev.sm_count * per_sm / q.groups));
    } else {
      c.auto_n = -1;
    }
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_decode_plans.size() >= 4096) g_decode_plans.clear();
    g_decode_plans[key] = c;
  }
  if (!c.ok) return false;
  p.G = p.Hq / p.Hkv;
  p.Hc = c.Hc;
  p.groups = c.groups;
  p.stages = c.stages;
  p.stage_bytes = c.stage_bytes;
  p.q_off = c.q_off;
  p.cum_off = c.cum_off;
  p.len_off = c.len_off;
  p.bar_off = c.bar_off;
  p.smem_bytes = c.smem_bytes;
  *auto_n = c.auto_n;
  return true;
}

// CTAs that the kernel can use at most: with every row as long as the window, the
// sinks and its pages allow, it takes this many (see the kernel's rule for q).
int useful_ctas(const vh::WindowDecodeParams& p, int max_pages_per_seq) {
  const long long all = (static_cast<long long>(max_pages_per_seq) * p.P + 15) / 16;
  const long long row = std::min(all, (p.sinks + 15LL) / 16 + (p.window + 15LL) / 16 + 1);
  const long long q = std::max(1L, static_cast<long>(std::sqrt(static_cast<float>(row) * (0.05f * p.G)) + 0.5f) - 1);
  return static_cast<int>(std::min<long long>(65535, (p.B * row + q - 1) / q));
}

// Scalars that every call of this file checks alike.
bool valid_cache(int B, int Hq, int Hkv, int D, int P, int64_t page_stride, int64_t token_stride, int64_t head_stride,
                 int num_pages, const int32_t* page_table, int max_pages_per_seq) {
  return valid_shape(B, Hq, Hkv, D, P) && num_pages >= 1 && page_stride >= 1 && token_stride >= 1 &&
         head_stride >= 1 && valid_paging(P, max_pages_per_seq) && !too_many_tiles(B, max_pages_per_seq, P) &&
         valid_table(page_table, B, max_pages_per_seq, num_pages);
}

bool aligned_cache(const void* k, const void* v, int64_t page_stride, int64_t token_stride, int64_t head_stride) {
  return aligned16(k) && aligned16(v) && page_stride % 8 == 0 && token_stride % 8 == 0 && head_stride % 8 == 0;
}

// The driver's tensor-map encoder, looked up once through the runtime.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    cudaGetLastError();
    return nullptr;
  }();
  return fn;
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides,
                    box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor maps of the prompt kernel.  A K or V box is a run of tokens that
// never crosses a page and divides a key tile of 128: all 128, or the largest
// power of two in the page size (a row's only page may end inside the box).
bool encode_prompt_maps(vh::PromptParams& p) {
  int box = 128;
  if (p.max_pages_per_seq > 1)
    while (p.P % box != 0) box /= 2;
  p.box = box;
  p.shift_box = __builtin_ctz(box);
  auto dim = [](long long x) { return static_cast<cuuint64_t>(x); };
  {
    const cuuint64_t dims[3] = {dim(p.D), dim(p.Hq), dim(p.T)}, strides[2] = {dim(2LL * p.D), dim(2LL * p.D * p.Hq)};
    const cuuint32_t b[3] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(128 / p.G)};
    if (!encode(&p.tmap_q, p.q, 3, dims, strides, b)) return false;
  }
  // token before head; if the encoder refuses strides in that order, head before token
  for (p.tm_tok_dim = 1; p.tm_tok_dim <= 2; ++p.tm_tok_dim) {
    const bool tf = p.tm_tok_dim == 1;
    const cuuint64_t dims[4] = {dim(p.D), dim(tf ? p.P : p.Hkv), dim(tf ? p.Hkv : p.P), dim(p.num_pages)};
    const cuuint64_t strides[3] = {dim(2 * (tf ? p.token_stride : p.head_stride)),
                                   dim(2 * (tf ? p.head_stride : p.token_stride)), dim(2 * p.page_stride)};
    const cuuint32_t b[4] = {64, static_cast<cuuint32_t>(tf ? box : 1), static_cast<cuuint32_t>(tf ? 1 : box), 1};
    if (encode(&p.tmap_k, p.k_cache, 4, dims, strides, b) && encode(&p.tmap_v, p.v_cache, 4, dims, strides, b)) return true;
  }
  return false;
}

// Blocks that T tokens of B rows make, with 2^shift tokens in a block (rows fill
// their last blocks by half, say; the kernel finds the number itself).
long long likely_blocks(int T, int B, int shift) {
  return ((static_cast<long long>(T) + (1 << shift) - 1) >> shift) + (B - 1) / 2;
}

// Small blocks (128 rows, both warpgroups on them) where they fit the SMs once: a
// prompt of 1000 tokens (16 / 8 heads, 128 such blocks, window 256) takes 10.0 us
// with them and 18.9 us with blocks of 256 rows, one of 2000 tokens (256) 15.4 and 14.1.
bool small_blocks(int T, int B, int G, int Hkv, const DeviceInfo& dev) {
  return likely_blocks(T, B, 7 - __builtin_ctz(G)) * Hkv <= dev.sm_count;
}

// CTAs that share a block's keys: as many as leave every cluster running at
// once, and two key tiles each at least.  (16 tokens over 4100 keys,
// 8 kv heads: 29 us with one CTA a block, 20, 15 and 14 us with 2, 4 and 8, and
// 25 us with 16, of which half the clusters wait for the others; over 300 keys 8.4
// us with one and 9.8 with 2; 128 tokens over 4200 30, 23 and 19 us with 1, 2 and 4,
// and 33 with 8.)
int prompt_splits(const vh::PromptParams& p, const int (&clusters)[5]) {
  const long long longest = std::min<long long>(static_cast<long long>(p.max_pages_per_seq) * p.P,
                                                static_cast<long long>(p.window) + p.sinks + (1 << p.shift_block));
  const long long blocks = likely_blocks(p.T, p.B, p.shift_block);
  int x = 0;
  while (x < 4 && blocks * p.Hkv <= clusters[x + 1] && (longest + 127) / 128 >= (2LL << (x + 1))) ++x;
  return 1 << x;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? VH_OK : VH_ECUDA; }

}  // namespace

extern "C" {

int vh_mrope_kv_append(const vh_e16* q, const vh_e16* k_new, const vh_e16* v_new, int64_t q_stride, int64_t k_stride,
                       int64_t v_stride, const float* cos_sin, int max_pos, const int32_t* positions,
                       const uint8_t* pair_axis, int num_axes, const float* q_norm_w, const float* k_norm_w,
                       float norm_eps, vh_e16* k_cache, vh_e16* v_cache, int64_t page_stride, int64_t token_stride,
                       int64_t head_stride, int num_pages, const int32_t* page_table, int max_pages_per_seq,
                       const int32_t* token_start, const int32_t* seq_lens, const int32_t* active, void* q_rot,
                       int32_t* err_flag, unsigned flags, int T, int B, int Hq, int Hkv, int D, int page_size,
                       void* stream) {
  if ((flags & ~(VH_FLAG_FP16 | VH_FLAG_ROPE_INTERLEAVED | VH_FLAG_Q16)) != 0 || T < 0 || max_pos < 1 ||
      num_axes < 1 || num_axes > 4 || !(norm_eps >= 0.f) || !(norm_eps < 1e30f) ||
      !valid_cache(B, Hq, Hkv, D, page_size, page_stride, token_stride, head_stride, num_pages, page_table,
                   max_pages_per_seq) ||
      (!token_start && T != B) || q_stride < static_cast<int64_t>(Hq) * D || k_stride < static_cast<int64_t>(Hkv) * D ||
      v_stride < static_cast<int64_t>(Hkv) * D)
    return VH_EINVAL;
  vh::MropeParams p{};
  if (pair_axis)
    for (int i = 0; i < D / 2; ++i) {
      if (pair_axis[i] >= num_axes) return VH_EINVAL;
      p.axis[i >> 5] |= static_cast<unsigned long long>(pair_axis[i]) << (2 * (i & 31));
    }
  if (T == 0) return VH_OK;
  if (!q || !k_new || !v_new || !cos_sin || !k_cache || !v_cache || !seq_lens || !active || !q_rot) return VH_EINVAL;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(cos_sin) || !aligned16(q_rot) ||
      !aligned16(q_norm_w) || !aligned16(k_norm_w) || q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 ||
      !aligned_cache(k_cache, v_cache, page_stride, token_stride, head_stride))
    return VH_EALIGN;
  if (!device_info()) return VH_ENODEV;
  p.q = q;
  p.k_new = k_new;
  p.v_new = v_new;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.cos_sin = cos_sin;
  p.max_pos = max_pos;
  p.positions = positions;
  p.num_axes = num_axes;
  p.q_norm_w = q_norm_w;
  p.k_norm_w = k_norm_w;
  p.norm_eps = norm_eps;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.page_stride = page_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.num_pages = num_pages;
  p.page_table = page_table;
  p.max_pages_per_seq = max_pages_per_seq;
  p.token_start = token_start;
  p.seq_lens = seq_lens;
  p.active = active;
  p.q_rot = q_rot;
  p.q16 = (flags & VH_FLAG_Q16) != 0;
  p.rope_interleaved = (flags & VH_FLAG_ROPE_INTERLEAVED) != 0;
  p.f16 = (flags & VH_FLAG_FP16) != 0;
  p.err_flag = err_flag;
  p.T = T;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.P = page_size;
  return status_of(vh::launch_mrope_kv_append(p, static_cast<cudaStream_t>(stream)));
}

int vh_window_decode_attn(const float* q_rot, const vh_e16* k_cache, const vh_e16* v_cache, int64_t page_stride,
                          int64_t token_stride, int64_t head_stride, int num_pages, const int32_t* page_table,
                          int max_pages_per_seq, const int32_t* seq_lens, const int32_t* active, int window, int sinks,
                          vh_e16* out, float sm_scale, int num_ctas, void* workspace, size_t workspace_bytes,
                          int32_t* err_flag, unsigned flags, int B, int Hq, int Hkv, int D, int page_size,
                          void* stream) try {
  if (!q_rot || !k_cache || !v_cache || !seq_lens || !active || !out ||
      (flags & ~(VH_FLAG_FP16 | VH_FLAG_PDL)) != 0 || window < 0 || sinks < 0 || num_ctas < 0 || num_ctas > 65535 ||
      !(sm_scale == sm_scale) ||
      !valid_cache(B, Hq, Hkv, D, page_size, page_stride, token_stride, head_stride, num_pages, page_table,
                   max_pages_per_seq))
    return VH_EINVAL;
  if (!aligned16(q_rot) || !aligned16(out) || !aligned_cache(k_cache, v_cache, page_stride, token_stride, head_stride))
    return VH_EALIGN;
  if (!workspace) return VH_EWORKSPACE;
  if (!aligned16(workspace)) return VH_EALIGN;
  const DeviceInfo* dev = device_info();
  if (!dev || !prepared(*dev)) return VH_ENODEV;
  vh::WindowDecodeParams p{};
  p.f16 = (flags & VH_FLAG_FP16) != 0;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.P = page_size;
  int auto_n = 0;
  if (!plan_decode(p, *dev, &auto_n)) return VH_EINVAL;
  p.window = window > 0 ? std::min(window, vh::kNoWindow) : vh::kNoWindow;
  p.sinks = std::min(sinks, vh::kNoWindow);
  p.N = num_ctas > 0 ? num_ctas : std::min(auto_n, useful_ctas(p, max_pages_per_seq));
  const vh::WsLayout w = vh::ws_layout(B, Hq, Hkv, D, p.N);
  if (workspace_bytes < w.total) return VH_EWORKSPACE;
  // the tensor maps are those of the other attention calls
  vh::AttnParams a{};
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.page_stride = page_stride;
  a.token_stride = token_stride;
  a.head_stride = head_stride;
  a.num_pages = num_pages;
  a.Hkv = Hkv;
  a.Hc = p.Hc;
  a.D = D;
  a.P = page_size;
  if (!vh::encode_cache_maps(a)) return VH_EINVAL;
  p.tmap_k = a.tmap_k;
  p.tmap_v = a.tmap_v;
  p.tmap_k8 = a.tmap_k8;
  p.tmap_v8 = a.tmap_v8;
  p.tm_tok_dim = a.tm_tok_dim;
  p.full_boxes = a.full_boxes;
  p.memory = {k_cache, v_cache, page_stride, token_stride, head_stride};
  p.q_rot = q_rot;
  p.num_pages = num_pages;
  p.page_table = page_table;
  p.max_pages_per_seq = max_pages_per_seq;
  p.seq_lens = seq_lens;
  p.active = active;
  p.out = out;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.counters = reinterpret_cast<int*>(ws + w.counters);
  p.part_lse = reinterpret_cast<float*>(ws + w.lse);
  p.part_o = reinterpret_cast<float*>(ws + w.o);
  p.err_flag = err_flag;
  const float scale = sm_scale > 0.f ? sm_scale : 1.0f / sqrtf(static_cast<float>(D));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.early = (flags & VH_FLAG_PDL) != 0;
  return status_of(vh::launch_window_decode(p, static_cast<cudaStream_t>(stream)));
} catch (...) {  // (a plan that the host has no memory for; no exception leaves a C function)
  return VH_ECUDA;
}

size_t vh_prompt_workspace_bytes(int T, int B, int Hq, int Hkv, int D) {
  return T < 0 || !valid_shape(B, Hq, Hkv, D, 16) ? 0 : 256;
}

int vh_window_prompt_attn(const vh_e16* q, const vh_e16* k_cache, const vh_e16* v_cache, int64_t page_stride,
                          int64_t token_stride, int64_t head_stride, int num_pages, const int32_t* page_table,
                          int max_pages_per_seq, const int32_t* token_start, const int32_t* seq_lens,
                          const int32_t* active, int window, int sinks, vh_e16* out, float sm_scale, int num_splits,
                          void* workspace, size_t workspace_bytes, int32_t* err_flag, unsigned flags, int T, int B,
                          int Hq, int Hkv, int D, int page_size, void* stream) {
  if ((flags & ~VH_FLAG_FP16) != 0 || T < 0 || window < 0 || sinks < 0 || num_splits < 0 || num_splits > 16 ||
      (num_splits & (num_splits - 1)) != 0 ||
      !(sm_scale == sm_scale) ||
      !valid_cache(B, Hq, Hkv, D, page_size, page_stride, token_stride, head_stride, num_pages, page_table,
                   max_pages_per_seq))
    return VH_EINVAL;
  if (T == 0) return VH_OK;
  if (!q || !k_cache || !v_cache || !token_start || !seq_lens || !active || !out) return VH_EINVAL;
  if (!aligned16(q) || !aligned16(out) || !aligned_cache(k_cache, v_cache, page_stride, token_stride, head_stride))
    return VH_EALIGN;
  if (!workspace) return VH_EWORKSPACE;
  if (!aligned16(workspace)) return VH_EALIGN;
  const DeviceInfo* dev = device_info();
  if (!dev || !prepared(*dev)) return VH_ENODEV;
  if (workspace_bytes < vh_prompt_workspace_bytes(T, B, Hq, Hkv, D)) return VH_EWORKSPACE;
  vh::PromptParams p{};
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.page_stride = page_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.num_pages = num_pages;
  p.page_table = page_table;
  p.max_pages_per_seq = max_pages_per_seq;
  p.token_start = token_start;
  p.seq_lens = seq_lens;
  p.active = active;
  p.window = window > 0 ? std::min(window, vh::kNoWindow) : vh::kNoWindow;
  p.sinks = std::min(sinks, vh::kNoWindow);
  p.out = out;
  const float scale = sm_scale > 0.f ? sm_scale : 1.0f / sqrtf(static_cast<float>(D));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.err_flag = err_flag;
  p.f16 = (flags & VH_FLAG_FP16) != 0;
  p.T = T;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.G = Hq / Hkv;
  p.P = page_size;
  const int(&clusters)[5] = g_prepared[dev->index].clusters;
  p.shift_g = __builtin_ctz(p.G);
  p.pair = small_blocks(T, B, p.G, Hkv, *dev);
  p.shift_block = (p.pair ? 7 : 8) - p.shift_g;
  p.splits = num_splits > 0 ? num_splits : prompt_splits(p, clusters);
  while (p.splits > 1 && clusters[__builtin_ctz(p.splits)] < 1) p.splits /= 2;
  const long long blocks = (static_cast<long long>(T) >> p.shift_block) + B, units = blocks * Hkv * p.splits;
  if (units > INT32_MAX / 2 || blocks * Hkv > (1LL << 32) / Hkv - 1 || !encode_prompt_maps(p)) return VH_EINVAL;
  p.shift_splits = __builtin_ctz(p.splits);
  p.shift_page = (page_size & (page_size - 1)) == 0 ? __builtin_ctz(page_size) : -1;
  p.hkv_inverse = Hkv == 1 ? 0u : static_cast<uint32_t>(((1ULL << 32) + Hkv - 1) / Hkv);
  p.blocks = static_cast<int>(blocks);
  // CTAs draw units one after the other; a cluster's CTAs have one each
  p.ctas = static_cast<int>(p.splits > 1 ? units : std::min<long long>(units, dev->sm_count));
  p.counter = static_cast<int*>(workspace);
  return status_of(vh::launch_window_prompt(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
