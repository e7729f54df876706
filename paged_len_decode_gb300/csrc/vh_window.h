// vh_window.h -- parameter blocks and launchers of the ragged-batch append,
// the windowed decode attention and the prompt attention (internal; the
// public interface is vh.h).
#pragma once

#include <cstdint>
#include <cuda.h>  // CUtensorMap (the type only)
#include <cuda_runtime.h>

#include "vh_kernels.h"

namespace vh {

// A window that never ends, for W = 0 (slots are below 2^24).
constexpr int kNoWindow = 1 << 28;

struct MropeParams {
  const uint16_t* q;
  const uint16_t* k_new;
  const uint16_t* v_new;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  const float* cos_sin;
  int max_pos;
  const int32_t* positions;    // [num_axes][T], or null (slot index)
  int num_axes;
  unsigned long long axis[2];  // 2 bits a rotation pair, pair 0 lowest
  const float* q_norm_w;       // [D], or null
  const float* k_norm_w;
  float norm_eps;
  uint16_t* k_cache;
  uint16_t* v_cache;
  long long page_stride, token_stride, head_stride;
  int num_pages;
  const int32_t* page_table;   // null: contiguous cache
  int max_pages_per_seq;
  const int32_t* token_start;  // [B + 1], or null (one token a row)
  const int32_t* seq_lens;
  const int32_t* active;
  void* q_rot;                 // float or 16-bit elements
  int q16;
  int rope_interleaved, f16;
  int32_t* err_flag;
  int T, B, Hq, Hkv, D, P;
  int warps;                   // that share a token
};

struct WindowDecodeParams {
  // K and V caches as 4-D tensors (see vh_kernels.h): boxes of 16 tokens x Hc
  // heads, and of 8 tokens x 1 head
  CUtensorMap tmap_k, tmap_v, tmap_k8, tmap_v8;
  int tm_tok_dim, full_boxes;
  CacheMemory memory;          // the same caches
  const float* q_rot;          // [B][Hq][D]
  int num_pages;
  const int32_t* page_table;   // null: contiguous cache
  int max_pages_per_seq;
  const int32_t* seq_lens;
  const int32_t* active;
  int window, sinks;           // window >= 1 (kNoWindow: none), sinks >= 0
  uint16_t* out;
  float scale_log2;            // softmax scale * log2(e)
  int* counters;               // [groups][B] pieces delivered per row; zero between calls
  float* part_o;               // [groups][N][2][Hc*G][D]
  float* part_lse;             // [groups][N][2][Hc*G], base 2
  int32_t* err_flag;
  int f16;
  int early;                   // VH_FLAG_PDL: lengths, flags and page ids are read before the dependency wait
  int B, Hq, Hkv, D, G, P;
  int Hc, groups, N, stages;
  int stage_bytes;             // K then V of one tile: [D/64][Hc][16 tokens][128 B swizzled] each
  int q_off, cum_off, len_off, bar_off, smem_bytes;
};

// The prompt kernel's ring of K and V stages and its shared memory: the
// queries of both row tiles, the stages, 32 KB through which outputs leave, and
// up to 1024 bytes to align them.
template <int D>
constexpr int kPromptStages = D == 128 ? 4 : 6;
template <int D>
constexpr int kPromptQueries = D == 128 ? 1 : 2;  // blocks of queries held at a time
template <int D>
constexpr int kPromptSmem = (2 * kPromptQueries<D> + kPromptStages<D>) * 128 * D * 2 + 32768 + 1024;

struct PromptParams {
  // queries as a 3-D tensor (head_dim, q head, token), boxes of 64 x G x 128/G;
  // K and V as 4-D tensors (see vh_kernels.h), boxes of 64 x `box` tokens x 1 head
  CUtensorMap tmap_q, tmap_k, tmap_v;
  int tm_tok_dim, box, shift_box;
  const uint16_t* q;           // [T][Hq][D]
  const uint16_t* k_cache;
  const uint16_t* v_cache;
  long long page_stride, token_stride, head_stride;
  int num_pages;
  const int32_t* page_table;   // null: contiguous cache
  int max_pages_per_seq;
  const int32_t* token_start;
  const int32_t* seq_lens;
  const int32_t* active;
  int window, sinks;
  uint16_t* out;
  float scale_log2;
  int32_t* err_flag;
  int f16;
  int T, B, Hq, Hkv, D, G, P;
  int pair;                    // blocks of 128 (token, head) rows, by both warpgroups; else of 256
  int shift_block;             // log2 of a block's tokens
  int blocks;                  // T >> shift_block, + B: an upper bound (rows fill their last block partly)
  int splits;                  // CTAs that share the keys of a block (a cluster): 1, 2, 4, 8 or 16
  int ctas;
  int shift_g, shift_splits, shift_page;  // log2 of G, splits and P (-1: not a power of two)
  uint32_t hkv_inverse;        // ceil(2^32 / Hkv), 0 for Hkv == 1: v / Hkv of v < 2^32 / Hkv is the high word of v times it
  int* counter;                // the next unit to be drawn (splits == 1); zero between calls
};

// The launch of kernels that begin with pdl_begin (vh_ragged.cuh).
template <typename P>
inline cudaError_t launch_dependent(void (*kernel)(P), const P& p, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                    int cluster = 1) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_mrope_kv_append(const MropeParams& p, cudaStream_t stream);
cudaError_t prepare_window_decode(int max_smem);  // once per device, every variant
cudaError_t window_decode_occupancy(const WindowDecodeParams& p, int* blocks_per_sm);
cudaError_t launch_window_decode(const WindowDecodeParams& p, cudaStream_t stream);
// once per device, every variant; clusters[x]: clusters of 2^x CTAs that run at a time
cudaError_t prepare_window_prompt(int (&clusters)[5]);
cudaError_t launch_window_prompt(const PromptParams& p, cudaStream_t stream);

}  // namespace vh
