// vh_quant.h -- parameter blocks and launchers of the calls on an 8-bit cache
// that are not in vh_window.h (internal; the public interface is vh.h).
#pragma once

#include "vh_window.h"

namespace vh {

// An 8-bit cache as memory: e4m3 values (strides in elements, bytes), and a scale
// for every slot and head (strides in floats; a page's slots follow one another).
struct QuantMemory {
  const uint8_t* k;
  const uint8_t* v;
  long long page_stride, token_stride, head_stride;
  const float* k_scale;
  const float* v_scale;
  long long scale_page, scale_head;
};

bool aligned_quant(const QuantMemory& m);  // (vh_window_api.cu)

struct QuantDecodeParams {
  // K and V as 4-D tensors (head_dim, token, kv head, page), boxes of D x 16 tokens x Hc heads,
  // and their scales as 3-D ones (token, kv head, page), boxes of 16 tokens x Hc heads; of 8
  // tokens where pages have 8
  CUtensorMap tmap_k, tmap_v, tmap_ks, tmap_vs;
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
  int f16;                     // of out
  int early;                   // VH_FLAG_PDL: lengths, flags and page ids are read before the dependency wait
  int B, Hq, Hkv, D, G, P;
  int Hc, groups, N, stages;
  int stage_bytes;             // K and V of one tile [Hc][16][D], their scales (scale_bytes each)
  int scale_bytes;
  int q_off, cum_off, len_off, bar_off, smem_bytes;
};

// What a row's piece costs in the merge, by q head of a kv head, in the time that a CTA takes for a
// tile.  (0.05, 0.1, 0.2 and 0.4: one row of up to 30000 tokens, 64 / 8 heads of 128, 40.1, 38.6, 36.9 and
// 41.8 us; 40 / 5 heads 30.8, 30.3, 31.9 and 37.9; four rows of 16000, 64 / 8 heads of 64, 52.4, 43.4, 45.1 and 47.6.)
constexpr float kQuantPiece = 0.1f;

struct QuantReadParams {
  QuantMemory memory;
  int num_pages;
  const int32_t* page_table;   // null: contiguous cache
  int max_pages_per_seq;
  const int32_t* seq_lens;
  const int32_t* active;
  const int32_t* first_slot;   // [B], or null (0)
  int sinks;
  uint16_t* k_out;
  uint16_t* v_out;
  long long out_page, out_token, out_head;  // strides
  int out_pages;
  const int32_t* out_table;
  int out_per_row;
  int32_t* err_flag;
  int f16;
  int B, Hkv, D, P, out_P;
  uint32_t hkv_inverse;        // ceil(2^32 / Hkv), 0 for Hkv == 1: y / Hkv of small y is the high word of y times it
};
inline size_t quant_read_smem(int B) { return 4 * (3 * static_cast<size_t>(B) + 1); }

cudaError_t prepare_quant_read(int max_smem);
cudaError_t launch_quant_read(const QuantReadParams& p, int sm_count, cudaStream_t stream);
cudaError_t prepare_quant_decode(int max_smem);  // once per device, every variant
cudaError_t quant_decode_occupancy(const QuantDecodeParams& p, int* blocks_per_sm);
cudaError_t launch_quant_decode(const QuantDecodeParams& p, cudaStream_t stream);

}  // namespace vh
