// Declarations of the serving operators (page tables, cache append, paged
// attention, the 8-bit LM head) shared by their kernels and their entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mds {

// status bits of mds.h beyond those of mds_device.h
constexpr uint32_t kStatusBadPage = 16u;
constexpr uint32_t kStatusNoPages = 32u;

// ------------------------------------------------- paged key/value cache --
struct PageTableArgs {
  int B, n_slots, max_pages, page_log2, n_pages, max_tokens, advance_add;
  const int32_t* idx_map;     // [B] state slot, < 0 padding; null: slot = b
  const int32_t* kv_len;      // [n_slots]
  const int32_t* advance;     // [B] or null
  const int32_t* chunk_len;   // [B]; < 0 releases the request's pages
  int32_t* block_table;       // [n_slots][max_pages]
  const int32_t* pages_held;  // [n_slots]
  int32_t* free_list;         // [n_pages]
  const int32_t* free_count;  // [1]
  int32_t* query_start;       // [B + 1]
  int32_t* seq_lens;          // [B]
  long long* positions;       // [max_tokens]
  long long* slot_map;        // [max_tokens]
  int32_t* kv_len_out;        // [n_slots], may be kv_len
  int32_t* pages_held_out;    // [n_slots], may be pages_held
  int32_t* free_count_out;    // [1], may be free_count
  uint32_t* status;
};
hipError_t launch_page_tables(const PageTableArgs& a, hipStream_t st);

struct KvAppendArgs {
  int T, Hkv, D, page_log2, n_pages, e4m3;
  const uint16_t* k;
  const uint16_t* v;
  long long src_ts[2], src_hs[2];    // keys, values: token and head strides (elements)
  void* k_pages;
  void* v_pages;
  long long ps[2], ts[2], hs[2];     // page, token and head strides (elements)
  const long long* slot_map;         // [T], < 0: the row is skipped
  const float* k_scale;              // [Hkv] (e4m3 pages)
  const float* v_scale;
  uint32_t* status;
};
hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t st);

struct PagedAttnArgs {
  int T, B, Hq, Hkv, G, D, page_log2, n_pages, n_slots, max_pages, e4m3, causal, window;
  const uint16_t* q;                 // bf16 [T][Hq][D]
  long long q_ts, q_hs;
  const void* k_pages;
  const void* v_pages;
  long long k_ps, k_ts, k_hs, v_ps, v_ts, v_hs;  // bytes
  const int32_t* block_table;        // [n_slots][max_pages]
  const int32_t* idx_map;            // [B] or null
  const int32_t* query_start;        // [B + 1]
  const int32_t* seq_lens;           // [B]
  float scale_log2;                  // softmax scale * log2(e)
  const float* k_scale;              // [Hkv] or null
  const float* v_scale;
  uint16_t* out;                     // bf16 [T][Hq][D]
  long long o_ts, o_hs;
  float* lse;                        // [T][Hq] or null
  // plan (attn_plan): row tiles and key chunks
  int tiles;                         // row tiles of the launch, over all requests
  int per_req;                       // row tiles per request (> 0), or 0: tile of a request by its row offset
  int by_length;                     // tiles in the order of falling sequence length (per_req > 0, B <= 128)
  int chunk, n_chunks;               // keys per chunk; the last chunk takes what is left
  float* part_o;                     // [n_chunks][tiles][Hkv][rows][D] (n_chunks > 1)
  float2* part_ml;                   // [n_chunks][tiles][Hkv][rows] (max, sum) in base 2
  uint32_t* status;
};
// Row tiles, chunks and workspace bytes of a call (host only).
struct AttnPlan {
  int rows, key_groups, tiles, per_req, chunk, n_chunks;
  bool by_length;
  size_t part_o, part_ml, total;  // workspace offsets and size
};
AttnPlan attn_plan(int T, int B, int Hkv, int G, int D, int max_q_len, long long max_seq_len, int window);
// Workspace bytes of a call of these sizes or smaller ones (host only).
size_t attn_workspace(int T, int B, int Hkv, int G, int D, int max_q_len, long long max_seq_len, int window);
hipError_t launch_paged_attention(const PagedAttnArgs& a, const AttnPlan& p, hipStream_t st);

// ------------------------------------------------------- 8-bit LM head --
// e4m3 operands in tiles of 16 rows by 128 columns, 2 KB each: element (r, c)
// of a tile at (c / 16) * 256 + r * 16 + c % 16, tiles of a 16-row block in
// column order (fp8_tile_index).
__host__ __device__ __forceinline__ size_t fp8_tile_index(long long row, int col, int H) {
  return (size_t)(row >> 4) * 16 * H + (size_t)(col >> 7) * 2048 + (size_t)((col & 127) >> 4) * 256 +
         (size_t)(row & 15) * 16 + (col & 15);
}
struct LmHeadFp8Args {
  int M, K, V, H;                // rows M = B*K, H a multiple of 128
  const uint16_t* hidden;        // bf16 [M][H]
  long long hidden_rs;
  const uint8_t* w;              // tiled e4m3 [ceil(V / 16)][16 H]
  const float* w_scale;          // [ceil(V / 128)][H / 128]
  int mb;                        // 16-row blocks of a row tile (lm_head_fp8_blocks)
  uint8_t* xq;                   // workspace: [row tiles][H / 128] stages of fp8_stage_bytes(mb): mb tiles of 2 KB (16
                                 // rows by 128 columns of codes, in the matrix's tile order), then the 16 mb row scales
  void* out;
  long long out_rs, out_ss;
  int out_bf16, vec_out;
};
// bytes of a row tile's quantised chunk of 128 columns: codes, scales, up to whole KB (the copies' size)
__host__ __device__ constexpr int fp8_stage_bytes(int mb) { return (mb * 2112 + 1023) / 1024 * 1024; }
int lm_head_fp8_blocks(int M);
hipError_t launch_lm_head_fp8(const LmHeadFp8Args& a, hipStream_t st);
hipError_t launch_tile_fp8(int V, int H, const uint8_t* codes, uint8_t* tiled, hipStream_t st);
hipError_t launch_quantize_fp8(int V, int H, const uint16_t* w, uint8_t* tiled, float* scales, hipStream_t st);

// Error reporting of the extern "C" layer: sets the thread's message, returns code.
int abi_fail(int code, const char* msg);
int abi_ok();

}  // namespace mds
