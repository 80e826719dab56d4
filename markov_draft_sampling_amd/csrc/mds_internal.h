// Host/device interface between the C-ABI layer (abi.hip) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mds {

// ------------------------------------------------------------ draft loop --
constexpr int kDraftMaxSlabs = 1024;    // column slabs (work-groups) per batch tile and step
constexpr int kDraftMinTilesPerSlab = 8;  // 16-column tiles per slab, at least
// Winner keys sit one 128-byte line apart: every work-group of a step merges
// into every request's key, and atomics on keys sharing a line serialise.
constexpr int kKeyStride = 16;  // u64 words from one (step, request) key to the next
__host__ __device__ __forceinline__ size_t key_index(int k, int B, int b) {
  return ((size_t)k * B + b) * kKeyStride;
}
// Every draft and top-k workspace starts with a region of kFixedKeys winner
// keys that each call leaves at zero (the finalize pass clears the keys it
// reads, and nothing else writes there), so a streaming call with
// K * B <= kFixedKeys needs no clearing launch whatever the workspace held
// before; larger calls keep theirs elsewhere and clear them first.
constexpr int kFixedKeys = 4096;

struct DraftStepArgs {
  int B, K, V, r, k, G, nMT, BT;
  int base_bf16, cache_bf16, vec_base, vec_cache;
  const void* base;
  long long base_rs, base_ss;
  const uint16_t* w1;
  const uint16_t* w2;
  const int32_t* anchor;
  const long long* anchor_pos;
  const float* temp;
  const long long* seeds;
  void* cache;
  long long cache_rs, cache_ss;
  unsigned long long* keys;  // [K][B] winner keys at key_index(k, B, b)
  float2* qpart;             // [K][B][Gq] (max, sum exp) of cache / T per slab
  int Gq;                    // partials per (step, request) row of qpart (>= G)
  uint32_t* status;
  int zero;                  // always 0 (an offset the compiler cannot fold)
  // request-state indexing (all null / B for the plain call)
  const int32_t* idx_map;    // [B][K] state slot of row b at step k, < 0 inert; null: slot = b
  const int32_t* row_map;    // [n_slots] cache row of a slot; null: row = slot
  const long long* sample_pos;  // [B][K] predicted position P (draw keyed by P - 1); null: anchor_pos + k
  int n_slots, n_rows;
  int fp64;                  // fp64 Gumbel option: float64 scores, 64-bit keys of the fp64 format
  int w2_tiled;              // w2 in the 16-row tile order of tile_w2_kernel (step kernels for r <= 256 only)
};

struct DraftFinalArgs {
  int B, K, G;               // G: q partials of each step after the first
  unsigned long long* keys;  // read, then cleared
  const float2* qpart;       // [K][B][Gq]
  const float* temp;
  int32_t* tokens;
  float* lse;
  const int32_t* idx_map;
  const int32_t* row_map;
  int n_slots, n_rows;
  int fp64;  // keys in the fp64 format
  int G0;    // q partials of step 0
  int Gq;    // partials per (step, request) row of qpart
};

// The state slot of batch row b at draft step k, or -1 when the row is inert
// there (past the batch, a negative slot, or a slot / cache row out of range,
// the last two flagged in the status word).
__device__ __forceinline__ int draft_slot(const int32_t* idx_map, const int32_t* row_map, int B, int K, int n_slots,
                                          int n_rows, uint32_t* status, int b, int k) {
  if (b >= B) return -1;
  if (!idx_map) return b;
  const int s = idx_map[(size_t)b * K + k];
  if (s < 0) return -1;
  const int row = s < n_slots ? (row_map ? row_map[s] : s) : -1;
  if (row < 0 || row >= n_rows) {
    if (status) atomicOr(status, 8u);
    return -1;
  }
  return s;
}
__device__ __forceinline__ int draft_slot(const DraftStepArgs& a, int b) {
  return draft_slot(a.idx_map, a.row_map, a.B, a.K, a.n_slots, a.n_rows, a.status, b, a.k);
}
// cache row of a live slot s of batch row b
__device__ __forceinline__ int draft_cache_row(const DraftStepArgs& a, int b, int s) {
  return !a.idx_map ? b : (a.row_map ? a.row_map[s] : s);
}
// key of the draw of batch row b (< B) at step k: the position before the predicted token
__device__ __forceinline__ long long draft_pos_key(const DraftStepArgs& a, int b) {
  return a.sample_pos ? a.sample_pos[(size_t)b * a.K + a.k] - 1 : a.anchor_pos[b] + a.k;
}

int draft_nb(int B, int r);
int draft_slabs(int V, int cus);
// Batch tiles up to which the wave kernel runs one work-group per CU over
// all of them (the fixed-count fast loop needs the CU to itself).
constexpr int kDraftFastTiles = 4;
int draft_wave_slabs(int V, int cus, int bt);
hipError_t launch_draft_init(unsigned long long* keys, int n, hipStream_t st);
hipError_t launch_draft_step(const DraftStepArgs& a, hipStream_t st);
// Wave-independent streaming step (rank <= 256); hipErrorNotSupported
// (nothing launched) for a larger rank.
size_t draft_wave_lds(int NB, int r);
// w2 [V, r] row-major -> the tiled order the step kernels read with 1 KB loads
// (w2_tiled_elems(V, r) bf16 elements, rows past V zero)
__host__ __forceinline__ size_t w2_tiled_elems(int V, int r) { return (size_t)((V + 15) / 16) * 16 * r; }
hipError_t launch_tile_w2(const uint16_t* w2, uint16_t* out, int V, int r, hipStream_t st);
hipError_t launch_draft_wave(const DraftStepArgs& a, hipStream_t st);
hipError_t launch_draft_finalize(const DraftFinalArgs& a, hipStream_t st);

// ------------------------------------------------- top-k Markov drafting --
constexpr int kTopkMax = 256;             // candidates per row, at most
constexpr int kTopkChunk = 8192;          // base-logit columns per selection work-group
constexpr int kTopkMergeKeys = 7168;      // chunk keys a row's merge holds on chip (chunks * k)

struct TopkArgs {
  int B, K, V, r, topk, NC;  // NC = chunks per row
  int base_bf16, cache_bf16, vec_base, vec_cache;
  const void* base;
  long long base_rs, base_ss;
  const uint16_t* w1;
  const uint16_t* w2;
  const int32_t* anchor;
  const float* temp;
  const long long* seeds;
  void* cache;
  long long cache_rs, cache_ss;
  int32_t* tokens;
  float* lse;
  unsigned long long* ckeys;  // [B*K][NC][topk] each chunk's k largest selection keys (0 = none)
  int32_t* cand;              // [B*K][topk] a row's candidate columns, increasing
  uint32_t* status;
  const int32_t* idx_map;     // as in DraftStepArgs
  const int32_t* row_map;
  const long long* sample_pos;  // [B][K], required
  int n_slots, n_rows;
  int fp64;
};
size_t topk_chunk_lds(int topk);

// ------------------------------------------------------ draft LM head --
struct LmHeadArgs {
  int M, K, V, H;             // rows M = B*K (row m = b*K + k), vocabulary, hidden size (a multiple of 256)
  const uint16_t* hidden;     // [M][H] bf16, row stride hidden_rs elements
  long long hidden_rs;
  const uint16_t* lm_head;    // [V][H] bf16, contiguous
  void* out;                  // row (b, k) at b*out_rs + k*out_ss elements, float32 or bf16
  long long out_rs, out_ss;
  int out_bf16, vec_out;
  int cus;                    // compute units of the device (the launch splits its last partial round)
};
// step0 non-null: the LM head also runs step 0 of the draft loop (M = B*K
// <= 256, B <= 32, rank <= 256, the fp32 Gumbel): the step-0 logit rows are not
// stored, and the q partials of step 0 take lm_head_work_groups(a) slots
hipError_t launch_lm_head(const LmHeadArgs& a, hipStream_t st, const DraftStepArgs* step0 = nullptr);
int lm_head_work_groups(const LmHeadArgs& a);
hipError_t launch_topk_select(const TopkArgs& a, hipStream_t st);
hipError_t launch_topk_merge(const TopkArgs& a, hipStream_t st);
hipError_t launch_topk_chain(const TopkArgs& a, hipStream_t st);

// ---------------------------------------------------------- verification --
// columns per statistics block: the pages' sampler uses 8192-column blocks;
// the block size only orders the summation, and 4096 measured faster here
// (37.1 against 38.7 us for the pass at V = 200064, B = 32, K = 7)
constexpr int kStatsChunk = 4096;

// Partials of one (row, block) are published as one 64-bit word: for a
// sampled row (max, sum exp) of x = logit / T as two floats (max in the low
// half), for a greedy row the winner key of the raw logits.
struct RowStat {  // combined statistics of one target row
  float m;        // max of x = logit / T (sampled rows)
  float lz;       // log of sum exp(x - m); NaN if the row held NaN
  unsigned long long key;  // winner key of the raw logits (greedy rows)
};

struct TopP {  // kept set of one target row: ord(t) > tau, or == tau and id <= cut
  uint32_t tau;
  int cut;
  float log_z;  // log of the kept mass sum exp(x - m)
  int on;
};

struct ReqState {  // the accept decision of one request, read by the residual draw
  int n_acc;   // accepted drafts; the final token is drawn from row n_acc
  int mode;    // 0 bonus from p_K, 1 residual of row n_acc, 2 greedy (done), 3 residual empty -> p
  float M, LZ; // row n_acc: max of logit / T and log of its (kept) mass
  float LQ;    // draft row n_acc: log sum exp of cache / T (mode 1)
  int pad;
  TopP tp;     // kept set of row n_acc (tp.on == 0 when no top-p)
};

// The kVerifyCounterBytes after the verify workspace's 256-byte status block
// hold one arrival counter and one 64-bit winner key per request. Every call
// leaves them at zero, so they sit at a fixed offset whatever (B, K, V) a
// call uses. The block is 2048 lines of 512 bytes: request b uses line
// b mod 2048, its counter is 32-bit word b / 2048 of the line's first 128
// bytes, its key 64-bit word b / 2048 of bytes [128, 384). With b < 65536
// (the largest batch a call accepts) b / 2048 < 32, so no key overlaps a
// counter and nothing leaves the line. Requests b and b + 2048 i share a
// line; any other two do not (many work-groups bumping counters of one line
// serialise on it).
constexpr size_t kVerifyCounterOffset = 256;
constexpr int kVerifyLines = 2048;
constexpr int kVerifyLineBytes = 512;
constexpr size_t kVerifyCounterBytes = (size_t)kVerifyLines * kVerifyLineBytes;
constexpr int kVerifyMaxB = kVerifyLines * 32;  // b / 2048 < 32
// index in 32-bit words from the start of the block
__host__ __device__ constexpr int verify_counter_index(int b) {
  return (b & (kVerifyLines - 1)) * (kVerifyLineBytes / 4) + (b >> 11);
}
// index in 64-bit words from the start of the block
__host__ __device__ constexpr int verify_key_index(int b) {
  return (b & (kVerifyLines - 1)) * (kVerifyLineBytes / 8) + 16 + (b >> 11);
}

struct VerifyArgs {
  int B, K, V, NC;
  const float* target;
  long long target_rs;
  const void* cache;
  int cache_bf16, vec_cache;
  long long cache_rs, cache_ss;
  const float* draft_lse;  // [B*K], or null: then the statistics pass also reads the cache rows
  const int32_t* draft;
  const float* temp;
  const float* top_p;
  const long long* seeds;
  const long long* anchor_pos;
  int32_t* out_tokens;
  int32_t* num_accepted;
  unsigned long long* tpart;  // [NC][B*(K+1)] packed partials of the target rows
  unsigned long long* qpart;  // [NC][B*K] packed partials of the cache rows (draft_lse null)
  RowStat* rowstat;           // [B*(K+1)]
  float* qlse;                // [B*K] draft log-normalisers (copied or combined)
  unsigned long long* tq;     // [B*K] (target, cache) logits at the draft tokens, packed
  TopP* topp;                 // [B*(K+1)] or null
  ReqState* req;              // [B]
  unsigned long long* rkey;   // winner keys of the final draws, at verify_key_index(b)
  unsigned* cnt;              // [B] arrival counters (zero between calls)
  uint32_t* status;
  int vec_target;
  int decide;                 // the statistics pass also takes the accept decision (no top-p)
  int NR;                     // residual blocks per request (kResCols columns each)
  // request-state indexing (null / B for the plain call)
  const int32_t* idx_map;     // [B] state slot of request b, < 0 padding; null: slot = b
  const int32_t* row_map;     // [n_slots] cache row of a slot; null: row = slot
  int n_slots, n_rows;
};

// The state slot of request b, or -1 for a padding request (a negative slot,
// or a slot / cache row out of range, the latter flagged in the status word).
__device__ __forceinline__ int verify_slot(const VerifyArgs& a, int b) {
  if (!a.idx_map) return b;
  const int s = a.idx_map[b];
  if (s < 0) return -1;
  const int row = s < a.n_slots ? (a.row_map ? a.row_map[s] : s) : -1;
  if (row < 0 || row >= a.n_rows) {
    if (a.status) atomicOr(a.status, 8u);
    return -1;
  }
  return s;
}
__device__ __forceinline__ int verify_cache_row(const VerifyArgs& a, int b, int s) {
  return !a.idx_map ? b : (a.row_map ? a.row_map[s] : s);
}

constexpr int kResCols = 2048;  // columns per residual work-group

// The statistics pass; launch_combine must follow it (it also decides when
// a.decide, i.e. without top-p).
hipError_t launch_verify_stats(const VerifyArgs& a, hipStream_t st);
hipError_t launch_combine(const VerifyArgs& a, hipStream_t st);
hipError_t launch_top_p(const VerifyArgs& a, hipStream_t st);
hipError_t launch_decide(const VerifyArgs& a, hipStream_t st);
hipError_t launch_residual(const VerifyArgs& a, hipStream_t st);

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
// Row tiles, chunks and workspace bytes of a call (host only); cus: compute units.
struct AttnPlan {
  int rows, tiles, per_req, chunk, n_chunks;
  bool by_length;
  size_t part_o, part_ml, total;  // workspace offsets and size
};
AttnPlan attn_plan(int T, int B, int Hkv, int G, int D, int max_q_len, long long max_seq_len, int window);
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
  int out_bf16, vec_out, cus;
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

// ----------------------------------------------------------------- debug --
hipError_t launch_debug_noise(int n, const int32_t* cols, long long seed, long long pos, uint32_t salt,
                              uint32_t* words, float* g, hipStream_t st);
hipError_t launch_debug_gumbel(int n, const uint32_t* words, float* g, hipStream_t st);
hipError_t launch_debug_top_p_out(int rows, const TopP* tp, uint32_t* tau, int32_t* cut, float* log_z, int32_t* on,
                                  hipStream_t st);

}  // namespace mds
