// extern "C" entry points of the serving operators (page tables, cache append,
// paged attention, the 8-bit LM head): argument checks on the host, then the
// kernels on the caller's stream. See include/mds.h for the contract.
#include "../../include/mds.h"
#include "mds_serve.h"

namespace {

using mds::abi_fail;
using mds::abi_ok;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int hip_fail(hipError_t e) { return abi_fail(MDS_ERR_HIP, hipGetErrorString(e)); }

// A dimension of one element is never stepped along: its stride may be anything, and counts as 0.
int64_t step(int64_t n, int64_t stride) { return n <= 1 ? 0 : stride; }

// log2 of a page size, or -1
int page_log2(int page_size) {
  for (int s = 4; s <= 10; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

int check_page(int page_size, int n_pages, int* lg) {
  *lg = page_log2(page_size);
  if (page_size < 1 || n_pages < 1) return abi_fail(MDS_ERR_INVALID_ARG, "page_size and n_pages must be >= 1");
  if (*lg < 0) return abi_fail(MDS_ERR_UNSUPPORTED, "page_size must be a power of two in [16, 1024]");
  if ((long long)n_pages * page_size > 0x7FFFFFFFFFLL) return abi_fail(MDS_ERR_INVALID_ARG, "the cache is too large");
  return MDS_OK;
}

// [n_pages][P][Hkv][D] pages of `es`-byte elements with a unit last stride: 16-byte aligned, strides that
// are whole 16-byte pieces and fit the kernels' 32-bit offsets inside a page
int check_pages(const void* p, int es, int64_t ps, int64_t ts, int64_t hs, int page_size) {
  const int64_t e16 = 16 / es;
  if (!aligned(p, 16) || ps % e16 || ts % e16 || hs % e16)
    return abi_fail(MDS_ERR_UNSUPPORTED, "pages must be 16-byte aligned with strides that are multiples of 16 bytes");
  if (ps < 0 || ts < 0 || hs < 0 || ps > (int64_t{1} << 40) || ts > (1 << 30) || hs > (int64_t{1} << 40) ||
      ts * es * page_size >= (1LL << 31))
    return abi_fail(MDS_ERR_INVALID_ARG, "page strides must be >= 0, and a page's slots span less than 2 GiB");
  return MDS_OK;
}

int check_heads(int Hkv, int D) {
  if (Hkv < 1 || Hkv > 1024) return abi_fail(MDS_ERR_INVALID_ARG, "key heads must be in [1, 1024]");
  if (D < 1) return abi_fail(MDS_ERR_INVALID_ARG, "the head dimension must be >= 1");
  return MDS_OK;
}

constexpr int kMaxBatch = 65535;
constexpr int kMaxSlots = 1 << 17;

int check_batch(int B, int n_slots, int max_pages, int lg, bool idx) {
  if (B < 1 || B > kMaxBatch) return abi_fail(MDS_ERR_INVALID_ARG, "B must be in [1, 65535]");
  if (n_slots < 1 || n_slots > kMaxSlots) return abi_fail(MDS_ERR_INVALID_ARG, "n_slots must be in [1, 2^17]");
  if (!idx && n_slots < B) return abi_fail(MDS_ERR_INVALID_ARG, "without idx_map: n_slots >= B");
  if (max_pages < 1 || ((long long)max_pages << lg) >= (1LL << 30))
    return abi_fail(MDS_ERR_INVALID_ARG, "max_pages must be >= 1 and max_pages * page_size below 2^30");
  return MDS_OK;
}

int check_cache_dtype(int dt) {
  if (dt != MDS_BF16 && dt != MDS_E4M3) return abi_fail(MDS_ERR_INVALID_ARG, "cache dtype must be MDS_BF16 or MDS_E4M3");
  return MDS_OK;
}

int check_attention(int T, int B, int Hq, int Hkv, int D, int max_q_len, int64_t max_seq_len, int window) {
  int rc;
  if (T < 0 || T > (1 << 24)) return abi_fail(MDS_ERR_INVALID_ARG, "T must be in [0, 2^24]");
  if (B < 1 || B > kMaxBatch) return abi_fail(MDS_ERR_INVALID_ARG, "B must be in [1, 65535]");
  if ((rc = check_heads(Hkv, D))) return rc;
  if (Hq < 1 || Hq > 1024 || Hq % Hkv) return abi_fail(MDS_ERR_INVALID_ARG, "query heads must be a multiple of key heads, at most 1024");
  if (D != 64 && D != 128) return abi_fail(MDS_ERR_UNSUPPORTED, "the head dimension must be 64 or 128");
  if (max_q_len < 0 || max_q_len > (1 << 24)) return abi_fail(MDS_ERR_INVALID_ARG, "max_q_len must be in [0, 2^24]");
  if (max_seq_len < 0 || max_seq_len > (1LL << 30)) return abi_fail(MDS_ERR_INVALID_ARG, "max_seq_len must be in [0, 2^30]");
  if (window < 0 || window > (1 << 30)) return abi_fail(MDS_ERR_INVALID_ARG, "window must be in [0, 2^30] (0: none)");
  if ((long long)T * (Hq / Hkv) > 0x3FFFFFFF) return abi_fail(MDS_ERR_UNSUPPORTED, "too many query rows");
  return MDS_OK;
}

// strides (elements) of a written array keep its elements apart: taken from the smallest stride up, each
// must step past everything below it
struct Dim {
  int64_t n, stride;
};
template <int N>
bool disjoint(Dim (&d)[N], int64_t inner) {
  for (int i = 1; i < N; ++i)
    for (int j = i; j > 0 && d[j].stride < d[j - 1].stride; --j) {
      const Dim t = d[j];
      d[j] = d[j - 1];
      d[j - 1] = t;
    }
  int64_t extent = inner;
  for (int i = 0; i < N; ++i) {
    if (d[i].n <= 1) continue;
    if (d[i].stride < extent) return false;
    if (d[i].stride > (int64_t{1} << 62) / d[i].n) return false;
    extent += (d[i].n - 1) * d[i].stride;
  }
  return true;
}

int check_lm_head_fp8(int V, int H) {
  if (V < 2 || V >= (1 << 24)) return abi_fail(MDS_ERR_INVALID_ARG, "V must be in [2, 2^24)");
  if (H < 128 || H > (1 << 16)) return abi_fail(MDS_ERR_INVALID_ARG, "H must be in [128, 65536]");
  if (H % 128) return abi_fail(MDS_ERR_UNSUPPORTED, "H must be a multiple of 128");
  return MDS_OK;
}

size_t tiled_fp8_bytes(int V, int H) { return (size_t)((V + 15) / 16) * 16 * H; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  return (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

int lm_head_fp8_rows(int B, int K, int* rows) {
  if (B < 1 || B > kMaxBatch) return abi_fail(MDS_ERR_INVALID_ARG, "B must be in [1, 65535]");
  if (K < 1 || K > 64) return abi_fail(MDS_ERR_INVALID_ARG, "K must be in [1, 64]");
  *rows = B * K;
  return MDS_OK;
}

size_t lm_head_fp8_ws(int rows, int H) {
  const int mb = mds::lm_head_fp8_blocks(rows);
  const size_t tiles = (size_t)((rows + 15) / 16 + mb - 1) / mb;
  return tiles * (H / 128) * mds::fp8_stage_bytes(mb);
}

}  // namespace

extern "C" {

int mds_lm_head_fp8_tiled_bytes(int V, int H, size_t* out_bytes) {
  int rc;
  if ((rc = check_lm_head_fp8(V, H))) return rc;
  if (!out_bytes) return abi_fail(MDS_ERR_INVALID_ARG, "out_bytes is NULL");
  *out_bytes = tiled_fp8_bytes(V, H);
  return abi_ok();
}

int mds_tile_lm_head_fp8(int V, int H, const void* codes, void* tiled, size_t tiled_bytes, void* stream) {
  int rc;
  if ((rc = check_lm_head_fp8(V, H))) return rc;
  if (!codes || !tiled) return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(codes, 16) || !aligned(tiled, 16)) return abi_fail(MDS_ERR_INVALID_ARG, "codes and tiled must be 16-byte aligned");
  const size_t need = tiled_fp8_bytes(V, H);
  if (tiled_bytes < need) return abi_fail(MDS_ERR_INVALID_ARG, "tiled is too small");
  if (overlap(codes, (size_t)V * H, tiled, need)) return abi_fail(MDS_ERR_INVALID_ARG, "codes and tiled overlap");
  const hipError_t e = mds::launch_tile_fp8(V, H, (const uint8_t*)codes, (uint8_t*)tiled, (hipStream_t)stream);
  return e == hipSuccess ? abi_ok() : hip_fail(e);
}

int mds_quantize_lm_head_fp8(int V, int H, const void* lm_head, void* tiled, size_t tiled_bytes, float* scales,
                             void* stream) {
  int rc;
  if ((rc = check_lm_head_fp8(V, H))) return rc;
  if (!lm_head || !tiled || !scales) return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(lm_head, 16) || !aligned(tiled, 16))
    return abi_fail(MDS_ERR_INVALID_ARG, "lm_head and tiled must be 16-byte aligned");
  const size_t need = tiled_fp8_bytes(V, H);
  if (tiled_bytes < need) return abi_fail(MDS_ERR_INVALID_ARG, "tiled is too small");
  if (overlap(lm_head, (size_t)V * H * 2, tiled, need)) return abi_fail(MDS_ERR_INVALID_ARG, "lm_head and tiled overlap");
  const hipError_t e =
      mds::launch_quantize_fp8(V, H, (const uint16_t*)lm_head, (uint8_t*)tiled, scales, (hipStream_t)stream);
  return e == hipSuccess ? abi_ok() : hip_fail(e);
}

int mds_lm_head_fp8_workspace_bytes(int B, int K, int V, int H, size_t* out_bytes) {
  int rc, rows;
  if ((rc = lm_head_fp8_rows(B, K, &rows)) || (rc = check_lm_head_fp8(V, H))) return rc;
  if (!out_bytes) return abi_fail(MDS_ERR_INVALID_ARG, "out_bytes is NULL");
  *out_bytes = lm_head_fp8_ws(rows, H);
  return abi_ok();
}

int mds_lm_head_fp8(int B, int K, int V, int H, const void* hidden, int64_t hidden_row_stride, const void* lm_head,
                    const float* scales, void* out, int out_dtype, int64_t out_req_stride, int64_t out_step_stride,
                    void* workspace, size_t workspace_bytes, void* stream) {
  int rc, rows;
  if ((rc = lm_head_fp8_rows(B, K, &rows)) || (rc = check_lm_head_fp8(V, H))) return rc;
  if (!hidden || !lm_head || !scales || !out || !workspace) return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  if (out_dtype != MDS_F32 && out_dtype != MDS_BF16) return abi_fail(MDS_ERR_INVALID_ARG, "out dtype must be MDS_F32 or MDS_BF16");
  if (rows == 1) hidden_row_stride = H;
  if (hidden_row_stride < H || hidden_row_stride % 8)
    return abi_fail(MDS_ERR_INVALID_ARG, "hidden_row_stride must be a multiple of 8, at least H");
  if (!aligned(hidden, 16) || !aligned(lm_head, 16)) return abi_fail(MDS_ERR_INVALID_ARG, "hidden and lm_head must be 16-byte aligned");
  out_req_stride = step(B, out_req_stride);
  out_step_stride = step(K, out_step_stride);
  Dim dims[2] = {{B, out_req_stride}, {K, out_step_stride}};
  if (out_req_stride < 0 || out_step_stride < 0 || !disjoint(dims, V))
    return abi_fail(MDS_ERR_INVALID_ARG, "out strides make rows overlap or are shorter than V");
  if (!aligned(workspace, 256)) return abi_fail(MDS_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (workspace_bytes < lm_head_fp8_ws(rows, H)) return abi_fail(MDS_ERR_WORKSPACE, "workspace too small for the LM head");
  mds::LmHeadFp8Args a{};
  a.M = rows;
  a.K = K;
  a.V = V;
  a.H = H;
  a.hidden = (const uint16_t*)hidden;
  a.hidden_rs = hidden_row_stride;
  a.w = (const uint8_t*)lm_head;
  a.w_scale = scales;
  a.mb = mds::lm_head_fp8_blocks(rows);
  a.xq = (uint8_t*)workspace;
  a.out = out;
  a.out_rs = out_req_stride;
  a.out_ss = out_step_stride;
  a.out_bf16 = out_dtype == MDS_BF16;
  a.vec_out = aligned(out, a.out_bf16 ? 8 : 16) && out_req_stride % 4 == 0 && out_step_stride % 4 == 0;
  const hipError_t e = mds::launch_lm_head_fp8(a, (hipStream_t)stream);
  return e == hipSuccess ? abi_ok() : hip_fail(e);
}

int mds_kv_page_tables(int B, int n_slots, int max_pages, int page_size, int n_pages, int max_tokens,
                       const int32_t* idx_map, const int32_t* kv_len, const int32_t* advance, int advance_add,
                       const int32_t* chunk_len, int32_t* block_table, const int32_t* pages_held,
                       int32_t* free_list, const int32_t* free_count, int32_t* query_start, int32_t* seq_lens,
                       int64_t* positions, int64_t* slot_map, int32_t* kv_len_out, int32_t* pages_held_out,
                       int32_t* free_count_out, uint32_t* status, void* stream) {
  int rc;
  mds::PageTableArgs a{};
  if ((rc = check_page(page_size, n_pages, &a.page_log2))) return rc;
  if ((rc = check_batch(B, n_slots, max_pages, a.page_log2, idx_map != nullptr))) return rc;
  if (max_tokens < 0 || max_tokens > (1 << 24)) return abi_fail(MDS_ERR_INVALID_ARG, "max_tokens must be in [0, 2^24]");
  if (!kv_len || !chunk_len || !block_table || !pages_held || !free_list || !free_count || !query_start || !seq_lens ||
      (max_tokens && (!positions || !slot_map)) || !kv_len_out || !pages_held_out || !free_count_out)
    return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  a.B = B;
  a.n_slots = n_slots;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.max_tokens = max_tokens;
  a.advance_add = advance_add;
  a.idx_map = idx_map;
  a.kv_len = kv_len;
  a.advance = advance;
  a.chunk_len = chunk_len;
  a.block_table = block_table;
  a.pages_held = pages_held;
  a.free_list = free_list;
  a.free_count = free_count;
  a.query_start = query_start;
  a.seq_lens = seq_lens;
  a.positions = (long long*)positions;
  a.slot_map = (long long*)slot_map;
  a.kv_len_out = kv_len_out;
  a.pages_held_out = pages_held_out;
  a.free_count_out = free_count_out;
  a.status = status;
  const hipError_t e = mds::launch_page_tables(a, (hipStream_t)stream);
  return e == hipSuccess ? abi_ok() : hip_fail(e);
}

int mds_kv_append(int T, int Hkv, int D, const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                  int64_t v_token_stride, int64_t v_head_stride, void* k_pages, void* v_pages, int cache_dtype,
                  int page_size, int n_pages, int64_t k_page_stride, int64_t k_slot_stride, int64_t k_pages_head_stride,
                  int64_t v_page_stride, int64_t v_slot_stride, int64_t v_pages_head_stride, const int64_t* slot_map,
                  const float* k_scale, const float* v_scale, uint32_t* status, void* stream) {
  int rc;
  mds::KvAppendArgs a{};
  if (T < 0 || T > (1 << 24)) return abi_fail(MDS_ERR_INVALID_ARG, "T must be in [0, 2^24]");
  if ((rc = check_heads(Hkv, D)) || (rc = check_cache_dtype(cache_dtype))) return rc;
  if (D % 16 || D > 1024) return abi_fail(MDS_ERR_UNSUPPORTED, "the head dimension must be a multiple of 16, at most 1024");
  if ((rc = check_page(page_size, n_pages, &a.page_log2))) return rc;
  a.e4m3 = cache_dtype == MDS_E4M3;
  if (!k_pages || !v_pages || (T && (!k || !v || !slot_map)) || (a.e4m3 && (!k_scale || !v_scale)))
    return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  const int es = a.e4m3 ? 1 : 2;
  k_page_stride = step(n_pages, k_page_stride);
  v_page_stride = step(n_pages, v_page_stride);
  k_pages_head_stride = step(Hkv, k_pages_head_stride);
  v_pages_head_stride = step(Hkv, v_pages_head_stride);
  k_token_stride = step(T, k_token_stride);
  v_token_stride = step(T, v_token_stride);
  k_head_stride = step(Hkv, k_head_stride);
  v_head_stride = step(Hkv, v_head_stride);
  if ((rc = check_pages(k_pages, es, k_page_stride, k_slot_stride, k_pages_head_stride, page_size)) ||
      (rc = check_pages(v_pages, es, v_page_stride, v_slot_stride, v_pages_head_stride, page_size)))
    return rc;
  Dim kd[3] = {{n_pages, k_page_stride}, {page_size, k_slot_stride}, {Hkv, k_pages_head_stride}};
  Dim vd[3] = {{n_pages, v_page_stride}, {page_size, v_slot_stride}, {Hkv, v_pages_head_stride}};
  if (!disjoint(kd, D) || !disjoint(vd, D)) return abi_fail(MDS_ERR_INVALID_ARG, "page strides make rows overlap");
  if (!aligned(k, 16) || !aligned(v, 16) || k_token_stride % 8 || k_head_stride % 8 || v_token_stride % 8 ||
      v_head_stride % 8)
    return abi_fail(MDS_ERR_UNSUPPORTED, "k and v must be 16-byte aligned with strides that are multiples of 8 elements");
  if (k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0)
    return abi_fail(MDS_ERR_INVALID_ARG, "strides must be >= 0");
  if ((long long)T * Hkv * (D / 8) >= 0x7FFFFFFFLL) return abi_fail(MDS_ERR_UNSUPPORTED, "too many elements in one call");
  if (T == 0) return abi_ok();
  a.T = T;
  a.Hkv = Hkv;
  a.D = D;
  a.n_pages = n_pages;
  a.k = (const uint16_t*)k;
  a.v = (const uint16_t*)v;
  a.src_ts[0] = k_token_stride;
  a.src_hs[0] = k_head_stride;
  a.src_ts[1] = v_token_stride;
  a.src_hs[1] = v_head_stride;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.ps[0] = k_page_stride;
  a.ts[0] = k_slot_stride;
  a.hs[0] = k_pages_head_stride;
  a.ps[1] = v_page_stride;
  a.ts[1] = v_slot_stride;
  a.hs[1] = v_pages_head_stride;
  a.slot_map = (const long long*)slot_map;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.status = status;
  const hipError_t e = mds::launch_kv_append(a, (hipStream_t)stream);
  return e == hipSuccess ? abi_ok() : hip_fail(e);
}

int mds_paged_attention_workspace_bytes(int T, int B, int Hq, int Hkv, int D, int max_q_len, int64_t max_seq_len,
                                        int window, size_t* out_bytes) {
  int rc;
  if ((rc = check_attention(T, B, Hq, Hkv, D, max_q_len, max_seq_len, window))) return rc;
  if (!out_bytes) return abi_fail(MDS_ERR_INVALID_ARG, "out_bytes is NULL");
  *out_bytes = mds::attn_workspace(T, B, Hkv, Hq / Hkv, D, max_q_len, max_seq_len, window);
  return abi_ok();
}

int mds_paged_attention(int T, int B, int Hq, int Hkv, int D, const void* q, int64_t q_token_stride,
                        int64_t q_head_stride, const void* k_pages, const void* v_pages, int cache_dtype,
                        int page_size, int n_pages, int64_t k_page_stride, int64_t k_slot_stride,
                        int64_t k_pages_head_stride, int64_t v_page_stride, int64_t v_slot_stride,
                        int64_t v_pages_head_stride, const int32_t* block_table, int n_slots, int max_pages,
                        const int32_t* idx_map, const int32_t* query_start, const int32_t* seq_lens, int max_q_len,
                        int64_t max_seq_len, float scale, int causal, int window, const float* k_scale,
                        const float* v_scale, void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                        void* workspace, size_t workspace_bytes, void* stream) {
  int rc;
  mds::PagedAttnArgs a{};
  if ((rc = check_attention(T, B, Hq, Hkv, D, max_q_len, max_seq_len, window)) ||
      (rc = check_cache_dtype(cache_dtype)) || (rc = check_page(page_size, n_pages, &a.page_log2)) ||
      (rc = check_batch(B, n_slots, max_pages, a.page_log2, idx_map != nullptr)))
    return rc;
  a.e4m3 = cache_dtype == MDS_E4M3;
  if ((T && (!q || !out)) || !k_pages || !v_pages || !block_table || !query_start || !seq_lens || !workspace)
    return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!a.e4m3 && (k_scale || v_scale)) return abi_fail(MDS_ERR_INVALID_ARG, "scales belong to an MDS_E4M3 cache");
  if (!(scale > 0.0f) || !(scale < 1e30f)) return abi_fail(MDS_ERR_INVALID_ARG, "scale must be positive and finite");
  if (causal != 0 && causal != 1) return abi_fail(MDS_ERR_INVALID_ARG, "causal must be 0 or 1");
  const int es = a.e4m3 ? 1 : 2;
  k_page_stride = step(n_pages, k_page_stride);
  v_page_stride = step(n_pages, v_page_stride);
  k_pages_head_stride = step(Hkv, k_pages_head_stride);
  v_pages_head_stride = step(Hkv, v_pages_head_stride);
  q_token_stride = step(T, q_token_stride);
  q_head_stride = step(Hq, q_head_stride);
  out_token_stride = step(T, out_token_stride);
  out_head_stride = step(Hq, out_head_stride);
  if ((rc = check_pages(k_pages, es, k_page_stride, k_slot_stride, k_pages_head_stride, page_size)) ||
      (rc = check_pages(v_pages, es, v_page_stride, v_slot_stride, v_pages_head_stride, page_size)))
    return rc;
  if (!aligned(q, 16) || !aligned(out, 16) || q_token_stride % 8 || q_head_stride % 8 || out_token_stride % 8 ||
      out_head_stride % 8)
    return abi_fail(MDS_ERR_UNSUPPORTED, "q and out must be 16-byte aligned with strides that are multiples of 8 elements");
  Dim dims[2] = {{T, out_token_stride}, {Hq, out_head_stride}};
  if (q_token_stride < 0 || q_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0 || !disjoint(dims, D))
    return abi_fail(MDS_ERR_INVALID_ARG, "strides must be >= 0, and those of out keep its rows apart");
  if (!aligned(workspace, 256)) return abi_fail(MDS_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (T == 0 || max_q_len == 0) return abi_ok();
  const mds::AttnPlan p = mds::attn_plan(T, B, Hkv, Hq / Hkv, D, max_q_len, max_seq_len, window);
  if (workspace_bytes < p.total) return abi_fail(MDS_ERR_WORKSPACE, "workspace too small for paged attention");
  if ((long long)p.tiles * Hkv * p.n_chunks > 0x7FFFFFFFLL) return abi_fail(MDS_ERR_UNSUPPORTED, "too many work-groups");
  a.T = T;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.D = D;
  a.n_pages = n_pages;
  a.n_slots = n_slots;
  a.max_pages = max_pages;
  a.causal = causal;
  a.window = window;
  a.q = (const uint16_t*)q;
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_ps = k_page_stride * es;
  a.k_ts = k_slot_stride * es;
  a.k_hs = k_pages_head_stride * es;
  a.v_ps = v_page_stride * es;
  a.v_ts = v_slot_stride * es;
  a.v_hs = v_pages_head_stride * es;
  a.block_table = block_table;
  a.idx_map = idx_map;
  a.query_start = query_start;
  a.seq_lens = seq_lens;
  a.scale_log2 = scale * 0x1.715476p+0f;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.out = (uint16_t*)out;
  a.o_ts = out_token_stride;
  a.o_hs = out_head_stride;
  a.lse = lse;
  a.tiles = p.tiles;
  a.per_req = p.per_req;
  a.by_length = p.by_length;
  a.chunk = p.chunk;
  a.n_chunks = p.n_chunks;
  a.part_o = (float*)((unsigned char*)workspace + p.part_o);
  a.part_ml = (float2*)((unsigned char*)workspace + p.part_ml);
  a.status = (uint32_t*)workspace;
  const hipError_t e = mds::launch_paged_attention(a, p, (hipStream_t)stream);
  return e == hipSuccess ? abi_ok() : hip_fail(e);
}

int mds_call_packed(int call, const int64_t* a, int n, void* stream) {
  // the calls' argument types: i int, l int64, p pointer, z size, f float
  static const char* const kTypes[] = {"iiiiiipppippppppppppppp", "iiipllpllppiiillllllpppp",
                                       "iiiiipllppiiillllllpiipppilfiipppllppz", "iiiiplpppillpz"};
  if (call < 0 || call > MDS_PACKED_LM_HEAD_FP8) return abi_fail(MDS_ERR_INVALID_ARG, "unknown call");
  if (!a) return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  const char* t = kTypes[call];
  for (int i = 0; i < n || t[i]; ++i) {
    if (i >= n || !t[i]) return abi_fail(MDS_ERR_INVALID_ARG, "wrong number of arguments");
    if ((t[i] == 'i' && a[i] != (int)a[i]) || (t[i] == 'z' && a[i] < 0))
      return abi_fail(MDS_ERR_INVALID_ARG, "an integer is out of its type's range");
  }
  auto real = [](int64_t x) {
    double d;
    static_assert(sizeof d == sizeof x, "8 bytes");
    __builtin_memcpy(&d, &x, sizeof d);
    return (float)d;
  };
  switch (call) {
    case MDS_PACKED_PAGE_TABLES:
      return mds_kv_page_tables((int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)a[4], (int)a[5],
                                (const int32_t*)a[6], (const int32_t*)a[7], (const int32_t*)a[8], (int)a[9],
                                (const int32_t*)a[10], (int32_t*)a[11], (const int32_t*)a[12], (int32_t*)a[13],
                                (const int32_t*)a[14], (int32_t*)a[15], (int32_t*)a[16], (int64_t*)a[17],
                                (int64_t*)a[18], (int32_t*)a[19], (int32_t*)a[20], (int32_t*)a[21],
                                (uint32_t*)a[22], stream);
    case MDS_PACKED_APPEND:
      return mds_kv_append((int)a[0], (int)a[1], (int)a[2], (const void*)a[3], a[4], a[5], (const void*)a[6], a[7],
                           a[8], (void*)a[9], (void*)a[10], (int)a[11], (int)a[12], (int)a[13], a[14], a[15], a[16],
                           a[17], a[18], a[19], (const int64_t*)a[20], (const float*)a[21], (const float*)a[22],
                           (uint32_t*)a[23], stream);
    case MDS_PACKED_ATTENTION:
      return mds_paged_attention((int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)a[4], (const void*)a[5], a[6],
                                 a[7], (const void*)a[8], (const void*)a[9], (int)a[10], (int)a[11], (int)a[12],
                                 a[13], a[14], a[15], a[16], a[17], a[18], (const int32_t*)a[19], (int)a[20],
                                 (int)a[21], (const int32_t*)a[22], (const int32_t*)a[23], (const int32_t*)a[24],
                                 (int)a[25], a[26], real(a[27]), (int)a[28], (int)a[29], (const float*)a[30],
                                 (const float*)a[31], (void*)a[32], a[33], a[34], (float*)a[35], (void*)a[36],
                                 (size_t)a[37], stream);
    default:
      return mds_lm_head_fp8((int)a[0], (int)a[1], (int)a[2], (int)a[3], (const void*)a[4], a[5], (const void*)a[6],
                             (const float*)a[7], (void*)a[8], (int)a[9], a[10], a[11], (void*)a[12],
                             (size_t)a[13], stream);
  }
}

}  // extern "C"
