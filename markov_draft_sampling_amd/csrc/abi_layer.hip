// extern "C" entry points of a layer's step between its projections and the
// logits (norm and rotation, with the append; the 4-bit LM head): argument
// checks on the host, then the kernels on the caller's stream. See
// include/mds.h for the contract.
#include <math.h>

#include "abi_checks.h"

using namespace mds::abi;
using mds::abi_fail;
using mds::abi_ok;

namespace {

int check_rows(const void* p, int64_t ts, int64_t hs) {
  if (!aligned(p, 16) || ts % 8 || hs % 8)
    return abi_fail(MDS_ERR_UNSUPPORTED, "rows must be 16-byte aligned with strides that are multiples of 8 elements");
  if (ts < 0 || hs < 0) return abi_fail(MDS_ERR_INVALID_ARG, "strides must be >= 0");
  return MDS_OK;
}

int check_out(const void* p, int T, int64_t ts, int H, int64_t hs, int D) {
  const int rc = check_rows(p, ts, hs);
  if (rc) return rc;
  Dim d[2] = {{T, ts}, {H, hs}};
  if (!disjoint(d, D)) return abi_fail(MDS_ERR_INVALID_ARG, "strides of an output make its rows overlap");
  return MDS_OK;
}

// The sizes of both rotations
int check_rope_sizes(int T, int Hq, int Hk, int D, int per_key_head) {
  int rc;
  if (T < 0 || T > (1 << 24)) return abi_fail(MDS_ERR_INVALID_ARG, "T must be in [0, 2^24]");
  if ((rc = check_heads(Hk, D))) return rc;
  if (Hq < 1 || Hq > 1024) return abi_fail(MDS_ERR_INVALID_ARG, "query heads must be in [1, 1024]");
  if (D % 16 || D > 256) return abi_fail(MDS_ERR_UNSUPPORTED, "the head dimension must be a multiple of 16, at most 256");
  const int heads = Hq + per_key_head * Hk;
  if ((long long)T * heads >= 0x7FFFFFFFLL || !launchable(256, ((long long)T * mds::rope_plan(T, heads, D).per_token + 3) / 4))
    return abi_fail(MDS_ERR_UNSUPPORTED, "too many heads in one call");
  return MDS_OK;
}

// What both calls have in common; fills a
int check_rope(mds::RopeArgs& a, int T, int Hq, int Hk, int D, int R, const void* q, int64_t q_ts, int64_t q_hs,
               const void* k, int64_t k_ts, int64_t k_hs, const int64_t* positions, const double* inv_freq,
               const void* q_weight, const void* k_weight, float eps, double rope_scale, int interleaved, void* q_out,
               int64_t qo_ts, int64_t qo_hs, int per_key_head) {
  int rc;
  if ((rc = check_rope_sizes(T, Hq, Hk, D, per_key_head))) return rc;
  if (R < 0 || R > D) return abi_fail(MDS_ERR_INVALID_ARG, "the rotated part must be in [0, D]");
  if (R % 16) return abi_fail(MDS_ERR_UNSUPPORTED, "the rotated part must be a multiple of 16");
  if ((T && (!q || !k || !q_out || !positions)) || (R && !inv_freq))
    return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!(eps >= 0.0f) || !(eps < 1e30f)) return abi_fail(MDS_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!(fabs(rope_scale) < 1e30)) return abi_fail(MDS_ERR_INVALID_ARG, "rope_scale must be finite");
  if (interleaved != 0 && interleaved != 1) return abi_fail(MDS_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(positions, 8) || !aligned(inv_freq, 8))
    return abi_fail(MDS_ERR_INVALID_ARG, "weights must be 16-byte aligned, positions and frequencies 8-byte aligned");
  a.q_ts = step(T, q_ts);
  a.q_hs = step(Hq, q_hs);
  a.k_ts = step(T, k_ts);
  a.k_hs = step(Hk, k_hs);
  a.qo_ts = step(T, qo_ts);
  a.qo_hs = step(Hq, qo_hs);
  if ((rc = check_rows(q, a.q_ts, a.q_hs)) || (rc = check_rows(k, a.k_ts, a.k_hs)) ||
      (rc = check_out(q_out, T, a.qo_ts, Hq, a.qo_hs, D)))
    return rc;
  a.T = T;
  a.Hq = Hq;
  a.Hk = Hk;
  a.D = D;
  a.R = R;
  a.interleaved = interleaved;
  a.q = (const uint16_t*)q;
  a.k = (const uint16_t*)k;
  a.positions = (const long long*)positions;
  a.inv_freq = inv_freq;
  a.q_weight = (const uint16_t*)q_weight;
  a.k_weight = (const uint16_t*)k_weight;
  a.eps = eps;
  a.rope_scale = rope_scale;
  a.q_out = (uint16_t*)q_out;
  return MDS_OK;
}

size_t mx_code_bytes(int V, int H) { return (size_t)((V + 15) / 16) * 8 * H; }
size_t mx_scale_bytes(int V, int H) { return (size_t)((V + 15) / 16) * 256 * ((H + 511) / 512); }

// A matrix whose tiles are made or read back in one launch: a work-group for 16 rows and 512 columns
int check_mx_matrix(int V, int H) {
  const int rc = check_lm_head_matrix(V, H);
  if (rc) return rc;
  if (!launchable(256, (long long)((V + 15) / 16) * ((H + 511) / 512))) return abi_fail(MDS_ERR_UNSUPPORTED, "the matrix is too large");
  return MDS_OK;
}

int check_mx_tiled(int V, int H, const void* tiled, size_t tiled_bytes, const void* tiled_scales, size_t scale_bytes) {
  if (!tiled || !tiled_scales) return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(tiled, 16) || !aligned(tiled_scales, 4))
    return abi_fail(MDS_ERR_INVALID_ARG, "tiled codes must be 16-byte aligned, their scales 4-byte aligned");
  if (tiled_bytes < mx_code_bytes(V, H) || scale_bytes < mx_scale_bytes(V, H))
    return abi_fail(MDS_ERR_INVALID_ARG, "tiled codes or scales are too small");
  if (overlap(tiled, mx_code_bytes(V, H), tiled_scales, mx_scale_bytes(V, H)))
    return abi_fail(MDS_ERR_INVALID_ARG, "tiled codes and scales overlap");
  return MDS_OK;
}

bool meets_tiled(const void* p, size_t n, int V, int H, const void* tiled, const void* tiled_scales) {
  return overlap(p, n, tiled, mx_code_bytes(V, H)) || overlap(p, n, tiled_scales, mx_scale_bytes(V, H));
}

}  // namespace

extern "C" {

int mds_qk_norm_rope(int T, int Hq, int Hkv, int D, int R, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                     const void* k, int64_t k_token_stride, int64_t k_head_stride, const int64_t* positions,
                     const double* inv_freq, const void* q_weight, const void* k_weight, float eps, double rope_scale,
                     int interleaved, void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                     int64_t k_out_token_stride, int64_t k_out_head_stride, void* stream) {
  int rc;
  mds::RopeArgs a{};
  if ((rc = check_rope(a, T, Hq, Hkv, D, R, q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, positions,
                       inv_freq, q_weight, k_weight, eps, rope_scale, interleaved, q_out, q_out_token_stride,
                       q_out_head_stride, 1)))
    return rc;
  if (T && !k_out) return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  a.ko_ts = step(T, k_out_token_stride);
  a.ko_hs = step(Hkv, k_out_head_stride);
  if ((rc = check_out(k_out, T, a.ko_ts, Hkv, a.ko_hs, D))) return rc;
  if (T == 0) return abi_ok();
  a.k_out = (uint16_t*)k_out;
  const hipError_t e = mds::launch_rope(a, (hipStream_t)stream);
  return e == hipSuccess ? abi_ok() : hip_fail(e);
}

int mds_qk_norm_rope_append(int T, int Hq, int Hkv, int D, int R, const void* q, int64_t q_token_stride,
                            int64_t q_head_stride, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                            const void* v, int64_t v_token_stride, int64_t v_head_stride, const int64_t* positions,
                            const double* inv_freq, const void* q_weight, const void* k_weight, float eps,
                            double rope_scale, int interleaved, void* q_out, int64_t q_out_token_stride,
                            int64_t q_out_head_stride, void* k_pages, void* v_pages, int cache_dtype, int page_size,
                            int n_pages, int64_t k_page_stride, int64_t k_slot_stride, int64_t k_pages_head_stride,
                            int64_t v_page_stride, int64_t v_slot_stride, int64_t v_pages_head_stride,
                            const int64_t* slot_map, const float* k_scale, const float* v_scale, uint32_t* status,
                            void* stream) {
  int rc;
  mds::RopeArgs a{};
  if ((rc = check_rope(a, T, Hq, Hkv, D, R, q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, positions,
                       inv_freq, q_weight, k_weight, eps, rope_scale, interleaved, q_out, q_out_token_stride,
                       q_out_head_stride, 2)) ||
      (rc = check_cache_dtype(cache_dtype)) || (rc = check_page(page_size, n_pages, &a.page_log2)))
    return rc;
  a.e4m3 = cache_dtype == MDS_E4M3;
  if (!k_pages || !v_pages || (T && (!v || !slot_map)) || (a.e4m3 && (!k_scale || !v_scale)))
    return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  const int es = a.e4m3 ? 1 : 2;
  a.v_ts = step(T, v_token_stride);
  a.v_hs = step(Hkv, v_head_stride);
  a.ps[0] = step(n_pages, k_page_stride);
  a.ts[0] = k_slot_stride;
  a.hs[0] = step(Hkv, k_pages_head_stride);
  a.ps[1] = step(n_pages, v_page_stride);
  a.ts[1] = v_slot_stride;
  a.hs[1] = step(Hkv, v_pages_head_stride);
  if ((rc = check_rows(v, a.v_ts, a.v_hs)) || (rc = check_pages(k_pages, es, a.ps[0], a.ts[0], a.hs[0], page_size)) ||
      (rc = check_pages(v_pages, es, a.ps[1], a.ts[1], a.hs[1], page_size)))
    return rc;
  for (int i = 0; i < 2; ++i) {
    Dim d[3] = {{n_pages, a.ps[i]}, {page_size, a.ts[i]}, {Hkv, a.hs[i]}};
    if (!disjoint(d, D)) return abi_fail(MDS_ERR_INVALID_ARG, "page strides make rows overlap");
  }
  if (T == 0) return abi_ok();
  a.n_pages = n_pages;
  a.v = (const uint16_t*)v;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.slot_map = (const long long*)slot_map;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.status = status;
  const hipError_t e = mds::launch_rope(a, (hipStream_t)stream);
  return e == hipSuccess ? abi_ok() : hip_fail(e);
}

int mds_debug_qk_norm_rope_plan(int T, int Hq, int Hkv, int D, int append, int32_t* out) {
  int rc;
  if ((rc = check_rope_sizes(T, Hq, Hkv, D, append ? 2 : 1))) return rc;
  if (!out) return abi_fail(MDS_ERR_INVALID_ARG, "out is NULL");
  const mds::RopePlan p = mds::rope_plan(T, Hq + (append ? 2 : 1) * Hkv, D);
  out[0] = p.lanes;
  out[1] = p.heads;
  return abi_ok();
}

int mds_lm_head_mxfp4_bytes(int V, int H, size_t* code_bytes, size_t* scale_bytes) {
  int rc;
  if ((rc = check_lm_head_matrix(V, H))) return rc;
  if (!code_bytes || !scale_bytes) return abi_fail(MDS_ERR_INVALID_ARG, "code_bytes or scale_bytes is NULL");
  *code_bytes = mx_code_bytes(V, H);
  *scale_bytes = mx_scale_bytes(V, H);
  return abi_ok();
}

int mds_tile_lm_head_mxfp4(int V, int H, const void* codes, const void* scales, void* tiled, size_t tiled_bytes,
                           void* tiled_scales, size_t tiled_scale_bytes, void* stream) {
  int rc;
  if ((rc = check_mx_matrix(V, H)) || (rc = check_mx_tiled(V, H, tiled, tiled_bytes, tiled_scales, tiled_scale_bytes)))
    return rc;
  if (!codes || !scales) return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(codes, 16)) return abi_fail(MDS_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  if (meets_tiled(codes, (size_t)V * (H / 2), V, H, tiled, tiled_scales) ||
      meets_tiled(scales, (size_t)V * (H / 32), V, H, tiled, tiled_scales))
    return abi_fail(MDS_ERR_INVALID_ARG, "the matrix and its tiles overlap");
  const hipError_t e = mds::launch_tile_mx(V, H, (const uint8_t*)codes, (const uint8_t*)scales, (uint8_t*)tiled,
                                           (uint8_t*)tiled_scales, (hipStream_t)stream);
  return e == hipSuccess ? abi_ok() : hip_fail(e);
}

int mds_quantize_lm_head_mxfp4(int V, int H, const void* lm_head, void* tiled, size_t tiled_bytes, void* tiled_scales,
                               size_t tiled_scale_bytes, void* stream) {
  int rc;
  if ((rc = check_mx_matrix(V, H)) || (rc = check_mx_tiled(V, H, tiled, tiled_bytes, tiled_scales, tiled_scale_bytes)))
    return rc;
  if (!lm_head) return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(lm_head, 16)) return abi_fail(MDS_ERR_INVALID_ARG, "lm_head must be 16-byte aligned");
  if (meets_tiled(lm_head, (size_t)V * H * 2, V, H, tiled, tiled_scales))
    return abi_fail(MDS_ERR_INVALID_ARG, "the matrix and its tiles overlap");
  const hipError_t e = mds::launch_quantize_mx(V, H, (const uint16_t*)lm_head, (uint8_t*)tiled, (uint8_t*)tiled_scales,
                                               (hipStream_t)stream);
  return e == hipSuccess ? abi_ok() : hip_fail(e);
}

int mds_unpack_lm_head_mxfp4(int V, int H, const void* tiled, const void* tiled_scales, void* lm_head, void* stream) {
  int rc;
  if ((rc = check_mx_matrix(V, H)) || (rc = check_mx_tiled(V, H, tiled, mx_code_bytes(V, H), tiled_scales, mx_scale_bytes(V, H))))
    return rc;
  if (!lm_head) return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(lm_head, 16)) return abi_fail(MDS_ERR_INVALID_ARG, "lm_head must be 16-byte aligned");
  if (meets_tiled(lm_head, (size_t)V * H * 2, V, H, tiled, tiled_scales))
    return abi_fail(MDS_ERR_INVALID_ARG, "the matrix and its tiles overlap");
  const hipError_t e = mds::launch_unpack_mx(V, H, (const uint8_t*)tiled, (const uint8_t*)tiled_scales, (uint16_t*)lm_head,
                                             (hipStream_t)stream);
  return e == hipSuccess ? abi_ok() : hip_fail(e);
}

int mds_lm_head_mxfp4(int B, int K, int V, int H, const void* hidden, int64_t hidden_row_stride, const void* lm_head,
                      const void* scales, void* out, int out_dtype, int64_t out_req_stride, int64_t out_step_stride,
                      void* stream) {
  int rc, rows;
  if ((rc = check_lm_head_rows(B, K, &rows)) || (rc = check_lm_head_matrix(V, H))) return rc;
  if (!hidden || !lm_head || !scales || !out) return abi_fail(MDS_ERR_INVALID_ARG, "a required pointer is NULL");
  if (out_dtype != MDS_F32 && out_dtype != MDS_BF16) return abi_fail(MDS_ERR_INVALID_ARG, "out dtype must be MDS_F32 or MDS_BF16");
  if (rows == 1) hidden_row_stride = H;
  if (hidden_row_stride < H || hidden_row_stride % 8)
    return abi_fail(MDS_ERR_INVALID_ARG, "hidden_row_stride must be a multiple of 8, at least H");
  // (112 rows are addressed with 32-bit offsets)
  if (hidden_row_stride > (1 << 22)) return abi_fail(MDS_ERR_UNSUPPORTED, "hidden_row_stride must be at most 2^22");
  if ((int64_t)((V + 63) / 64) * ((rows + 15) / 16) > (1 << 30)) return abi_fail(MDS_ERR_UNSUPPORTED, "too many work-groups");
  const mds::LmHeadMxPlan plan = mds::lm_head_mx_plan(rows, V);
  if (!plan.few && !launchable(256, (int64_t)(plan.v_tiles + 7) / 8 * 8 * plan.row_tiles))
    return abi_fail(MDS_ERR_UNSUPPORTED, "too many work-groups");
  if (!aligned(hidden, 16) || !aligned(lm_head, 16) || !aligned(scales, 4))
    return abi_fail(MDS_ERR_INVALID_ARG, "hidden and lm_head must be 16-byte aligned, scales 4-byte aligned");
  out_req_stride = step(B, out_req_stride);
  out_step_stride = step(K, out_step_stride);
  Dim dims[2] = {{B, out_req_stride}, {K, out_step_stride}};
  if (out_req_stride < 0 || out_step_stride < 0 || !disjoint(dims, V))
    return abi_fail(MDS_ERR_INVALID_ARG, "out strides make rows overlap or are shorter than V");
  mds::LmHeadMxArgs a{};
  a.M = rows;
  a.K = K;
  a.V = V;
  a.H = H;
  a.hidden = (const uint16_t*)hidden;
  a.hidden_rs = hidden_row_stride;
  a.w = (const uint8_t*)lm_head;
  a.w_scale = (const uint8_t*)scales;
  a.out = out;
  a.out_rs = out_req_stride;
  a.out_ss = out_step_stride;
  a.out_bf16 = out_dtype == MDS_BF16;
  a.vec_out = aligned(out, a.out_bf16 ? 8 : 16) && out_req_stride % 4 == 0 && out_step_stride % 4 == 0;
  const hipError_t e = mds::launch_lm_head_mx(a, (hipStream_t)stream);
  return e == hipSuccess ? abi_ok() : hip_fail(e);
}

int mds_debug_lm_head_mxfp4_plan(int B, int K, int V, int H, int32_t* out) {
  int rc, rows;
  if ((rc = check_lm_head_rows(B, K, &rows)) || (rc = check_lm_head_matrix(V, H))) return rc;
  if (!out) return abi_fail(MDS_ERR_INVALID_ARG, "out is NULL");
  const mds::LmHeadMxPlan p = mds::lm_head_mx_plan(rows, V);
  out[0] = p.few;
  out[1] = p.height;
  out[2] = p.nbw;
  return abi_ok();
}

}  // extern "C"
