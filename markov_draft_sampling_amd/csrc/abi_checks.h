// Checks of the serving entry points' arguments on the host, shared by their
// files (abi_serve.hip, abi_layer.hip).
#pragma once

#include "../../include/mds.h"
#include "mds_serve.h"

namespace mds {
namespace abi {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline int hip_fail(hipError_t e) { return abi_fail(MDS_ERR_HIP, hipGetErrorString(e)); }

// A launch's threads are counted in 32 bits.
inline bool launchable(int threads, long long groups) { return groups < ((1LL << 32) + threads - 1) / threads; }

// A dimension of one element is never stepped along: its stride may be anything, and counts as 0.
inline int64_t step(int64_t n, int64_t stride) { return n <= 1 ? 0 : stride; }

// log2 of a page size, or -1
inline int page_log2(int page_size) {
  for (int s = 4; s <= 10; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

inline int check_page(int page_size, int n_pages, int* lg) {
  *lg = page_log2(page_size);
  if (page_size < 1 || n_pages < 1) return abi_fail(MDS_ERR_INVALID_ARG, "page_size and n_pages must be >= 1");
  if (*lg < 0) return abi_fail(MDS_ERR_UNSUPPORTED, "page_size must be a power of two in [16, 1024]");
  if ((long long)n_pages * page_size > 0x7FFFFFFFFFLL) return abi_fail(MDS_ERR_INVALID_ARG, "the cache is too large");
  return MDS_OK;
}

// [n_pages][P][Hkv][D] pages of `es`-byte elements with a unit last stride: 16-byte aligned, strides that
// are whole 16-byte pieces and fit the kernels' 32-bit offsets inside a page
inline int check_pages(const void* p, int es, int64_t ps, int64_t ts, int64_t hs, int page_size) {
  const int64_t e16 = 16 / es;
  if (!aligned(p, 16) || ps % e16 || ts % e16 || hs % e16)
    return abi_fail(MDS_ERR_UNSUPPORTED, "pages must be 16-byte aligned with strides that are multiples of 16 bytes");
  if (ps < 0 || ts < 0 || hs < 0 || ps > (int64_t{1} << 40) || ts > (1 << 30) || hs > (int64_t{1} << 40) ||
      ts * es * page_size >= (1LL << 31))
    return abi_fail(MDS_ERR_INVALID_ARG, "page strides must be >= 0, and a page's slots span less than 2 GiB");
  return MDS_OK;
}

inline int check_heads(int Hkv, int D) {
  if (Hkv < 1 || Hkv > 1024) return abi_fail(MDS_ERR_INVALID_ARG, "key heads must be in [1, 1024]");
  if (D < 1) return abi_fail(MDS_ERR_INVALID_ARG, "the head dimension must be >= 1");
  return MDS_OK;
}

inline constexpr int kMaxBatch = 65535;
inline constexpr int kMaxSlots = 1 << 17;

inline int check_batch(int B, int n_slots, int max_pages, int lg, bool idx) {
  if (B < 1 || B > kMaxBatch) return abi_fail(MDS_ERR_INVALID_ARG, "B must be in [1, 65535]");
  if (n_slots < 1 || n_slots > kMaxSlots) return abi_fail(MDS_ERR_INVALID_ARG, "n_slots must be in [1, 2^17]");
  if (!idx && n_slots < B) return abi_fail(MDS_ERR_INVALID_ARG, "without idx_map: n_slots >= B");
  if (max_pages < 1 || ((long long)max_pages << lg) >= (1LL << 30))
    return abi_fail(MDS_ERR_INVALID_ARG, "max_pages must be >= 1 and max_pages * page_size below 2^30");
  return MDS_OK;
}

inline int check_cache_dtype(int dt) {
  if (dt != MDS_BF16 && dt != MDS_E4M3) return abi_fail(MDS_ERR_INVALID_ARG, "cache dtype must be MDS_BF16 or MDS_E4M3");
  return MDS_OK;
}

inline int check_attention(int T, int B, int Hq, int Hkv, int D, int max_q_len, int64_t max_seq_len, int window) {
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

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  return (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

inline int check_lm_head_matrix(int V, int H) {
  if (V < 2 || V >= (1 << 24)) return abi_fail(MDS_ERR_INVALID_ARG, "V must be in [2, 2^24)");
  if (H < 128 || H > (1 << 16)) return abi_fail(MDS_ERR_INVALID_ARG, "H must be in [128, 65536]");
  if (H % 128) return abi_fail(MDS_ERR_UNSUPPORTED, "H must be a multiple of 128");
  return MDS_OK;
}

inline int check_lm_head_rows(int B, int K, int* rows) {
  if (B < 1 || B > kMaxBatch) return abi_fail(MDS_ERR_INVALID_ARG, "B must be in [1, 65535]");
  if (K < 1 || K > 64) return abi_fail(MDS_ERR_INVALID_ARG, "K must be in [1, 64]");
  *rows = B * K;
  return MDS_OK;
}

// Keys that may be seen behind the window, as far as the plan of the work goes: in whole blocks of 64, as the window is.
inline int sinks_window(int window, int sinks) {
  if (window <= 0 || sinks <= 0) return window;
  const int64_t n = (int64_t)window + ((sinks + 63) & ~63);
  return n > (1 << 30) ? 1 << 30 : (int)n;
}

inline int check_sinks(int sinks) {
  if (sinks < 0 || sinks > (1 << 29)) return abi_fail(MDS_ERR_INVALID_ARG, "sinks must be in [0, 2^29]");
  return MDS_OK;
}

}  // namespace abi
}  // namespace mds
