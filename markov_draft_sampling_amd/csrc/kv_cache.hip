// The paged key/value cache's bookkeeping and writes: page tables, slot map
// and positions of a step's new tokens, and the append of their keys and
// values.
//
// Page tables. With P tokens a page, request b on state slot s holds
// held[s] pages for a context of ctx = kv_len[s] + advance[b] + advance_add
// tokens and is given n = chunk_len[b] new ones: it needs
// max(0, ceil((ctx + n) / P) - held[s]) pages more. Where each request's
// tokens and pages start are two prefix sums over the batch (held in 64 bits),
// so one work-group does them: the whole plan is a few KB and bound by the
// latency of its dependent loads (idx_map, then the slot's state, then the
// free list), not by bytes. Tokens are then filled in by the same work-group
// for small steps, by a second launch for large ones.
//
// Append. Every element is read once and written once, 16 bytes a lane
// (two reads and one write for an 8-bit cache): bound by HBM for long
// prompts, by the launch for a decoding step.
#include "mds_device.h"
#include "mds_internal.h"

namespace mds {
namespace {

constexpr int kPlanThreads = 1024;
// Tokens up to which the plan's own work-group writes positions and slots:
// 4096 is four tokens a thread; past that one CU's stores cost more than a launch.
constexpr int kPlanFillTokens = 4096;

// Exclusive prefix sums of two values over the work-group, and the totals.
// s_w: [2][16] wave totals.
__device__ __forceinline__ void block_scan2(long long a, long long b, long long& ea, long long& eb, long long& ta,
                                            long long& tb, long long (*s_w)[16]) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  long long ia = a, ib = b;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const long long ua = __shfl_up(ia, off), ub = __shfl_up(ib, off);
    if (lane >= off) {
      ia += ua;
      ib += ub;
    }
  }
  __syncthreads();  // the wave totals of an earlier scan have been read
  if (lane == 63) {
    s_w[0][w] = ia;
    s_w[1][w] = ib;
  }
  __syncthreads();
  ea = ia - a;
  eb = ib - b;
  ta = tb = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / 64; ++i) {
    const long long x = s_w[0][i], y = s_w[1][i];
    if (i < w) {
      ea += x;
      eb += y;
    }
    ta += x;
    tb += y;
  }
}

// Position and slot of token t: its request is the first whose end is past t.
__device__ __forceinline__ void fill_token(const PageTableArgs& a, int t) {
  const int total = a.query_start[a.B];
  if (t >= total) {
    a.positions[t] = 0;
    a.slot_map[t] = -1;
    return;
  }
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.query_start[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  const int s = a.idx_map ? a.idx_map[lo] : lo;
  const long long pos = (long long)a.kv_len_out[s] + (t - a.query_start[lo]);
  a.positions[t] = pos;
  long long slot = -1;
  if (a.seq_lens[lo] > 0) {  // 0: the request was refused
    const int pg = a.block_table[(size_t)s * a.max_pages + (pos >> a.page_log2)];
    if (pg >= 0 && pg < a.n_pages)
      slot = ((long long)pg << a.page_log2) + (pos & ((1 << a.page_log2) - 1));
    else
      set_status(a.status, kStatusBadPage);
  }
  a.slot_map[t] = slot;
}

__global__ __launch_bounds__(kPlanThreads) void page_plan_kernel(PageTableArgs a, int fill) {
  extern __shared__ uint32_t s_bits[];  // [2][words]: slots seen, slots seen twice
  __shared__ long long s_w[2][16];
  __shared__ long long s_at[kPlanThreads];  // where a request's released or new pages start
  __shared__ int s_n[kPlanThreads], s_held[kPlanThreads], s_slot[kPlanThreads];
  __shared__ long long s_taken;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int words = (a.n_slots + 31) >> 5;
  const int P = 1 << a.page_log2;
  int bad = 0;
  if (tid == 0) s_taken = 0;

  // a slot that two rows name belongs to neither: both are padding
  if (a.idx_map) {
    for (int i = tid; i < 2 * words; i += kPlanThreads) s_bits[i] = 0;
    __syncthreads();
    for (int b = tid; b < a.B; b += kPlanThreads) {
      const int s = a.idx_map[b];
      if (s < 0) continue;
      if (s >= a.n_slots) {
        bad |= kStatusBadIndex;
        continue;
      }
      if (atomicOr(&s_bits[s >> 5], 1u << (s & 31)) & (1u << (s & 31))) {
        atomicOr(&s_bits[words + (s >> 5)], 1u << (s & 31));
        bad |= kStatusBadIndex;
      }
    }
    __syncthreads();
  }
  auto live_slot = [&](int b) {
    if (b >= a.B) return -1;
    if (!a.idx_map) return b;
    const int s = a.idx_map[b];
    if (s < 0 || s >= a.n_slots || (s_bits[words + (s >> 5)] >> (s & 31) & 1u)) return -1;
    return s;
  };
  auto clamp_held = [&](int h) {
    if (h < 0 || h > a.max_pages) {
      bad |= kStatusBadIndex;
      return h < 0 ? 0 : a.max_pages;
    }
    return h;
  };

  // pages of finished requests go to the end of the free list, in batch order
  long long count = a.free_count[0];
  if (count < 0 || count > a.n_pages) {
    bad |= kStatusBadIndex;
    count = count < 0 ? 0 : a.n_pages;
  }
  long long back = 0;
  int any = 0;
  for (int b = tid; b < a.B; b += kPlanThreads) any |= a.chunk_len[b] < 0;
  if (__syncthreads_or(any)) {
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
      const int b = b0 + tid;
      const int s = live_slot(b);
      const bool done = s >= 0 && a.chunk_len[b] < 0;
      const int held = done ? clamp_held(a.pages_held[s]) : 0;
      long long e, e2, t, t2;
      block_scan2(held, 0, e, e2, t, t2, s_w);
      s_at[tid] = back + e;
      s_n[tid] = held;
      s_slot[tid] = s;
      __syncthreads();
      const int m = min(kPlanThreads, a.B - b0);
      for (int r = w; r < m; r += kPlanThreads / 64) {
        const int n = s_n[r];
        const int32_t* row = a.block_table + (size_t)(n ? s_slot[r] : 0) * a.max_pages;
        for (int i = lane; i < n; i += 64) {
          const long long at = count + s_at[r] + i;
          if (at < a.n_pages)
            a.free_list[at] = row[i];
          else
            bad |= kStatusBadIndex;
        }
      }
      __syncthreads();
      if (done) {
        a.pages_held_out[s] = 0;
        a.kv_len_out[s] = 0;
        a.seq_lens[b] = 0;
      }
      back += t;
    }
  }
  const long long avail = min(count + back, (long long)a.n_pages);
  __threadfence_block();
  __syncthreads();

  long long tok0 = 0, need0 = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const int s = live_slot(b);
    const int n_in = b < a.B ? a.chunk_len[b] : 0;
    const bool here = s >= 0 && n_in >= 0;
    const int n = here ? n_in : 0;
    long long ctx = 0;
    int held = 0;
    if (here) {
      ctx = (long long)a.kv_len[s] + (a.advance ? (long long)a.advance[b] + a.advance_add : 0);
      if (ctx < 0 || ctx > 0x7FFFFFFF) {
        bad |= kStatusBadIndex;
        ctx = ctx < 0 ? 0 : 0x7FFFFFFF;
      }
      held = clamp_held(a.pages_held[s]);
    }
    const long long want = (ctx + n + P - 1) >> a.page_log2;
    long long te, ne, tt, nt, dummy0, dummy1;
    block_scan2(n, 0, te, dummy0, tt, dummy1, s_w);
    const long long t_end = tok0 + te + n;
    const bool fits = here && want <= a.max_pages && t_end <= a.max_tokens;
    const long long need = fits && want > held ? want - held : 0;
    block_scan2(need, 0, ne, dummy0, nt, dummy1, s_w);
    const long long from = need0 + ne;
    const bool granted = fits && (need == 0 || from + need <= avail);
    if (here && !granted) bad |= kStatusNoPages;
    if (b < a.B) {
      if (b == 0) a.query_start[0] = 0;
      a.query_start[b + 1] = (int)min(t_end, (long long)a.max_tokens);
      if (n_in >= 0 || s < 0) a.seq_lens[b] = granted ? (int)(ctx + n) : 0;
      if (here) {
        a.kv_len_out[s] = (int)ctx;
        a.pages_held_out[s] = held + (granted ? (int)need : 0);
      }
    }
    if (granted && need) atomicMax((unsigned long long*)&s_taken, (unsigned long long)(from + need));
    s_at[tid] = from;
    s_n[tid] = granted ? (int)need : 0;
    s_held[tid] = held;
    s_slot[tid] = s;
    const int more = __syncthreads_or(granted && need > 2);
    // new page i of the step is the free list's i-th from its end
    if (!more) {
      for (int i = 0; i < s_n[tid]; ++i)
        a.block_table[(size_t)s * a.max_pages + held + i] = a.free_list[avail - 1 - from - i];
    } else {
      const int m = min(kPlanThreads, a.B - b0);
      for (int r = w; r < m; r += kPlanThreads / 64) {
        const int k = s_n[r];
        int32_t* row = a.block_table + (size_t)(k ? s_slot[r] : 0) * a.max_pages + s_held[r];
        for (int i = lane; i < k; i += 64) row[i] = a.free_list[avail - 1 - s_at[r] - i];
      }
    }
    __syncthreads();
    tok0 += tt;
    need0 += nt;
  }
  if (tid == 0) a.free_count_out[0] = (int)(avail - s_taken);
  if (bad && a.status) atomicOr(a.status, (uint32_t)bad);
  if (!fill) return;
  __threadfence_block();
  __syncthreads();
  for (int t = tid; t < a.max_tokens; t += kPlanThreads) fill_token(a, t);
}

__global__ __launch_bounds__(256) void page_fill_kernel(PageTableArgs a) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t < a.max_tokens) fill_token(a, t);
}

// 8 bf16 -> 8 e4m3 codes: round to nearest even of the float32 quotient by
// the head's scale, past the largest value to the largest; NaN stays NaN.
__device__ __forceinline__ u32x2 quant8(u32x4 x, float scale) {
  uint32_t o[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t wd = x[h * 2 + (i >> 1)];
      const float y = __uint_as_float(i & 1 ? wd & 0xFFFF0000u : wd << 16) / scale;
      f[i] = y != y ? y : fminf(fmaxf(y, -448.0f), 448.0f);
    }
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    o[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], p, true);
  }
  return u32x2{o[0], o[1]};
}

// blockIdx.y: 0 keys, 1 values. A thread moves 8 elements (bf16 pages) or 16
// (e4m3 pages); consecutive threads run through a row's heads and columns.
template <bool E4M3>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a) {
  constexpr int EPT = E4M3 ? 16 : 8;
  const unsigned i = blockIdx.x * 256u + threadIdx.x;  // fewer than 2^31 pieces (checked on the host)
  const unsigned per_head = (unsigned)(a.D / EPT);
  const unsigned per_row = (unsigned)a.Hkv * per_head;
  const int t = (int)(i / per_row);
  if (t >= a.T) return;
  const unsigned r = i - (unsigned)t * per_row;
  const int h = (int)(r / per_head);
  const int c = (int)(r - (unsigned)h * per_head) * EPT;
  const long long slot = a.slot_map[t];
  if (slot < 0) return;
  const long long pg = slot >> a.page_log2;
  if (pg >= a.n_pages) {
    set_status(a.status, kStatusBadPage);
    return;
  }
  const long long in_pg = slot & ((1 << a.page_log2) - 1);
  const int kv = blockIdx.y;
  const uint16_t* src = (kv ? a.v : a.k) + t * a.src_ts[kv] + h * a.src_hs[kv] + c;
  char* dst = (char*)(kv ? a.v_pages : a.k_pages) +
              (pg * a.ps[kv] + in_pg * a.ts[kv] + h * a.hs[kv] + c) * (E4M3 ? 1 : 2);
  if constexpr (E4M3) {
    const float sc = (kv ? a.v_scale : a.k_scale)[h];
    const u32x2 lo = quant8(*(const u32x4*)src, sc), hi = quant8(*(const u32x4*)(src + 8), sc);
    *(u32x4*)dst = u32x4{lo[0], lo[1], hi[0], hi[1]};
  } else {
    *(u32x4*)dst = *(const u32x4*)src;
  }
}

}  // namespace

hipError_t launch_page_tables(const PageTableArgs& a, hipStream_t st) {
  const bool fill = a.max_tokens <= kPlanFillTokens;
  const size_t lds = a.idx_map ? (size_t)((a.n_slots + 31) / 32) * 8 : 0;
  hipLaunchKernelGGL(page_plan_kernel, dim3(1), dim3(kPlanThreads), lds, st, a, fill ? 1 : 0);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || fill) return e;
  hipLaunchKernelGGL(page_fill_kernel, dim3((a.max_tokens + 255) / 256), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t st) {
  const long long n = (long long)a.T * a.Hkv * (a.D / (a.e4m3 ? 16 : 8));
  const dim3 grid((unsigned)((n + 255) / 256), 2);
  if (a.e4m3)
    hipLaunchKernelGGL(kv_append_kernel<true>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(kv_append_kernel<false>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace mds
