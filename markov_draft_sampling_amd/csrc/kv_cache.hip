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
// free list), not by bytes: 32 requests of 8 tokens 4.8 us, 1024 requests with
// prompts and releases 21 us and 5 us for the tokens. Tokens are filled in by
// the same work-group for small steps, by a second launch for large ones.
//
// Append. Every element is read once and written once, 16 bytes a lane
// (two reads and one write for an 8-bit cache): bound by HBM for long
// prompts (16384 tokens of 8 heads of 128: 134 MB in 24.5 us, 5.5 TB/s), by the
// launch for a decoding step (3.8 us).
#include "mds_device.h"
#include "mds_serve.h"

namespace mds {
namespace {

// Tokens up to which the plan's own work-group writes positions and slots: past that one CU's stores cost more
// than a launch.
constexpr int kPlanFillTokens = 4096;
// Threads of the plan: 256 keep its barriers and scans short (32 requests of 8 tokens: 4.8 us a launch, 12.7 us with
// 1024 and scans through LDS); 1024 take large batches in fewer tiles.
constexpr int kPlanSmall = 256, kPlanLarge = 1024;

// Inclusive prefix sum over the wave (its total stays below 2^32): shifts within rows of 16 lanes, then the
// rows' last lanes broadcast to the rows behind them.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_add(uint32_t v) {
  return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v = dpp_add<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);  // lane 15 of rows 0 and 2 to rows 1 and 3
  return dpp_add<0x143, 0xC>(v);  // lane 31 to rows 2 and 3
}

// Exclusive prefix sum over the work-group, and the total, in 64 bits. s_w: a word per wave.
template <int NT>
__device__ __forceinline__ void block_scan(uint32_t a, long long& before, long long& total, uint32_t* s_w) {
  const int w = threadIdx.x >> 6;
  const uint32_t in = wave_scan(a);
  __syncthreads();  // the wave totals of an earlier scan have been read
  if ((threadIdx.x & 63) == 63) s_w[w] = in;
  __syncthreads();
  before = (long long)in - a;
  total = 0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) {
    const uint32_t x = s_w[i];
    if (i < w) before += x;
    total += x;
  }
}

// Position pos of a request on state slot s: its cache slot, -1 for a refused request.
__device__ __forceinline__ long long cache_slot(const PageTableArgs& a, int s, long long pos, bool refused) {
  if (refused) return -1;
  const int pg = a.block_table[(size_t)s * a.max_pages + (pos >> a.page_log2)];
  if (pg < 0 || pg >= a.n_pages) {
    set_status(a.status, kStatusBadPage);
    return -1;
  }
  return ((long long)pg << a.page_log2) + (pos & ((1 << a.page_log2) - 1));
}

// fill: this work-group also writes every token's position and slot
template <int kPlanThreads>
__global__ __launch_bounds__(kPlanThreads) void page_plan_kernel(PageTableArgs a, int fill) {
  extern __shared__ uint32_t s_bits[];  // [2][words]: slots seen, slots seen twice
  __shared__ uint32_t s_w[kPlanThreads / 64];
  __shared__ long long s_at[kPlanThreads];  // where a request's released or new pages start
  __shared__ int s_n[kPlanThreads], s_held[kPlanThreads], s_slot[kPlanThreads];
  __shared__ int s_end[kPlanThreads], s_ctx[kPlanThreads], s_seq[kPlanThreads];
  __shared__ long long s_taken;
  const int tid = threadIdx.x;
  const int words = (a.n_slots + 31) >> 5;
  const int P = 1 << a.page_log2;
  int bad = 0;
  if (tid == 0) s_taken = 0;
  // the first tile's inputs and the free list's length, asked for together: the rest of the plan is a chain of
  // loads that wait for each other
  int slot_in = -1, n_first = 0;
  long long adv_first = 0;
  if (tid < a.B) {
    slot_in = a.idx_map ? a.idx_map[tid] : tid;
    n_first = a.chunk_len[tid];
    adv_first = a.advance ? (long long)a.advance[tid] + a.advance_add : 0;
  }
  long long count = a.free_count[0];

  // a slot that two rows name belongs to neither: both are padding
  if (a.idx_map) {
    for (int i = tid; i < 2 * words; i += kPlanThreads) s_bits[i] = 0;
    __syncthreads();
    for (int b = tid; b < a.B; b += kPlanThreads) {
      const int s = b == tid ? slot_in : a.idx_map[b];
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
    const int s = b == tid ? slot_in : a.idx_map[b];
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
  if (count < 0 || count > a.n_pages) {
    bad |= kStatusBadIndex;
    count = count < 0 ? 0 : a.n_pages;
  }
  long long back = 0;
  int any = n_first < 0;
  for (int b = tid + kPlanThreads; b < a.B; b += kPlanThreads) any |= a.chunk_len[b] < 0;
  if (__syncthreads_or(any)) {
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
      const int b = b0 + tid;
      const int s = live_slot(b);
      const bool done = s >= 0 && a.chunk_len[b] < 0;
      const int held = done ? clamp_held(a.pages_held[s]) : 0;
      long long e, t;
      block_scan<kPlanThreads>((uint32_t)held, e, t, s_w);
      // the requests that give pages back, side by side
      long long at_list, m;
      block_scan<kPlanThreads>(held > 0, at_list, m, s_w);
      if (held > 0) {
        s_at[at_list] = back + e;
        s_n[at_list] = held;
        s_slot[at_list] = s;
      }
      __syncthreads();
      // sixteen lanes a request, 32 pages a lane in flight
      for (int r = tid >> 4; r < m; r += kPlanThreads / 16) {
        const int n = s_n[r];
        const int32_t* row = a.block_table + (size_t)s_slot[r] * a.max_pages;
        for (int i0 = tid & 15; i0 < n; i0 += 512) {
          int pg[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) pg[k] = row[min(i0 + 16 * k, n - 1)];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const long long at = count + s_at[r] + i0 + 16 * k;
            if (i0 + 16 * k >= n) break;
            if (at < a.n_pages)
              a.free_list[at] = pg[k];
            else
              bad |= kStatusBadIndex;
          }
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
    __threadfence_block();
    __syncthreads();
  }
  const long long avail = min(count + back, (long long)a.n_pages);

  long long tok0 = 0, need0 = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const int s = live_slot(b);
    const int n_in = b >= a.B ? 0 : b0 == 0 ? n_first : a.chunk_len[b];
    const bool here = s >= 0 && n_in >= 0;
    const int n = here ? n_in : 0;
    long long ctx = 0;
    int held = 0;
    if (here) {
      ctx = a.kv_len[s] + (b0 == 0 ? adv_first : a.advance ? (long long)a.advance[b] + a.advance_add : 0);
      held = a.pages_held[s];
      if (ctx < 0 || ctx > 0x7FFFFFFF) {
        bad |= kStatusBadIndex;
        ctx = ctx < 0 ? 0 : 0x7FFFFFFF;
      }
      held = clamp_held(held);
    }
    const long long want = (ctx + n + P - 1) >> a.page_log2;
    long long te, ne, tt, nt;
    // (a request of more tokens than there is room for counts as one too many: it is refused either way, and
    // what stands behind it starts past the end)
    const uint32_t nc = (uint32_t)min(n, a.max_tokens + 1);
    block_scan<kPlanThreads>(nc, te, tt, s_w);
    const long long t_end = tok0 + te + nc;
    const bool fits = here && want <= a.max_pages && t_end <= a.max_tokens;
    const long long need = fits && want > held ? want - held : 0;
    block_scan<kPlanThreads>((uint32_t)need, ne, nt, s_w);
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
    s_end[tid] = (int)min(t_end, (long long)a.max_tokens);
    s_ctx[tid] = (int)ctx;
    s_seq[tid] = granted;
    const int more = __syncthreads_or(granted && need > 2);
    // new page i of the step is the free list's i-th from its end
    if (!more) {
      for (int i = 0; i < s_n[tid]; ++i)
        a.block_table[(size_t)s * a.max_pages + held + i] = a.free_list[avail - 1 - from - i];
    } else {
      const int m = min(kPlanThreads, a.B - b0);
      for (int r = tid >> 4; r < m; r += kPlanThreads / 16) {
        const int k = s_n[r];
        int32_t* row = a.block_table + (size_t)(k ? s_slot[r] : 0) * a.max_pages + s_held[r];
#pragma unroll 8
        for (int i = tid & 15; i < k; i += 16) row[i] = a.free_list[avail - 1 - s_at[r] - i];
      }
    }
    __threadfence_block();
    __syncthreads();
    if (fill) {
      // the tile's tokens; a token's request is the first whose end is past it
      const int m = min(kPlanThreads, a.B - b0);
      const int t0 = (int)min(tok0, (long long)a.max_tokens), t1 = s_end[m - 1];
      for (int t = t0 + tid; t < t1; t += kPlanThreads) {
        int lo = 0, hi = m - 1;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (s_end[mid] > t)
            hi = mid;
          else
            lo = mid + 1;
        }
        const long long pos = (long long)s_ctx[lo] + (t - (lo ? s_end[lo - 1] : t0));
        a.positions[t] = pos;
        a.slot_map[t] = cache_slot(a, s_slot[lo], pos, !s_seq[lo]);
      }
      __syncthreads();
    }
    tok0 += tt;
    need0 += nt;
  }
  if (tid == 0) a.free_count_out[0] = (int)(avail - s_taken);
  if (bad && a.status) atomicOr(a.status, (uint32_t)bad);
  if (!fill) return;
  for (int t = (int)min(tok0, (long long)a.max_tokens) + tid; t < a.max_tokens; t += kPlanThreads) {
    a.positions[t] = 0;
    a.slot_map[t] = -1;
  }
}

// Token t from the plan's outputs: its request is the first whose end is past it.
__global__ __launch_bounds__(256) void page_fill_kernel(PageTableArgs a) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= a.max_tokens) return;
  if (t >= a.query_start[a.B]) {
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
  a.slot_map[t] = cache_slot(a, s, pos, a.seq_lens[lo] <= 0);
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
  if (a.B <= kPlanSmall)
    hipLaunchKernelGGL(page_plan_kernel<kPlanSmall>, dim3(1), dim3(kPlanSmall), lds, st, a, fill ? 1 : 0);
  else
    hipLaunchKernelGGL(page_plan_kernel<kPlanLarge>, dim3(1), dim3(kPlanLarge), lds, st, a, fill ? 1 : 0);
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
