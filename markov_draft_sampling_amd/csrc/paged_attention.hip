// Attention of a chunk of new tokens of every request over its paged
// key/value cache: one token (decoding), the K + 1 tokens that verification
// scores, a draft block whose tokens see each other both ways, or a chunk of
// a prompt.
//
// o = softmax(scale q k^T + mask) v, the softmax in one pass over the keys
// with a running maximum m and sum l in float32 and base 2: a block's
// p = 2^(x - m), l += sum p, o += p v; when a block's maximum passes m by more
// than 8, o and l are scaled by 2^(m - m') first (below that p stays under
// 2^8, which costs no precision in floating point). p is rounded to bf16 for
// the second product (within 2^-8 of each, the products' own input type, as v
// has; with the output's rounding 0.0020 to 0.0023 of the outputs' norm from 64
// bits, where that rounding alone gives 0.0016 to 0.0018; a second bf16 part of p
// would be one product more for every two); l sums the unrounded p.
//
// Rows. The G query heads of one key head read the same keys, so a request's
// rows are its (token, head in group) pairs, token-major, in tiles of 16, 32,
// 64 or 128 rows: every key and value is read from HBM once per tile, and a
// tile's work-group is one (request, rows, key head).
//
// Waves. A work-group is RG row groups of 32 rows (16 in the smallest tile)
// by KG key groups of waves. Key group g takes blocks g, g + KG, .. of KB keys.
// Few rows are bound by the cache's bytes: one row group, four key groups, a
// work-group to a CU with 128 KB of LDS to keep reads in flight (or, over short
// sequences of many requests, fewer key groups in two or four work-groups). Up to 64 rows
// take two by two (or by one or four), a prompt's 128 rows four row groups that share every block;
// both with two work-groups to a CU, so that one's softmax runs beside the
// other's products. The key groups' (m, l, o) are joined through LDS at the end.
//
// Split. Fewer tiles than CUs: the keys are cut into chunks of work-groups as
// well, whose (m, l, o) a second kernel joins (attn_plan has the rule). More
// work-groups than the CUs hold: the longest sequences go first.
//
// Block. Keys and values are copied straight into LDS (16 bytes a lane, no
// registers), two to four blocks ahead, 16-byte slots XOR-swizzled by row. A key
// group of one wave needs no barrier, one of several has one a block. Both
// products are computed transposed on the matrix cores (16x16x32 bf16): the
// scores as S^T = K Q^T, whose result layout (lane: one row, 4 keys of each
// 16) is the operand layout of P^T once the keys of a block are taken in the
// order {4 g .. 4 g + 3, 16 + 4 g ..}: no lane exchanges probabilities. Values
// are read column-wise from LDS by the transposing LDS reads in that order.
// 8-bit caches are widened to bf16 (exactly) after the LDS read; the key scale
// joins the softmax scale, the value scale the final division.
//
// Measured (32 query heads, 8 key heads, D = 128, the reads of each key and
// value once): one request of 131072 keys 105 us, 5.1 TB/s, bound by HBM; 32
// requests of 8 tokens over 100 .. 8192 keys 128 us, 4.5 TB/s, the last CUs to
// finish; 128 requests over an 8-bit cache 135 us, 4.2 TB/s; a chunk of
// 2048 prompt tokens over 14336 keys 515 us, 0.98 PFLOP/s, bound by the vector
// unit (the exponentials) and the matrix cores in turn; one token over 1037
// keys 9.6 us, two launches' latency. (The pairs at the rules below are from one
// run each; cards differ by up to 8%.)
#include <type_traits>

#include "mds_device.h"
#include "mds_serve.h"

namespace mds {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#define MDS_LDS __attribute__((address_space(3)))

constexpr float kLn2 = 0x1.62e430p-1f;
constexpr float kRescale = 8.0f;  // a maximum's growth (base 2) up to which the running one stays

// One request's row tile: which rows, and which keys its rows can see.
struct Tile {
  int b, slot, q0, n, r0, rows;  // request, state slot, first token, tokens, first row, rows (0: nothing to do)
  int seq, lim;                  // sequence length, and that within the block table
  int lo, hi;                    // keys that some row sees: [lo, hi)
  int base;                      // lo rounded down to a block of 64 (SINKS: 0)
  // SINKS: the first s keys are seen too. Places of keys, in whose blocks and chunks the tile is worked on, are the keys'
  // own numbers up to sb, a multiple of 64, and gap (one too) less than those from there on
  int s, sb, gap;
  int chunks;                    // chunks with keys (at least 1)
  int at;                        // number of the tile in the batch's own order: its place in the partials
};

// keys [lo, hi) that token t of the request sees
__device__ __forceinline__ void token_keys(const PagedAttnArgs& a, const Tile& t, int tok, int& lo, int& hi) {
  const int pos = t.seq - t.n + tok;
  hi = a.causal ? min(pos + 1, t.lim) : t.lim;
  lo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
}

__device__ __forceinline__ int clamp_tok(const PagedAttnArgs& a, int q, uint32_t& bad) {
  if (q < 0 || q > a.T) {
    bad |= kStatusBadIndex;
    return q < 0 ? 0 : a.T;
  }
  return q;
}

// The request with the n-th longest sequence (B <= 128; every wave ranks them all, about a microsecond), or -1 if it
// surely has no key past the first `least` (the quick way out of a chunk that only longer sequences have).
__device__ __forceinline__ int nth_longest(const PagedAttnArgs& a, int n, long long least) {
  const int lane = threadIdx.x & 63;
  // length above request number: all different (beyond 2^24 keys only the order may suffer)
  constexpr int kTop = (1 << 24) - 1;
  int key[2], rank[2] = {0, 0}, longer = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int b = lane + 64 * i;
    const int len = b < a.B ? min(max(a.seq_lens[b], 0), kTop) : 0;
    key[i] = b < a.B ? len * 128 + 127 - b : -1;
    longer += __popcll(__ballot(len > least));
  }
  if (least > 0 && least < kTop && n >= longer) return -1;
  for (int b = 0; b < min(a.B, 64); ++b) {
    const int k = __builtin_amdgcn_readlane(key[0], b);
    rank[0] += k > key[0];
    rank[1] += k > key[1];
  }
  for (int b = 64; b < a.B; ++b) {
    const int k = __builtin_amdgcn_readlane(key[1], b - 64);
    rank[0] += k > key[0];
    rank[1] += k > key[1];
  }
  const unsigned long long m0 = __ballot(key[0] >= 0 && rank[0] == n), m1 = __ballot(key[1] >= 0 && rank[1] == n);
  return m0 ? __ffsll(m0) - 1 : m1 ? 63 + __ffsll(m1) : 0;
}

// c: the chunk it is wanted for
template <int ROWS, bool SINKS>
__device__ __forceinline__ Tile find_tile(const PagedAttnArgs& a, int tile, int c, uint32_t& bad) {
  Tile t;
  t.rows = 0;
  if (a.per_req > 0) {
    t.b = tile / a.per_req;
    t.r0 = (tile - t.b * a.per_req) * ROWS;
    t.at = tile;
    if (a.by_length) {
      const int b = nth_longest(a, t.b, (long long)c * a.chunk);
      if (b < 0) return t;
      t.at += (b - t.b) * a.per_req;
      t.b = b;
    }
  } else {
    // Request b's tiles start at floor(q0 G / ROWS) + b: enough for its rows, since ceil(x) of its rows is at most
    // the step to the next request's start. The last request that starts at or before the tile, 64 probes a round.
    t.at = tile;
    const int lane = threadIdx.x & 63;
    int step = 1;
    while (step * 64 < a.B) step *= 64;
    t.b = 0;
    for (; step > 0; step >>= 6) {
      const int b = t.b + lane * step;
      uint32_t dummy = 0;
      const int q = clamp_tok(a, a.query_start[min(b, a.B - 1)], dummy);
      const int k = __popcll(__ballot(b < a.B && (int)((unsigned)q * (unsigned)a.G / ROWS) + b <= tile));
      if (k == 0) {  // no request starts that early, or query_start falls somewhere
        t.b = 0;
        break;
      }
      t.b += (k - 1) * step;
    }
  }
  t.b = __builtin_amdgcn_readfirstlane(t.b);
  const int qa = __builtin_amdgcn_readfirstlane(a.query_start[t.b]);
  const int qb = __builtin_amdgcn_readfirstlane(a.query_start[t.b + 1]);
  const int sl = __builtin_amdgcn_readfirstlane(a.seq_lens[t.b]);
  t.slot = a.idx_map ? __builtin_amdgcn_readfirstlane(a.idx_map[t.b]) : t.b;
  t.q0 = clamp_tok(a, qa, bad);
  t.n = clamp_tok(a, qb, bad) - t.q0;
  if (t.n < 0) bad |= kStatusBadIndex;
  if (a.per_req > 0) {
    if (t.n * (long long)a.G > (long long)a.per_req * ROWS) bad |= kStatusBadIndex;  // more tokens than max_q_len
  } else {
    t.r0 = (tile - ((int)((unsigned)t.q0 * (unsigned)a.G / ROWS) + t.b)) * ROWS;
  }
  if (t.r0 < 0) bad |= kStatusBadIndex;  // query_start falls somewhere
  t.rows = min(ROWS, t.n * a.G - t.r0);
  if (t.n <= 0 || t.rows <= 0 || t.r0 < 0) {
    t.rows = 0;
    return t;
  }
  t.seq = max(sl, 0);
  const long long cap = (long long)a.max_pages << a.page_log2;
  t.lim = (int)min((long long)t.seq, cap);
  if (t.lim < t.seq) bad |= kStatusBadIndex;
  if (t.slot < 0 || t.slot >= a.n_slots) {  // a padding request has no keys
    if (t.slot >= a.n_slots) bad |= kStatusBadIndex;
    t.lim = 0;
    t.slot = 0;
  }
  int h0, l1;
  token_keys(a, t, t.r0 / a.G, t.lo, h0);
  token_keys(a, t, (t.r0 + t.rows - 1) / a.G, l1, t.hi);
  t.hi = max(t.hi, 0);
  t.lo = min(t.lo, t.hi);
  t.base = t.lo & ~63;
  t.s = t.sb = t.gap = 0;
  if constexpr (SINKS) {
    t.s = min(a.sinks, t.hi);
    t.sb = (t.s + 63) & ~63;
    t.gap = max(t.base - t.sb, 0);
    t.base = 0;
  }
  t.chunks = min(max((t.hi - t.gap - t.base + a.chunk - 1) / a.chunk, 1), a.n_chunks);
  return t;
}

// Writes 8 (or 4) columns of one output row: o / l, scaled, in bf16; a row without keys is zero.
template <int NC>
__device__ __forceinline__ void store_row(const PagedAttnArgs& a, const Tile& t, int r, int h, int d0,
                                          const float (&o)[NC], float m, float l) {
  const int R = t.r0 + r;
  const int tok = R / a.G, hq = h * a.G + (R - tok * a.G);
  const float inv = l == 0.0f ? 0.0f : (a.v_scale ? a.v_scale[h] : 1.0f) / l;
  uint16_t* p = a.out + (long long)(t.q0 + tok) * a.o_ts + hq * a.o_hs + d0;
  uint32_t w[NC / 2];
#pragma unroll
  for (int i = 0; i < NC / 2; ++i) {
    const bf16x2 b = {(__bf16)(o[2 * i] * inv), (__bf16)(o[2 * i + 1] * inv)};
    w[i] = __builtin_bit_cast(uint32_t, b);
  }
  if constexpr (NC == 8)
    *(u32x4*)p = u32x4{w[0], w[1], w[2], w[3]};
  else
    *(u32x2*)p = u32x2{w[0], w[1]};
  if (a.lse && d0 == 0)
    a.lse[(long long)(t.q0 + tok) * a.Hq + hq] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Transposing LDS reads, a group of 16 lanes reading 4 (8) keys of 16 columns: a lane gets its column's.
__device__ __forceinline__ s16x4 read_tr16(uint32_t at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((MDS_LDS s16x4*)(uintptr_t)at);
}
__device__ __forceinline__ i32x2 read_tr8(uint32_t at) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((MDS_LDS i32x2*)(uintptr_t)at);
}

// Infinities and NaN among a lane's eight values of a block that some rows see only in part. nonfinite: all
// bits of their elements set.
__device__ __forceinline__ bf16x8 nonfinite(bf16x8 v) {
  const u32x4 x = __builtin_bit_cast(u32x4, v);
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (x[i] & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u;
    const uint32_t hi = (x[i] & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u;
    r[i] = lo | hi;
  }
  return __builtin_bit_cast(bf16x8, r);
}
__device__ __forceinline__ bool any_bits(bf16x8 v) {
  const u32x4 x = __builtin_bit_cast(u32x4, v);
  return (x[0] | x[1] | x[2] | x[3]) != 0;
}
__device__ __forceinline__ bf16x8 without(bf16x8 v, bf16x8 mask) {
  return __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, v) & ~__builtin_bit_cast(u32x4, mask));
}
// Adds them to the rows that do see them: how many +inf and -inf (a NaN counts as both) each row and column meets
// is a product of ones; key: the lane's first key, its others follow the block's order.
template <int NB, int ND>
__device__ __forceinline__ void add_nonfinite(bf16x8 v, bf16x8 inf, int key, const int (&mlo)[NB], const int (&mhi)[NB],
                                              int sinks, floatx4 (&O)[NB][ND], int db) {
  const u32x4 x = __builtin_bit_cast(u32x4, v), f = __builtin_bit_cast(u32x4, inf);
  u32x4 pos, neg;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t p = 0, n = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t e = x[i] >> (16 * h) & 0xFFFFu;
      const bool bad = (f[i] >> (16 * h) & 1u) != 0, nan = (e & 0x7Fu) != 0, minus = (e & 0x8000u) != 0;
      p |= bad && (nan || !minus) ? 0x3F80u << (16 * h) : 0u;
      n |= bad && (nan || minus) ? 0x3F80u << (16 * h) : 0u;
    }
    pos[i] = p;
    neg[i] = n;
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    bf16x8 seen;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = key + (e & 3) + 16 * (e >> 2);
      seen[e] = (__bf16)((((k >= mlo[nb]) | (k < sinks)) & (k < mhi[nb])) ? 1.0f : 0.0f);
    }
    const floatx4 zero = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    const floatx4 np = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, pos), seen, zero, 0, 0, 0);
    const floatx4 nn = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, neg), seen, zero, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      O[nb][db][i] += (np[i] > 0.0f ? INFINITY : 0.0f) + (nn[i] > 0.0f ? -INFINITY : 0.0f);
  }
}

// 16 bytes a lane straight into LDS at `lds` (uniform) + 16 * lane, from base (uniform) + off. As assembly:
// every wait for these copies is the kernel's own, and the compiler, which cannot tell the copies in flight
// apart, would wait for all of them before each LDS read. (m0, the LDS address, has no other use here; the load may read
// it one wait state after the scalar write at the earliest.)
__device__ __forceinline__ void copy_1k(const char* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_copies() {  // at most N of this wave's copies are still in flight
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// D: head dimension; E4M3: 8-bit cache; NB: 16-row blocks a wave; RG x KG waves: RG groups of rows, KG of keys;
// KB: keys of a block; LB: KB of LDS for the ring
template <int D, bool E4M3, int NB, int RG, int KG, int KB, int LB>
struct AttnShape {
  static constexpr int kRows = NB * 16 * RG;
  static constexpr int RB = D * (E4M3 ? 1 : 2);  // bytes of a key (or value)
  static constexpr int kPart = KB * RB;          // bytes of a block's keys
  static constexpr int kStage = 2 * kPart;       // a block of keys and values
  // blocks in flight per key group: what fits, four at most
  static constexpr int NST = KG * kStage * 4 <= LB * 1024 ? 4 : KG * kStage * 3 <= LB * 1024 ? 3 : 2;
  static constexpr int kRing = KG * kStage * NST;
  static constexpr int kJoin = RG * KG * 16 * D * 4;  // the waves' o, 16 rows each
  static constexpr int kLds = kRing > kJoin ? kRing : kJoin;
};

// SINKS: the first a.sinks keys are seen outside the window too; EU: waves of a SIMD at once
template <int D, bool E4M3, int NB, int RG, int KG, int KB, int LB, bool SINKS, int EU>
__global__ __launch_bounds__(64 * RG * KG) __attribute__((amdgpu_waves_per_eu(EU, EU))) void attn_kernel(
    PagedAttnArgs a) {
  using Sh = AttnShape<D, E4M3, NB, RG, KG, KB, LB>;
  constexpr int ROWS = Sh::kRows, RB = Sh::RB, kPart = Sh::kPart, kStage = Sh::kStage, NST = Sh::NST;
  constexpr int SPR = RB / 16;                 // 16-byte slots of a key
  constexpr int RPI = 64 / SPR;                // keys per copy (1 KB)
  constexpr int NI = KB / RPI;                 // copies of a block's keys (as many for its values)
  constexpr int NH = KB / 16;                  // half blocks of 16 keys, each in one page
  constexpr int NP = 64 / NH;                  // blocks whose page ids a wave holds
  constexpr int kMine = (NI + RG - 1) / RG;    // of them, a wave's (the RG waves of a key group share a block)
  constexpr int NS = D / 32;                   // 32-wide slices of the first product
  constexpr int ND = D / 16;                   // 16-wide column blocks of the second
  __shared__ __attribute__((aligned(16))) unsigned char s_kv[Sh::kLds];
  __shared__ float s_m[KG][ROWS], s_l[KG][ROWS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rg = w % RG, kg = w / RG;
  const int lr = lane & 15, lg = lane >> 4;
  const int h = blockIdx.x % (unsigned)a.Hkv;
  const int ct = blockIdx.x / (unsigned)a.Hkv;
  const int c = ct / a.tiles, tile = ct - c * a.tiles;

  uint32_t bad = 0;
  const Tile t = find_tile<ROWS, SINKS>(a, tile, c, bad);
  if (t.rows <= 0 || c >= t.chunks) {
    if (bad && tid == 0) set_status(a.status, bad);
    return;
  }
  const int c0 = t.base + c * a.chunk;
  // SINKS: lo and hi are the tile's, and end is the chunk's last place
  const int end = c == a.n_chunks - 1 ? t.hi - t.gap : min(t.hi - t.gap, c0 + a.chunk);
  const int lo = SINKS ? t.lo : max(t.lo, c0), hi = SINKS ? t.hi : end;
  const int nblk = end > (SINKS ? c0 : lo) ? (end - c0 + KB - 1) / KB : 0;
  const int sinks = SINKS ? t.s : 0;
  auto key_at = [&](int place) { return SINKS && place >= t.sb ? place + t.gap : place; };  // (of a block, or a piece of it)
  // Keys that a copy of the 16 keys from k on may read, [lo, hi) without SINKS. Those outside repeat the nearest inside:
  // what lies behind a sequence's end, or in a page of which no row sees a key, is never read. Their probability is zero.
  auto piece_lo = [&](int k) { return SINKS && k < sinks ? 0 : lo; };
  auto piece_hi = [&](int k) { return SINKS && k < sinks && k + 16 <= lo ? sinks : hi; };
  auto nearest = [&](int k, int of) { return min(max(k, piece_lo(of)), piece_hi(of) - 1); };
  const int nit = (nblk + KG - 1) / KG;                 // rounds; key group kg takes blocks kg, kg + KG, ..
  const int nmy = nblk > kg ? (nblk - kg + KG - 1) / KG : 0;  // of them, its own

  // the wave's rows: row R of the request is head R % G of token R / G; rows past the tile repeat the last
  const int r0 = t.r0 + min(rg * NB * 16, t.rows - 1), r1 = t.r0 + min((rg + 1) * NB * 16, t.rows) - 1;
  bf16x8 Q[NB][NS];
  int mlo[NB], mhi[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int R = min(t.r0 + (rg * NB + nb) * 16 + lr, t.r0 + t.rows - 1);
    const int tok = R / a.G, hq = h * a.G + (R - tok * a.G);
    const uint16_t* qp = a.q + (long long)(t.q0 + tok) * a.q_ts + hq * a.q_hs;
#pragma unroll
    for (int s = 0; s < NS; ++s)
      Q[nb][s] = *(const bf16x8*)(qp + (E4M3 ? 64 * (s >> 1) + 16 * lg + 8 * (s & 1) : 32 * s + 8 * lg));
    int klo, khi;
    token_keys(a, t, tok, klo, khi);
    mlo[nb] = max(klo, lo);
    mhi[nb] = min(khi, hi);
  }
  // keys that some row of the wave sees, and those that every row sees (blocks inside need no mask)
  int any_lo, any_hi, all_lo, all_hi;
  token_keys(a, t, r0 / a.G, any_lo, all_hi);
  token_keys(a, t, r1 / a.G, all_lo, any_hi);
  all_lo = max(all_lo, lo);
  all_hi = min(all_hi, hi);
  const float sc = a.scale_log2 * (a.k_scale ? a.k_scale[h] : 1.0f);

  // copies: copy p of a block's keys fills keys RPI p .. of it; lane l lands in row r = RPI p + l / SPR,
  // slot l % SPR, which holds the row's slot (l % SPR) ^ swizzle(r)
  auto kswz = [](int r) { return SPR == 16 ? r & 15 : SPR == 8 ? (r >> 1) & 7 : (r >> 2) & 3; };
  auto vswz = [](int r) {
    return E4M3 ? (SPR == 8 ? ((r >> 1) & 3) | ((r >> 2) & 4) : ((r >> 2) & 1) | ((r >> 3) & 2))
                : (SPR == 16 ? (r & 7) * 2 : ((r >> 1) & 3) * 2);
  };
  const int lrow = lane / SPR, lslot = lane % SPR;
  const uint32_t ring = (uint32_t)(uintptr_t)(MDS_LDS const void*)s_kv + kg * NST * kStage;
  const int32_t* trow = a.block_table + (size_t)t.slot * a.max_pages;
  const char* kb_h = (const char*)a.k_pages + h * a.k_hs;
  const char* vb_h = (const char*)a.v_pages + h * a.v_hs;
  const int pmask = (1 << a.page_log2) - 1;
  // this wave's copies of a block: numbers rg + RG m of its keys and of its values. Offsets of a lane's 16 bytes
  // from the first of the 16 keys (which lie in one page) that the copy is part of
  uint32_t ko[kMine], vo[kMine];
#pragma unroll
  for (int m = 0; m < kMine; ++m) {
    const int r = ((rg + RG * m) * RPI + lrow) % KB;
    ko[m] = (uint32_t)((r & 15) * (int)a.k_ts) + (uint32_t)((lslot ^ kswz(r)) * 16);
    vo[m] = (uint32_t)((r & 15) * (int)a.v_ts) + (uint32_t)((lslot ^ vswz(r)) * 16);
  }
  // Page ids of the key group's blocks i0 .. i0 + NP - 1: lane NH (i - i0) + j has the page of 16-key piece j of
  // block i.
  int pages = 0;
  auto load_pages = [&](int i0) {
    const int kh = key_at(c0 + (kg + KG * (i0 + lane / NH)) * KB + 16 * (lane % NH));
    pages = trow[nearest(kh, kh) >> a.page_log2];
    if ((unsigned)pages >= (unsigned)a.n_pages) {
      pages = 0;
      bad |= kStatusBadPage;
    }
  };
  auto copy_block = [&](int i, int st) {
    if (i && i % NP == 0) load_pages(i);
    const int k0 = key_at(c0 + (kg + KG * i) * KB);
    const bool inside = (k0 >= lo && k0 + KB <= hi) || (SINKS && k0 + KB <= sinks);
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int p = rg + RG * m, j = p * RPI / 16;  // copy p lies in 16-key piece j
      if (NI % RG != 0 && p >= NI) break;
      const int kc = nearest(k0 + 16 * j, k0 + 16 * j);
      const int pg = __builtin_amdgcn_readlane(pages, NH * (i % NP) + j);
      const char* kp = kb_h + pg * a.k_ps + (kc & pmask) * (int)a.k_ts;
      const char* vp = vb_h + pg * a.v_ps + (kc & pmask) * (int)a.v_ts;
      uint32_t kof = ko[m], vof = vo[m];
      if (!inside) {
        const int r = (p * RPI + lrow) & 15;
        const int d = nearest(k0 + 16 * j + r, k0 + 16 * j) - kc - r;  // from the row's own place to the key copied
        kof = (uint32_t)((int)kof + d * (int)a.k_ts);
        vof = (uint32_t)((int)vof + d * (int)a.v_ts);
      }
      copy_1k(kp, kof, ring + st * kStage + p * 1024);
      copy_1k(vp, vof, ring + st * kStage + kPart + p * 1024);
    }
  };

  // LDS offsets of a lane's reads: key slices of its row, and column reads of the values by block of 16 columns
  uint32_t va[ND];
#pragma unroll
  for (int db = 0; db < ND; ++db) {
    if constexpr (E4M3) {
      const int j = lr >> 1, r = (j & 4) * 4 + 4 * lg + (j & 3);
      va[db] = r * RB + (db ^ vswz(r)) * 16 + (lr & 1) * 8;
    } else {
      // keys r and r + 16 have the same swizzle
      const int r = 4 * lg + (lr >> 2);
      va[db] = r * RB + ((2 * db + ((lr >> 1) & 1)) ^ vswz(r)) * 16 + (lr & 1) * 8;
    }
  }

  floatx4 O[NB][ND];
  float l[NB];          // the lane's part of the row sum
  float m[NB], mc[NB];  // running maximum (base 2, scaled), and what is subtracted: it, or 0 before any key
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m[nb] = -INFINITY;
    mc[nb] = 0.0f;
    l[nb] = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) O[nb][d] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  auto widen = [](uint32_t v, bool up) {
    return up ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
  };
  // Wave priorities, where two work-groups share a CU and so each SIMD holds two waves that need the matrix cores and
  // the vector unit in turn: softmax and values go ahead of the other wave's scores, which would otherwise be cut into
  // (2048 prompt tokens: 491 us against 530 us). Where the key groups of a work-group wait for each other only
  // at its end, every second batch of work-groups also goes ahead as a whole, so that the two do not
  // keep in step (128 requests over an 8-bit cache: 135 us, with the first rule alone 141 us, without either 146 us).
  const bool ahead = KG > 1 && (blockIdx.x & 256) != 0;
  auto low = [&]() {
    if constexpr (RG > 1) {
      if (ahead)
        __builtin_amdgcn_s_setprio(1);
      else
        __builtin_amdgcn_s_setprio(0);
    }
  };
  auto high = [&]() {
    if constexpr (RG > 1) {
      if (ahead)
        __builtin_amdgcn_s_setprio(2);
      else
        __builtin_amdgcn_s_setprio(1);
    }
  };
  constexpr int NK = KB / 16;
  auto block = [&](int st, int i) {
    const int k0 = key_at(c0 + (kg + KG * i) * KB);
    const unsigned char* buf = s_kv + (kg * NST + st) * kStage;
    floatx4 S[NK][NB];
#pragma unroll
    for (int kb = 0; kb < NK; ++kb) {
      const int r = kb * 16 + lr;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[kb][nb] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
      bf16x8 K[NS];
      if constexpr (E4M3) {
#pragma unroll
        for (int p = 0; p < NS / 2; ++p) {
          const u32x4 x = *(const u32x4*)(buf + r * RB + ((4 * p + lg) ^ kswz(r)) * 16);
          K[2 * p] = __builtin_bit_cast(
              bf16x8, u32x4{widen(x[0], false), widen(x[0], true), widen(x[1], false), widen(x[1], true)});
          K[2 * p + 1] = __builtin_bit_cast(
              bf16x8, u32x4{widen(x[2], false), widen(x[2], true), widen(x[3], false), widen(x[3], true)});
        }
      } else {
#pragma unroll
        for (int s = 0; s < NS; ++s) K[s] = *(const bf16x8*)(buf + r * RB + ((4 * s + lg) ^ kswz(r)) * 16);
      }
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          S[kb][nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(K[s], Q[nb][s], S[kb][nb], 0, 0, 0);
    }
    high();
    // lane: row lr of each nb, keys k0 + 16 kb + 4 lg + i
    const bool masked = (k0 < all_lo && !(SINKS && k0 + KB <= sinks)) || k0 + KB > all_hi;
    if (masked) {
#pragma unroll
      for (int kb = 0; kb < NK; ++kb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = k0 + 16 * kb + 4 * lg + e;
            const bool late = SINKS ? (key >= mlo[nb]) | (key < sinks) : key >= mlo[nb];
            S[kb][nb][e] = (late & (key < mhi[nb])) ? S[kb][nb][e] : -INFINITY;
          }
    }
    float top[NB];
    bool grow = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float x = S[0][nb][0];
#pragma unroll
      for (int e = 1; e < 4 * NK; ++e) x = fmaxf(x, S[e >> 2][nb][e & 3]);
      top[nb] = x * sc;
      grow |= top[nb] > m[nb] + kRescale;
    }
    if (__any(grow)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float x = fmaxf(m[nb], top[nb]);
        x = fmaxf(x, __shfl_xor(x, 16));
        x = fmaxf(x, __shfl_xor(x, 32));
        const float f = x == m[nb] ? 1.0f : __builtin_amdgcn_exp2f(m[nb] - x);
        m[nb] = x;
        mc[nb] = x == -INFINITY ? 0.0f : x;
        l[nb] *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) O[nb][d] *= f;
      }
    }
    // values: lane column d = 16 db + lr, keys 4 lg + (0 .. 3) and 16 + 4 lg + (0 .. 3) of each 32
    const uint32_t vb = ring + st * kStage + kPart;
    auto value = [&](int k2, int db) {
      const uint32_t at = vb + k2 * 32 * RB + va[db];
      if constexpr (E4M3) {
        const i32x2 x = read_tr8(at);
        return __builtin_bit_cast(
            bf16x8, u32x4{widen(x[0], false), widen(x[0], true), widen(x[1], false), widen(x[1], true)});
      } else {
        const s16x4 x = read_tr16(at), y = read_tr16(at + 16 * RB);
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    };
#pragma unroll
    for (int k2 = 0; k2 < NK / 2; ++k2) {
      bf16x8 V[ND], P[NB];
#pragma unroll
      for (int db = 0; db < ND; ++db) V[db] = value(k2, db);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[2 * k2 + (e >> 2)][nb][e & 3], sc, -mc[nb]));
        l[nb] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
#pragma unroll
        for (int e = 0; e < 8; ++e) P[nb][e] = (__bf16)p[e];
      }
      if (masked) {
        // a value that some rows do not see must not reach them, but 0 times an infinity or NaN would
#pragma unroll
        for (int db = 0; db < ND; ++db) {
          const bf16x8 inf = nonfinite(V[db]);
          if (__any(any_bits(inf))) {
            add_nonfinite<NB, ND>(V[db], inf, k0 + 32 * k2 + 4 * lg, mlo, mhi, sinks, O, db);
            V[db] = without(V[db], inf);
          }
        }
      }
#pragma unroll
      for (int db = 0; db < ND; ++db)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          O[nb][db] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(V[db], P[nb], O[nb][db], 0, 0, 0);
    }
    low();
  };

  low();
  if (nmy > 0) load_pages(0);
  if constexpr (RG == 1) {
    // a key group is one wave: its ring is its own, no barrier
#pragma unroll
    for (int i = 0; i < NST; ++i)
      if (i < nmy) copy_block(i, i);
    int st = 0;
#pragma nounroll
    for (int i = 0; i < nmy; ++i) {
      // block i has landed: at most the NST - 1 blocks after it are still in flight
      if (i + NST <= nmy)
        wait_copies<(NST - 1) * 2 * NI>();
      else
        wait_copies<0>();  // near the end: all of them
      block(st, i);
      if (i + NST < nmy) {
        // the block's LDS reads have returned (their values were used): its place is free
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        copy_block(i + NST, st);
      }
      st = st + 1 == NST ? 0 : st + 1;
    }
  } else {
    // the RG waves of a key group share its blocks: one barrier a round, after which block i is there for all of
    // them and the place of block i - 1 is free
    constexpr int kLeast = 2 * (NI / RG);  // copies that every wave of the group makes of a block
#pragma unroll
    for (int i = 0; i < NST - 1; ++i)
      if (i < nmy) copy_block(i, i);
    int st = 0;
#pragma nounroll
    for (int i = 0; i < nit; ++i) {
      if (i + NST - 1 <= nmy)
        wait_copies<(NST - 2) * kLeast>();
      else
        wait_copies<0>();
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (i + NST - 1 < nmy) copy_block(i + NST - 1, st == 0 ? NST - 1 : st - 1);
      if (i < nmy) {
        const int k0 = key_at(c0 + (kg + KG * i) * KB);
        if (k0 < any_hi && (k0 + KB > any_lo || (SINKS && k0 < sinks))) block(st, i);  // else no row of this wave sees a key of it
      }
      st = st + 1 == NST ? 0 : st + 1;
    }
  }
  if (bad) set_status(a.status, bad);

  // join the key groups, 16 rows of each row group at a time: o scaled to the common maximum through LDS, summed
  // by the threads that share a row, 8 columns each
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    l[nb] += __shfl_xor(l[nb], 16);
    l[nb] += __shfl_xor(l[nb], 32);
    if (lg == 0) {
      s_m[kg][(rg * NB + nb) * 16 + lr] = m[nb];
      s_l[kg][(rg * NB + nb) * 16 + lr] = l[nb];
    }
  }
  __syncthreads();
  float* so = (float*)s_kv + (rg * KG) * 16 * D;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int row0 = (rg * NB + nb) * 16;
    float M = s_m[0][row0 + lr];
#pragma unroll
    for (int i = 1; i < KG; ++i) M = fmaxf(M, s_m[i][row0 + lr]);
    const float f = m[nb] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[nb] - M);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      const floatx4 x = m[nb] == -INFINITY && !(l[nb] != l[nb]) ? floatx4{0.0f, 0.0f, 0.0f, 0.0f} : O[nb][d] * f;
      *(floatx4*)(so + kg * 16 * D + lr * D + (((4 * d + lg) ^ lr) * 4)) = x;
    }
    __syncthreads();
    for (int it = kg * 64 + lane; it < 16 * (D / 8); it += 64 * KG) {
      const int rr = it / (D / 8), od = (it % (D / 8)) * 8, row = row0 + rr;
      if (row >= t.rows) continue;
      float Mr = s_m[0][row];
#pragma unroll
      for (int i = 1; i < KG; ++i) Mr = fmaxf(Mr, s_m[i][row]);
      float L = 0.0f;
#pragma unroll
      for (int i = 0; i < KG; ++i) {
        const float li = s_l[i][row];
        L += s_m[i][row] == -INFINITY && li == li ? 0.0f : li * __builtin_amdgcn_exp2f(s_m[i][row] - Mr);
      }
      float o[8];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        floatx4 x = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < KG; ++i) x += *(const floatx4*)(so + i * 16 * D + rr * D + (((od / 4 + q) ^ rr) * 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) o[q * 4 + e] = x[e];
      }
      if (t.chunks == 1) {
        store_row(a, t, row, h, od, o, Mr, L);
      } else {
        const size_t pr = (((size_t)c * a.tiles + t.at) * a.Hkv + h) * ROWS + row;
        float* po = a.part_o + pr * D + od;
        *(floatx4*)po = floatx4{o[0], o[1], o[2], o[3]};
        *(floatx4*)(po + 4) = floatx4{o[4], o[5], o[6], o[7]};
        if (od == 0) a.part_ml[pr] = make_float2(Mr, L);
      }
    }
    __syncthreads();
  }
}

// Joins the chunks of a row: o = sum 2^(m_c - M) o_c / sum 2^(m_c - M) l_c. Four groups of 16 lanes take the chunks in
// turn, up to four of them in flight each, with a running maximum of their own, and are joined at the end.
template <int D, int ROWS>
__device__ __forceinline__ void join_row(const PagedAttnArgs& a, const Tile& t, int row, int h) {
  const int lane = threadIdx.x & 63;
  const size_t step = (size_t)a.tiles * a.Hkv * ROWS;
  const size_t pr = ((size_t)t.at * a.Hkv + h) * ROWS + row;
  constexpr int NC = D / 16;
  const int g = lane >> 4, od = (lane & 15) * NC;
  float M = -INFINITY, L = 0.0f, o[NC];
#pragma unroll
  for (int e = 0; e < NC; ++e) o[e] = 0.0f;
  auto scale_to = [&](float x) {  // from M to x >= M
    const float f = M == x ? 1.0f : __builtin_amdgcn_exp2f(M - x);
    M = x;
    L *= f;
#pragma unroll
    for (int e = 0; e < NC; ++e) o[e] *= f;
  };
  auto take = [&](auto in_flight, int c0) {
    constexpr int NL = decltype(in_flight)::value;
    float2 ml[NL];
    floatx4 x[NL][NC / 4];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int c = c0 + 4 * i + g;
      const size_t p = pr + min(c, t.chunks - 1) * step;
      ml[i] = a.part_ml[p];
#pragma unroll
      for (int q = 0; q < NC / 4; ++q) x[i][q] = *(const floatx4*)(a.part_o + p * D + od + q * 4);
      if (c >= t.chunks) ml[i] = make_float2(-INFINITY, 0.0f);
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < NL; ++i) top = fmaxf(top, ml[i].x);
    scale_to(top);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      // a chunk without keys of the row has (-inf, 0)
      const bool none = ml[i].x == -INFINITY && ml[i].y == ml[i].y;
      const float f = none ? 0.0f : __builtin_amdgcn_exp2f(ml[i].x - M);
      L += ml[i].y * f;
#pragma unroll
      for (int q = 0; q < NC / 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[q * 4 + e] += none ? 0.0f : x[i][q][e] * f;
    }
  };
  if (t.chunks <= 4) {
    take(std::integral_constant<int, 1>{}, 0);
  } else {
#pragma nounroll
    for (int c0 = 0; c0 < t.chunks; c0 += 16) take(std::integral_constant<int, 4>{}, c0);
  }
  scale_to(fmaxf(M, fmaxf(__shfl_xor(M, 16), fmaxf(__shfl_xor(M, 32), __shfl_xor(M, 48)))));
#pragma unroll
  for (int e = 0; e < NC; ++e) {
    o[e] += __shfl_xor(o[e], 16);
    o[e] += __shfl_xor(o[e], 32);
  }
  L += __shfl_xor(L, 16);
  L += __shfl_xor(L, 32);
  if (g == 0) store_row(a, t, row, h, od, o, M, L);
}

template <int D, int ROWS, bool SINKS>
__global__ __launch_bounds__(256) void attn_join_kernel(PagedAttnArgs a) {
  uint32_t bad = 0;
  const Tile t = find_tile<ROWS, SINKS>(a, blockIdx.x / (unsigned)a.Hkv, 0, bad);  // (in the batch's own order)
  int row = blockIdx.y * 4 + (threadIdx.x >> 6);
  if (row >= t.rows || t.chunks <= 1) return;
#pragma nounroll
  do {
    join_row<D, ROWS>(a, t, row, blockIdx.x % (unsigned)a.Hkv);
    row += 4 * gridDim.y;
  } while (row < t.rows);
}

template <int D, bool E4M3, bool SINKS, int NB, int RG, int KG, int KB, int LB, int EU = (RG > 1 ? 2 : 1)>
hipError_t launch_shape(const PagedAttnArgs& a, hipStream_t st) {
  constexpr int ROWS = AttnShape<D, E4M3, NB, RG, KG, KB, LB>::kRows;
  const long long wgs = (long long)a.tiles * a.Hkv;
  hipLaunchKernelGGL((attn_kernel<D, E4M3, NB, RG, KG, KB, LB, SINKS, EU>), dim3((unsigned)(wgs * a.n_chunks)), dim3(64 * RG * KG), 0,
                     st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.n_chunks == 1) return e;
  // few tiles: a wave a row; many, most of which have nothing to join: some rows a wave
  PagedAttnArgs j = a;
  j.by_length = 0;
  const unsigned per_tile = (unsigned)(wgs >= 4096 ? 1 : wgs * (ROWS / 4) <= 4096 ? ROWS / 4 : 4096 / wgs);
  hipLaunchKernelGGL((attn_join_kernel<D, ROWS, SINKS>), dim3((unsigned)wgs, per_tile), dim3(256), 0, st, j);
  return hipGetLastError();
}

// With first tokens, up to 32 rows over an 8-bit cache: half the LDS and two work-groups to a CU, since a block is half as
// long in bytes and its chain of LDS reads, widening, exponentials and products is not (8 key heads of 128, sequences of up
// to twice the window; us with two work-groups to a CU / with one: 128 requests of one token, window 300 26 / 35, 2000
// 91 / 117, 4000 168 / 187; 64 requests, 1000 28 / 39; 32 requests, 8000 98 / 105; 32 of 8 tokens, 4000 51 / 58; 8 of one
// token, whose keys are split, 8000 27 / 29. Heads of 64: 24 / 31, 76 / 93, 135 / 148; 28 / 34; 71 / 72; 43 / 43; 27 / 27).
// Calls without first tokens, windowed or not, keep one.
template <int D, bool E4M3, bool SINKS>
hipError_t launch_d(const PagedAttnArgs& a, int rows, int key_groups, hipStream_t st) {
  if constexpr (E4M3 && SINKS) {
    switch (rows * 10 + key_groups) {
      case 162: return launch_shape<D, E4M3, SINKS, 1, 1, 2, 32, 32, 2>(a, st);
      case 164: return launch_shape<D, E4M3, SINKS, 1, 1, 4, 32, 64, 2>(a, st);
      case 322: return launch_shape<D, E4M3, SINKS, 2, 1, 2, 32, 32, 2>(a, st);
      case 324: return launch_shape<D, E4M3, SINKS, 2, 1, 4, 32, 64, 2>(a, st);
    }
  } else {
    switch (rows * 10 + key_groups) {
      case 161: return launch_shape<D, E4M3, SINKS, 1, 1, 1, 32, 32>(a, st);
      case 162: return launch_shape<D, E4M3, SINKS, 1, 1, 2, 32, 64>(a, st);
      case 164: return launch_shape<D, E4M3, SINKS, 1, 1, 4, 32, 128>(a, st);
      case 321: return launch_shape<D, E4M3, SINKS, 2, 1, 1, 32, 32>(a, st);
      case 322: return launch_shape<D, E4M3, SINKS, 2, 1, 2, 32, 64>(a, st);
      case 324: return launch_shape<D, E4M3, SINKS, 2, 1, 4, 32, 128>(a, st);
    }
  }
  switch (rows * 10 + key_groups) {
    case 641: return launch_shape<D, E4M3, SINKS, 2, 2, 1, 32, 32>(a, st);
    case 642: return launch_shape<D, E4M3, SINKS, 2, 2, 2, 32, 64>(a, st);
    case 644: return launch_shape<D, E4M3, SINKS, 2, 2, 4, 32, 128>(a, st);
    default: return launch_shape<D, E4M3, SINKS, 2, 4, 1, 64, 64>(a, st);
  }
}

}  // namespace

AttnPlan attn_plan(int T, int B, int Hkv, int G, int D, int max_q_len, long long max_seq_len, int window, bool sinks,
                   bool e4m3) {
  AttnPlan p;
  const long long most = (long long)max_q_len * G;  // rows of the longest request
  // Keys a tile reads at most (a window's first block starts up to 63 keys before it).
  long long span = max_seq_len;
  if (window > 0) span = span < (long long)window + max_q_len + 63 ? span : (long long)window + max_q_len + 63;
  auto direct = [&](int rows) { return (most + rows - 1) / rows; };
  auto by_rows = [&](int rows) { return (long long)T * G / rows + B; };
  auto work_groups = [&](int rows) {
    const long long d = direct(rows) * B, r = by_rows(rows);
    return (d < r ? d : r) * Hkv;
  };
  // Rows of a tile. All of a request's rows, up to 64, so that its keys are read once; for prompts 128 where that fills
  // the CUs twice, with the keys cut into chunks of 1024 or more, or where 64 would more than fill them, else 64 (8 key
  // heads, 32 heads, 128 / 64 rows: 1024 tokens over 4096 keys 111 / 130 us; 1024 tokens over none 36 / 29 us; 4 times 300
  // tokens over 1000 keys 55 / 64 us). Over short sequences, where the
  // time is that of the longest chain of one work-group, the smallest tile that leaves every work-group its own CU
  // (128 tokens over none: 7.4 us with 16 rows, 9.7 with 32, 10.5 with 64, 13.3 with 128; 2 times 290 tokens, 4 key
  // heads, 12 heads: 12.6 us with 32, 17.0 with 16 in two rounds, 18.5 with 64).
  if (most <= 16 || (span <= 1024 && work_groups(16) <= 256))
    p.rows = 16;
  else if (most <= 32 || (span <= 1024 && work_groups(32) <= 256))
    p.rows = 32;
  else
    p.rows = most > 64 && (work_groups(64) > 512 || work_groups(128) * (span < 2048 ? 1 : span / 1024) >= 512) ? 128 : 64;
  p.per_req = direct(p.rows) * B <= by_rows(p.rows) ? (int)direct(p.rows) : 0;
  p.tiles = (int)(p.per_req ? direct(p.rows) * B : by_rows(p.rows));
  // Chunks of keys. A split costs its partials and the join's launch, so fewer tiles than CUs are cut only into as many
  // work-groups as run at once (one a CU with up to 32 rows, two above, the second only for chunks of 1024 or more),
  // into chunks of at least 256 keys: one more would wait for a second round (217 tiles of 290 keys: 12.6 us
  // whole, 23.8 us in two chunks). And no chunk is so long that the rest waits for its CU: with tiles bound by
  // the cache's bytes, 4608 keys of 128 (of 32 requests with 8 key heads, over 100 to 8192 keys: 129 us, whole 136 us;
  // one of 30000 keys among 500: 87 us, in chunks of 16384 200 us; the price where all are as long, 8000 keys: 203 us,
  // whole 187 us), as many times longer as a CU has other tiles to run; with 128-row tiles, whose partials are
  // larger and whose length hides in their products, 16384 (2048 prompt tokens over 14336: 500 us whole, 560 us in
  // chunks of 4096). At most 8 chunks of a guess that is far too long, each of which costs a work-group that finds
  // nothing (128 requests of 2000 8-bit keys and a guess of 131072: 155 us, without that 181 us).
  const long long wgs = (long long)p.tiles * Hkv;
  // Key groups of up to 32 rows: four share a long sequence and end together. Over short ones, with more tiles than
  // CUs, the start and end of a work-group count, and two or four smaller ones to a CU hide them (8 key heads, 128
  // requests of one token: over 50 keys 13.5 us to 42.3 us with one key group, over 1 to 1024 keys 61 us to 77 us; 64
  // requests over 1 to 512 keys 21.5 us to 26.5 us with two; 128 over 1 to 4096 keys 243 us to 209 us).
  p.key_groups = p.rows > 64 ? 1 : p.rows > 32 ? 2 : 4;
  if (p.rows <= 32 && !sinks) {
    if (span <= 1024 && wgs > 512) p.key_groups = 1;
    if (span <= 512 && wgs > 256 && wgs <= 512) p.key_groups = 2;
  }
  // Sequences beyond a window all have as many keys to read, so the places beside a work-group matter up to longer ones.
  // That is so of any window; it is looked at for calls with first tokens only, and a window without them keeps the rule
  // above (128 requests of one token over an 8-bit cache, 8 key heads, window 2000, up to twice as many keys: 91 us with
  // first tokens and 114 us without; 64 over a bf16 cache, window 512: 28 and 34). (One token, 8 key heads, sequences of up to
  // twice the window; us with one / two / four key groups:
  // 64 requests, window 300 30 / 22 / 27, 1000 57 / 42 / 48, 4000 172 / 162 / 163; 128 requests, 300 35 / 39 / 59,
  // 2000 165 / 164 / 166, 4000 293 / 301 / 287; over 8-bit caches, whose work-groups are two to a CU already, 128
  // requests with two / four, 300 25 / 31, 1000 48 / 48, 2000 108 / 101).
  if (p.rows <= 32 && sinks) {
    if (e4m3)
      p.key_groups = wgs > 512 && span <= 1280 ? 2 : 4;
    else if (wgs > 256)
      p.key_groups = wgs <= 512 ? 2 : span <= 2560 ? 1 : 4;
  }
  long long want = wgs < 256 ? 256 / wgs : 1, cap = 16384;
  if (p.rows > 32) {
    long long twice = wgs < 512 ? 512 / wgs : 1;
    if (twice > span / 1024) twice = span / 1024;
    if (want < twice) want = twice;
  }
  if (p.rows <= 64) {
    cap = 4608 * 128 / D * (wgs > 1024 ? wgs / 1024 : 1);
    if (cap < span / 8) cap = span / 8;
  }
  long long chunk = (span + want - 1) / want;
  if (chunk > cap) chunk = cap;
  chunk = (chunk + 127) / 128 * 128;
  // (with first tokens 128 keys where every chunk then has a CU: one token, window 1000 10.3 us to 11.4 us)
  const long long least = sinks && p.rows <= 32 && span > 256 && wgs * ((span + 127) / 128) <= 256 ? 128 : 256;
  if (chunk < least) chunk = least;
  long long n = (span + chunk - 1) / chunk;
  if (n < 1) n = 1;
  // 64 rows: two key groups and two work-groups a CU, but four and one where there is no second one (512 prompt tokens
  // over none 15.6 us to 18.1 us; more work-groups than that: 1024 tokens 35 us to 30 us), and one over short
  // sequences of many requests (128 of 8 tokens and 64 heads over 60 keys: 26 us to 37 us)
  if (p.rows == 64 && wgs * n <= 256) p.key_groups = 4;
  if (p.rows == 64 && span <= 1024 && wgs >= 1024) p.key_groups = 1;
  p.chunk = (int)chunk;
  p.n_chunks = (int)n;
  // more work-groups than the CUs hold at once: the longest sequences go first, so that none starts last
  // (128 requests of 1 to 4096 keys over an 8-bit cache: 134 us against 173 us in the batch's order)
  p.by_length = p.per_req > 0 && B > 1 && B <= 128 && wgs * n > 256;
  const size_t rows = (size_t)p.n_chunks * p.tiles * Hkv * p.rows;
  p.part_o = 256;
  p.part_ml = p.part_o + (n > 1 ? (rows * D * 4 + 255) / 256 * 256 : 0);
  p.total = p.part_ml + (n > 1 ? (rows * 8 + 255) / 256 * 256 : 0);
  return p;
}

// Bytes that are enough for attn_plan of these sizes and of all smaller ones (its workspace alone is not: fewer tokens
// may be cut into more chunks). A plan's partials are n_chunks * tiles * Hkv * rows rows. Chunks that fill the CUs have 256
// keys (128 with first tokens) or more and leave at most 256 work-groups (up to 32 rows) or 512. Chunks that bound a work-group's length are at
// most nine (an eighth of the keys rounds down) of 4608 * 128 / D keys or more in tiles that hold a request's rows; lower
// tiles than that are chosen for short sequences or few work-groups, of which such chunks leave 512 at most. 128-row tiles
// have chunks of 16384 keys.
size_t attn_workspace(int T, int B, int Hkv, int G, int D, int max_q_len, long long max_seq_len, int window, bool sinks) {
  const long long most = max_q_len > 0 ? (long long)max_q_len * G : G;
  long long span = max_seq_len, rows = 0;
  if (window > 0) span = span < (long long)window + max_q_len + 63 ? span : (long long)window + max_q_len + 63;
  auto chunks = [&](long long keys) { return (span + keys - 1) / keys; };
  for (int r = 16; r <= 128; r *= 2) {
    const long long direct = (most + r - 1) / r * r * B, by_rows = (long long)T * G + (long long)r * B;
    const long long padded = (direct < by_rows ? direct : by_rows) * Hkv;
    long long fill = (r <= 32 ? 256 : 512) * (long long)r;
    const long long most_chunks = chunks(sinks ? 128 : 256);
    if (fill > padded * most_chunks) fill = padded * most_chunks;
    if (most_chunks > 1 && rows < fill) rows = fill;
    long long n = r == 128 ? chunks(16384) : chunks(4608 * 128 / D);
    if (r < 128 && n > 9) n = 9;
    const long long bound = n * (r == 128 ? padded : (long long)r * B * Hkv);
    if (n > 1 && rows < bound) rows = bound;
    if (most <= r) break;
  }
  const size_t o = (size_t)rows * D * 4, ml = (size_t)rows * 8;
  return 256 + (o + 255) / 256 * 256 + (ml + 255) / 256 * 256;
}

template <bool SINKS>
static hipError_t launch(const PagedAttnArgs& a, const AttnPlan& p, hipStream_t st) {
  if (a.D == 128)
    return a.e4m3 ? launch_d<128, true, SINKS>(a, p.rows, p.key_groups, st)
                  : launch_d<128, false, SINKS>(a, p.rows, p.key_groups, st);
  return a.e4m3 ? launch_d<64, true, SINKS>(a, p.rows, p.key_groups, st)
                : launch_d<64, false, SINKS>(a, p.rows, p.key_groups, st);
}
hipError_t launch_paged_attention(const PagedAttnArgs& a, const AttnPlan& p, hipStream_t st) {
  return a.sinks > 0 ? launch<true>(a, p, st) : launch<false>(a, p, st);
}

}  // namespace mds
