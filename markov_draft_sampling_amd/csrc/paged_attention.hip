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
// the second product (relative 2^-9 each, the products' own input type); l
// sums the unrounded p.
//
// Rows. The G query heads of one key head read the same keys, so a request's
// rows are its (token, head in group) pairs, token-major: tiles of up to 64
// rows, and every key and value is read from HBM once per tile.
//
// Split. Few rows means few work-groups, so the keys are cut into chunks of
// work-groups as well, whose (m, l, o) a second kernel joins.
//
// Wave. Four waves of a work-group take the chunk's blocks of 32 keys in turn,
// each with its own part of LDS and without a barrier: a block's keys and
// values are copied straight into LDS (16 bytes a lane, no registers), two to
// four blocks in flight per wave, 16-byte slots XOR-swizzled by row. Both
// products are computed transposed on the matrix cores (16x16x32 bf16): the
// scores as S^T = K Q^T, whose result layout (lane: one row, 4 keys of each
// 16) is the operand layout of P^T once the keys of a block are taken in the
// order {4 g .. 4 g + 3, 16 + 4 g ..}: no lane exchanges probabilities. Values
// are read column-wise from LDS by the transposing LDS reads in that order.
// 8-bit caches are widened to bf16 (exactly) after the LDS read; the key scale
// joins the softmax scale, the value scale the final division.
#include "mds_device.h"
#include "mds_internal.h"

namespace mds {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#define MDS_LDS __attribute__((address_space(3)))
#define MDS_GLOBAL __attribute__((address_space(1)))

constexpr float kLn2 = 0x1.62e430p-1f;
constexpr float kRescale = 8.0f;  // a maximum's growth (base 2) up to which the running one stays

// One request's row tile: which rows, and which keys its rows can see.
struct Tile {
  int b, slot, q0, n, r0, rows;  // request, state slot, first token, tokens, first row, rows (0: nothing to do)
  int seq, lim;                  // sequence length, and that within the block table
  int lo, hi;                    // keys that some row sees: [lo, hi)
  int base;                      // lo rounded down to a block
  int chunks;                    // chunks with keys (at least 1)
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

template <int ROWS>
__device__ __forceinline__ Tile find_tile(const PagedAttnArgs& a, int tile, uint32_t& bad) {
  Tile t;
  t.rows = 0;
  if (a.per_req > 0) {
    t.b = tile / a.per_req;
    t.r0 = (tile - t.b * a.per_req) * ROWS;
  } else {
    // request b's tiles start at floor(q0 G / ROWS) + b: enough for its rows,
    // since ceil(x) of its rows is at most the step to the next request's start
    const int lane = threadIdx.x & 63;
    int cnt = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
      const int b = b0 + lane;
      uint32_t dummy = 0;
      const int q = clamp_tok(a, a.query_start[min(b, a.B - 1)], dummy);
      const bool before = b < a.B && (int)((unsigned)q * (unsigned)a.G / ROWS) + b <= tile;
      cnt += __popcll(__ballot(before));
    }
    if (cnt == 0) return t;
    t.b = cnt - 1;
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
  t.rows = min(ROWS, t.n * a.G - t.r0);
  if (t.n <= 0 || t.rows <= 0) {
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
  t.base = t.lo & ~31;
  t.chunks = min(max((t.hi - t.base + a.chunk - 1) / a.chunk, 1), a.n_chunks);
  return t;
}

// Writes 8 (or D / 16) columns of one output row: o / l, scaled, in bf16; a row without keys is zero.
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

// Transposing LDS reads, a group of 16 lanes reading 4 (8) keys of 16 columns, and the wait for them: as
// one asm block, since the compiler would have the intrinsics wait for every copy in flight.
// F[q]: the 4 keys at a[q] and the 4 at a[q] + OFF.
template <int OFF>
__device__ __forceinline__ void read_tr16(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, bf16x8 (&F)[4]) {
  u32x2 x[8];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8\n\t"
      "ds_read_b64_tr_b16 %1, %8 offset:%12\n\t"
      "ds_read_b64_tr_b16 %2, %9\n\t"
      "ds_read_b64_tr_b16 %3, %9 offset:%12\n\t"
      "ds_read_b64_tr_b16 %4, %10\n\t"
      "ds_read_b64_tr_b16 %5, %10 offset:%12\n\t"
      "ds_read_b64_tr_b16 %6, %11\n\t"
      "ds_read_b64_tr_b16 %7, %11 offset:%12\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
      : "v"(a0), "v"(a1), "v"(a2), "v"(a3), "n"(OFF)
      : "memory");
#pragma unroll
  for (int q = 0; q < 4; ++q)
    F[q] = __builtin_bit_cast(bf16x8, u32x4{x[2 * q][0], x[2 * q][1], x[2 * q + 1][0], x[2 * q + 1][1]});
}
__device__ __forceinline__ void read_tr8(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, i32x2 (&x)[4]) {
  asm volatile(
      "ds_read_b64_tr_b8 %0, %4\n\t"
      "ds_read_b64_tr_b8 %1, %5\n\t"
      "ds_read_b64_tr_b8 %2, %6\n\t"
      "ds_read_b64_tr_b8 %3, %7\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
      : "v"(a0), "v"(a1), "v"(a2), "v"(a3)
      : "memory");
}

// D: head dimension; E4M3: 8-bit cache; NB: 16-row blocks of the row tile
template <int D, bool E4M3, int NB>
__global__ __launch_bounds__(256, 1) void attn_kernel(PagedAttnArgs a) {
  constexpr int ROWS = NB * 16;
  constexpr int RB = D * (E4M3 ? 1 : 2);       // bytes of a key (or value)
  constexpr int SPR = RB / 16;                 // 16-byte slots of it
  constexpr int RPI = 64 / SPR;                // keys per copy instruction (1 KB)
  constexpr int NI = 32 / RPI;                 // copy instructions for a block's keys (as many for its values)
  constexpr int kPart = 32 * RB;               // bytes of a block's keys
  constexpr int kStage = 2 * kPart;
  constexpr int NST = kStage >= 16384 ? 2 : 4; // blocks in flight per wave
  constexpr int NS = D / 32;                   // 32-wide slices of the first product
  constexpr int ND = D / 16;                   // 16-wide column blocks of the second
  // one array per block in flight: the copies into one are not taken for writes to another
  __shared__ __attribute__((aligned(16))) unsigned char s0[4 * kStage], s1[4 * kStage];
  __shared__ __attribute__((aligned(16))) unsigned char s2[NST > 2 ? 4 * kStage : 16], s3[NST > 2 ? 4 * kStage : 16];
  __shared__ float s_m[4][ROWS], s_l[4][ROWS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int h = blockIdx.x % (unsigned)a.Hkv;
  const int ct = blockIdx.x / (unsigned)a.Hkv;
  const int c = ct / a.tiles, tile = ct - c * a.tiles;

  uint32_t bad = 0;
  const Tile t = find_tile<ROWS>(a, tile, bad);
  if (t.rows <= 0 || c >= t.chunks) {
    if (bad && tid == 0) set_status(a.status, bad);
    return;
  }
  const int c0 = t.base + c * a.chunk;
  const int lo = max(t.lo, c0), hi = c == a.n_chunks - 1 ? t.hi : min(t.hi, c0 + a.chunk);
  const int nblk = hi > lo ? (hi - c0 + 31) >> 5 : 0;
  const int nmy = nblk > w ? (nblk - w + 3) >> 2 : 0;  // this wave's blocks: w, w + 4, ..

  // the rows: row R of the request is head R % G of token R / G; rows past the tile repeat the last
  bf16x8 Q[NB][NS];
  int mlo[NB], mhi[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int R = t.r0 + min(nb * 16 + lr, t.rows - 1);
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
  // keys that every row sees: blocks inside need no mask
  int all_lo, all_hi, x0, x1;
  token_keys(a, t, (t.r0 + t.rows - 1) / a.G, all_lo, x1);
  token_keys(a, t, t.r0 / a.G, x0, all_hi);
  all_lo = max(all_lo, lo);
  all_hi = min(all_hi, hi);
  const float sc = a.scale_log2 * (a.k_scale ? a.k_scale[h] : 1.0f);

  // copies: instruction p of a block fills keys RPI p .. of it; lane l lands in row r = RPI p + l / SPR,
  // slot l % SPR, which holds the row's slot (l % SPR) ^ swizzle(r)
  auto kswz = [](int r) { return SPR == 16 ? r & 15 : SPR == 8 ? (r >> 1) & 7 : (r >> 2) & 3; };
  auto vswz = [](int r) {
    return E4M3 ? (SPR == 8 ? ((r >> 1) & 3) | ((r >> 2) & 4) : ((r >> 2) & 1) | ((r >> 3) & 2))
                : (SPR == 16 ? (r & 7) * 2 : ((r >> 1) & 3) * 2);
  };
  const int lrow = lane / SPR, lslot = lane % SPR;
  uint32_t ko[NI], vo[NI];
#pragma unroll
  for (int p = 0; p < NI; ++p) {
    const int r = p * RPI + lrow;
    ko[p] = (uint32_t)((r & 15) * (int)a.k_ts) + (uint32_t)((lslot ^ kswz(r)) * 16);
    vo[p] = (uint32_t)((r & 15) * (int)a.v_ts) + (uint32_t)((lslot ^ vswz(r)) * 16);
  }
  const int32_t* trow = a.block_table + (size_t)t.slot * a.max_pages;
  const char* kb_h = (const char*)a.k_pages + h * a.k_hs;
  const char* vb_h = (const char*)a.v_pages + h * a.v_hs;
  const int pmask = (1 << a.page_log2) - 1;
  // Page ids of the wave's blocks i0 .. i0 + 31: lane 2 (i - i0) + j has the page of half j (16 keys, in one
  // page) of block i. Keys outside [lo, hi) repeat the nearest one inside: what lies behind a sequence's end
  // is never read, and their probability is zero.
  int pages = 0;
  auto load_pages = [&](int i0) {
    const int kh = c0 + (w + 4 * (i0 + (lane >> 1))) * 32 + 16 * (lane & 1);
    pages = trow[min(max(kh, lo), hi - 1) >> a.page_log2];
    if ((unsigned)pages >= (unsigned)a.n_pages) {
      pages = 0;
      bad |= kStatusBadPage;
    }
  };
  auto copy_one = [&](const char* p, unsigned char* to) {
    __builtin_amdgcn_global_load_lds((const MDS_GLOBAL void*)p, (MDS_LDS void*)to, 16, 0, 0);
  };
  auto copy_block = [&](unsigned char* buf, int i) {
    if (i && (i & 31) == 0) load_pages(i);
    const int k0 = c0 + (w + 4 * i) * 32;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int kh = k0 + 16 * j;
      const int kc = min(max(kh, lo), hi - 1);
      const int pg = __builtin_amdgcn_readlane(pages, 2 * (i & 31) + j);
      const char* kp = kb_h + pg * a.k_ps + (kc & pmask) * a.k_ts;
      const char* vp = vb_h + pg * a.v_ps + (kc & pmask) * a.v_ts;
      unsigned char* to = buf + j * (NI / 2) * 1024;
      if (k0 >= lo && k0 + 32 <= hi) {
#pragma unroll
        for (int p = 0; p < NI / 2; ++p) {
          copy_one(kp + ko[j * (NI / 2) + p], to + p * 1024);
          copy_one(vp + vo[j * (NI / 2) + p], to + kPart + p * 1024);
        }
      } else {
#pragma unroll
        for (int p = 0; p < NI / 2; ++p) {
          const int q = j * (NI / 2) + p, r = (q * RPI + lrow) & 15;
          const int d = min(max(kh + r, lo), hi - 1) - kc - r;  // from the row's own place to the key copied
          copy_one(kp + (uint32_t)((int)ko[q] + d * (int)a.k_ts), to + p * 1024);
          copy_one(vp + (uint32_t)((int)vo[q] + d * (int)a.v_ts), to + kPart + p * 1024);
        }
      }
    }
  };

  // LDS offsets of a lane's column reads of the values, by block of 16 columns
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
  float m[NB], l[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m[nb] = -INFINITY;
    l[nb] = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) O[nb][d] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  auto widen = [](uint32_t v, bool up) {
    return up ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
  };
  auto block = [&](const unsigned char* buf, int i) {
    const int k0 = c0 + (w + 4 * i) * 32;
    floatx4 S[2][NB];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
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
    // lane: row lr of each nb, keys k0 + 16 kb + 4 lg + i
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[kb][nb] *= sc;
    if (k0 < all_lo || k0 + 32 > all_hi) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = k0 + 16 * kb + 4 * lg + e;
            S[kb][nb][e] = ((key >= mlo[nb]) & (key < mhi[nb])) ? S[kb][nb][e] : -INFINITY;
          }
    }
    float top[NB];
    bool grow = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const floatx4 x = S[0][nb], y = S[1][nb];
      top[nb] = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])));
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
        l[nb] *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) O[nb][d] *= f;
      }
    }
    bf16x8 P[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float mm = m[nb] == -INFINITY ? 0.0f : m[nb];  // a row without keys so far: every p is 0
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(S[e >> 2][nb][e & 3] - mm);
      l[nb] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
#pragma unroll
      for (int e = 0; e < 8; ++e) P[nb][e] = (__bf16)p[e];
    }
    // values: lane column d = 16 db + lr, keys 4 lg + (0 .. 3) and 16 + 4 lg + (0 .. 3)
    const uint32_t vb = (uint32_t)(uintptr_t)(MDS_LDS const void*)buf + kPart;
#pragma unroll
    for (int d0 = 0; d0 < ND; d0 += 4) {
      bf16x8 Vf[4];
      if constexpr (E4M3) {
        i32x2 x[4];
        read_tr8(vb + va[d0], vb + va[d0 + 1], vb + va[d0 + 2], vb + va[d0 + 3], x);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          Vf[q] = __builtin_bit_cast(bf16x8, u32x4{widen(x[q][0], false), widen(x[q][0], true), widen(x[q][1], false),
                                                   widen(x[q][1], true)});
      } else {
        read_tr16<16 * RB>(vb + va[d0], vb + va[d0 + 1], vb + va[d0 + 2], vb + va[d0 + 3], Vf);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          O[nb][d0 + q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(Vf[q], P[nb], O[nb][d0 + q], 0, 0, 0);
    }
  };

  unsigned char* const buf[4] = {s0 + w * kStage, s1 + w * kStage, NST > 2 ? s2 + w * kStage : s0,
                                 NST > 2 ? s3 + w * kStage : s1};
  if (nmy > 0) load_pages(0);
#pragma unroll
  for (int i = 0; i < NST; ++i)
    if (i < nmy) copy_block(buf[i], i);
#pragma nounroll
  for (int i0 = 0; i0 < nmy; i0 += NST) {
#pragma unroll
    for (int j = 0; j < NST; ++j) {
      const int i = i0 + j;
      if (i < nmy) {
        // block i has landed: at most the NST - 1 blocks after it are still in flight
        constexpr int N = (NST - 1) * 2 * NI;
        asm volatile("" ::: "memory");
        if (i + NST <= nmy)
          __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
        else
          __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));  // near the end: all of them
        asm volatile("" ::: "memory");
        block(buf[j], i);
        if (i + NST < nmy) {
          // the block's LDS reads have returned (their values were used): its place is free
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          copy_block(buf[j], i + NST);
        }
      }
    }
  }
  if (bad) set_status(a.status, bad);

  // join the four waves, 16 rows at a time: o scaled to the common maximum through LDS, summed by
  // 16 threads a row
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    l[nb] += __shfl_xor(l[nb], 16);
    l[nb] += __shfl_xor(l[nb], 32);
    if (lg == 0) {
      s_m[w][nb * 16 + lr] = m[nb];
      s_l[w][nb * 16 + lr] = l[nb];
    }
  }
  __syncthreads();
  const int orow = tid >> 4, od = (tid & 15) * (D / 16);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    if (nb * 16 >= t.rows) break;
    const float M = fmaxf(fmaxf(s_m[0][nb * 16 + lr], s_m[1][nb * 16 + lr]),
                          fmaxf(s_m[2][nb * 16 + lr], s_m[3][nb * 16 + lr]));
    const float f = m[nb] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[nb] - M);
    float* so = (float*)(s0 + w * kStage);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      const floatx4 x = m[nb] == -INFINITY && !(l[nb] != l[nb]) ? floatx4{0.0f, 0.0f, 0.0f, 0.0f} : O[nb][d] * f;
      *(floatx4*)(so + lr * D + (((4 * d + lg) ^ lr) * 4)) = x;
    }
    __syncthreads();
    const int row = nb * 16 + orow;
    if (row < t.rows) {
      const float Mr = fmaxf(fmaxf(s_m[0][row], s_m[1][row]), fmaxf(s_m[2][row], s_m[3][row]));
      float L = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float li = s_l[i][row];
        L += s_m[i][row] == -INFINITY && li == li ? 0.0f : li * __builtin_amdgcn_exp2f(s_m[i][row] - Mr);
      }
      float o[D / 16];
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        floatx4 x = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x += *(const floatx4*)((const float*)(s0 + i * kStage) + orow * D + (((od / 4 + q) ^ orow) * 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) o[q * 4 + e] = x[e];
      }
      if (a.n_chunks == 1 || t.chunks == 1) {
        store_row<D / 16>(a, t, row, h, od, o, Mr, L);
      } else {
        const size_t pr = ((size_t)ct * a.Hkv + h) * ROWS + row;
        float* po = a.part_o + pr * D + od;
#pragma unroll
        for (int q = 0; q < D / 64; ++q) *(floatx4*)(po + q * 4) = floatx4{o[q * 4], o[q * 4 + 1], o[q * 4 + 2], o[q * 4 + 3]};
        if ((tid & 15) == 0) a.part_ml[pr] = make_float2(Mr, L);
      }
    }
    __syncthreads();
  }
}

// Joins the chunks of a row tile: o = sum 2^(m_c - M) o_c / sum 2^(m_c - M) l_c.
template <int D, int ROWS>
__global__ __launch_bounds__(256) void attn_join_kernel(PagedAttnArgs a) {
  const int tid = threadIdx.x;
  const int h = blockIdx.x % (unsigned)a.Hkv;
  const int tile = blockIdx.x / (unsigned)a.Hkv;
  uint32_t bad = 0;
  const Tile t = find_tile<ROWS>(a, tile, bad);
  if (t.rows <= 0 || t.chunks <= 1) return;
  const int od = (tid & 15) * (D / 16);
  const size_t step = (size_t)a.tiles * a.Hkv * ROWS;
  for (int row = blockIdx.y * 16 + (tid >> 4); row < t.rows; row += 16 * gridDim.y) {
    const size_t pr = ((size_t)tile * a.Hkv + h) * ROWS + row;
    float M = -INFINITY;
    for (int c = 0; c < t.chunks; ++c) M = fmaxf(M, a.part_ml[pr + c * step].x);
    float L = 0.0f, o[D / 16];
#pragma unroll
    for (int e = 0; e < D / 16; ++e) o[e] = 0.0f;
    for (int c = 0; c < t.chunks; ++c) {
      const float2 ml = a.part_ml[pr + c * step];
      if (ml.x == -INFINITY && ml.y == ml.y) continue;  // no keys of the row in this chunk
      const float f = __builtin_amdgcn_exp2f(ml.x - M);
      L += ml.y * f;
      const float* po = a.part_o + (pr + c * step) * D + od;
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        const floatx4 x = *(const floatx4*)(po + q * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[q * 4 + e] += x[e] * f;
      }
    }
    store_row<D / 16>(a, t, row, h, od, o, M, L);
  }
}

template <int D, bool E4M3, int NB>
hipError_t launch_nb(const PagedAttnArgs& a, hipStream_t st) {
  const long long wgs = (long long)a.tiles * a.Hkv;
  hipLaunchKernelGGL((attn_kernel<D, E4M3, NB>), dim3((unsigned)(wgs * a.n_chunks)), dim3(256), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.n_chunks == 1) return e;
  hipLaunchKernelGGL((attn_join_kernel<D, NB * 16>), dim3((unsigned)wgs, NB), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <int D, bool E4M3>
hipError_t launch_d(const PagedAttnArgs& a, int rows, hipStream_t st) {
  switch (rows) {
    case 16: return launch_nb<D, E4M3, 1>(a, st);
    case 32: return launch_nb<D, E4M3, 2>(a, st);
    default: return launch_nb<D, E4M3, 4>(a, st);
  }
}

}  // namespace

AttnPlan attn_plan(int T, int B, int Hkv, int G, int D, int max_q_len, long long max_seq_len, int window) {
  AttnPlan p;
  const long long most = (long long)max_q_len * G;  // rows of the longest request
  p.rows = most <= 16 ? 16 : most <= 32 ? 32 : 64;
  const long long direct = (most + p.rows - 1) / p.rows;
  const long long by_rows = (long long)T * G / p.rows + B;
  p.per_req = direct * B <= by_rows ? (int)direct : 0;
  p.tiles = (int)(p.per_req ? direct * B : by_rows);
  // keys a tile reads at most, cut so that about four work-groups a CU result
  long long span = max_seq_len;
  if (window > 0) span = span < (long long)window + max_q_len ? span : (long long)window + max_q_len;
  const long long wgs = (long long)p.tiles * Hkv;
  long long want = (4 * 256 + wgs - 1) / wgs;
  long long chunk = (span + 32 + want - 1) / want;
  chunk = (chunk + 127) / 128 * 128;
  if (chunk < 256) chunk = 256;
  long long n = (span + 31 + chunk - 1) / chunk;
  if (n < 1) n = 1;
  p.chunk = (int)chunk;
  p.n_chunks = (int)n;
  const size_t rows = (size_t)p.n_chunks * p.tiles * Hkv * p.rows;
  p.part_o = 256;
  p.part_ml = p.part_o + (n > 1 ? (rows * D * 4 + 255) / 256 * 256 : 0);
  p.total = p.part_ml + (n > 1 ? (rows * 8 + 255) / 256 * 256 : 0);
  return p;
}

hipError_t launch_paged_attention(const PagedAttnArgs& a, const AttnPlan& p, hipStream_t st) {
  if (a.D == 128) return a.e4m3 ? launch_d<128, true>(a, p.rows, st) : launch_d<128, false>(a, p.rows, st);
  return a.e4m3 ? launch_d<64, true>(a, p.rows, st) : launch_d<64, false>(a, p.rows, st);
}

}  // namespace mds
