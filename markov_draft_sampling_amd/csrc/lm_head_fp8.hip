// LM head from an 8-bit matrix: logits[m, v] = sum over blocks j of 128
// columns of sx[m, j] sw[v / 128, j] sum_c qx[m, 128 j + c] qw[v, 128 j + c],
// with qw e4m3 and one float32 scale for each 128 x 128 block of the matrix,
// and the hidden rows quantised on the way in: for each row and 128 columns
// sx = max(amax, 2^-100) / 448 and qx = e4m3(x / sx), nearest even.
//
// Codes widen to bf16 exactly and their products are summed by the bf16 matrix
// instruction, whose sums are float32: the 8-bit one, twice as fast, drops low
// bits of its products before they are added (measured on 16 x 16 x 128 of
// normal codes: 1.5e-5 of the result's norm off, against 9e-9 here), which
// a float32 logit shows. A block's sum (of up to 32 rows: each half block's, of
// 64 columns) is scaled and added to the float32 total.
//
// The matrix is kept in tiles of 16 rows by 128 columns in operand order
// (fp8_tile_index): a wave copies its operands as 1 KB runs into its own part
// of LDS and widens them in registers; which columns a lane holds does not
// matter as long as both operands agree. The quantising
// kernel writes the hidden rows' codes in the same order, chunk (128 columns)
// by chunk with the rows' scales behind, so that a chunk goes into LDS as one
// linear copy without registers, shared by the waves.
//
// For few rows the call is bound by the matrix's V * H bytes (7 rows, H = 4096:
// 145 us and 5.7 TB/s at V = 200064, 29.4 us at V = 32000, 4 of them the hidden
// rows' launch); at 224 rows by the matrix cores and the operand reads from LDS
// (V = 200064: 367 to 375 us, 0.98 to 1.0 PFLOP/s), which is why a wave takes 64
// vocabulary rows: every hidden operand serves four products. (The pairs at the
// rules below are from one run each; cards differ by up to 8%.)
#include "mds_device.h"
#include "mds_serve.h"

namespace mds {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 0x1p-100f;  // a block of zeros gets a scale it can be divided by
constexpr int kStagger = 5;  // chunk offset between consecutive work-groups

__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d) {
  const int p = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, p, true);
}
// Values past the largest (the quotient by a rounded scale) go to the largest; NaN stays NaN.
__device__ __forceinline__ float clamp_e4m3(float y) {
  return y != y ? y : fminf(fmaxf(y, -kE4m3Max), kE4m3Max);
}

// Two codes of a word to two bf16 (exact: every e4m3 value is one)
__device__ __forceinline__ uint32_t widen(uint32_t v, bool up) {
  return up ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true))
            : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
}
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi) {
  return __builtin_bit_cast(bf16x8, u32x4{widen(lo, false), widen(lo, true), widen(hi, false), widen(hi, true)});
}

// Hidden rows: a wave per 4 rows and 128 columns, a lane 8 columns of a row (the call waits for it: short rows of
// divisions a lane, 4.7 us with 32 columns).
__global__ __launch_bounds__(256) void quant_rows_kernel(LmHeadFp8Args a) {
  const int HB = a.H >> 7, MBt = (a.M + 15) >> 4;
  // a work-group per 16 rows and 128 columns
  const int mb = blockIdx.x % (unsigned)MBt, j = blockIdx.x / (unsigned)MBt;
  const int r = threadIdx.x >> 4, m = mb * 16 + r, c0 = (threadIdx.x & 15) * 8;
  const int mt = mb / a.mb, mi = mb - mt * a.mb;
  uint8_t* stage = a.xq + ((size_t)mt * HB + j) * fp8_stage_bytes(a.mb);
  float x[8];
  u32x4 v = u32x4{0, 0, 0, 0};
  if (m < a.M) v = *(const u32x4*)(a.hidden + (long long)m * a.hidden_rs + j * 128 + c0);
  float am = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v[i] << 16);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    am = fmaxf(am, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
  }
#pragma unroll
  for (int i = 1; i < 16; i *= 2) am = fmaxf(am, __shfl_xor(am, i));
  const float s = am / kE4m3Max;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = clamp_e4m3(x[i] / s);
  *(u32x2*)(stage + mi * 2048 + (c0 >> 4) * 256 + r * 16 + (c0 & 8)) =
      u32x2{quant4(x[0], x[1], x[2], x[3]), quant4(x[4], x[5], x[6], x[7])};
  if (c0 == 0) ((float*)(stage + a.mb * 2048))[mi * 16 + r] = s;
}

// Work-group barrier once this wave's copies of the next chunk have landed in
// LDS: at most N newer memory operations stay in flight.
template <int N>
__device__ __forceinline__ void chunk_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// buffer descriptor of n bytes from p (raw bytes: word 3), kept in scalar registers
__device__ __forceinline__ u32x4 words_at(const uint8_t* p, int n) {
  const uint64_t q = (uint64_t)p;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)q),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(q >> 32)),
               (uint32_t)__builtin_amdgcn_readfirstlane(n), 0x00020000u};
}
// 16 bytes a lane straight into LDS, as assembly: every wait for these copies is the kernels' own, and the compiler, which
// cannot tell the copies in flight apart, would wait for all of them before every LDS read. (m0, the LDS address, has no
// other use in these kernels; the load may read it one wait state after the scalar write at the earliest.) r: a
// descriptor's four words; ONCE: not kept in the caches.
template <bool ONCE>
__device__ __forceinline__ void copy_1k_asm(u32x4 r, const uint8_t* to, int lane_off, int off) {
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)to;
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
                 :: "s"(lds), "v"(lane_off), "s"(r), "s"(off) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(lds), "v"(lane_off), "s"(r), "s"(off) : "memory");
}

// acc += (sx of the row * sw) * (A times the hidden operands of 64 columns at xb, a block every 2 KB). One row
// block after the other, operand reads one block ahead, scaling one block behind (the order is pinned: left alone
// the compiler holds every block's sums at once).
template <int MB>
__device__ __forceinline__ void scaled_products(const uint8_t* xb, const float* sx, float sw, const bf16x8 (&A)[2],
                                                floatx4 (&acc)[MB]) {
  u32x4 raw = *(const u32x4*)xb;
  float s = sx[0], sp = 0.0f;
  floatx4 z, zp;
#pragma unroll
  for (int mb = 0; mb <= MB; ++mb) {
    u32x4 rn = raw;
    float sn = s;
    if (mb + 1 < MB) {
      rn = *(const u32x4*)(xb + (mb + 1) * 2048);
      sn = sx[(mb + 1) * 16];
    }
    if (mb < MB) {
      const bf16x8 b0 = widen8(raw[0], raw[1]), b1 = widen8(raw[2], raw[3]);
      z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[0], b0, floatx4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
      z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[1], b1, z, 0, 0, 0);
    }
    if (mb > 0) {
      const float f = sp * sw;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[mb - 1][i] = __builtin_fmaf(zp[i], f, acc[mb - 1][i]);
    }
    __builtin_amdgcn_sched_barrier(0);
    raw = rn;
    sp = s;
    s = sn;
    zp = z;
  }
}

// lane: vocabulary rows 4 lg + (0 .. 3) of each of its blocks for hidden row lr of each row block
template <int MB, int NBW>
__device__ __forceinline__ void store_logits(const LmHeadFp8Args& a, const floatx4 (&acc)[NBW][MB], int mb0, int vb0) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int m = (mb0 + mb) * 16 + lr;
    if (m >= a.M) continue;
    const int b = m / a.K, k = m - b * a.K;
    const long long off = (long long)b * a.out_rs + (long long)k * a.out_ss;
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb) {
      const int v = (vb0 + nb) * 16 + lg * 4;
      const floatx4 z = acc[nb][mb];
      if (a.out_bf16) {
        uint16_t* o = (uint16_t*)a.out + off + v;
        uint32_t hh[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) hh[i] = f32_to_bf16_bits(z[i]);
        if (a.vec_out && v + 3 < a.V) {
          *(u32x2*)o = u32x2{hh[0] | (hh[1] << 16), hh[2] | (hh[3] << 16)};
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (v + i < a.V) o[i] = (uint16_t)hh[i];
        }
      } else {
        float* o = (float*)a.out + off + v;
        if (a.vec_out && v + 3 < a.V) {
          *(f32x4*)o = f32x4{z[0], z[1], z[2], z[3]};
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (v + i < a.V) o[i] = z[i];
        }
      }
    }
  }
}

// Up to 32 hidden rows (MB 16-row blocks): four waves, each with all the rows and a 16-row block of the vocabulary.
// Bound by the matrix, of which a wave copies its own 2 KB a chunk (128 columns) into LDS; the hidden rows' chunk is
// shared. Both stand in a ring of NST chunks, NST - 1 of them in flight, two work-groups to a CU or more (7 rows, H = 4096,
// rings of 4 / 6 / 7 chunks: V = 32000 29.8 / 30.8 / 31.3 us, V = 50017 44.4 / 46.3 / 47.2 us).
//
// What the waits count: copies alone. Every load between the first copy and the last barrier is one of copy_1k_asm's,
// which the compiler can neither drop nor turn into another kind (a plain load counted here once became a scalar one,
// and others of the last chunks were dropped). The matrix's scales go into LDS ahead of them.
template <int MB>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void lm_head_fp8_kernel(LmHeadFp8Args a) {
  constexpr int NW = 4, NST = 4;
  constexpr int kStage = fp8_stage_bytes(MB);       // a chunk's hidden rows and their scales
  constexpr int kCopy = kStage / 1024;              // 1 KB copies of it, dealt to the waves in turn
  constexpr int kQ = (kCopy + NW - 1) / NW;
  constexpr int kMine = kQ + 2;                     // copies a wave makes of a chunk, each wave as many
  __shared__ __attribute__((aligned(16))) uint8_t s_x[NST][kStage];
  __shared__ __attribute__((aligned(16))) uint8_t s_w[NST][NW][2048];
  __shared__ float s_ws[512];  // the scales of the work-group's rows, by chunk (H <= 65536)
  static_assert(sizeof s_x + sizeof s_w + sizeof s_ws <= 80 * 1024, "two work-groups a CU");
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15;
  const int HB = a.H >> 7, VB = (a.V + 15) >> 4;
  const int vt0 = blockIdx.x * NW, vb0 = vt0 + w;  // 16-row blocks of the work-group (all in one scale block), of this wave
  const int coff = (int)((blockIdx.x * (unsigned)kStagger) % (unsigned)HB);
  auto chunk_of = [&](int c) { return c + coff >= HB ? c + coff - HB : c + coff; };
  for (int i = tid; i < HB; i += 64 * NW) s_ws[i] = a.w_scale[(size_t)min(vt0 >> 3, (a.V - 1) >> 7) * HB + i];
  const u32x4 xrs = words_at(a.xq + (size_t)blockIdx.y * HB * kStage, HB * kStage);
  const u32x4 wrs = words_at(a.w + (size_t)min(vb0, VB - 1) * HB * 2048, HB * 2048);  // (past the last: that again)
  auto copy = [&](int st, int c) {
    const int j = chunk_of(c);
#pragma unroll
    for (int p = 0; p < 2; ++p) copy_1k_asm<true>(wrs, s_w[st][w] + p * 1024, lane * 16, j * 2048 + p * 1024);
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const int p = min(q * NW + w, kCopy - 1);  // the last piece may be copied twice
      copy_1k_asm<false>(xrs, s_x[st] + p * 1024, lane * 16, j * kStage + p * 1024);
    }
  };
  floatx4 acc[1][MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) acc[0][mb] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
  for (int i = 0; i < NST - 1; ++i)
    if (i < HB) copy(i, i);
  int st = 0;
#pragma nounroll
  for (int c = 0; c < HB; ++c) {
    // Chunk c has landed for all waves: of each wave's copies at most those of the NST - 2 chunks after it are in flight
    // (near the end, where fewer were made: none). And all have read chunk c - 1, whose place is free.
    if (c + NST - 1 <= HB)
      chunk_barrier<(NST - 2) * kMine>();
    else
      chunk_barrier<0>();
    if (c + NST - 1 < HB) copy(st == 0 ? NST - 1 : st - 1, c + NST - 1);
    const uint8_t* cur = s_x[st];
    const float sw = s_ws[chunk_of(c)];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const u32x4 x = *(const u32x4*)(s_w[st][w] + p * 1024 + lane * 16);
      const bf16x8 A[2] = {widen8(x[0], x[1]), widen8(x[2], x[3])};
      scaled_products<MB>(cur + p * 1024 + lane * 16, (const float*)(cur + MB * 2048) + lr, sw, A, acc[0]);
    }
    st = st + 1 == NST ? 0 : st + 1;
  }
  store_logits<MB, 1>(a, acc, blockIdx.y * MB, vb0);
}

// More rows: a work-group of four waves has MB 16-row blocks of them, a wave all of these and NBW vocabulary blocks of
// its own. A chunk (128 columns) at a time: the hidden rows two chunks deep in LDS, shared; the wave's part of the
// matrix (2 KB a block and chunk) one deep in a part of LDS of its own, widened into registers at the chunk's start,
// after which the next chunk is copied over it. One barrier a chunk. A chunk's sums are scaled once, since the vector
// unit would be the bound otherwise. The row tiles of a vocabulary tile run on the same XCD next to each other, so that
// the later ones find the matrix in the caches. Four waves, two work-groups a CU: against eight waves and one, 77 us to
// 104 us at V = 32000 and 284 us to 317 us at V = 151936, whose last round would be short of work-groups, and as fast
// where the rounds come out even (H = 4096, 224 rows, NBW = 4).
constexpr int kWideWaves = 4;
template <int MB, int NBW>
__global__ __launch_bounds__(64 * kWideWaves) __attribute__((amdgpu_waves_per_eu(2, 2))) void lm_head_fp8_wide_kernel(
    LmHeadFp8Args a, int v_tiles, int m_tiles) {
  constexpr int NW = kWideWaves;
  constexpr int kScales = (NW * NBW + 7) / 8;  // scale blocks (8 vocabulary blocks) of a work-group
  constexpr int kStage = fp8_stage_bytes(MB);
  constexpr int kCopy = kStage / 1024;
  constexpr int kQ = (kCopy + NW - 1) / NW;
  __shared__ __attribute__((aligned(16))) uint8_t s_x[2][kStage];
  __shared__ __attribute__((aligned(16))) uint8_t s_w[NW][NBW * 2048];
  __shared__ float s_ws[kScales][512];  // the scale blocks' scales, by chunk (H <= 65536)
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15;
  const int HB = a.H >> 7, VB = (a.V + 15) >> 4;
  // work-groups go to the eight XCDs in turn: row tile after row tile of eight vocabulary tiles
  const int grp = blockIdx.x / (8u * (unsigned)m_tiles), in = blockIdx.x - grp * 8 * m_tiles;
  const int vt = grp * 8 + (in & 7), mt = in >> 3;
  if (vt >= v_tiles) return;
  const int vt0 = vt * NW * NBW;
  const int coff = __builtin_amdgcn_readfirstlane((int)(((unsigned)vt * (unsigned)kStagger) % (unsigned)HB));
  auto chunk_of = [&](int c) { return c + coff >= HB ? c + coff - HB : c + coff; };
  for (int i = tid; i < kScales * HB; i += 64 * NW) {
    const int b = i / HB;
    s_ws[b][i - b * HB] = a.w_scale[(size_t)min((vt0 >> 3) + b, (a.V - 1) >> 7) * HB + i - b * HB];
  }
  const u32x4 xrs = words_at(a.xq + (size_t)mt * HB * kStage, HB * kStage);
  // the wave's rows of the matrix: 4 blocks of HB * 2 KB (those past the last repeat it)
  const int vb0 = vt0 + w * NBW, vbc = min(vb0, VB - 1);
  const int nblk = __builtin_amdgcn_readfirstlane(min(NBW, VB - vbc));
  const u32x4 wrs = words_at(a.w + (size_t)vbc * HB * 2048, nblk * HB * 2048);
  auto copy_x = [&](uint8_t* buf, int c) {
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const int p = min(q * NW + w, kCopy - 1);
      copy_1k_asm<false>(xrs, buf + p * 1024, lane * 16, chunk_of(c) * kStage + p * 1024);
    }
  };
  auto copy_w = [&](int c) {
#pragma unroll
    for (int p = 0; p < 2 * NBW; ++p)  // 1 KB run p of the wave's chunk: half p % 2 of block p / 2
      copy_1k_asm<true>(wrs, s_w[w] + p * 1024, lane * 16,
                        min(p >> 1, nblk - 1) * HB * 2048 + chunk_of(c) * 2048 + (p & 1) * 1024);
  };
  floatx4 acc[NBW][MB];
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  copy_x(s_x[0], 0);
  copy_w(0);
  chunk_barrier<0>();
#pragma nounroll
  for (int c = 0; c < HB; ++c) {
    const uint8_t* cur = s_x[c & 1];
    bf16x8 A[NBW][4];
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const u32x4 x = *(const u32x4*)(s_w[w] + nb * 2048 + p * 1024 + lane * 16);
        A[nb][2 * p] = widen8(x[0], x[1]);
        A[nb][2 * p + 1] = widen8(x[2], x[3]);
      }
    const float sw = s_ws[kScales == 1 ? 0 : w * NBW >> 3][chunk_of(c)];
    // the wave has read its part of the matrix: its next chunk may land on it
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (c + 1 < HB) {
      copy_w(c + 1);
      copy_x(s_x[(c + 1) & 1], c + 1);
    }
    const uint8_t* xb = cur + lane * 16;
    const float* sx = (const float*)(cur + MB * 2048) + lr;
    auto operand = [&](int mb, int p) { return *(const u32x4*)(xb + mb * 2048 + p * 1024); };
    // one row block after the other, operand reads one block ahead, scaling one block behind (the order is
    // pinned: left alone the compiler holds every block's sums at once)
    // ahead of the SIMD's other wave from here on, which then widens and copies between these products (358 us against
    // 374 us at V = 200064, 224 rows)
    __builtin_amdgcn_s_setprio(1);
    u32x4 b[2] = {operand(0, 0), operand(0, 1)};
    float s = sx[0], sp = 0.0f;
    floatx4 z[NBW], zp[NBW];
#pragma unroll
    for (int mb = 0; mb <= MB; ++mb) {
      float sn = s;
      if (mb < MB) {
        if (mb + 1 < MB) sn = sx[(mb + 1) * 16];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const bf16x8 b0 = widen8(b[p][0], b[p][1]), b1 = widen8(b[p][2], b[p][3]);
          if (mb + 1 < MB) b[p] = operand(mb + 1, p);
#pragma unroll
          for (int nb = 0; nb < NBW; ++nb)
            z[nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[nb][2 * p], b0, p ? z[nb] : floatx4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
          for (int nb = 0; nb < NBW; ++nb)
            z[nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[nb][2 * p + 1], b1, z[nb], 0, 0, 0);
        }
      }
      if (mb > 0) {
        const float f = sp * sw;
#pragma unroll
        for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[nb][mb - 1][i] = __builtin_fmaf(zp[nb][i], f, acc[nb][mb - 1][i]);
      }
      // the block's order: operand reads, then every product followed by two of the vector unit's instructions
      // (without it: 142 us against 118 us for V = 65536, 224 rows)
      if (mb < MB) {
        if (mb + 1 < MB) __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
#pragma unroll
        for (int k = 0; k < 4 * NBW; ++k) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      sp = s;
      s = sn;
#pragma unroll
      for (int nb = 0; nb < NBW; ++nb) zp[nb] = z[nb];
    }
    // the sums are finished here: otherwise they sink past the branches, with all their addends kept alive
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) asm volatile("" : "+v"(acc[nb][mb]));
    __builtin_amdgcn_s_setprio(0);
    chunk_barrier<0>();  // chunk c + 1 has landed
  }
  store_logits<MB, NBW>(a, acc, mt * MB, vb0);
}

// Row-major codes [V][H] into the tiles, 16 bytes a thread; rows past V are zero.
__global__ __launch_bounds__(256) void tile_fp8_kernel(int V, int H, const uint8_t* codes, uint8_t* tiled) {
  const int HB = H >> 7;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;  // piece of the tiled array
  const size_t n = (size_t)((V + 15) >> 4) * H;
  if (i >= n) return;
  const int r = (int)(i & 15), q = (int)(i >> 4 & 7);
  const size_t tile = i >> 7;
  const int j = (int)(tile % (unsigned)HB);
  const size_t v = tile / (unsigned)HB * 16 + r;
  u32x4 x = u32x4{0, 0, 0, 0};
  if (v < (size_t)V) x = *(const u32x4*)(codes + v * H + j * 128 + q * 16);
  *(u32x4*)(tiled + i * 16) = x;
}

// One 128 x 128 block of a bf16 matrix: its largest magnitude, its scale, its codes in tiles.
__global__ __launch_bounds__(256) void quant_blocks_kernel(int V, int H, const uint16_t* wm, uint8_t* tiled,
                                                           float* scales) {
  __shared__ float s_max[4];
  const int tid = threadIdx.x, HB = H >> 7;
  const int j = blockIdx.x % (unsigned)HB, vb = blockIdx.x / (unsigned)HB;
  // a thread has 16 columns of rows r + 32 i: pieces of 32 bytes, consecutive threads along a row
  const int q = tid & 7, r = tid >> 3;
  float x[4][16], am = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = vb * 128 + i * 32 + r;
    u32x4 lo = u32x4{0, 0, 0, 0}, hi = lo;
    if (v < V) {
      const uint16_t* p = wm + (size_t)v * H + j * 128 + q * 16;
      lo = *(const u32x4*)p;
      hi = *(const u32x4*)(p + 8);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[i][2 * e] = __uint_as_float(lo[e] << 16);
      x[i][2 * e + 1] = __uint_as_float(lo[e] & 0xFFFF0000u);
      x[i][8 + 2 * e] = __uint_as_float(hi[e] << 16);
      x[i][8 + 2 * e + 1] = __uint_as_float(hi[e] & 0xFFFF0000u);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) am = fmaxf(am, fabsf(x[i][e]));
  }
  am = wave_max_f32(am);
  if ((tid & 63) == 0) s_max[tid >> 6] = am;
  __syncthreads();
  am = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  const float s = am / kE4m3Max;
  if (tid == 0) scales[(size_t)vb * HB + j] = s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = vb * 128 + i * 32 + r;
    if ((v >> 4) >= (V + 15) >> 4) continue;
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = quant4(clamp_e4m3(x[i][4 * e] / s), clamp_e4m3(x[i][4 * e + 1] / s), clamp_e4m3(x[i][4 * e + 2] / s),
                    clamp_e4m3(x[i][4 * e + 3] / s));
    *(u32x4*)(tiled + fp8_tile_index(v, j * 128 + q * 16, H)) = u32x4{o[0], o[1], o[2], o[3]};
  }
}

template <int MB>
hipError_t launch_mb(const LmHeadFp8Args& a, hipStream_t st) {
  const int VB = (a.V + 15) >> 4, MBt = (a.M + 15) >> 4;
  const dim3 grid((unsigned)((VB + 3) / 4), (unsigned)((MBt + MB - 1) / MB));
  hipLaunchKernelGGL(lm_head_fp8_kernel<MB>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

// Vocabulary blocks a wave: four, so that every hidden operand serves four products, where that leaves more than a
// work-group to a CU; else two, down to half a work-group to a CU, and one below that (H = 4096, us with four / two /
// one: V = 65536, 224 rows 115 / 137 / 180, 112 rows 82 / 72 / 95; V = 32000, 224 rows 76 / 69 / 88, 66 rows 57 / 40 / 38;
// V = 4099, 66 rows 55 / 35 / 29).
constexpr long long kWide4 = 256 * kWideWaves * 4, kWide2 = 256 * kWideWaves * 2;  // 16-row blocks, all row tiles

template <int MB>
hipError_t launch_wide(const LmHeadFp8Args& a, hipStream_t st) {
  const int VB = (a.V + 15) >> 4, mt = (((a.M + 15) >> 4) + MB - 1) / MB;
  auto launch = [&](auto kernel, int nbw) {
    const int tiles = (VB + kWideWaves * nbw - 1) / (kWideWaves * nbw);
    hipLaunchKernelGGL(kernel, dim3((unsigned)((tiles + 7) / 8 * 8 * mt)), dim3(64 * kWideWaves), 0, st, a, tiles, mt);
    return hipGetLastError();
  };
  const long long blocks = (long long)VB * mt;
  if (blocks > kWide4) return launch(lm_head_fp8_wide_kernel<MB, 4>, 4);
  if (blocks >= kWide2) return launch(lm_head_fp8_wide_kernel<MB, 2>, 2);
  return launch(lm_head_fp8_wide_kernel<MB, 1>, 1);
}

}  // namespace

hipError_t launch_lm_head_fp8(const LmHeadFp8Args& a, hipStream_t st) {
  const int MBt = (a.M + 15) >> 4, HB = a.H >> 7;
  hipLaunchKernelGGL(quant_rows_kernel, dim3((unsigned)(HB * MBt)), dim3(256), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  switch (a.mb) {
    case 1: return launch_mb<1>(a, st);
    case 2:
      // 32 rows, H = 4096, wide / few: V = 32000 32.4 / 32.1 us, 50017 45.7 / 52.4, 65536 57.7 / 58.9, 200064 164 / 162
      return (a.V + 15) >> 4 >= kWide2 ? launch_wide<2>(a, st) : launch_mb<2>(a, st);
    case 3: return launch_wide<3>(a, st);
    case 4: return launch_wide<4>(a, st);
    case 5: return launch_wide<5>(a, st);
    case 6: return launch_wide<6>(a, st);
    default: return launch_wide<7>(a, st);
  }
}

// Row tiles of at most 7 blocks, all of one height (126 rows in 4 + 4 blocks, V = 200064: 288 us, in 7 + 1 359 us).
int lm_head_fp8_blocks(int M) {
  const int n = (M + 15) >> 4, tiles = (n + 6) / 7;
  return (n + tiles - 1) / tiles;
}

hipError_t launch_tile_fp8(int V, int H, const uint8_t* codes, uint8_t* tiled, hipStream_t st) {
  const size_t n = (size_t)((V + 15) >> 4) * H;
  hipLaunchKernelGGL(tile_fp8_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, V, H, codes, tiled);
  return hipGetLastError();
}

hipError_t launch_quantize_fp8(int V, int H, const uint16_t* w, uint8_t* tiled, float* scales, hipStream_t st) {
  const unsigned n = (unsigned)((V + 127) >> 7) * (unsigned)(H >> 7);
  hipLaunchKernelGGL(quant_blocks_kernel, dim3(n), dim3(256), 0, st, V, H, w, tiled, scales);
  return hipGetLastError();
}

}  // namespace mds
