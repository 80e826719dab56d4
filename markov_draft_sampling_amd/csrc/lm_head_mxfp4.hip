// LM head from a microscaled 4-bit matrix: logits[m, v] = sum over c of
// x[m, c] w[v, c], w[v, c] = code[v, c] 2^(s[v, c / 32] - 127), code an e2m1
// value (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), s a byte for 32
// columns of a row (255: NaN), x the bf16 hidden rows as they are.
//
// Every weight is a bf16 value (unless it is so large that bf16 has none), so
// codes are widened to bf16 with their scale in one instruction for two, and
// the bf16 matrix instruction's products are exact and its sums float32.
// Hidden rows are not rounded: the matrix instructions that take 4-bit codes
// as they are want the rows in 8 bits or fewer.
//
// Tiles of 16 rows by 128 columns, 1 KB, in operand order: lane l = r + 16 g of a
// wave has the 32 codes of row r, columns 32 g on - one scale a lane and tile.
// Which columns a matrix instruction takes together does not matter as long as both
// operands agree: its slice s has columns 32 g + 8 s .. + 7 of each g. Scales of
// four tiles in a row of tiles are the bytes of a lane's word.
//
// Up to some 50 rows the call is bound by the matrix's 17 / 32 V H bytes (H = 4096: one row, V = 200064 72 us and 6.1
// TB/s; 7 rows, V = 151936 59 us; 32 rows, V = 200064 89 us), above by the matrix cores, the widening and the operand
// reads from LDS (224 rows: V = 200064 284 us and 1.29 PFLOP/s, V = 151936 227 us). Small vocabularies take a
// work-group's start and its chain of loads (7 rows, V = 4099 7 us). (Times at the rules below are of this code on one
// card, the two sides in turn; those of what is not kept are of the build that had it. Cards differ by up to 8%.)
#include <type_traits>

#include "mds_device.h"
#include "mds_serve.h"

namespace mds {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Slice s (8 codes) of a lane's 16 bytes of a tile, as bf16. scale: 2^(s - 127) (its exponent counts; 255: NaN)
__device__ __forceinline__ bf16x8 widen(uint32_t codes, float scale) {
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  return __builtin_bit_cast(bf16x8, r);
}
// Byte i of a lane's word of scales, as the float whose exponent it is
__device__ __forceinline__ float scale_of(uint32_t word, int i) { return __uint_as_float((word >> (8 * i) & 0xFFu) << 23); }

// Logits go out by way of LDS, as rows of consecutive columns (four floats of padding keep rows apart in the banks): a
// row's run of them in one piece, also where rows are not aligned and every logit is a store of its own (when it was built: 224
// rows, V = 100003 163 us, by stores of a lane's own four logits 201; V = 151936 221 and 228).
template <int COLS>
constexpr int kOutStride = COLS + 4;

// A wave's LDS operations keep their order, and so must the compiler where lanes read what others of the wave wrote.
__device__ __forceinline__ void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

// Where a hidden row's logits start
__device__ __forceinline__ long long row_at(const LmHeadMxArgs& a, int m) {
  const int b = m / a.K;
  return (long long)b * a.out_rs + (long long)(m - b * a.K) * a.out_ss;
}

// The i-th of n threads stores its part of `rows` rows of COLS logits from column v0 on. at(r): where row r starts;
// z(r, c, n): its n logits from column c on (n: 4 or 1, as a type).
template <int COLS, typename At, typename Z>
__device__ __forceinline__ void store_rows(const LmHeadMxArgs& a, int i, int n, int rows, int v0, At at, Z z) {
  if (a.vec_out) {
    for (int e = i; e < rows * (COLS / 4); e += n) {
      const int r = e / (COLS / 4), c = e % (COLS / 4) * 4, v = v0 + c;
      if (v >= a.V) continue;
      const floatx4 x = z(r, c, std::integral_constant<int, 4>{});
      const long long off = at(r) + v;
      if (a.out_bf16) {
        uint16_t* o = (uint16_t*)a.out + off;
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = f32_to_bf16_bits(x[k]);
        if (v + 3 < a.V) {
          *(u32x2*)o = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (v + k < a.V) o[k] = (uint16_t)h[k];
        }
      } else {
        float* o = (float*)a.out + off;
        if (v + 3 < a.V) {
          *(floatx4*)o = x;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (v + k < a.V) o[k] = x[k];
        }
      }
    }
  } else {
    for (int e = i; e < rows * COLS; e += n) {
      const int r = e / COLS, c = e % COLS, v = v0 + c;
      if (v >= a.V) continue;
      const float x = z(r, c, std::integral_constant<int, 1>{});
      const long long off = at(r) + v;
      if (a.out_bf16)
        ((uint16_t*)a.out)[off] = (uint16_t)f32_to_bf16_bits(x);
      else
        ((float*)a.out)[off] = x;
    }
  }
}

// Few hidden rows, up to 4 NG: the four waves of a work-group have the same NBW vocabulary blocks and divide the columns,
// 512 (four tiles, a word of scales) at a time; their sums are joined through LDS at the end. So a hidden row is read once
// a work-group, no wave waits for another before the end, and both operands go from memory into registers, NP tiles
// ahead. The hidden rows are read along themselves (a wave 4 rows of 256 bytes at a time: as operands, 16 bytes of
// every row at a time, four times as many cache lines are touched) and change places in a part of LDS of the wave's own.
template <int NG, int NBW>
__global__ __launch_bounds__(256) void lm_head_mx_kernel(LmHeadMxArgs a) {
  constexpr int MB = (NG + 3) / 4;
  constexpr int NP = 2;  // (three, four: 16 rows, V = 200064, H = 4096 108 and 107 us against 93; V = 32000 22 and 22 against 19: fewer waves a CU)
  constexpr int kOut = kOutStride<NBW * 16>;
  constexpr int kX = NG * 1024, kZ = NG * 4 * kOut * 4;  // a wave's hidden rows of a tile; in the end its sums
  __shared__ __attribute__((aligned(16))) unsigned char s[4 * (kX > kZ ? kX : kZ)];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int HB = a.H >> 7, G = (HB + 3) >> 2, VB = (a.V + 15) >> 4;
  unsigned char* s_x = s + w * kX;
  const int vb0 = blockIdx.x * NBW;
  // the wave's tiles: words w, w + 4, .. of each row of tiles, of which only the last may be short
  const int words = G > w ? (G - w + 3) >> 2 : 0;
  const int n = words ? 4 * words - ((words - 1) * 4 + w == G - 1 ? 4 * G - HB : 0) : 0;
  const uint8_t* wp[NBW];
  const uint8_t* sp[NBW];
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb) {
    const size_t vb = (size_t)min(vb0 + nb, VB - 1);
    wp[nb] = a.w + vb * HB * 1024;
    sp[nb] = a.w_scale + vb * G * 256;
  }
  const uint32_t lane16 = lane * 16, lane4 = lane * 4;
  // rows past the last repeat it; row r's 16-byte slot p stands at slot p ^ (r % 16)
  const uint16_t* xp[NG];
  uint32_t put[NG], get[MB];
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int r = 4 * i + lg;
    xp[i] = a.hidden + (long long)min(r, a.M - 1) * a.hidden_rs + 8 * lr;
    put[i] = r * 256 + (lr ^ (r & 15)) * 16;
  }
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) get[mb] = min(mb * 16 + lr, NG * 4 - 1);
  floatx4 acc[NBW][MB];
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  u32x4 W[NP][NBW], X[NP][NG];
  uint32_t S[NP][NBW];
  auto load = [&](int p, int i) {
    const int c = min(i, n - 1);
    const int t = ((c >> 2) * 4 + w) * 4 + (c & 3);
#pragma unroll
    for (int j = 0; j < NG; ++j) X[p][j] = *(const u32x4*)(xp[j] + t * 128);
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb) {
      W[p][nb] = __builtin_nontemporal_load((const u32x4*)(wp[nb] + (size_t)t * 1024 + lane16));
      S[p][nb] = *(const uint32_t*)(sp[nb] + (t >> 2) * 256 + lane4);
    }
  };
  if (n > 0) {
#pragma unroll
    for (int p = 0; p < NP; ++p) load(p, p);
#pragma nounroll
    for (int i0 = 0; i0 < n; i0 += NP) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int i = i0 + p;
        if (i < n) {
#pragma unroll
          for (int j = 0; j < NG; ++j) *(u32x4*)(s_x + put[j]) = X[p][j];
          wave_lds();
          float sc[NBW];
#pragma unroll
          for (int nb = 0; nb < NBW; ++nb) sc[nb] = scale_of(S[p][nb], i & 3);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            bf16x8 x[MB];
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
              x[mb] = *(const bf16x8*)(s_x + get[mb] * 256 + ((4 * lg + k) ^ (get[mb] & 15)) * 16);
#pragma unroll
            for (int nb = 0; nb < NBW; ++nb) {
              const bf16x8 A = widen(W[p][nb][k], sc[nb]);
#pragma unroll
              for (int mb = 0; mb < MB; ++mb)
                acc[nb][mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, x[mb], acc[nb][mb], 0, 0, 0);
            }
          }
          wave_lds();
        }
        load(p, i + NP);
      }
    }
  }
  __syncthreads();  // all waves have read their hidden rows
  auto z_of = [&](int wave, int r, int c) { return s + wave * kZ + (r * kOut + c) * 4; };
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb)
      if (mb * 16 + lr < NG * 4) *(floatx4*)z_of(w, mb * 16 + lr, nb * 16 + lg * 4) = acc[nb][mb];
  __syncthreads();
  store_rows<NBW * 16>(
      a, threadIdx.x, 256, a.M, vb0 * 16, [&](int r) { return row_at(a, r); },
      [&](int r, int c, auto cols) {
        using T = typename std::conditional<decltype(cols)::value == 4, floatx4, float>::type;
        auto part = [&](int k) { return *(const T*)z_of(k, r, c); };
        return (part(0) + part(1)) + (part(2) + part(3));
      });
}

// 16 bytes a lane straight into LDS at `lds` (uniform) + 16 * lane, from base (uniform) + off, as assembly: the waits for
// these copies are the kernel's own. (m0, the LDS address, has no other use here; the load may read it one wait state
// after the scalar write at the earliest.)
__device__ __forceinline__ void copy_1k(const char* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory");
}

// More rows: a work-group of four waves has MB 16-row blocks of them, a wave all of these and NBW vocabulary blocks of
// its own; two work-groups a CU. A tile's columns (128) at a time: the hidden rows in LDS, two of these deep and shared,
// 16-byte slots XOR-swizzled by row; the matrix in registers, asked for one ahead. The row tiles of a vocabulary tile run
// on the same XCD next to each other, so that the later ones find the matrix in the caches. (Not kept: eight waves that
// share three stages, and runs of the vocabulary in uneven passes that fill every CU, 239 us against 223 for 224 rows,
// V = 151936: a pass costs as much as one more block; one work-group of four waves with eight blocks a wave, 256 us; four
// tiles asked for ahead where a tile is little work, 20 rows, V = 32000 23.0 us to 25.7, in the same source at 2 to 4% of
// the large calls.)
template <int MB, int NBW>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void lm_head_mx_wide_kernel(
    LmHeadMxArgs a, int v_tiles, int m_tiles) {
  constexpr int NW = 4;
  constexpr int kStage = MB * 4096;  // the hidden rows' 128 columns
  // The order within a tile: operand reads one row block ahead, the next slice's widening between this one's products (224
  // rows, H = 4096: V = 131072 183 us against 196 as the compiler has it, four blocks at V = 200064 288 against 308). With five blocks there are no registers for it.
  constexpr bool kPinned = NBW <= 4;
  constexpr int kOut = kOutStride<NBW * 16>;
  constexpr int kOutWave = 16 * kOut * 4;  // a wave's logits of 16 rows, in the same place in the end
  __shared__ __attribute__((aligned(16))) unsigned char s_x[2 * kStage > NW * kOutWave ? 2 * kStage : NW * kOutWave];
  __shared__ long long s_at[MB * 16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int HB = a.H >> 7, G = (HB + 3) >> 2, VB = (a.V + 15) >> 4;
  // work-groups go to the eight XCDs in turn: row tile after row tile of eight vocabulary tiles
  const int grp = blockIdx.x / (8u * (unsigned)m_tiles), in = blockIdx.x - grp * 8 * m_tiles;
  const int vt = grp * 8 + (in & 7), mt = in >> 3;
  if (vt >= v_tiles) return;
  const int vb0 = (vt * NW + w) * NBW, m0 = mt * MB * 16;
  if (tid < MB * 16) s_at[tid] = row_at(a, min(m0 + tid, a.M - 1));
  const uint8_t* wp[NBW];
  const uint8_t* sp[NBW];
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb) {
    const size_t vb = (size_t)min(vb0 + nb, VB - 1);
    wp[nb] = a.w + vb * HB * 1024 + lane * 16;
    sp[nb] = a.w_scale + vb * G * 256 + lane * 4;
  }
  // this wave's copies: 4 rows of 256 bytes each, rows 4 (w + 4 q) on; lane l lands in row l / 16, slot l % 16, which
  // holds the row's slot (l % 16) ^ (row % 16)
  const char* xb = (const char*)(a.hidden + (long long)m0 * a.hidden_rs);
  uint32_t xo[MB];
#pragma unroll
  for (int q = 0; q < MB; ++q) {
    const int r = 4 * (w + 4 * q) + lg;
    xo[q] = (uint32_t)(min(r, a.M - 1 - m0) * (int)a.hidden_rs * 2) + (uint32_t)((lr ^ (r & 15)) * 16);
  }
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)s_x;
  auto copy_x = [&](int st, int c) {
#pragma unroll
    for (int q = 0; q < MB; ++q) copy_1k(xb + c * 256, xo[q], lds + st * kStage + (w + 4 * q) * 1024);
  };
  u32x4 W[NBW];
  uint32_t S[NBW];
  auto load_w = [&](int c) {
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb) {
      W[nb] = *(const u32x4*)(wp[nb] + (size_t)c * 1024);
      S[nb] = *(const uint32_t*)(sp[nb] + (c >> 2) * 256);
    }
  };
  floatx4 acc[NBW][MB];
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  copy_x(0, 0);
  load_w(0);
#pragma nounroll
  for (int c = 0; c < HB; ++c) {
    // tile c's columns are there for all waves, which are done with those before it
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    u32x4 cw[NBW];
    float sc[NBW];
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb) {
      cw[nb] = W[nb];
      sc[nb] = scale_of(S[nb], c & 3);
    }
    if (c + 1 < HB) {
      copy_x((c + 1) & 1, c + 1);
      load_w(c + 1);
    }
    const unsigned char* cur = s_x + (c & 1) * kStage + lr * 256;
    auto operand = [&](int mb, int s) { return *(const bf16x8*)(cur + mb * 4096 + ((4 * lg + s) ^ lr) * 16); };
    __builtin_amdgcn_s_setprio(1);
    if constexpr (kPinned) {
      bf16x8 A[2][NBW];
#pragma unroll
      for (int nb = 0; nb < NBW; ++nb) A[0][nb] = widen(cw[nb][0], sc[nb]);
      bf16x8 x = operand(0, 0);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          bf16x8 xn = x;
          const bool more = s < 3 || mb + 1 < MB;
          if (more) xn = mb + 1 < MB ? operand(mb + 1, s) : operand(0, s + 1);
          if (s < 3) {
#pragma unroll
            for (int nb = 0; nb < NBW; ++nb)
              if (nb * MB / NBW == mb) A[(s + 1) & 1][nb] = widen(cw[nb][s + 1], sc[nb]);
          }
#pragma unroll
          for (int nb = 0; nb < NBW; ++nb)
            acc[nb][mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[s & 1][nb], x, acc[nb][mb], 0, 0, 0);
          if (more) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
          for (int nb = 0; nb < NBW; ++nb) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
          x = xn;
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8 A[NBW];
#pragma unroll
        for (int nb = 0; nb < NBW; ++nb) A[nb] = widen(cw[nb][s], sc[nb]);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const bf16x8 x = operand(mb, s);
#pragma unroll
          for (int nb = 0; nb < NBW; ++nb)
            acc[nb][mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[nb], x, acc[nb][mb], 0, 0, 0);
        }
      }
    }
    __builtin_amdgcn_s_setprio(0);
  }
  __syncthreads();  // the hidden rows have been read
  float* so = (float*)(s_x + w * kOutWave);
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb) *(floatx4*)(so + lr * kOut + nb * 16 + lg * 4) = acc[nb][mb];
    wave_lds();
    store_rows<NBW * 16>(
        a, lane, 64, min(16, a.M - m0 - mb * 16), vb0 * 16, [&](int r) { return s_at[mb * 16 + r]; },
        [&](int r, int c, auto cols) {
          using T = typename std::conditional<decltype(cols)::value == 4, floatx4, float>::type;
          return *(const T*)(so + r * kOut + c);
        });
    if (mb + 1 < MB) wave_lds();
  }
}

// Row-major codes [V][H / 2] and scales [V][H / 32] into the tiles: a thread per 16 codes' bytes; rows past V and
// columns past H are zero.
__global__ __launch_bounds__(256) void tile_mx_kernel(int V, int H, const uint8_t* codes, const uint8_t* scales,
                                                      uint8_t* tiled, uint8_t* tiled_scales) {
  const int HB = H >> 7, G = (HB + 3) >> 2, VB = (V + 15) >> 4;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;  // lane of a tile, the scales' short words included
  const int lane = (int)(i & 63), r = lane & 15, g = lane >> 4;
  const size_t tile = i >> 6;
  const size_t vb = tile / (unsigned)(4 * G);
  const int c = (int)(tile - vb * (unsigned)(4 * G));
  if (vb >= (size_t)VB) return;
  const size_t v = vb * 16 + r;
  const bool in = v < (size_t)V && c < HB;
  if (c < HB) {
    u32x4 x = u32x4{0, 0, 0, 0};
    if (in) x = *(const u32x4*)(codes + v * (H / 2) + c * 64 + g * 16);
    *(u32x4*)(tiled + (vb * HB + c) * 1024 + lane * 16) = x;
  }
  tiled_scales[(vb * G + (c >> 2)) * 256 + lane * 4 + (c & 3)] = in ? scales[v * (H / 32) + c * 4 + g] : 0;
}

__device__ __forceinline__ bf16x2 two_of(uint32_t word) { return __builtin_bit_cast(bf16x2, word); }

// Largest magnitude's bits over the four lanes of a quad
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, false));
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, false));
}

// A bf16 matrix to codes and scales: a wave per 4 rows and 512 columns, a lane 8 columns of a row and a quarter of
// these, so that a quad has a block of 32 columns.
__global__ __launch_bounds__(256) void quantize_mx_kernel(int V, int H, const uint16_t* wm, uint8_t* tiled,
                                                          uint8_t* tiled_scales) {
  const int HB = H >> 7, G = (HB + 3) >> 2, VB = (V + 15) >> 4;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  // a work-group per 16 rows and word of scales
  const unsigned gi = blockIdx.x % (unsigned)G;
  const size_t vb = blockIdx.x / (unsigned)G;
  const int r = 4 * w + (lane >> 4), g = lane >> 2 & 3, piece = lane & 3;
  const size_t v = vb * 16 + r;
  if (vb >= (size_t)VB) return;
  u32x4 x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = (int)gi * 4 + k;
    x[k] = u32x4{0, 0, 0, 0};
    if (v < (size_t)V && c < HB) x[k] = __builtin_nontemporal_load((const u32x4*)(wm + v * H + c * 128 + (lane & 15) * 8));
  }
  uint32_t word = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = (int)gi * 4 + k;
    uint32_t top = 0;  // magnitudes of bf16 compare as their bits do, infinities and NaN above all
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(x[k][i] & 0x7FFFu, x[k][i] >> 16 & 0x7FFFu));
    top = quad_max(top);
    const uint32_t e = top >> 7;  // exponent of the largest, at least 2^-100's; 6 = 1.5 2^2 is the largest code's value
    const uint32_t s = e == 255u ? 255u : max(e, 27u) - 2u;
    const float scale = __uint_as_float(s << 23);
    uint32_t codes = 0;
    if (s != 255u) {
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, two_of(x[k][0]), scale, 0);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, two_of(x[k][1]), scale, 1);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, two_of(x[k][2]), scale, 2);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, two_of(x[k][3]), scale, 3);
    }
    if (c < HB) {
      *(uint32_t*)(tiled + (vb * HB + c) * 1024 + g * 256 + r * 16 + piece * 4) = codes;
      word |= (v < (size_t)V ? s : 0u) << (8 * k);
    }
  }
  if (piece == 0) *(uint32_t*)(tiled_scales + (vb * G + gi) * 256 + (g * 16 + r) * 4) = word;
}

// Back to bf16: the same lanes, 8 columns each
__global__ __launch_bounds__(256) void unpack_mx_kernel(int V, int H, const uint8_t* tiled, const uint8_t* tiled_scales,
                                                        uint16_t* out) {
  const int HB = H >> 7, G = (HB + 3) >> 2;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const unsigned gi = blockIdx.x % (unsigned)G;
  const size_t vb = blockIdx.x / (unsigned)G;
  const int r = 4 * w + (lane >> 4), g = lane >> 2 & 3, piece = lane & 3;
  const size_t v = vb * 16 + r;
  if (v >= (size_t)V) return;
  const uint32_t word = *(const uint32_t*)(tiled_scales + (vb * G + gi) * 256 + (g * 16 + r) * 4);
  uint32_t x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = (int)gi * 4 + k;
    x[k] = c < HB ? *(const uint32_t*)(tiled + (vb * HB + c) * 1024 + g * 256 + r * 16 + piece * 4) : 0u;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = (int)gi * 4 + k;
    if (c < HB)
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4, widen(x[k], scale_of(word, k))),
                                  (u32x4*)(out + v * H + c * 128 + (lane & 15) * 8));
  }
}

template <int NG, int NBW>
hipError_t launch_few(const LmHeadMxArgs& a, hipStream_t st) {
  const int VB = (a.V + 15) >> 4;
  hipLaunchKernelGGL((lm_head_mx_kernel<NG, NBW>), dim3((unsigned)((VB + NBW - 1) / NBW)), dim3(256), 0, st, a);
  return hipGetLastError();
}
// Vocabulary blocks of a work-group: four, so that the hidden rows are read less often, but fewer where that leaves CUs
// without one, and for up to 4 rows, which cost little (us with one / two / four: H = 4096, 16 rows, V = 4099 8.7 / 7.8 / 9.4,
// V = 32000 28 / 22 / 19; H = 2048, 4 rows, V = 151936 34 / 33 / 36, one row 30 / 29 / 35).
int few_blocks(int VB, int ng) { return VB <= 512 ? 1 : ng == 1 || VB <= 1024 ? 2 : 4; }
template <int NG>
hipError_t launch_few_rows(const LmHeadMxArgs& a, int nbw, hipStream_t st) {
  if (nbw == 1) return launch_few<NG, 1>(a, st);
  if constexpr (NG > 1)
    if (nbw == 4) return launch_few<NG, 4>(a, st);
  return launch_few<NG, 2>(a, st);
}

template <int MB, int NBW>
hipError_t launch_wide(const LmHeadMxArgs& a, int tiles, int mt, hipStream_t st) {
  hipLaunchKernelGGL((lm_head_mx_wide_kernel<MB, NBW>), dim3((unsigned)((tiles + 7) / 8 * 8 * mt)), dim3(256), 0, st, a, tiles,
                     mt);
  return hipGetLastError();
}

// What a launch of the wide kernel takes, in units that a pass over a row of the matrix with one more block would add: the
// CUs take 512 work-groups a round, each of a time that grows with its blocks of the vocabulary beside what a tile of the
// hidden rows costs (as much as one of them); 256 or fewer at the end have a CU each and take about 0.7 of it.
// (H = 4096, us with 1 / 2 / 3 / 4 / 5 blocks a wave, and 6 / 7 up to 64 rows; the rule's choice: 32 rows, V = 151936
// 104 / 83 / 75 / 90 / 65 / 67 / 72, 5; 32 rows, V = 200064 144 / 110 / 108 / 103 / 106 / 113 / 88, 7; 112 rows, V = 32000
// 41 / 41 / 45 / 54 / 67, 1; 112 rows, V = 100003 143 / 108 / 119 / 92 / 117, 4; 224 rows, V = 200064 440 / 329 / 303 / 289 /
// 285, 5.)
float wide_cost(int VB, int mt, int nbw) {
  const long long wgs = (long long)((VB + 4 * nbw - 1) / (4 * nbw)) * mt, rest = wgs % 512;
  return (float)(wgs / 512) * (float)(1 + nbw) + (rest == 0 ? 0.0f : rest <= 256 ? 0.7f : 1.0f) * (float)(1 + nbw);
}
int wide_blocks(int VB, int mt, int mb) {
  int best = 1;
  for (int nbw = 2; nbw <= (mb <= 4 ? 7 : 5); ++nbw)  // (what the registers hold)
    if (wide_cost(VB, mt, nbw) < wide_cost(VB, mt, best)) best = nbw;
  return best;
}
// Row tiles of at most 7 blocks, all of one height; lower ones while every work-group keeps a CU to itself (112 rows,
// V = 4099, H = 4096: 29 us in one tile, three of 3 blocks 19 us; seven of one, which share CUs, would take 15.5).
int wide_row_tiles(int VB, int n) {
  const int least = (n + 6) / 7, alone = 256 / ((VB + 3) / 4);
  return alone > n ? n : alone > least ? alone : least;
}

template <int MB>
hipError_t launch_rows(const LmHeadMxArgs& a, const LmHeadMxPlan& p, hipStream_t st) {
  if constexpr (MB <= 4) {
    if (p.nbw == 6) return launch_wide<MB, 6>(a, p.v_tiles, p.row_tiles, st);
    if (p.nbw == 7) return launch_wide<MB, 7>(a, p.v_tiles, p.row_tiles, st);
  }
  switch (p.nbw) {
    case 1: return launch_wide<MB, 1>(a, p.v_tiles, p.row_tiles, st);
    case 2: return launch_wide<MB, 2>(a, p.v_tiles, p.row_tiles, st);
    case 3: return launch_wide<MB, 3>(a, p.v_tiles, p.row_tiles, st);
    case 4: return launch_wide<MB, 4>(a, p.v_tiles, p.row_tiles, st);
    default: return launch_wide<MB, 5>(a, p.v_tiles, p.row_tiles, st);
  }
}

}  // namespace

LmHeadMxPlan lm_head_mx_plan(int M, int V) {
  const int VB = (V + 15) >> 4, n = (M + 15) >> 4;
  const int tiles = wide_row_tiles(VB, n), mb = (n + tiles - 1) / tiles, mt = (n + mb - 1) / mb;
  const int nbw = wide_blocks(VB, mt, mb);
  // Up to 32 rows either kernel: the few rows' takes a start and a time by the vocabulary that grows with the rows, in
  // wide_cost's units (H = 4096, us few / wide, the rule's choice: 7 rows, V = 151936 61 / 59, wide, V = 200064 79 / 79, wide;
  // 16 rows, V = 32000 19 / 24, few, V = 100003 51 / 48, few; 32 rows, V = 4099 12 / 15, few, V = 32000 23.5 / 24.9, wide,
  // V = 200064 112 / 89, wide. It misses by up to 15% where the wide one's work-groups just fill a round and the bytes bound
  // it: 8 rows, V = 128256 52 / 60, wide).
  if (M <= 32) {
    const float few = 0.5f + (M <= 4 ? 0.55e-3f : M <= 8 ? 0.61e-3f : M <= 16 ? 0.71e-3f : 0.88e-3f) * (float)VB;
    const int ng = M <= 4 ? 1 : M <= 8 ? 2 : M <= 16 ? 4 : 8;
    if (few < wide_cost(VB, mt, nbw)) return {true, ng, few_blocks(VB, ng), 0, 0};
  }
  return {false, mb, nbw, mt, (VB + 4 * nbw - 1) / (4 * nbw)};
}

hipError_t launch_lm_head_mx(const LmHeadMxArgs& a, hipStream_t st) {
  const LmHeadMxPlan p = lm_head_mx_plan(a.M, a.V);
  if (p.few) {
    if (p.height == 1) return launch_few_rows<1>(a, p.nbw, st);
    if (p.height == 2) return launch_few_rows<2>(a, p.nbw, st);
    return p.height == 4 ? launch_few_rows<4>(a, p.nbw, st) : launch_few_rows<8>(a, p.nbw, st);
  }
  switch (p.height) {
    case 1: return launch_rows<1>(a, p, st);
    case 2: return launch_rows<2>(a, p, st);
    case 3: return launch_rows<3>(a, p, st);
    case 4: return launch_rows<4>(a, p, st);
    case 5: return launch_rows<5>(a, p, st);
    case 6: return launch_rows<6>(a, p, st);
    default: return launch_rows<7>(a, p, st);
  }
}

hipError_t launch_tile_mx(int V, int H, const uint8_t* codes, const uint8_t* scales, uint8_t* tiled, uint8_t* tiled_scales,
                          hipStream_t st) {
  const size_t n = (size_t)((V + 15) >> 4) * (((H >> 7) + 3) / 4 * 4);  // tiles, a wave each
  hipLaunchKernelGGL(tile_mx_kernel, dim3((unsigned)((n + 3) / 4)), dim3(256), 0, st, V, H, codes, scales, tiled, tiled_scales);
  return hipGetLastError();
}

hipError_t launch_quantize_mx(int V, int H, const uint16_t* w, uint8_t* tiled, uint8_t* tiled_scales, hipStream_t st) {
  const size_t n = (size_t)((V + 15) >> 4) * (((H >> 7) + 3) / 4);
  hipLaunchKernelGGL(quantize_mx_kernel, dim3((unsigned)n), dim3(256), 0, st, V, H, w, tiled, tiled_scales);
  return hipGetLastError();
}

hipError_t launch_unpack_mx(int V, int H, const uint8_t* tiled, const uint8_t* tiled_scales, uint16_t* out, hipStream_t st) {
  const size_t n = (size_t)((V + 15) >> 4) * (((H >> 7) + 3) / 4);
  hipLaunchKernelGGL(unpack_mx_kernel, dim3((unsigned)n), dim3(256), 0, st, V, H, tiled, tiled_scales, out);
  return hipGetLastError();
}

}  // namespace mds
