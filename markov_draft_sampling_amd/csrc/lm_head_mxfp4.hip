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

// lane: vocabulary rows 4 lg + (0 .. 3) of 16-row block vb for hidden row lr of row block mb
__device__ __forceinline__ void store_block(const LmHeadMxArgs& a, floatx4 z, int mb, int vb) {
  const int lane = threadIdx.x & 63, m = mb * 16 + (lane & 15), v = vb * 16 + (lane >> 4) * 4;
  if (m >= a.M || v >= a.V) return;
  const int b = m / a.K, k = m - b * a.K;
  const long long off = (long long)b * a.out_rs + (long long)k * a.out_ss + v;
  if (a.out_bf16) {
    uint16_t* o = (uint16_t*)a.out + off;
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = f32_to_bf16_bits(z[i]);
    if (a.vec_out && v + 3 < a.V) {
      *(u32x2*)o = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (v + i < a.V) o[i] = (uint16_t)h[i];
    }
  } else {
    float* o = (float*)a.out + off;
    if (a.vec_out && v + 3 < a.V) {
      *(f32x4*)o = f32x4{z[0], z[1], z[2], z[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (v + i < a.V) o[i] = z[i];
    }
  }
}

// Few hidden rows (MB 16-row blocks): the four waves of a work-group have the same NBW vocabulary blocks and divide the
// columns, 512 (four tiles, a word of scales) at a time; their sums are joined through LDS at the end. So a
// hidden row is read once a work-group, no wave waits for another before the end, and both operands go from memory into
// registers, NP tiles ahead.
template <int MB, int NBW>
__global__ __launch_bounds__(256) void lm_head_mx_kernel(LmHeadMxArgs a) {
  constexpr int NP = 2;
  __shared__ floatx4 s_z[4][NBW * MB][64];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int HB = a.H >> 7, G = (HB + 3) >> 2, VB = (a.V + 15) >> 4;
  const int vb0 = blockIdx.x * NBW, mb0 = blockIdx.y * MB;
  // the wave's tiles: words w, w + 4, .. of each row of tiles, of which only the last may be short
  const int words = G > w ? (G - w + 3) >> 2 : 0;
  const int n = words ? 4 * words - ((words - 1) * 4 + w == G - 1 ? 4 * G - HB : 0) : 0;
  const uint8_t* wp[NBW];
  const uint8_t* sp[NBW];
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb) {
    const size_t vb = (size_t)min(vb0 + nb, VB - 1);
    wp[nb] = a.w + vb * HB * 1024 + lane * 16;
    sp[nb] = a.w_scale + vb * G * 256 + lane * 4;
  }
  const uint16_t* xp[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) xp[mb] = a.hidden + (long long)min((mb0 + mb) * 16 + lr, a.M - 1) * a.hidden_rs + 32 * lg;
  floatx4 acc[NBW][MB];
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  u32x4 W[NP][NBW];
  uint32_t S[NP][NBW];
  bf16x8 X[NP][MB][4];
  auto tile_of = [&](int i) { return ((i >> 2) * 4 + w) * 4 + (i & 3); };
  auto load = [&](int p, int i) {
    const int c = tile_of(min(i, n - 1));
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb) {
      W[p][nb] = __builtin_nontemporal_load((const u32x4*)(wp[nb] + (size_t)c * 1024));
      S[p][nb] = *(const uint32_t*)(sp[nb] + (c >> 2) * 256);
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int s = 0; s < 4; ++s) X[p][mb][s] = *(const bf16x8*)(xp[mb] + c * 128 + 8 * s);
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
          for (int nb = 0; nb < NBW; ++nb) {
            const float sc = scale_of(S[p][nb], i & 3);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const bf16x8 A = widen(W[p][nb][s], sc);
#pragma unroll
              for (int mb = 0; mb < MB; ++mb)
                acc[nb][mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, X[p][mb][s], acc[nb][mb], 0, 0, 0);
            }
          }
        }
        load(p, i + NP);
      }
    }
  }
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) s_z[w][nb * MB + mb][lane] = acc[nb][mb];
  __syncthreads();
  for (int u = w; u < NBW * MB; u += 4) {
    const floatx4 z = (s_z[0][u][lane] + s_z[1][u][lane]) + (s_z[2][u][lane] + s_z[3][u][lane]);
    store_block(a, z, mb0 + u % MB, vb0 + u / MB);
  }
}

// 16 bytes a lane straight into LDS at `lds` (uniform) + 16 * lane, from base (uniform) + off, as assembly: the waits for
// these copies are the kernel's own. (m0, the LDS address, has no other use here; the load may read it one wait state
// after the scalar write at the earliest.)
__device__ __forceinline__ void copy_1k(const char* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory");
}

// More rows: a work-group of four waves has MB 16-row blocks of them, a wave all of these and NBW vocabulary blocks of
// its own. A tile's columns (128) at a time: the hidden rows in LDS, two of these deep and shared, 16-byte slots
// XOR-swizzled by row; the matrix in registers, loaded one ahead. The row tiles of a vocabulary tile run on
// the same XCD next to each other, so that the later ones find the matrix in the caches.
template <int MB, int NBW>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void lm_head_mx_wide_kernel(
    LmHeadMxArgs a, int v_tiles, int m_tiles) {
  constexpr int NW = 4;
  constexpr int kStage = MB * 4096;  // the hidden rows' 128 columns
  __shared__ __attribute__((aligned(16))) unsigned char s_x[2][kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int HB = a.H >> 7, G = (HB + 3) >> 2, VB = (a.V + 15) >> 4;
  // work-groups go to the eight XCDs in turn: row tile after row tile of eight vocabulary tiles
  const int grp = blockIdx.x / (8u * (unsigned)m_tiles), in = blockIdx.x - grp * 8 * m_tiles;
  const int vt = grp * 8 + (in & 7), mt = in >> 3;
  if (vt >= v_tiles) return;
  const int vb0 = (vt * NW + w) * NBW, m0 = mt * MB * 16;
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
    const unsigned char* cur = s_x[c & 1] + lr * 256;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8 A[NBW];
#pragma unroll
      for (int nb = 0; nb < NBW; ++nb) A[nb] = widen(cw[nb][s], sc[nb]);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const bf16x8 x = *(const bf16x8*)(cur + mb * 4096 + ((4 * lg + s) ^ lr) * 16);
#pragma unroll
        for (int nb = 0; nb < NBW; ++nb)
          acc[nb][mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[nb], x, acc[nb][mb], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb) store_block(a, acc[nb][mb], mt * MB + mb, vb0 + nb);
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

template <int MB, int NBW>
hipError_t launch_few(const LmHeadMxArgs& a, hipStream_t st) {
  const int VB = (a.V + 15) >> 4, MBt = (a.M + 15) >> 4;
  hipLaunchKernelGGL((lm_head_mx_kernel<MB, NBW>), dim3((unsigned)((VB + NBW - 1) / NBW), (unsigned)((MBt + MB - 1) / MB)),
                     dim3(256), 0, st, a);
  return hipGetLastError();
}
template <int MB, int NBW>
hipError_t launch_wide(const LmHeadMxArgs& a, hipStream_t st) {
  const int VB = (a.V + 15) >> 4, mt = (((a.M + 15) >> 4) + MB - 1) / MB;
  const int tiles = (VB + 4 * NBW - 1) / (4 * NBW);
  hipLaunchKernelGGL((lm_head_mx_wide_kernel<MB, NBW>), dim3((unsigned)((tiles + 7) / 8 * 8 * mt)), dim3(256), 0, st, a,
                     tiles, mt);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lm_head_mx(const LmHeadMxArgs& a, hipStream_t st) {
  // row tiles of at most 7 blocks, all of one height
  const int n = (a.M + 15) >> 4, tiles = (n + 6) / 7, mb = (n + tiles - 1) / tiles;
  switch (mb) {
    case 1: return launch_few<1, 4>(a, st);
    case 2: return launch_few<2, 4>(a, st);
    case 3: return launch_wide<3, 4>(a, st);
    case 4: return launch_wide<4, 4>(a, st);
    case 5: return launch_wide<5, 4>(a, st);
    case 6: return launch_wide<6, 4>(a, st);
    default: return launch_wide<7, 4>(a, st);
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
