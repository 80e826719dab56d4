// LM head from an 8-bit matrix: logits[m, v] = sum over blocks j of 128
// columns of sx[m, j] sw[v / 128, j] sum_c qx[m, 128 j + c] qw[v, 128 j + c],
// with qw e4m3 and one float32 scale for each 128 x 128 block of the matrix,
// and the hidden rows quantised on the way in: for each row and 128 columns
// sx = max(amax, 2^-100) / 448 and qx = e4m3(x / sx), nearest even.
//
// Products of codes are exact and summed in float32 by the matrix cores
// (16x16x128 of 8-bit operands, twice the bf16 rate); each block's sum is
// scaled once and added to the float32 total.
//
// The call is bound by the matrix: V * H bytes, read once from HBM for up to
// 256 rows. It is kept in tiles of 16 rows by 128 columns in operand order
// (fp8_tile_index), so that a wave reads its operands straight into registers
// as two 1 KB runs and no LDS pass is needed; which 16 columns a lane holds
// does not matter as long as both operands agree. The quantised hidden rows
// are written in the same tiles by the quantising kernel and copied chunk by
// chunk into LDS, three chunks deep, shared by the work-group's eight waves.
#include "mds_device.h"
#include "mds_internal.h"

namespace mds {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 0x1p-100f;  // a block of zeros gets a scale it can be divided by
constexpr int kStagger = 5;  // chunk offset between consecutive work-groups
constexpr int kUnitScales = 0x7F7F7F7F;  // 2^0 for every operand block of the scaled matrix instruction

__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d) {
  const int p = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, p, true);
}
// Values past the largest (the quotient by a rounded scale) go to the largest; NaN stays NaN.
__device__ __forceinline__ float clamp_e4m3(float y) {
  return y != y ? y : fminf(fmaxf(y, -kE4m3Max), kE4m3Max);
}

// Hidden rows: a wave per 16 rows and 128 columns, a lane 32 columns of a row.
__global__ __launch_bounds__(256) void quant_rows_kernel(LmHeadFp8Args a) {
  const int HB = a.H >> 7, MBt = (a.M + 15) >> 4;
  const int wv = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (wv >= HB * MBt) return;
  const int lane = threadIdx.x & 63;
  const int mb = wv % MBt, j = wv / MBt;
  const int r = lane >> 2, m = mb * 16 + r, c0 = (lane & 3) * 32;
  const int mt = mb / a.mb, mi = mb - mt * a.mb;
  uint8_t* stage = a.xq + ((size_t)mt * HB + j) * fp8_stage_bytes(a.mb);
  uint8_t* dst = stage + mi * 2048 + r * 16;
  float* xs = (float*)(stage + a.mb * 2048) + mi * 16 + r;
  const int p0 = (lane & 3) * 2;
  if (m >= a.M) {
    *(u32x4*)(dst + p0 * 256) = u32x4{0, 0, 0, 0};
    *(u32x4*)(dst + p0 * 256 + 256) = u32x4{0, 0, 0, 0};
    if ((lane & 3) == 0) *xs = 0.0f;
    return;
  }
  const uint16_t* src = a.hidden + (long long)m * a.hidden_rs + j * 128 + c0;
  float x[32];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const u32x4 v = *(const u32x4*)(src + q * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[q * 8 + 2 * i] = __uint_as_float(v[i] << 16);
      x[q * 8 + 2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
  }
  float am = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < 32; ++i) am = fmaxf(am, fabsf(x[i]));
  am = fmaxf(am, __shfl_xor(am, 1));
  am = fmaxf(am, __shfl_xor(am, 2));
  const float s = am / kE4m3Max;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = quant4(clamp_e4m3(x[4 * i] / s), clamp_e4m3(x[4 * i + 1] / s), clamp_e4m3(x[4 * i + 2] / s),
                  clamp_e4m3(x[4 * i + 3] / s));
  *(u32x4*)(dst + p0 * 256) = u32x4{w[0], w[1], w[2], w[3]};
  *(u32x4*)(dst + p0 * 256 + 256) = u32x4{w[4], w[5], w[6], w[7]};
  if ((lane & 3) == 0) *xs = s;
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

// 16 x 16 sums over 128 columns of e4m3 codes
__device__ __forceinline__ floatx4 product(i32x8 a, i32x8 b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, floatx4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, kUnitScales,
                                                          0, kUnitScales);
}

// 16 bytes a lane straight into LDS
__device__ __forceinline__ void copy_1k(__amdgpu_buffer_rsrc_t rs, uint8_t* to, int lane_off, int off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)to, 16, lane_off, off, 0, 0);
}

// MB: 16-row blocks of hidden rows; NBW: 16-row vocabulary blocks per wave; eight waves.
template <int MB, int NBW>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void lm_head_fp8_kernel(LmHeadFp8Args a) {
  constexpr int NW = 8;
  constexpr int kStage = fp8_stage_bytes(MB);    // a chunk's hidden rows and their scales
  constexpr int kCopy = kStage / 1024;           // 1 KB copies of it, dealt to the waves in turn
  constexpr int kQ = (kCopy + NW - 1) / NW;
  constexpr int kLoads = 2 * NBW + 1;            // a wave's loads of a chunk of the matrix
  __shared__ __attribute__((aligned(16))) uint8_t s_x0[kStage], s_x1[kStage], s_x2[kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int HB = a.H >> 7, VB = (a.V + 15) >> 4;
  const int mb0 = blockIdx.y * MB;
  const int vb0 = (blockIdx.x * NW + w) * NBW;   // first 16-row block of this wave
  const int coff = (int)((blockIdx.x * (unsigned)kStagger) % (unsigned)HB);
  auto chunk_of = [&](int c) { return c + coff >= HB ? c + coff - HB : c + coff; };

  const uint8_t* wp[NBW];
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb) wp[nb] = a.w + (size_t)min(vb0 + nb, VB - 1) * HB * 2048 + lane * 16;
  const float* wsp = a.w_scale + (size_t)min(vb0 >> 3, (a.V - 1) >> 7) * HB;
  // copies as buffer loads: the compiler would have the flat form wait for every load in flight
  const __amdgpu_buffer_rsrc_t xrs = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.xq + (size_t)blockIdx.y * HB * kStage), (short)0, HB * kStage, 0x00020000);  // word 3: raw bytes
  auto copy = [&](uint8_t* buf, int c) {
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const int p = min(q * NW + w, kCopy - 1);  // every wave as many: the last piece may be copied twice
      copy_1k(xrs, buf + p * 1024, lane * 16, chunk_of(c) * kStage + p * 1024);
    }
  };
  i32x8 A[3][NBW];
  float ws[3];
  auto aload = [&](int slot, int c) {
    const int j = chunk_of(c);
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb) {
      const u32x4 a0 = __builtin_nontemporal_load((const u32x4*)(wp[nb] + (size_t)j * 2048));
      const u32x4 a1 = __builtin_nontemporal_load((const u32x4*)(wp[nb] + (size_t)j * 2048 + 1024));
      A[slot][nb] = i32x8{(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
    }
    ws[slot] = wsp[j];
  };
  floatx4 acc[NBW][MB];
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  // chunk c: its hidden rows in LDS buffer c % 3, its matrix tiles in register slot c % 3; the copies and
  // loads of chunk c + 2 go out at the start of chunk c
  copy(s_x0, 0);
  aload(0, 0);
  __builtin_amdgcn_sched_barrier(0);
  copy(s_x1, min(1, HB - 1));
  aload(1, min(1, HB - 1));
  __builtin_amdgcn_sched_barrier(0);
  chunk_barrier<kQ + 2 * kLoads>();
  auto chunk = [&](int c, int cc, const uint8_t* cur, uint8_t* nxt) {
    const int ch = min(c + 2, HB - 1);  // the last chunk is requested again at the end, never used
    copy(nxt, ch);
    aload((cc + 2) % 3, ch);
    __builtin_amdgcn_sched_barrier(0);
    const float sw = ws[cc];
    // one row block after the other: its operand reads one block ahead, its scaling one block behind the
    // products (the order is pinned: left alone the compiler holds every block's products at once)
    const float* sx = (const float*)(cur + MB * 2048) + lr;
    auto operand = [&](int mb) {
      const u32x4 b0 = *(const u32x4*)(cur + mb * 2048 + lane * 16);
      const u32x4 b1 = *(const u32x4*)(cur + mb * 2048 + 1024 + lane * 16);
      return i32x8{(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
    };
    i32x8 b = operand(0);
    float s = sx[0], sp = 0.0f;
    floatx4 z[NBW], zp[NBW];
#pragma unroll
    for (int mb = 0; mb <= MB; ++mb) {
      i32x8 bn = b;
      float sn = s;
      if (mb + 1 < MB) {
        bn = operand(mb + 1);
        sn = sx[(mb + 1) * 16];
      }
      if (mb < MB) {
#pragma unroll
        for (int nb = 0; nb < NBW; ++nb)
          z[nb] = product(A[cc][nb], b);
      }
      if (mb > 0) {
        const float f = sp * sw;
#pragma unroll
        for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[nb][mb - 1][i] = __builtin_fmaf(zp[nb][i], f, acc[nb][mb - 1][i]);
      }
      __builtin_amdgcn_sched_barrier(0);
      b = bn;
      sp = s;
      s = sn;
#pragma unroll
      for (int nb = 0; nb < NBW; ++nb) zp[nb] = z[nb];
    }
    // chunk c + 1's copies have landed: newer are its loads, and chunk c + 2's copies and loads
    chunk_barrier<kQ + 2 * kLoads>();
  };
  int c = 0;
#pragma nounroll
  for (; c + 3 <= HB; c += 3) {
    chunk(c, 0, s_x0, s_x2);
    chunk(c + 1, 1, s_x1, s_x0);
    chunk(c + 2, 2, s_x2, s_x1);
  }
  if (c < HB) chunk(c, 0, s_x0, s_x2);
  if (c + 1 < HB) chunk(c + 1, 1, s_x1, s_x0);
  // lane: vocabulary rows 4 lg + (0 .. 3) of its blocks for hidden row lr of each block
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

template <int MB, int NBW>
hipError_t launch_mb(const LmHeadFp8Args& a, hipStream_t st) {
  const int VB = (a.V + 15) >> 4, MBt = (a.M + 15) >> 4;
  const dim3 grid((unsigned)((VB + 8 * NBW - 1) / (8 * NBW)), (unsigned)((MBt + MB - 1) / MB));
  hipLaunchKernelGGL((lm_head_fp8_kernel<MB, NBW>), grid, dim3(512), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lm_head_fp8(const LmHeadFp8Args& a, hipStream_t st) {
  const int MBt = (a.M + 15) >> 4, HB = a.H >> 7;
  hipLaunchKernelGGL(quant_rows_kernel, dim3((unsigned)((HB * MBt + 3) / 4)), dim3(256), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  switch (a.mb) {
    case 1: return launch_mb<1, 2>(a, st);
    case 2: return launch_mb<2, 2>(a, st);
    case 4: return launch_mb<4, 2>(a, st);
    case 8: return launch_mb<8, 2>(a, st);
    case 12: return launch_mb<12, 2>(a, st);
    default: return launch_mb<14, 2>(a, st);
  }
}

int lm_head_fp8_blocks(int M) {
  const int n = (M + 15) >> 4;
  return n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : n <= 8 ? 8 : n <= 12 ? 12 : 14;
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
