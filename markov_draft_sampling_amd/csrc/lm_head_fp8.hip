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
// a float32 logit shows. Each half block of 64 columns is scaled and added to
// the float32 total.
//
// The matrix is kept in tiles of 16 rows by 128 columns in operand order
// (fp8_tile_index): a wave reads its operands straight into registers as 1 KB
// runs, a chunk (128 columns) or more ahead, and widens them there; which
// columns a lane holds does not matter as long as both operands agree. The
// quantising kernel writes the hidden rows' codes, widened to bf16, in the
// same order, chunk by chunk with the rows' scales behind, so that a chunk goes
// into LDS as one linear copy without registers, shared by the waves.
//
// Bound by the matrix's V * H bytes for few rows; at 224 rows by the matrix
// cores and the LDS reads of the hidden rows, which is why a wave takes 64
// vocabulary rows (every hidden operand serves four products) and two waves
// share a vocabulary tile, each with half the hidden rows.
#include "mds_device.h"
#include "mds_internal.h"

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

// Hidden rows: a wave per 16 rows and 128 columns, a lane 32 columns of a row.
// Column c of row r of a block goes to 1 KB run c / 64 * 2 + c / 8 % 2, lane (c / 16 % 4) * 16 + r of it.
__global__ __launch_bounds__(256) void quant_rows_kernel(LmHeadFp8Args a) {
  const int HB = a.H >> 7, MBt = (a.M + 15) >> 4;
  const int wv = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (wv >= HB * MBt) return;
  const int lane = threadIdx.x & 63;
  const int mb = wv % MBt, j = wv / MBt;
  const int r = lane >> 2, m = mb * 16 + r, c0 = (lane & 3) * 32;
  const int mt = mb / a.mb, mi = mb - mt * a.mb;
  uint8_t* stage = a.xq + ((size_t)mt * HB + j) * fp8_stage_bytes(a.mb);
  uint8_t* dst = stage + mi * 4096 + (c0 >> 6) * 2048 + ((c0 >> 4 & 3) * 16 + r) * 16;
  float* xs = (float*)(stage + a.mb * 4096) + mi * 16 + r;
  float x[32];
  if (m < a.M) {
    const uint16_t* src = a.hidden + (long long)m * a.hidden_rs + j * 128 + c0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u32x4 v = *(const u32x4*)(src + q * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[q * 8 + 2 * i] = __uint_as_float(v[i] << 16);
        x[q * 8 + 2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = 0.0f;
  }
  float am = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < 32; ++i) am = fmaxf(am, fabsf(x[i]));
  am = fmaxf(am, __shfl_xor(am, 1));
  am = fmaxf(am, __shfl_xor(am, 2));
  const float s = am / kE4m3Max;
  // 16 columns (two runs) from c0, 16 from c0 + 16 (the next 16 lanes of the same runs)
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float* y = x + q * 16 + e * 8;
      const uint32_t lo = quant4(clamp_e4m3(y[0] / s), clamp_e4m3(y[1] / s), clamp_e4m3(y[2] / s), clamp_e4m3(y[3] / s));
      const uint32_t hi = quant4(clamp_e4m3(y[4] / s), clamp_e4m3(y[5] / s), clamp_e4m3(y[6] / s), clamp_e4m3(y[7] / s));
      *(bf16x8*)(dst + e * 1024 + q * 256) = widen8(lo, hi);
    }
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

// 16 bytes a lane straight into LDS
__device__ __forceinline__ void copy_1k(__amdgpu_buffer_rsrc_t rs, uint8_t* to, int lane_off, int off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)to, 16, lane_off, off, 0, 0);
}

// A work-group has MW x VW waves: wave (wm, wv) takes MB 16-row blocks of hidden rows from wm * MB and NBW
// 16-row blocks of the vocabulary. NST chunks of hidden rows in LDS, R chunks of the matrix in registers.
template <int MB, int NBW, int MW, int VW, int NST, int R>
__global__ __launch_bounds__(64 * MW * VW) __attribute__((amdgpu_waves_per_eu(2, 2))) void lm_head_fp8_kernel(
    LmHeadFp8Args a) {
  static_assert((NST == 2 || NST == 4) && NST % R == 0 && 8 % NBW == 0, "ring sizes, one scale block a wave");
  constexpr int NW = MW * VW;
  constexpr int kStage = fp8_stage_bytes(MB * MW);  // a chunk's hidden rows and their scales
  constexpr int kCopy = kStage / 1024;              // 1 KB copies of it, dealt to the waves in turn
  constexpr int kQ = (kCopy + NW - 1) / NW;
  constexpr int kLoads = 2 * NBW + 1;               // a wave's loads of a chunk of the matrix
  // newer operations than the copies of the next chunk: its loads, and all of the chunks after it
  constexpr int kNewer = kLoads + (NST - 2) * (kQ + kLoads);
  __shared__ __attribute__((aligned(16))) uint8_t s_x0[kStage], s_x1[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t s_x2[NST > 2 ? kStage : 16], s_x3[NST > 2 ? kStage : 16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / VW, wv = w % VW;
  const int lr = lane & 15, lg = lane >> 4;
  const int HB = a.H >> 7, VB = (a.V + 15) >> 4;
  const int mb0 = (blockIdx.y * MW + wm) * MB;
  const int vb0 = (blockIdx.x * VW + wv) * NBW;  // first 16-row block of this wave
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
  u32x4 raw[R][2][NBW];  // codes of 64 columns each
  float ws[R];
  auto load = [&](int slot, int p, int c) {
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb)
      raw[slot][p][nb] = __builtin_nontemporal_load((const u32x4*)(wp[nb] + (size_t)chunk_of(c) * 2048 + p * 1024));
  };
  floatx4 acc[NBW][MB];
#pragma unroll
  for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  // chunk c: hidden rows in LDS stage c % NST, matrix in register slot c % R. At its start the copies of chunk
  // c + NST - 1 go out; each half's registers are loaded with chunk c + R once they are widened.
  auto stage_of = [&](int i) { return i == 0 ? s_x0 : i == 1 ? s_x1 : i == 2 ? s_x2 : s_x3; };
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) {
    copy(stage_of(i), min(i, HB - 1));
    if (i < R) {
      load(i, 0, min(i, HB - 1));
      load(i, 1, min(i, HB - 1));
      ws[i] = wsp[chunk_of(min(i, HB - 1))];
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  if constexpr (R == NST) {
    load(R - 1, 0, min(R - 1, HB - 1));
    load(R - 1, 1, min(R - 1, HB - 1));
    ws[R - 1] = wsp[chunk_of(min(R - 1, HB - 1))];
    __builtin_amdgcn_sched_barrier(0);
  }
  chunk_barrier<kLoads>();
  auto chunk = [&](int c, int st, int slot) {
    const uint8_t* cur = stage_of(st) + wm * MB * 4096;
    const float* sx = (const float*)(stage_of(st) + MB * MW * 4096) + wm * MB * 16 + lr;
    copy(stage_of((st + NST - 1) % NST), min(c + NST - 1, HB - 1));  // the last chunk again at the end, never used
    const float sw = ws[slot];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      bf16x8 A[NBW][2];
#pragma unroll
      for (int nb = 0; nb < NBW; ++nb) {
        const u32x4 x = raw[slot][p][nb];
        A[nb][0] = widen8(x[0], x[1]);
        A[nb][1] = widen8(x[2], x[3]);
      }
      load(slot, p, min(c + R, HB - 1));
      if (p == 1) ws[slot] = wsp[chunk_of(min(c + R, HB - 1))];
      __builtin_amdgcn_sched_barrier(0);
      // one row block after the other, operand reads one block ahead, scaling one block behind (the order is
      // pinned: left alone the compiler holds every block's sums at once)
      const uint8_t* xb = cur + p * 2048 + lane * 16;
      bf16x8 b0 = *(const bf16x8*)xb, b1 = *(const bf16x8*)(xb + 1024);
      float s = sx[0], sp = 0.0f;
      floatx4 z[NBW], zp[NBW];
#pragma unroll
      for (int mb = 0; mb <= MB; ++mb) {
        bf16x8 n0 = b0, n1 = b1;
        float sn = s;
        if (mb + 1 < MB) {
          n0 = *(const bf16x8*)(xb + (mb + 1) * 4096);
          n1 = *(const bf16x8*)(xb + (mb + 1) * 4096 + 1024);
          sn = sx[(mb + 1) * 16];
        }
        if (mb < MB) {
#pragma unroll
          for (int nb = 0; nb < NBW; ++nb)
            z[nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[nb][0], b0, floatx4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
          for (int nb = 0; nb < NBW; ++nb) z[nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[nb][1], b1, z[nb], 0, 0, 0);
        }
        if (mb > 0) {
          const float f = sp * sw;
#pragma unroll
          for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nb][mb - 1][i] = __builtin_fmaf(zp[nb][i], f, acc[nb][mb - 1][i]);
        }
        __builtin_amdgcn_sched_barrier(0);
        b0 = n0;
        b1 = n1;
        sp = s;
        s = sn;
#pragma unroll
        for (int nb = 0; nb < NBW; ++nb) zp[nb] = z[nb];
      }
    }
    chunk_barrier<kNewer>();  // chunk c + 1's copies have landed
  };
  int c = 0;
#pragma nounroll
  for (; c + NST <= HB; c += NST)
#pragma unroll
    for (int i = 0; i < NST; ++i) chunk(c + i, i, i % R);
#pragma unroll
  for (int i = 0; i + 1 < NST; ++i)
    if (c + i < HB) chunk(c + i, i, i % R);
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

template <int MB, int NBW, int MW, int VW, int NST, int R>
hipError_t launch_mb(const LmHeadFp8Args& a, hipStream_t st) {
  const int VB = (a.V + 15) >> 4, MBt = (a.M + 15) >> 4;
  const dim3 grid((unsigned)((VB + VW * NBW - 1) / (VW * NBW)), (unsigned)((MBt + MB * MW - 1) / (MB * MW)));
  hipLaunchKernelGGL((lm_head_fp8_kernel<MB, NBW, MW, VW, NST, R>), grid, dim3(64 * MW * VW), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lm_head_fp8(const LmHeadFp8Args& a, hipStream_t st) {
  const int MBt = (a.M + 15) >> 4, HB = a.H >> 7;
  hipLaunchKernelGGL(quant_rows_kernel, dim3((unsigned)((HB * MBt + 3) / 4)), dim3(256), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  switch (a.mb) {
    case 1: return launch_mb<1, 1, 1, 4, 4, 4>(a, st);
    case 2: return launch_mb<2, 1, 1, 4, 4, 4>(a, st);
    case 4: return launch_mb<4, 2, 1, 4, 4, 4>(a, st);
    case 7: return launch_mb<7, 4, 1, 4, 2, 1>(a, st);
    default: return launch_mb<7, 4, 2, 4, 2, 1>(a, st);
  }
}

int lm_head_fp8_blocks(int M) {
  const int n = (M + 15) >> 4;
  return n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : n <= 7 ? 7 : 14;
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
