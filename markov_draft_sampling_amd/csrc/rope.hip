// Norm and rotation of the queries and keys of new tokens, and the append of
// the keys and values to the paged cache in the same pass.
//
// Per head of D columns, with the weights w where they are given,
//   y = x w / sqrt(mean(x^2) + eps),
// and for pair i of the R / 2 pairs of the first R columns, (i, i + R / 2) or
// (2 i, 2 i + 1), at the angle a = position * inv_freq[i],
//   (y1, y2) -> s (y1 cos a - y2 sin a, y2 cos a + y1 sin a);
// columns from R on keep y. All in float32 from the bf16 inputs, rounded once
// where it is written (bf16, or e4m3 of the quotient by the head's scale).
// Angles, sines and cosines are float64 until they are rounded to float32: at
// position 10^6 a float32 angle is a sixteenth of a radian off.
//
// An e4m3 code is a sixteenth of its value: where the quotient is next to the
// border of two codes, the last bit of float32 decides. So that float32 decides
// alike wherever a key is computed, sines and cosines here are the float32
// nearest to those of the float64 angle, at far positions too, and 1 / sqrt that
// nearest to the root of the float32 mean (but where float64 cannot tell which of
// two is nearer, some 1 in 10^7), products are rounded one by one and squares are
// summed fours in turn and then neighbours. (That is the columns' order, except
// where a part of a head is turned in halves: there a lane's two eights of columns
// are R / 2 apart, and the sum may differ in its last bits.) (Heads of 128: with
// float32 sines and fused products three codes in a million fell on the other side
// than by separate operations, now none of 43 million; the prompt below takes
// 76.1 us and took 75.3.)
//
// A wave takes some heads of one token, LPH lanes a head and 16 columns a lane:
// two pieces of 16 bytes, which in either layout are whole pairs (columns 8 j
// and R / 2 + 8 j on, or 16 j on), so that no lane needs another's columns and
// the sum of squares is the only exchange. The 64 lanes compute the token's
// sines and cosines once, a pair each, and read their eight pairs from LDS.
//
// Bound by HBM for prompts, every element read and written once (16384 tokens of
// 32 query and 8 key heads of 128 with their values, 403 MB: 76 us, 5.3 TB/s),
// by the launch for a decoding step (one token 3.3 us, 256 tokens 4.2 us).
#include "mds_device.h"
#include "mds_serve.h"

namespace mds {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kMaxPairs = 128;  // of a head (D <= 256)

enum RopeTo { kRows, kPages, kPages8 };  // keys (and values) go to rows, bf16 pages, e4m3 pages

template <int CTRL>
__device__ __forceinline__ float dpp_sum(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
}
// Sum over groups of LPH lanes, in each of them
template <int LPH>
__device__ __forceinline__ float group_sum(float x) {
  x = dpp_sum<0xB1>(x);                           // neighbours
  x = dpp_sum<0x4E>(x);                           // pairs of a quad
  if constexpr (LPH > 4) x = dpp_sum<0x141>(x);   // quads of eight: the mirrored lane has the other one's sum
  if constexpr (LPH > 8) x = dpp_sum<0x140>(x);   // eights of a row
  return x;
}

__device__ __forceinline__ void unpack8(u32x4 v, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v[i] << 16);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ u32x4 pack8(const float* x) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16x2 b = {(__bf16)x[2 * i], (__bf16)x[2 * i + 1]};
    r[i] = __builtin_bit_cast(uint32_t, b);
  }
  return r;
}
// 8 e4m3 codes: nearest even of the float32 quotient, past the largest value to the largest; NaN stays NaN
__device__ __forceinline__ u32x2 quant8(const float* x, float scale) {
  u32x2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float y = x[4 * h + i] / scale;
      f[i] = y != y ? y : fminf(fmaxf(y, -448.0f), 448.0f);
    }
    const int p = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    o[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], p, true);
  }
  return o;
}

// U: heads a lane takes; a wave takes 64 / LPH * U of a token
template <int LPH, int U, int TO>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, int per_token) {
  __shared__ float2 s_turn[4][kMaxPairs];  // a wave's token: cosine and sine of each pair
  constexpr int HPW = 64 / LPH;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const unsigned unit = blockIdx.x * 4u + (unsigned)w;
  const int t = (int)(unit / (unsigned)per_token), part = (int)(unit - (unsigned)t * (unsigned)per_token);
  if (t >= a.T) return;
  const int g = lane / LPH, j = lane % LPH;
  const int heads = a.Hq + (TO == kRows ? a.Hk : 2 * a.Hk);
  const int lanes = a.D >> 4;                    // lanes of a head that have columns
  const bool turned = j < a.R >> 4;
  const bool split = turned && !a.interleaved;   // the lane's pieces are R / 2 columns apart
  const int c0 = split ? 8 * j : 16 * j, c1 = split ? 8 * j + (a.R >> 1) : 16 * j + 8;

  const bool halves = a.R == a.D && !a.interleaved;  // every lane's pieces are half a head apart

  const double pos = (double)a.positions[t];
  u32x4 x[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = (part * U + u) * HPW + g;
    if (h >= heads || j >= lanes) continue;
    const uint16_t* p = h < a.Hq ? a.q + t * a.q_ts + h * a.q_hs
                        : h < a.Hq + a.Hk ? a.k + t * a.k_ts + (h - a.Hq) * a.k_hs
                                          : a.v + t * a.v_ts + (h - a.Hq - a.Hk) * a.v_hs;
    x[u][0] = *(const u32x4*)(p + c0);
    x[u][1] = *(const u32x4*)(p + c1);
  }
  long long slot = 0;
  if constexpr (TO != kRows) slot = a.slot_map[t];
  for (int i = lane; i < a.R >> 1; i += 64) {
    // The angle's turns without the whole ones. An angle is rounded once, its turns are not: the product with 1 / (2 pi)
    // is a sum of two, so that a far position's sine is that of its angle. (Fused, the difference would have the rest already.)
#pragma clang fp contract(off)
    constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnRest = -0x1.6b01ec5417056p-57;
    const double angle = pos * a.inv_freq[i], turns = angle * kTurn;
    const double rest = __builtin_fma(angle, kTurnRest, __builtin_fma(angle, kTurn, -turns));
    double s, c;
    sincospi(2.0 * ((turns - __builtin_rint(turns)) + rest), &s, &c);
    s_turn[w][i] = make_float2((float)(c * a.rope_scale), (float)(s * a.rope_scale));
  }
  // (a wave's LDS operations keep their order)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  float cs[8], sn[8];
  if (turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = s_turn[w][8 * j + i];
      cs[i] = f.x;
      sn[i] = f.y;
    }
  }
  bool keep = true;
  long long page = 0, in_page = 0;
  if constexpr (TO != kRows) {
    page = slot >> a.page_log2;
    in_page = slot & ((1 << a.page_log2) - 1);
    keep = slot >= 0;
    if (page >= a.n_pages) {
      keep = false;
      if (lane == 0) set_status(a.status, kStatusBadPage);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = (part * U + u) * HPW + g;
    const bool here = h < heads && j < lanes;
    const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hk;
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = 0.0f;
    if (here) {
      unpack8(x[u][0], y);
      unpack8(x[u][1], y + 8);
    }
    const uint16_t* weight = is_q ? a.q_weight : a.k_weight;
    if (a.q_weight || a.k_weight) {
      float sum[4];  // of four columns each, whose squares float32 holds exactly
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* z = y + 4 * i;
        sum[i] = ((z[0] * z[0] + z[1] * z[1]) + z[2] * z[2]) + z[3] * z[3];
      }
      float lo = sum[0] + sum[1], hi = sum[2] + sum[3];
      if (!halves) {
        lo += hi;
        hi = 0.0f;
      }
      const float ss = group_sum<LPH>(lo) + group_sum<LPH>(hi);
      if (here && weight && !is_v) {
        const float r = (float)rsqrt((double)(ss / (float)a.D + a.eps));
        float f[16];
        unpack8(*(const u32x4*)(weight + c0), f);
        unpack8(*(const u32x4*)(weight + c1), f + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = y[i] * r * f[i];
      }
    }
    if (!here) continue;
    if (turned && !is_v) {
#pragma clang fp contract(off)
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = y[2 * i], q = y[2 * i + 1];
          y[2 * i] = p * cs[i] - q * sn[i];
          y[2 * i + 1] = q * cs[i] + p * sn[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = y[i], q = y[8 + i];
          y[i] = p * cs[i] - q * sn[i];
          y[8 + i] = q * cs[i] + p * sn[i];
        }
      }
    }
    if (is_q || TO == kRows) {
      uint16_t* o = is_q ? a.q_out + t * a.qo_ts + h * a.qo_hs : a.k_out + t * a.ko_ts + (h - a.Hq) * a.ko_hs;
      *(u32x4*)(o + c0) = pack8(y);
      *(u32x4*)(o + c1) = pack8(y + 8);
      continue;
    }
    if (!keep) continue;
    const int hk = is_v ? h - a.Hq - a.Hk : h - a.Hq;
    const long long at = is_v ? page * a.ps[1] + in_page * a.ts[1] + hk * a.hs[1]
                              : page * a.ps[0] + in_page * a.ts[0] + hk * a.hs[0];
    if constexpr (TO == kPages8) {
      uint8_t* o = (uint8_t*)(is_v ? a.v_pages : a.k_pages) + at;
      const float sc = (is_v ? a.v_scale : a.k_scale)[hk];
      *(u32x2*)(o + c0) = quant8(y, sc);
      *(u32x2*)(o + c1) = quant8(y + 8, sc);
    } else {
      uint16_t* o = (uint16_t*)(is_v ? a.v_pages : a.k_pages) + at;
      *(u32x4*)(o + c0) = is_v ? x[u][0] : pack8(y);
      *(u32x4*)(o + c1) = is_v ? x[u][1] : pack8(y + 8);
    }
  }
}

template <int LPH, int U, int TO>
hipError_t launch(const RopeArgs& a, const RopePlan& p, hipStream_t st) {
  const long long n = (long long)a.T * p.per_token;
  hipLaunchKernelGGL((rope_kernel<LPH, U, TO>), dim3((unsigned)((n + 3) / 4)), dim3(256), 0, st, a, p.per_token);
  return hipGetLastError();
}
template <int LPH, int TO>
hipError_t launch_lanes(const RopeArgs& a, const RopePlan& p, hipStream_t st) {
  return p.heads == 2 ? launch<LPH, 2, TO>(a, p, st) : launch<LPH, 1, TO>(a, p, st);
}
template <int TO>
hipError_t launch_to(const RopeArgs& a, hipStream_t st) {
  const RopePlan p = rope_plan(a.T, a.Hq + (TO == kRows ? a.Hk : 2 * a.Hk), a.D);
  if (p.lanes == 4) return launch_lanes<4, TO>(a, p, st);
  return p.lanes == 8 ? launch_lanes<8, TO>(a, p, st) : launch_lanes<16, TO>(a, p, st);
}

}  // namespace

RopePlan rope_plan(int T, int heads, int D) {
  RopePlan p;
  p.lanes = D <= 64 ? 4 : D <= 128 ? 8 : 16;
  const int waves = (heads * p.lanes + 63) / 64;  // of a token, at one head a lane
  // Two heads a lane once the waves fill the CUs: sines, cosines and positions serve two, and twice the bytes are in flight
  // (us with one and two: 32 + 2 x 8 heads of 128, 24576 waves 21.5 and 19.4, 6144 7.5 and 7.5; 16 + 2 x 4 of 256, 6144
  // 7.9 and 7.7; 8 + 2 x 2 of 128, 4096 5.0 and 5.2; 27 of 64, 4096 4.6 and 4.6, 2048 3.4 and 3.7. With three the
  // prompt above takes 79 against 76).
  p.heads = (long long)T * waves > 4096 ? 2 : 1;
  p.per_token = (waves + p.heads - 1) / p.heads;
  return p;
}

hipError_t launch_rope(const RopeArgs& a, hipStream_t st) {
  if (!a.k_pages) return launch_to<kRows>(a, st);
  return a.e4m3 ? launch_to<kPages8>(a, st) : launch_to<kPages>(a, st);
}

}  // namespace mds
