// A block of the store expanded to the values it stands for, by one warp, in fp32.
//
// Lane 4g + t reads its fragment-order words as they lie (16 bytes a lane, conflict-free and
// coalesced).  Step j = 0..3 covers channels 32j .. 32j + 31 and gives the lane
//   keys    x[m][h][e] = token g + 8h, channel 32j + 16m + 4t + e
//   values  x[m][h][e] = token {2t, 2t + 1, 2t + 8, 2t + 9}[e], channel 32j + 16m + 8h + g
// The dithered store regenerates its dither: four channels of a token come from one Philox call,
// which is what a lane's keys need; values need one channel of four tokens, so the warp forms the
// step's 16 x 32 dithers once in a scratch of its own and picks them out.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace witcert {

constexpr int kXsPitch = 36;                     // floats per token: value dithers fall on distinct banks
constexpr int kXsFloats = kBlk * kXsPitch;       // scratch of one warp (dithered store only)

// Integer to float by placing bits, without conversions (which share a pipe with the dither's XORs):
// 2^23 + byte minus 2^23 + 128 is the code.  m, the upper 24 random bits, read as a float is m 2^-149
// (numbers below 2^-125 are evenly spaced, subnormal or not), so one FMA gives -xi = 1/2 - m 2^-24, exact.
__device__ __forceinline__ float code_i8(uint32_t w, int e) {
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | (uint32_t)e)) - 8388736.0f;
}
__device__ __forceinline__ float neg_xi24(uint32_t u) { return __fmaf_rn(__uint_as_float(u >> 8), -0x1p125f, 0.5f); }
__device__ __forceinline__ float4 neg_dither4_24(const StoreArgs& s, int h, int t, int quad, int tensor) {
  const uint4 u = philox4x32_10_rk(make_uint4((uint32_t)t, (uint32_t)quad | ((uint32_t)tensor << 16),
                                              (uint32_t)h | ((uint32_t)s.layer << 16), 0u), s.rk0, s.rk1);
  return make_float4(neg_xi24(u.x), neg_xi24(u.y), neg_xi24(u.z), neg_xi24(u.w));
}
__device__ __forceinline__ void e4m3x4(uint32_t w, float (&x)[4]) {
  const float2 lo = __half22float2(bits_h2(e4m3x2_lo(w))), hi = __half22float2(bits_h2(e4m3x2_hi(w)));
  x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
}
__device__ __forceinline__ void bf16x4(uint32_t a, uint32_t b, float (&x)[4]) {
  x[0] = __uint_as_float(a << 16); x[1] = __uint_as_float(a & 0xFFFF0000u);
  x[2] = __uint_as_float(b << 16); x[3] = __uint_as_float(b & 0xFFFF0000u);
}
__device__ __forceinline__ float half_at(const uint8_t* p) { return __half2float(*reinterpret_cast<const __half*>(p)); }
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Keys of step j; tb is the position of the block's first token (dither).
template <int SCH>
__device__ __forceinline__ void block_keys(const StoreArgs& s, const uint8_t* bp, int h, int tb, int j, int lane,
                                           float (&x)[2][2][4]) {
  const int g = lane >> 2, t = lane & 3;
  if constexpr (int8_layout(SCH)) {
    const uint4 w = *reinterpret_cast<const uint4*>(bp + Int8Layout::KC + j * 512 + lane * 16);
    const float sc[2] = {half_at(bp + Int8Layout::KS + (g * 4 + j) * 2), half_at(bp + Int8Layout::KS + ((g + 8) * 4 + j) * 2)};
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float4 nx = make_float4(0.f, 0.f, 0.f, 0.f);
        if (SCH == kInt8) nx = neg_dither4_24(s, h, tb + g + 8 * r, 8 * j + 4 * m + t, 0);
        const float n4[4] = {nx.x, nx.y, nx.z, nx.w};
        const uint32_t c = word_of(w, 2 * m + r);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[m][r][e] = (code_i8(c, e) + n4[e]) * sc[r];
      }
  } else if constexpr (SCH == kFp8) {
    const uint4 w = *reinterpret_cast<const uint4*>(bp + Fp8Layout::KC + j * 512 + lane * 16);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) e4m3x4(word_of(w, 2 * m + r), x[m][r]);
  } else if constexpr (SCH == kKivi) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(bp + KiviLayout::KC + lane * 16 + j * 4);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint8_t* kp = bp + KiviLayout::KP + (t * 32 + (2 * j + m) * 4) * 2;
      const uint2 su = *reinterpret_cast<const uint2*>(kp), zu = *reinterpret_cast<const uint2*>(kp + 256);
      const float2 s01 = __half22float2(bits_h2(su.x)), s23 = __half22float2(bits_h2(su.y));
      const float2 z01 = __half22float2(bits_h2(zu.x)), z23 = __half22float2(bits_h2(zu.y));
      const float sc[4] = {s01.x, s01.y, s23.x, s23.y}, zr[4] = {z01.x, z01.y, z23.x, z23.y};
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int bit = 2 * (m * 4 + r + 2 * (e >> 1)) + 16 * (e & 1);
          x[m][r][e] = __fmaf_rn(sc[e], (float)((w >> bit) & 3u), zr[e]);
        }
    }
  } else {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint4 w = *reinterpret_cast<const uint4*>(bp + BboxLayout::KH + ((2 * j + m) * 32 + lane) * 16);
      bf16x4(w.x, w.z, x[m][0]);
      bf16x4(w.y, w.w, x[m][1]);
    }
  }
}

// Exact key rows (a repaired block's, or KIVI's unfinished block's) in place of the codes' values.
__device__ __forceinline__ void exact_keys(const StoreArgs& s, const void* rows, bool bf16, int j, int lane,
                                           float (&x)[2][2][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const size_t o = (size_t)(g + 8 * r) * kD + 32 * j + 16 * m + 4 * t;
      if (bf16) {
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(rows) + o);
        bf16x4(u.x, u.y, x[m][r]);
      } else {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(rows) + o);
        x[m][r][0] = v.x; x[m][r][1] = v.y; x[m][r][2] = v.z; x[m][r][3] = v.w;
      }
    }
}
// Where the exact rows of block blk lie: the exact pool if it is repaired, the tail if it is
// KIVI's unfinished block (len tokens held), null otherwise.
template <int SCH>
__device__ __forceinline__ const void* exact_rows(const StoreArgs& s, int i, int h, int blk, int len, bool& bf16) {
  const size_t sh = (size_t)i * s.Hkv + h;
  bf16 = s.is_bf16 != 0;
  const int slot = s.slots ? s.slots[sh * s.nblk_max + blk] : -1;
  if (slot >= 0) return static_cast<const uint8_t*>(s.pool) + (size_t)slot * kBlk * kD * (bf16 ? 2 : 4);
  if (SCH == kKivi && blk == len / kBlk) {
    bf16 = false;
    return s.kivi_tail + sh * kBlk * kD;
  }
  return nullptr;
}

// Values of step j (xs: the warp's scratch, used by the dithered store).
template <int SCH>
__device__ __forceinline__ void block_values(const StoreArgs& s, const uint8_t* bp, int h, int tb, int j, int lane,
                                             float* xs, float (&x)[2][2][4]) {
  const int g = lane >> 2, t = lane & 3;
  if constexpr (int8_layout(SCH)) {
    if constexpr (SCH == kInt8) {
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 4 * k + (lane >> 3), quad = lane & 7;
        *reinterpret_cast<float4*>(xs + r * kXsPitch + quad * 4) =
            neg_dither4_24(s, h, tb + r, 8 * j + quad, 1);
      }
      __syncwarp();
    }
    const uint4 w = *reinterpret_cast<const uint4*>(bp + Int8Layout::VC + j * 512 + lane * 16);
    const uint2 su = *reinterpret_cast<const uint2*>(bp + Int8Layout::VS + (j * 16 + 4 * t) * 2);
    const float2 s01 = __half22float2(bits_h2(su.x)), s23 = __half22float2(bits_h2(su.y));
    const float sc[4] = {s01.x, s01.y, s23.x, s23.y};
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t c = word_of(w, 2 * m + r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float nx = SCH == kInt8 ? xs[(2 * t + (e & 1) + 8 * (e >> 1)) * kXsPitch + 16 * m + 8 * r + g] : 0.f;
          x[m][r][e] = (code_i8(c, e) + nx) * sc[e];
        }
      }
  } else if constexpr (SCH == kFp8) {
    const uint4 w = *reinterpret_cast<const uint4*>(bp + Fp8Layout::VC + j * 512 + lane * 16);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) e4m3x4(word_of(w, 2 * m + r), x[m][r]);
  } else if constexpr (SCH == kKivi) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(bp + KiviLayout::VC + lane * 16 + j * 4);
    float sc[4], zr[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int tok = 2 * t + (e & 1) + 8 * (e >> 1);
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(bp + KiviLayout::VP + (tok * 4 + j) * 4));
      sc[e] = p.x; zr[e] = p.y;
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int bit = 2 * (m * 4 + r + 2 * (e >> 1)) + 16 * (e & 1);
          x[m][r][e] = __fmaf_rn(sc[e], (float)((w >> bit) & 3u), zr[e]);
        }
  } else {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint4 w = *reinterpret_cast<const uint4*>(bp + BboxLayout::VH + ((2 * j + m) * 32 + lane) * 16);
      bf16x4(w.x, w.z, x[m][0]);
      bf16x4(w.y, w.w, x[m][1]);
    }
  }
}

}  // namespace witcert
