// Tensor-core operand images from the compressed store: 128-token tiles of keys and values as the
// MMAs of the chunk attention read them from shared memory.
//
// Both images are K-major with the 128-byte swizzle: panels of 64 elements (128 bytes) a row, 128
// rows a panel, 16-byte piece c of row r at piece c ^ (r mod 8).
//   keys    row = token place, elements = channels, two panels
//   values  row = channel place, elements = token places, two panels: the transpose
// Orders inside a tile are free as long as both products agree, and are chosen so that every lane's
// codes are one 16-byte piece and a warp's pieces fall on distinct banks:
//   token 16 b + r of a group of 32 (two blocks) sits at place 8 ((r mod 8) / 2) + 4 (r mod 2) +
//   2 (r / 8) + b: eight value codes of a lane, four of either block, are adjacent, and nothing has
//   to be transposed.  The logits come out in this order.
//   channel 32 j + 16 m + 4 t + e of a key sits at element 32 j + 8 t + 4 m + e (so do the queries)
//   channel c of a value sits at row 8 (c / 8) + 4 (c mod 2) + (c mod 8) / 2 (the output's columns)
// Elements are fp16 (2^-11 rounding of the decoded value; beyond 65504 they saturate), or bf16 for
// the black-box store, which is exact.  Places past the sequence's length are zero.
#pragma once
#include "dequant.cuh"

namespace witcert {

__device__ __forceinline__ uint32_t half2_sat(__half2 v) {
  const __half2 lim = __half2half2(__ushort_as_half(0x7BFF));
  return h2_bits(__hmax2_nan(__hmin2_nan(v, lim), __hneg2(lim)));
}
// Two decoded values as an operand pair.
template <int SCH> __device__ __forceinline__ uint32_t operand2(float a, float b) {
  if (SCH == kBbox) return bf2_bits(__floats2bfloat162_rn(a, b));
  return half2_sat(__floats2half2_rn(a, b));
}

// Keys of step j of a block as operand pairs: w[m][r][p] = channels 32j + 16m + 4t + 2p, + 1 of token
// g + 8r.  The undithered stores are decoded in fp16 with a single rounding.
template <int SCH>
__device__ __forceinline__ void key_words(const StoreArgs& s, const uint8_t* bp, int h, int tb, int j, int lane,
                                          uint32_t (&w)[2][2][2]) {
  const int g = lane >> 2, t = lane & 3;
  if constexpr (SCH == kFp8) {
    const uint4 c = *reinterpret_cast<const uint4*>(bp + Fp8Layout::KC + j * 512 + lane * 16);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        w[m][r][0] = e4m3x2_lo(word_of(c, 2 * m + r));
        w[m][r][1] = e4m3x2_hi(word_of(c, 2 * m + r));
      }
  } else if constexpr (SCH == kRtn) {
    const uint4 c = *reinterpret_cast<const uint4*>(bp + Int8Layout::KC + j * 512 + lane * 16);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const __half2 sc = __half2half2(*reinterpret_cast<const __half*>(bp + Int8Layout::KS + ((g + 8 * r) * 4 + j) * 2));
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        w[m][r][0] = half2_sat(__hmul2(bits_h2(i8x2_lo(word_of(c, 2 * m + r))), sc));
        w[m][r][1] = half2_sat(__hmul2(bits_h2(i8x2_hi(word_of(c, 2 * m + r))), sc));
      }
    }
  } else if constexpr (SCH == kKivi) {
    const uint32_t c = *reinterpret_cast<const uint32_t*>(bp + KiviLayout::KC + lane * 16 + j * 4);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint8_t* kp = bp + KiviLayout::KP + (t * 32 + (2 * j + m) * 4) * 2;
      const uint2 sc = *reinterpret_cast<const uint2*>(kp), zr = *reinterpret_cast<const uint2*>(kp + 256);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        w[m][r][0] = half2_sat(__hfma2(bits_h2(u2x2(c, m * 4 + r)), bits_h2(sc.x), bits_h2(zr.x)));
        w[m][r][1] = half2_sat(__hfma2(bits_h2(u2x2(c, m * 4 + r + 2)), bits_h2(sc.y), bits_h2(zr.y)));
      }
    }
  } else if constexpr (SCH == kBbox) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint4 c = *reinterpret_cast<const uint4*>(bp + BboxLayout::KH + ((2 * j + m) * 32 + lane) * 16);
      w[m][0][0] = c.x; w[m][0][1] = c.z; w[m][1][0] = c.y; w[m][1][1] = c.w;
    }
  } else {
    float x[2][2][4];
    block_keys<SCH>(s, bp, h, tb, j, lane, x);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        w[m][r][0] = operand2<SCH>(x[m][r][0], x[m][r][1]);
        w[m][r][1] = operand2<SCH>(x[m][r][2], x[m][r][3]);
      }
  }
}

// Values of step j of a block as operand pairs: w[m][r][p] = tokens 2t + 8p, 2t + 8p + 1 of channel
// 32j + 16m + 8r + g.
template <int SCH>
__device__ __forceinline__ void value_words(const StoreArgs& s, const uint8_t* bp, int h, int tb, int j, int lane,
                                            float* xs, uint32_t (&w)[2][2][2]) {
  const int t = lane & 3;
  if constexpr (SCH == kFp8) {
    const uint4 c = *reinterpret_cast<const uint4*>(bp + Fp8Layout::VC + j * 512 + lane * 16);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        w[m][r][0] = e4m3x2_lo(word_of(c, 2 * m + r));
        w[m][r][1] = e4m3x2_hi(word_of(c, 2 * m + r));
      }
  } else if constexpr (SCH == kRtn) {
    const uint4 c = *reinterpret_cast<const uint4*>(bp + Int8Layout::VC + j * 512 + lane * 16);
    const uint2 sc = *reinterpret_cast<const uint2*>(bp + Int8Layout::VS + (j * 16 + 4 * t) * 2);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        w[m][r][0] = half2_sat(__hmul2(bits_h2(i8x2_lo(word_of(c, 2 * m + r))), bits_h2(sc.x)));
        w[m][r][1] = half2_sat(__hmul2(bits_h2(i8x2_hi(word_of(c, 2 * m + r))), bits_h2(sc.y)));
      }
  } else if constexpr (SCH == kKivi) {
    const uint32_t c = *reinterpret_cast<const uint32_t*>(bp + KiviLayout::VC + lane * 16 + j * 4);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      // (scale, zero) of tokens 2t + 8p and 2t + 8p + 1
      const __half2 a = *reinterpret_cast<const __half2*>(bp + KiviLayout::VP + ((2 * t + 8 * p) * 4 + j) * 4);
      const __half2 b = *reinterpret_cast<const __half2*>(bp + KiviLayout::VP + ((2 * t + 8 * p + 1) * 4 + j) * 4);
      const __half2 sc = __lows2half2(a, b), zr = __highs2half2(a, b);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) w[m][r][p] = half2_sat(__hfma2(bits_h2(u2x2(c, m * 4 + r + 2 * p)), sc, zr));
    }
  } else if constexpr (SCH == kBbox) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint4 c = *reinterpret_cast<const uint4*>(bp + BboxLayout::VH + ((2 * j + m) * 32 + lane) * 16);
      w[m][0][0] = c.x; w[m][0][1] = c.z; w[m][1][0] = c.y; w[m][1][1] = c.w;
    }
  } else {
    float x[2][2][4];
    block_values<SCH>(s, bp, h, tb, j, lane, xs, x);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        w[m][r][0] = operand2<SCH>(x[m][r][0], x[m][r][1]);
        w[m][r][1] = operand2<SCH>(x[m][r][2], x[m][r][3]);
      }
  }
}

// Two blocks of a tile (token group pr = 0..3, first token at position-in-sequence tb), and half of
// their channels (steps 2 jh, 2 jh + 1), by one warp.  Blocks past the sequence may be anything.
struct BlockPair {
  const uint8_t* bp[2];
  const void* exact[2];          // exact key rows instead of the codes, or null
  bool ebf[2];
  int h, tb, len, pr, jh, lane;
};
// The blocks' exact rows (see exact_rows), looked up where the sequence i holds the block.
template <int SCH>
__device__ __forceinline__ void find_exact(const StoreArgs& s, int i, BlockPair& x) {
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    x.exact[b] = nullptr;
    x.ebf[b] = false;
    if ((s.slots || SCH == kKivi) && x.tb + b * kBlk < x.len)
      x.exact[b] = exact_rows<SCH>(s, i, x.h, x.tb / kBlk + b, x.len, x.ebf[b]);
  }
}
template <int SCH>
__device__ __forceinline__ void expand_keys(const StoreArgs& s, const BlockPair& x, uint8_t* img) {
  const int g = x.lane >> 2, t = x.lane & 3;
  const bool tail = x.tb + 2 * kBlk > x.len;
#pragma unroll 1
  for (int j = 2 * x.jh; j < 2 * x.jh + 2; ++j)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t w[2][2][2];
      if (x.exact[b]) {
        float v[2][2][4];
        exact_keys(s, x.exact[b], x.ebf[b], j, x.lane, v);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int p = 0; p < 2; ++p) w[m][r][p] = operand2<SCH>(v[m][r][2 * p], v[m][r][2 * p + 1]);
      } else {
        key_words<SCH>(s, x.bp[b], x.h, s.pos0 + x.tb + b * kBlk, j, x.lane, w);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 32 * x.pr + 8 * (g >> 1) + 4 * (g & 1) + 2 * r + b;
        uint4 v = make_uint4(w[0][r][0], w[0][r][1], w[1][r][0], w[1][r][1]);
        if (tail && x.tb + b * kBlk + g + 8 * r >= x.len) v = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(img + (j >> 1) * (kTileTok * 128) + row * 128 + (((4 * (j & 1) + t) ^ (row & 7)) << 4)) = v;
      }
    }
}
template <int SCH>
__device__ __forceinline__ void expand_values(const StoreArgs& s, const BlockPair& x, float* xs, uint8_t* img) {
  const int g = x.lane >> 2, t = x.lane & 3;
  const bool tail = x.tb + 2 * kBlk > x.len;
#pragma unroll 1
  for (int j = 2 * x.jh; j < 2 * x.jh + 2; ++j) {
    uint32_t w[2][2][2][2];                                  // [b][m][r][p]
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      value_words<SCH>(s, x.bp[b], x.h, s.pos0 + x.tb + b * kBlk, j, x.lane, xs, w[b]);
      if (tail) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int tok = x.tb + b * kBlk + 2 * t + 8 * p;
          const uint32_t keep = tok + 1 < x.len ? 0xFFFFFFFFu : tok < x.len ? 0xFFFFu : 0u;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r) w[b][m][r][p] &= keep;
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 32 * j + 16 * m + 8 * r + 4 * (g & 1) + (g >> 1);
        const uint4 v = make_uint4(__byte_perm(w[0][m][r][0], w[1][m][r][0], 0x5410), __byte_perm(w[0][m][r][1], w[1][m][r][1], 0x5410),
                                   __byte_perm(w[0][m][r][0], w[1][m][r][0], 0x7632), __byte_perm(w[0][m][r][1], w[1][m][r][1], 0x7632));
        *reinterpret_cast<uint4*>(img + (x.pr >> 1) * (kD * 128) + row * 128 + (((4 * (x.pr & 1) + t) ^ (row & 7)) << 4)) = v;
      }
  }
}

}  // namespace witcert
