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

// The dithered store's operand: s (code - xi) = code s + (-xi) s with one rounding of the sum; -xi is
// 1.5 - (1 + its upper 23 random bits), rounded to fp16 (2^-13 s), without an integer-to-float conversion,
// and so is its product with s (2^-12 s; 2^-25 where it is subnormal).  Both stay under what the store itself
// is off by, s / sqrt 12; formed in fp32 they would take two conversions and two FMAs an element.
__device__ __forceinline__ uint32_t neg_xi2(uint32_t u0, uint32_t u1) {
  return h2_bits(__floats2half2_rn(1.5f - __uint_as_float(__funnelshift_r(u0, 0x7Fu, 9)),
                                   1.5f - __uint_as_float(__funnelshift_r(u1, 0x7Fu, 9))));
}
__device__ __forceinline__ uint4 dither_words(const StoreArgs& s, int h, int t, int quad, int tensor) {
  return philox4x32_10_rk(make_uint4((uint32_t)t, (uint32_t)quad | ((uint32_t)tensor << 16),
                                     (uint32_t)h | ((uint32_t)s.layer << 16), 0u), s.rk0, s.rk1);
}
// -xi of step j of a block's keys, n[m][r][p] = channels 32j + 16m + 4t + 2p, + 1 of token g + 8r.
__device__ __forceinline__ void key_dither(const StoreArgs& s, int h, int tb, int j, int lane, uint32_t (&n)[2][2][2]) {
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint4 u = dither_words(s, h, tb + (lane >> 2) + 8 * r, 8 * j + 4 * m + (lane & 3), 0);
      n[m][r][0] = neg_xi2(u.x, u.y);
      n[m][r][1] = neg_xi2(u.z, u.w);
    }
}
// -xi of step j of its values, n[m][r][p] = tokens 2t + 8p, 2t + 8p + 1 of channel 32j + 16m + 8r + g.  One
// Philox call gives four channels of a token: a lane forms two tokens of a channel quad at a time in
// the warp's scratch xs, and picks out its own channels' pairs.
constexpr int kXwPitch = 40;                       // words per token pair: a lane's picks fall on distinct banks
constexpr int kXwWords = 8 * kXwPitch;             // scratch of one warp
__device__ __forceinline__ void value_dither(const StoreArgs& s, int h, int tb, int j, int lane, uint32_t* xs,
                                             uint32_t (&n)[2][2][2]) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int pr = 4 * k + (lane >> 3), q = lane & 7;      // tokens 2 pr, 2 pr + 1
    const uint4 u = dither_words(s, h, tb + 2 * pr, 8 * j + q, 1), v = dither_words(s, h, tb + 2 * pr + 1, 8 * j + q, 1);
    *reinterpret_cast<uint4*>(xs + pr * kXwPitch + 4 * q) =
        make_uint4(neg_xi2(u.x, v.x), neg_xi2(u.y, v.y), neg_xi2(u.z, v.z), neg_xi2(u.w, v.w));
  }
  __syncwarp();
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int p = 0; p < 2; ++p) n[m][r][p] = xs[((lane & 3) + 4 * p) * kXwPitch + 16 * m + 8 * r + (lane >> 2)];
}
// The dither depends on position, head and layer, not on the sequence: where several sequences are
// read, it is formed once, in the lanes' order, and fetched (dither_kernel in expand.cu).  Place of
// (tile, head, keys or values, token group, step, block) in 16-byte pieces, two a lane.
__device__ __forceinline__ size_t dither_at(int Hkv, int tile, int h, int values, int pr, int j, int b, int lane) {
  return (((((((size_t)tile * Hkv + h) * 2 + values) * 4 + pr) * 4 + j) * 2 + b) * 2) * 32 + lane;
}
__device__ __forceinline__ void load_dither(const uint4* table, size_t at, uint32_t (&n)[2][2][2]) {
  const uint4 lo = table[at], hi = table[at + 32];
  n[0][0][0] = lo.x; n[0][0][1] = lo.y; n[0][1][0] = lo.z; n[0][1][1] = lo.w;
  n[1][0][0] = hi.x; n[1][0][1] = hi.y; n[1][1][0] = hi.z; n[1][1][1] = hi.w;
}
__device__ __forceinline__ uint32_t dithered2(uint32_t code2, uint32_t nxi2, __half2 sc) {
  return half2_sat(__hfma2(bits_h2(code2), sc, __hmul2(bits_h2(nxi2), sc)));
}

// Four E4M3 codes as two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi) : "r"(w));
}

// kSteps steps of a block's keys from step j0 on as a lane reads them: codes and what decodes them.
// Decoding follows separately, so that the codes' buffer can be given back in between.
//   words(jj, n): step j0 + jj as operand pairs, w[m][r][p] = channels 32j + 16m + 4t + 2p, + 1 of token g + 8r
//   (n: its -xi, dithered store)
// The stores are decoded in fp16, the undithered ones with a single rounding.  The dithered store
// takes the steps one by one: its integer work, not memory, bounds it.
template <int SCH> constexpr int kSteps = SCH == kInt8 ? 1 : 2;

template <int SCH> struct KeyCodes {
  static constexpr int S = kSteps<SCH>;
  uint4 c[SCH == kBbox ? 4 : S];         // black box: (step, m)
  __half2 sc[S][2];                      // INT8: the steps' scales of tokens g and g + 8, twice
  __device__ __forceinline__ void load(const uint8_t* bp, int j0, int lane) {
    if constexpr (SCH == kBbox) {
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = *reinterpret_cast<const uint4*>(bp + BboxLayout::KH + ((2 * j0 + k) * 32 + lane) * 16);
    } else {
      static_assert(Int8Layout::KC == Fp8Layout::KC, "one place for the codes");
#pragma unroll
      for (int jj = 0; jj < S; ++jj) {
        c[jj] = *reinterpret_cast<const uint4*>(bp + Int8Layout::KC + (j0 + jj) * 512 + lane * 16);
        if constexpr (int8_layout(SCH)) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
            sc[jj][r] = __half2half2(*reinterpret_cast<const __half*>(bp + Int8Layout::KS + (((lane >> 2) + 8 * r) * 4 + j0 + jj) * 2));
        }
      }
    }
  }
  __device__ __forceinline__ void words(int jj, const uint32_t (&n)[2][2][2], uint32_t (&w)[2][2][2]) const {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if constexpr (SCH == kBbox) {
          const uint4& x = c[2 * jj + m];
          w[m][r][0] = r ? x.y : x.x;
          w[m][r][1] = r ? x.w : x.z;
        } else if constexpr (SCH == kFp8) {
          e4m3x4_pairs(word_of(c[jj], 2 * m + r), w[m][r][0], w[m][r][1]);
        } else {
          const uint32_t x = word_of(c[jj], 2 * m + r);
          if constexpr (SCH == kInt8) {
            w[m][r][0] = dithered2(i8x2_lo(x), n[m][r][0], sc[jj][r]);
            w[m][r][1] = dithered2(i8x2_hi(x), n[m][r][1], sc[jj][r]);
          } else {
            w[m][r][0] = half2_sat(__hmul2(bits_h2(i8x2_lo(x)), sc[jj][r]));
            w[m][r][1] = half2_sat(__hmul2(bits_h2(i8x2_hi(x)), sc[jj][r]));
          }
        }
      }
  }
};
template <> struct KeyCodes<kKivi> {
  uint2 c;
  uint4 sc[2], zr[2];                    // (step, m): four channels' scales and zeros
  __device__ __forceinline__ void load(const uint8_t* bp, int j0, int lane) {
    c = *reinterpret_cast<const uint2*>(bp + KiviLayout::KC + lane * 16 + j0 * 4);
    const uint8_t* kp = bp + KiviLayout::KP + ((lane & 3) * 32 + 2 * j0 * 4) * 2;
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      sc[jj] = *reinterpret_cast<const uint4*>(kp + 16 * jj);
      zr[jj] = *reinterpret_cast<const uint4*>(kp + 256 + 16 * jj);
    }
  }
  __device__ __forceinline__ void words(int jj, const uint32_t (&)[2][2][2], uint32_t (&w)[2][2][2]) const {
    const uint32_t x = jj ? c.y : c.x;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int p = 0; p < 2; ++p)
          w[m][r][p] = half2_sat(__hfma2(bits_h2(u2x2(x, m * 4 + r + 2 * p)), bits_h2(word_of(sc[jj], 2 * m + p)),
                                         bits_h2(word_of(zr[jj], 2 * m + p))));
  }
};

// The same for values: w[m][r][p] = tokens 2t + 8p, 2t + 8p + 1 of channel 32j + 16m + 8r + g.
template <int SCH> struct ValueCodes {
  static constexpr int S = kSteps<SCH>;
  uint4 c[SCH == kBbox ? 4 : S];
  uint2 sc[S];                           // INT8: the step's scales of the lane's four tokens
  __device__ __forceinline__ void load(const uint8_t* bp, int j0, int lane) {
    if constexpr (SCH == kBbox) {
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = *reinterpret_cast<const uint4*>(bp + BboxLayout::VH + ((2 * j0 + k) * 32 + lane) * 16);
    } else {
      static_assert(Int8Layout::VC == Fp8Layout::VC, "one place for the codes");
#pragma unroll
      for (int jj = 0; jj < S; ++jj) {
        c[jj] = *reinterpret_cast<const uint4*>(bp + Int8Layout::VC + (j0 + jj) * 512 + lane * 16);
        if constexpr (int8_layout(SCH)) sc[jj] = *reinterpret_cast<const uint2*>(bp + Int8Layout::VS + ((j0 + jj) * 16 + 4 * (lane & 3)) * 2);
      }
    }
  }
  __device__ __forceinline__ void words(int jj, const uint32_t (&n)[2][2][2], uint32_t (&w)[2][2][2]) const {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if constexpr (SCH == kBbox) {
          const uint4& x = c[2 * jj + m];
          w[m][r][0] = r ? x.y : x.x;
          w[m][r][1] = r ? x.w : x.z;
        } else if constexpr (SCH == kFp8) {
          e4m3x4_pairs(word_of(c[jj], 2 * m + r), w[m][r][0], w[m][r][1]);
        } else {
          const uint32_t x = word_of(c[jj], 2 * m + r);
          const __half2 lo = bits_h2(sc[jj].x), hi = bits_h2(sc[jj].y);
          if constexpr (SCH == kInt8) {
            w[m][r][0] = dithered2(i8x2_lo(x), n[m][r][0], lo);
            w[m][r][1] = dithered2(i8x2_hi(x), n[m][r][1], hi);
          } else {
            w[m][r][0] = half2_sat(__hmul2(bits_h2(i8x2_lo(x)), lo));
            w[m][r][1] = half2_sat(__hmul2(bits_h2(i8x2_hi(x)), hi));
          }
        }
      }
  }
};
template <> struct ValueCodes<kKivi> {
  uint2 c, sz[4];                        // tokens 2t, 2t + 1, 2t + 8, 2t + 9: the steps' (scale, zero) pairs
  __device__ __forceinline__ void load(const uint8_t* bp, int j0, int lane) {
    c = *reinterpret_cast<const uint2*>(bp + KiviLayout::VC + lane * 16 + j0 * 4);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      sz[e] = *reinterpret_cast<const uint2*>(bp + KiviLayout::VP + ((2 * (lane & 3) + (e & 1) + 8 * (e >> 1)) * 4 + j0) * 4);
  }
  __device__ __forceinline__ void words(int jj, const uint32_t (&)[2][2][2], uint32_t (&w)[2][2][2]) const {
    const uint32_t x = jj ? c.y : c.x;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const __half2 a = bits_h2(jj ? sz[2 * p].y : sz[2 * p].x), b = bits_h2(jj ? sz[2 * p + 1].y : sz[2 * p + 1].x);
      const __half2 sc = __lows2half2(a, b), zr = __highs2half2(a, b);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) w[m][r][p] = half2_sat(__hfma2(bits_h2(u2x2(x, m * 4 + r + 2 * p)), sc, zr));
    }
  }
};

// Two blocks of a tile (token group pr = 0..3, first token at position-in-sequence tb) for one warp.
// Blocks past the sequence may be anything.
struct BlockPair {
  const uint8_t* bp[2];
  const void* exact[2];          // exact key rows instead of the codes, or null
  bool ebf[2];
  int h, tb, len, pr, lane;
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
// Steps j0 and j0 + 1 (j0 = 0 or 2: one panel of the key image) of the two blocks into the key image,
// or the value image.  got() is called when the last codes are in registers, ready() before the first
// store: false gives up.  What is decoded together is decoded before any of it is stored: loads do
// not pass stores that might alias them.
template <int SCH, typename F, typename G>
__device__ __forceinline__ bool expand_keys(const StoreArgs& s, const BlockPair& x, int j0, uint8_t* img, F got, G ready) {
  constexpr int S = kSteps<SCH>;
  const int g = x.lane >> 2, t = x.lane & 3;
  const bool tail = x.tb + 2 * kBlk > x.len;
#pragma unroll 1
  for (int ja = 0; ja < 2; ja += S) {
    uint32_t n[2][2][2][2], w[S][2][2][2][2];                // [b][m][r][p]; [jj][b][m][r][p]
    if constexpr (SCH == kInt8) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (s.dither) load_dither(s.dither, dither_at(s.Hkv, x.tb / kTileTok, x.h, 0, x.pr, j0 + ja, b, x.lane), n[b]);
        else key_dither(s, x.h, s.pos0 + x.tb + b * kBlk, j0 + ja, x.lane, n[b]);
      }
    }
    KeyCodes<SCH> codes[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) codes[b].load(x.bp[b], j0 + ja, x.lane);
    if (ja + S == 2) got();
#pragma unroll
    for (int jj = 0; jj < S; ++jj)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (x.exact[b]) {
          float v[2][2][4];
          exact_keys(s, x.exact[b], x.ebf[b], j0 + ja + jj, x.lane, v);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int p = 0; p < 2; ++p) w[jj][b][m][r][p] = operand2<SCH>(v[m][r][2 * p], v[m][r][2 * p + 1]);
        } else {
          codes[b].words(jj, n[b], w[jj][b]);
        }
      }
    if (ja == 0 && !ready()) return false;
#pragma unroll
    for (int jj = 0; jj < S; ++jj)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = 32 * x.pr + 8 * (g >> 1) + 4 * (g & 1) + 2 * r + b;
          uint4 v = make_uint4(w[jj][b][0][r][0], w[jj][b][0][r][1], w[jj][b][1][r][0], w[jj][b][1][r][1]);
          if (tail && x.tb + b * kBlk + g + 8 * r >= x.len) v = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(img + (j0 >> 1) * (kTileTok * 128) + row * 128 + (((4 * (ja + jj) + t) ^ (row & 7)) << 4)) = v;
        }
  }
  return true;
}
template <int SCH, typename F, typename G>
__device__ __forceinline__ bool expand_values(const StoreArgs& s, const BlockPair& x, int j0, uint32_t* xs, uint8_t* img, F got,
                                              G ready) {
  constexpr int S = kSteps<SCH>;
  const int g = x.lane >> 2, t = x.lane & 3;
  const bool tail = x.tb + 2 * kBlk > x.len;
#pragma unroll 1
  for (int ja = 0; ja < 2; ja += S) {
    uint32_t n[2][2][2][2], w[S][2][2][2][2];                // [b][m][r][p]; [jj][b][m][r][p]
    if constexpr (SCH == kInt8) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (s.dither) load_dither(s.dither, dither_at(s.Hkv, x.tb / kTileTok, x.h, 1, x.pr, j0 + ja, b, x.lane), n[b]);
        else value_dither(s, x.h, s.pos0 + x.tb + b * kBlk, j0 + ja, x.lane, xs, n[b]);
      }
    }
    ValueCodes<SCH> codes[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) codes[b].load(x.bp[b], j0 + ja, x.lane);
    if (ja + S == 2) got();
#pragma unroll
    for (int jj = 0; jj < S; ++jj)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        codes[b].words(jj, n[b], w[jj][b]);
        if (tail) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int tok = x.tb + b * kBlk + 2 * t + 8 * p;
            const uint32_t keep = tok + 1 < x.len ? 0xFFFFFFFFu : tok < x.len ? 0xFFFFu : 0u;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int r = 0; r < 2; ++r) w[jj][b][m][r][p] &= keep;
          }
        }
      }
    if (ja == 0 && !ready()) return false;
#pragma unroll
    for (int jj = 0; jj < S; ++jj)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t (&a)[2] = w[jj][0][m][r], (&b)[2] = w[jj][1][m][r];
          const int row = 32 * (j0 + ja + jj) + 16 * m + 8 * r + 4 * (g & 1) + (g >> 1);
          *reinterpret_cast<uint4*>(img + (x.pr >> 1) * (kD * 128) + row * 128 + (((4 * (x.pr & 1) + t) ^ (row & 7)) << 4)) =
              make_uint4(__byte_perm(a[0], b[0], 0x5410), __byte_perm(a[1], b[1], 0x5410), __byte_perm(a[0], b[0], 0x7632),
                         __byte_perm(a[1], b[1], 0x7632));
        }
  }
  return true;
}

}  // namespace witcert
