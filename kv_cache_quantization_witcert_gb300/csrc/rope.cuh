// Rotary positions: shared by the standalone kernel (rope.cu) and the rotating cache writers.
//
// Pair p of a head's first `rot` channels turns by pos f_p radians.  The angle is kept as a
// fraction of a turn in 64-bit fixed point, turn_p = f_p / (2 pi) mod 1 to the nearest multiple of
// 2^-64, so pos turn_p, wrapped by the integer product, is the reduced angle of any 64-bit position to
// within |pos| 2^-65 turns (no fp64, no table of positions).  The nearest quarter turn is taken
// off before the remainder (at most 1/8 turn) becomes fp32, which leaves 2^-27 half turns.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace witcert {

// gain cos, gain sin of pos turn.
__device__ __forceinline__ void rope_cs(uint64_t turn, int64_t pos, float gain, float& c, float& s) {
  const uint64_t phase = (uint64_t)pos * turn;
  const uint64_t near = phase + (1ull << 61);
  const int quarter = (int)(near >> 62);
  const float r = __fmul_rn((float)(int32_t)((phase - ((uint64_t)quarter << 62)) >> 32), 0x1p-31f);   // half turns
  // Taylor series at pi r, |pi r| <= pi / 4: the first terms left out are below 2^-29 and 2^-33
  const float t = __fmul_rn(r, 3.14159265358979f), q = __fmul_rn(t, t);
  float sr = __fmaf_rn(q, 1.0f / 362880.0f, -1.0f / 5040.0f);
  sr = __fmaf_rn(q, sr, 1.0f / 120.0f);
  sr = __fmaf_rn(q, sr, -1.0f / 6.0f);
  sr = __fmaf_rn(__fmul_rn(q, sr), t, t);
  float cr = __fmaf_rn(q, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  cr = __fmaf_rn(q, cr, -1.0f / 720.0f);
  cr = __fmaf_rn(q, cr, 1.0f / 24.0f);
  cr = __fmaf_rn(q, cr, -0.5f);
  cr = __fmaf_rn(q, cr, 1.0f);
  const float cs = quarter & 1 ? sr : cr, sn = quarter & 1 ? cr : sr;
  // quarter 0: (c, s), 1: (-s, c), 2: (-c, -s), 3: (s, -c)
  c = __fmul_rn(gain, quarter == 1 || quarter == 2 ? -cs : cs);
  s = __fmul_rn(gain, quarter >= 2 ? -sn : sn);
}
// The pair (a, b) turned: a c - b s and b c + a s, each with two roundings.
__device__ __forceinline__ float rope_first(float a, float b, float c, float s) { return __fmaf_rn(a, c, -__fmul_rn(b, s)); }
__device__ __forceinline__ float rope_second(float a, float b, float c, float s) { return __fmaf_rn(b, c, __fmul_rn(a, s)); }

}  // namespace witcert
