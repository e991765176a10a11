// Operand images of a compressed cache for the chunk attention: 128-token tiles of keys and
// values as the tensor cores read them from shared memory, so that the attention kernel fetches a
// tile by one bulk copy.
//
// Both images are K-major with the 128-byte swizzle: panels of 64 elements (128 bytes) per row,
// 128 rows a panel, the 16-byte piece c of row r at piece c ^ (r mod 8).
//   keys    row = token place, elements = channels (two panels)
//   values  row = channel, elements = token places (two panels): the transpose, formed here
// The place of token r within its 16-token block is 4 pv_lane(r) + pv_slot(r), the order in which
// the store keeps its value codes: a lane's four value codes of a word are then adjacent places of
// a row, and nothing has to be transposed.  The attention's logits come out in that order.
// Elements are fp16 (2^-12 rounding of the decoded fp32 value; beyond 65504 they saturate), bf16
// for the black-box store, which is exact.  Rows past the sequence's length are zero.
//
// One warp per 16-token block; bound by HBM (codes in, 64 KB a tile and head out) and, for the
// dithered store, by the integer work of its dither.
#include "dequant.cuh"

namespace witcert {

namespace {

// Two values as an operand pair.
template <bool BF16>
__device__ __forceinline__ uint32_t operand2(float a, float b) {
  if (BF16) return bf2_bits(__floats2bfloat162_rn(a, b));
  const __half2 lim = __half2half2(__ushort_as_half(0x7BFF));
  return h2_bits(__hmax2_nan(__hmin2_nan(__floats2half2_rn(a, b), lim), __hneg2(lim)));
}

template <int SCH>
__global__ void __launch_bounds__(256) expand_kernel(const __grid_constant__ AttendArgs a) {
  __shared__ float scratch[SCH == kInt8 ? 8 : 1][SCH == kInt8 ? kXsFloats : 1];
  constexpr bool kBf = SCH == kBbox;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.x % a.s.Hkv, tile_all = blockIdx.x / a.s.Hkv;
  int k = 0;
  while (a.tile_off[k + 1] <= tile_all) ++k;
  const int i = a.seq[k], len = a.len[k];
  const int blk = (tile_all - a.tile_off[k]) * 8 + warp, tb = blk * kBlk;
  uint8_t* kimg = a.images + ((size_t)tile_all * a.s.Hkv + h) * 2 * kTileBytes;
  uint8_t* vimg = kimg + kTileBytes;
  const bool any = tb < len;
  const uint8_t* bp = nullptr;
  const void* exact = nullptr;
  bool ebf = false;
  if (any) {
    bp = a.s.blocks + block_index(a.s.table, a.s.Hkv, a.s.nblk_max, i, h, blk) * block_bytes(SCH);
    exact = exact_rows<SCH>(a.s, i, h, blk, len, ebf);
  }
  float* xs = scratch[SCH == kInt8 ? warp : 0];
#pragma unroll 1
  for (int j = 0; j < 4; ++j) {
    float x[2][2][4] = {};
    if (any) {
      if (exact) exact_keys(a.s, exact, ebf, j, lane, x);
      else block_keys<SCH>(a.s, bp, h, a.s.pos0 + tb, j, lane, x);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tok = g + 8 * r, row = warp * kBlk + 4 * pv_lane(tok) + pv_slot(tok);
        const int c = 32 * j + 16 * m + 4 * t;
        const bool in = tb + tok < len;
        const uint2 v = make_uint2(operand2<kBf>(in ? x[m][r][0] : 0.f, in ? x[m][r][1] : 0.f),
                                   operand2<kBf>(in ? x[m][r][2] : 0.f, in ? x[m][r][3] : 0.f));
        *reinterpret_cast<uint2*>(kimg + (c >> 6) * (kTileTok * 128) + row * 128 +
                                  ((((c & 63) >> 3) ^ (row & 7)) << 4) + (c & 4) * 2) = v;
      }
    float y[2][2][4] = {};
    if (any) block_values<SCH>(a.s, bp, h, a.s.pos0 + tb, j, lane, xs, y);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 32 * j + 16 * m + 8 * r + g, place = warp * kBlk + 4 * t;
        float z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = tb + 2 * t + (e & 1) + 8 * (e >> 1) < len ? y[m][r][e] : 0.f;
        *reinterpret_cast<uint2*>(vimg + (place >> 6) * (kD * 128) + row * 128 +
                                  ((((place & 63) >> 3) ^ (row & 7)) << 4) + (place & 4) * 2) =
            make_uint2(operand2<kBf>(z[0], z[1]), operand2<kBf>(z[2], z[3]));
      }
  }
}

}  // namespace

cudaError_t launch_expand(int scheme, const AttendArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)(a.tile_off[a.n_seq] * a.s.Hkv);
  if (grid == 0) return cudaSuccess;
  switch (scheme) {
    case kInt8: expand_kernel<kInt8><<<grid, 256, 0, st>>>(a); break;
    case kRtn: expand_kernel<kRtn><<<grid, 256, 0, st>>>(a); break;
    case kFp8: expand_kernel<kFp8><<<grid, 256, 0, st>>>(a); break;
    case kKivi: expand_kernel<kKivi><<<grid, 256, 0, st>>>(a); break;
    default: expand_kernel<kBbox><<<grid, 256, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace witcert
