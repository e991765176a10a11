// The keys and values a compressed cache stands for, as rows of the cache's dtype.
//
// One warp per (sequence, KV head, 16-token block), or, where that leaves the GPU empty, one per
// quarter of its channels (128 blocks of the dithered store: 12.2 us by whole blocks).  Bound by HBM: codes in, rows out (272 B and
// 512 B a token and head for INT8 caches of bf16 rows); the dithered store adds the regeneration
// of its dither, 2 x 32 Philox calls a token and head on the integer units.
//
// A lane's keys are four adjacent channels of a token: one 8-byte store, four lanes a sector.  Its
// values are four tokens of one channel, so bf16 values are packed in token pairs, transposed
// (movmatrix) into channel pairs of one token and exchanged between neighbour lanes into
// 8-byte pieces; fp32 values go out as they are, eight lanes a sector.
#include <type_traits>

#include "dequant.cuh"

namespace witcert {

namespace {

constexpr int kWarps = 4;
constexpr long long kFewUnits = 4096;            // about the warps the GPU holds at once

template <int SCH, bool BF16, bool QUARTERS>
__global__ void __launch_bounds__(kWarps * 32, SCH == kInt8 ? 9 : 8) read_kernel(const __grid_constant__ ReadArgs a) {
  __shared__ float scratch[SCH == kInt8 ? kWarps : 1][SCH == kInt8 ? kXsFloats : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  static_assert(kWarps == 4, "a warp a quarter");
  const long long unit = QUARTERS ? (long long)blockIdx.x : (long long)blockIdx.x * kWarps + warp;   // block * Hkv + head
  const int first = QUARTERS ? warp : 0;
  const int bidx = (int)(unit / a.s.Hkv), h = (int)(unit % a.s.Hkv);
  if (bidx >= a.blk_off[a.n_seq]) return;
  int lo = 0, hi = a.n_seq - 1;                                      // the k with blk_off[k] <= bidx < blk_off[k + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.blk_off[mid] <= bidx) lo = mid; else hi = mid - 1;
  }
  const int i = a.seq[lo], t0 = a.t0[lo], n = a.n[lo], blk = t0 / kBlk + (bidx - a.blk_off[lo]);
  const int tb = blk * kBlk;
  const uint8_t* bp = a.s.blocks + block_index(a.s.table, a.s.Hkv, a.s.nblk_max, i, h, blk) * block_bytes(SCH);
  bool ebf;
  const void* exact = exact_rows<SCH>(a.s, i, h, blk, a.len[lo], ebf);
  using T = typename std::conditional<BF16, __nv_bfloat16, float>::type;
  // element offset of token r of the block; used only where keep(r)
  auto row = [&](int r) { return ((a.row0[lo] + (tb + r - t0)) * a.s.Hkv + h) * kD; };
  auto keep = [&](int r) { return tb + r >= t0 && tb + r < t0 + n; };
  float* xs = scratch[SCH == kInt8 ? warp : 0];
  T* K = static_cast<T*>(a.K);
  T* V = static_cast<T*>(a.V);
#pragma unroll 1
  for (int j = first; j < (QUARTERS ? first + 1 : 4); ++j) {
    float x[2][2][4];
    if (exact) exact_keys(a.s, exact, ebf, j, lane, x);
    else block_keys<SCH>(a.s, bp, h, a.s.pos0 + tb, j, lane, x);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (!keep(g + 8 * r)) continue;
        T* o = K + row(g + 8 * r) + 32 * j + 16 * m + 4 * t;
        if constexpr (BF16)
          *reinterpret_cast<uint2*>(o) = make_uint2(bf2_bits(__floats2bfloat162_rn(x[m][r][0], x[m][r][1])),
                                                    bf2_bits(__floats2bfloat162_rn(x[m][r][2], x[m][r][3])));
        else
          *reinterpret_cast<float4*>(o) = make_float4(x[m][r][0], x[m][r][1], x[m][r][2], x[m][r][3]);
      }
    block_values<SCH>(a.s, bp, h, a.s.pos0 + tb, j, lane, xs, x);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int c0 = 32 * j + 16 * m;
      if constexpr (BF16) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {                                // tokens 0..7, 8..15 of the block
          const uint32_t b0 = movmatrix_trans(bf2_bits(__floats2bfloat162_rn(x[m][0][2 * u], x[m][0][2 * u + 1])));
          const uint32_t b1 = movmatrix_trans(bf2_bits(__floats2bfloat162_rn(x[m][1][2 * u], x[m][1][2 * u + 1])));
          // token g + 8u: b0 channels 2t, 2t + 1, b1 channels 8 + 2t, 9 + 2t
          const uint32_t got = __shfl_xor_sync(0xffffffffu, t & 1 ? b0 : b1, 1);
          if (keep(g + 8 * u))
            *reinterpret_cast<uint2*>(V + row(g + 8 * u) + c0 + (t & 1 ? 6 + 2 * t : 2 * t)) =
                t & 1 ? make_uint2(got, b1) : make_uint2(b0, got);
        }
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = 2 * t + (e & 1) + 8 * (e >> 1);
            if (keep(tok)) V[row(tok) + c0 + 8 * r + g] = x[m][r][e];
          }
      }
    }
  }
}

template <int SCH>
cudaError_t launch_s(const ReadArgs& a, cudaStream_t st) {
  const long long units = (long long)a.blk_off[a.n_seq] * a.s.Hkv;
  if (units < kFewUnits) {
    if (a.s.is_bf16) read_kernel<SCH, true, true><<<(unsigned)units, kWarps * 32, 0, st>>>(a);
    else read_kernel<SCH, false, true><<<(unsigned)units, kWarps * 32, 0, st>>>(a);
  } else {
    const unsigned grid = (unsigned)((units + kWarps - 1) / kWarps);
    if (a.s.is_bf16) read_kernel<SCH, true, false><<<grid, kWarps * 32, 0, st>>>(a);
    else read_kernel<SCH, false, false><<<grid, kWarps * 32, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_read(int scheme, const ReadArgs& a, cudaStream_t st) {
  if (a.blk_off[a.n_seq] == 0) return cudaSuccess;
  switch (scheme) {
    case kInt8: return launch_s<kInt8>(a, st);
    case kRtn: return launch_s<kRtn>(a, st);
    case kFp8: return launch_s<kFp8>(a, st);
    case kKivi: return launch_s<kKivi>(a, st);
    default: return launch_s<kBbox>(a, st);
  }
}

}  // namespace witcert
