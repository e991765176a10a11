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
#include <algorithm>
#include <climits>
#include <type_traits>

#include "dequant.cuh"

namespace witcert {

namespace {

constexpr int kWarps = 4;
constexpr long long kFewUnits = 4096;            // about the warps the GPU holds at once
constexpr int kSharedCtas = 1216;                // CTAs that fill the GPU
constexpr int kShare = 2;                        // sequences a dither serves, on average, for sharing it

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

// ------------------------------------------------------------------ a dither for several sequences
// The dither of step j's keys, taken off (dithered store): the same for every sequence.
__device__ __forceinline__ void key_dither(const StoreArgs& s, int h, int tb, int j, int lane, float (&nx)[2][2][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float4 d = neg_dither4_24(s, h, tb + g + 8 * r, 8 * j + 4 * m + t, 0);
      nx[m][r][0] = d.x; nx[m][r][1] = d.y; nx[m][r][2] = d.z; nx[m][r][3] = d.w;
    }
}
// Keys of step j of a dithered block, nx from key_dither.
__device__ __forceinline__ void dithered_keys(const uint8_t* bp, int j, int lane, const float (&nx)[2][2][4],
                                              float (&x)[2][2][4]) {
  const int g = lane >> 2;
  const uint4 w = *reinterpret_cast<const uint4*>(bp + Int8Layout::KC + j * 512 + lane * 16);
  const float sc[2] = {half_at(bp + Int8Layout::KS + (g * 4 + j) * 2), half_at(bp + Int8Layout::KS + ((g + 8) * 4 + j) * 2)};
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[m][r][e] = (code_i8(word_of(w, 2 * m + r), e) + nx[m][r][e]) * sc[r];
}

// The dither of step j's values, taken off, in the warp's scratch (dithered store): the same for every sequence.
__device__ __forceinline__ void value_dither(const StoreArgs& s, int h, int tb, int j, int lane, float* xs) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = 4 * k + (lane >> 3), quad = lane & 7;
    *reinterpret_cast<float4*>(xs + r * kXsPitch + quad * 4) = neg_dither4_24(s, h, tb + r, 8 * j + quad, 1);
  }
  __syncwarp();
}
// Values of step j of a dithered block, xs from value_dither.
__device__ __forceinline__ void dithered_values(const uint8_t* bp, int j, int lane, const float* xs, float (&x)[2][2][4]) {
  const int g = lane >> 2, t = lane & 3;
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
        const float nx = xs[(2 * t + (e & 1) + 8 * (e >> 1)) * kXsPitch + 16 * m + 8 * r + g];
        x[m][r][e] = (code_i8(c, e) + nx) * sc[e];
      }
    }
}

// Keys x of step j of the block whose first token is at tb, as output rows of sequence k of the launch.
template <bool BF16>
__device__ __forceinline__ void store_keys(const ReadArgs& a, int k, int h, int tb, int j, int lane, const float (&x)[2][2][4]) {
  using T = typename std::conditional<BF16, __nv_bfloat16, float>::type;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int tok = tb + g + 8 * r - a.t0[k];
      if (tok < 0 || tok >= a.n[k]) continue;
      T* o = static_cast<T*>(a.K) + ((a.row0[k] + tok) * a.s.Hkv + h) * kD + 32 * j + 16 * m + 4 * t;
      if constexpr (BF16)
        *reinterpret_cast<uint2*>(o) = make_uint2(bf2_bits(__floats2bfloat162_rn(x[m][r][0], x[m][r][1])),
                                                  bf2_bits(__floats2bfloat162_rn(x[m][r][2], x[m][r][3])));
      else
        *reinterpret_cast<float4*>(o) = make_float4(x[m][r][0], x[m][r][1], x[m][r][2], x[m][r][3]);
    }
}
template <bool BF16>
__device__ __forceinline__ void store_values(const ReadArgs& a, int k, int h, int tb, int j, int lane, const float (&x)[2][2][4]) {
  using T = typename std::conditional<BF16, __nv_bfloat16, float>::type;
  const int g = lane >> 2, t = lane & 3;
  // element offset of token r of the block; used only where keep(r)
  auto row = [&](int r) { return ((a.row0[k] + (tb + r - a.t0[k])) * a.s.Hkv + h) * kD; };
  auto keep = [&](int r) { return tb + r >= a.t0[k] && tb + r < a.t0[k] + a.n[k]; };
  T* V = static_cast<T*>(a.V);
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int c0 = 32 * j + 16 * m;
    if constexpr (BF16) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {                                  // tokens 0..7, 8..15 of the block
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

// Dithered blocks that stand at the same place of several sequences (beams of a prompt, a batch): a CTA takes a
// place and head, its warps a quarter of the channels each, forms the dither once and walks through the
// sequences of its part (the grid's second dimension), the next block's codes on their way.  Shared / formed by
// each, us, 8 heads, bf16: 16 sequences of 4099 tokens 79.9 / 137.5 (93.2 without the prefetch; 411 MB, 5.1 TB/s), 4 of
// 4096 28.7 / 41.0, 2 of 4096 16.5 / 22.6, 2 of 1000 8.3 / 8.5.
template <bool BF16>
__global__ void __launch_bounds__(kWarps * 32, 8) read_shared_kernel(const __grid_constant__ ReadArgs a, int blk0, int per) {
  __shared__ float scratch[kWarps][kXsFloats];
  const int j = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blk = blk0 + blockIdx.x / a.s.Hkv, h = blockIdx.x % a.s.Hkv, tb = blk * kBlk;
  float nx[2][2][4];
  key_dither(a.s, h, a.s.pos0 + tb, j, lane, nx);
  float* xs = scratch[j];
  value_dither(a.s, h, a.s.pos0 + tb, j, lane, xs);
  const int end = min(a.n_seq, (int)(blockIdx.y + 1) * per);
  // the next sequence of the part that has the place, and its block; the block's codes are on their way
  auto next = [&](int k, const uint8_t*& bp) {
    while (k < end && (tb + kBlk <= a.t0[k] || tb >= a.t0[k] + a.n[k])) ++k;
    if (k < end) {
      bp = a.s.blocks + block_index(a.s.table, a.s.Hkv, a.s.nblk_max, a.seq[k], h, blk) * block_bytes(kInt8);
      asm volatile("prefetch.global.L1 [%0];" ::"l"(bp + Int8Layout::KC + j * 512 + lane * 16));
      asm volatile("prefetch.global.L1 [%0];" ::"l"(bp + Int8Layout::VC + j * 512 + lane * 16));
      if (lane < 8) asm volatile("prefetch.global.L1 [%0];" ::"l"(bp + Int8Layout::KS + lane * 32));
    }
    return k;
  };
  const uint8_t* bp = nullptr;
#pragma unroll 1
  for (int k = next(blockIdx.y * per, bp); k < end;) {
    const uint8_t* bp_next = nullptr;
    const int k_next = next(k + 1, bp_next);
    bool ebf;
    const void* exact = exact_rows<kInt8>(a.s, a.seq[k], h, blk, a.len[k], ebf);
    float x[2][2][4];
    if (exact) exact_keys(a.s, exact, ebf, j, lane, x);
    else dithered_keys(bp, j, lane, nx, x);
    store_keys<BF16>(a, k, h, tb, j, lane, x);
    dithered_values(bp, j, lane, xs, x);
    store_values<BF16>(a, k, h, tb, j, lane, x);
    k = k_next;
    bp = bp_next;
  }
}

template <int SCH>
cudaError_t launch_s(const ReadArgs& a, cudaStream_t st) {
  const long long units = (long long)a.blk_off[a.n_seq] * a.s.Hkv;
  if constexpr (SCH == kInt8) {
    int from = INT_MAX, to = 0;
    for (int k = 0; k < a.n_seq; ++k) {
      from = std::min(from, a.t0[k] / kBlk);
      to = std::max(to, (a.t0[k] + a.n[k] - 1) / kBlk + 1);
    }
    const long long places = (long long)(to - from) * a.s.Hkv;
    const int parts = (int)std::min<long long>(a.n_seq, (kSharedCtas + places - 1) / places), per = (a.n_seq + parts - 1) / parts;
    if (per > 1 && units >= places * parts * kShare && places <= INT_MAX) {
      const dim3 grid((unsigned)places, (a.n_seq + per - 1) / per);
      if (a.s.is_bf16) read_shared_kernel<true><<<grid, kWarps * 32, 0, st>>>(a, from, per);
      else read_shared_kernel<false><<<grid, kWarps * 32, 0, st>>>(a, from, per);
      return cudaGetLastError();
    }
  }
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
