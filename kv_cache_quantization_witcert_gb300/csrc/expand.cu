// Operand images of a compressed cache in device memory (layout in expand.cuh), for row tiles that
// share them: the attention kernel then fetches a tile by one bulk copy.
//
// A CTA per (128-token tile, KV head), a warp per two blocks and half of the channels.  Bound by HBM
// (codes in, 64 KB a tile and head out) and, for the dithered store, by the integer work of its
// dither.
#include "attend.cuh"
#include "expand.cuh"

namespace witcert {

namespace {

template <int SCH>
__global__ void __launch_bounds__(256, SCH == kInt8 ? 4 : 3) expand_kernel(const __grid_constant__ AttendArgs a) {
  __shared__ __align__(16) uint32_t scratch[SCH == kInt8 ? 8 : 1][SCH == kInt8 ? kXwWords : 1];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  const int tile_all = blockIdx.x / a.s.Hkv;
  int k = 0;
  while (a.tile_off[k + 1] <= tile_all) ++k;
  const int i = a.seq[k];
  BlockPair x;
  x.h = blockIdx.x % a.s.Hkv;
  x.pr = warp >> 1; x.lane = threadIdx.x & 31;
  x.tb = (tile_all - a.tile_off[k]) * kTileTok + x.pr * 2 * kBlk;
  x.len = a.len[k];
  uint8_t* img = a.images + ((size_t)tile_all * a.s.Hkv + x.h) * 2 * kTileBytes;
  // past the sequence the tile's first block stands in (its codes are dropped)
  const int first = (tile_all - a.tile_off[k]) * (kTileTok / kBlk);
#pragma unroll
  for (int b = 0; b < 2; ++b)
    x.bp[b] = a.s.blocks + block_index(a.s.table, a.s.Hkv, a.s.nblk_max, i, x.h,
                                       x.tb + b * kBlk < x.len ? x.tb / kBlk + b : first) * block_bytes(SCH);
  find_exact<SCH>(a.s, i, x);
  expand_keys<SCH>(a.s, x, 2 * (warp & 1), img, [] {}, [] { return true; });
  expand_values<SCH>(a.s, x, 2 * (warp & 1), scratch[SCH == kInt8 ? warp : 0], img + kTileBytes, [] {}, [] { return true; });
}

// The dither of a tile and head in the order the expanding lanes fetch it; a quarter of it a CTA (keys
// or values, one step of a warp's two), as there are few tiles: 128 tiles and heads 6.2 us by whole ones.
__global__ void __launch_bounds__(256) dither_kernel(const __grid_constant__ StoreArgs s, uint4* table) {
  __shared__ __align__(16) uint32_t scratch[8][kXwWords];
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x % s.Hkv, tile = blockIdx.x / s.Hkv, pr = warp >> 1, j0 = 2 * (warp & 1);
#pragma unroll 1
  for (int b = 0; b < 2; ++b) {
    const int values = blockIdx.y >> 1, j = j0 + (blockIdx.y & 1), tb = s.pos0 + tile * kTileTok + (2 * pr + b) * kBlk;
    uint32_t n[2][2][2];
    if (values) value_dither(s, h, tb, j, lane, scratch[warp], n);
    else key_dither(s, h, tb, j, lane, n);
    uint4* to = table + dither_at(s.Hkv, tile, h, values, pr, j, b, lane);
    to[0] = make_uint4(n[0][0][0], n[0][0][1], n[0][1][0], n[0][1][1]);
    to[32] = make_uint4(n[1][0][0], n[1][0][1], n[1][1][0], n[1][1][1]);
  }
}

}  // namespace

cudaError_t launch_dither_table(const StoreArgs& s, uint4* table, int tiles, cudaStream_t st) {
  dither_kernel<<<dim3((unsigned)(tiles * s.Hkv), 4), 256, 0, st>>>(s, table);
  return cudaGetLastError();
}

cudaError_t launch_expand(int scheme, const AttendArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)(a.tile_off[a.n_seq] * a.s.Hkv);
  if (grid == 0) return cudaSuccess;
  switch (scheme) {
    case kInt8: return launch_after(expand_kernel<kInt8>, dim3(grid), 256, 0, st, a);
    case kRtn: return launch_after(expand_kernel<kRtn>, dim3(grid), 256, 0, st, a);
    case kFp8: return launch_after(expand_kernel<kFp8>, dim3(grid), 256, 0, st, a);
    case kKivi: return launch_after(expand_kernel<kKivi>, dim3(grid), 256, 0, st, a);
    default: return launch_after(expand_kernel<kBbox>, dim3(grid), 256, 0, st, a);
  }
}

}  // namespace witcert
