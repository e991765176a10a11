// Sequences that take each other's state, and pages that get a holder of their own.
//
// A map i <- parent(i) over the sequences of a cache, in place.  The host turns it into a list of moves
// in which no move reads what an earlier one has written (fork_moves in runtime.cu): sequences that
// nobody reads any more come first, and a cycle saves its first row in a register (`kept`) and hands
// it out last.  So each thread takes one 32-byte column of every row, layer and head alike, and runs down the
// whole list alone: no scratch memory, no barrier between threads, loads of kBatch moves in flight, and a
// source that several sequences take in a row is loaded once.
//
// Bound by HBM: every source block read once, every moved one written once.  Two prompts of 4099 tokens each to
// seven other beams (dithered INT8, 8 heads, 2 layers: 319 MB) 50 us, 6.4 TB/s; 8 beams of 8192 tokens that
// change places (black box, 8 heads, 2 layers: 1.14 GB) 176 us, 6.5 TB/s: 0.94 and 0.95 of the measured copy.
#include "common.cuh"
#include "kernels.h"

namespace witcert {

namespace {

constexpr int kRowThreads = 256;
// Below this many blocks the groups of moves run side by side, us, side by side / one after another: 64 sequences
// of 8 beams, 4 layers, two-bit, rotated: 100 tokens x 4 heads (32 blocks) 15.7 / 30.8 (the host 15), 300 x 8 (192) 26.7 /
// 47.0, FP8 (352) 59.5 / 72.7; above it 1000 x 8, two-bit (576) 110 / 101, FP8 (1152) 205 / 193.
constexpr int kManyBlocks = 456;
constexpr int kBatch = 4;                        // moves whose loads are in flight: 4 x 32 bytes a thread

struct alignas(32) Vec { uint32_t w[8]; };
__device__ __forceinline__ Vec load32(const uint8_t* p) {
  Vec v;
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
               : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store32(uint8_t* p, const Vec& v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]),
               "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7]) : "memory");
}

// GROUPS: the grid's second dimension counts heads and groups of moves; else the heads, and a thread runs down all.
// Four blocks an SM (64 registers) against three at 70: 8 beams' rotation of 4096 tokens 96.6 against 111 us.
template <bool GROUPS>
__global__ void __launch_bounds__(kRowThreads, 4) move_rows_kernel(const __grid_constant__ MoveRows a) {
  int k = 0;
  while (k + 1 < a.n_streams && blockIdx.x >= a.s[k + 1].block0) ++k;
  const MoveStream& s = a.s[k];
  const long long at = ((long long)(blockIdx.x - s.block0) * kRowThreads + threadIdx.x) * 32;
  const int head = GROUPS ? blockIdx.y / a.group.n : blockIdx.y, group = GROUPS ? blockIdx.y % a.group.n : 0;
  const int end = GROUPS ? a.group.first[group + 1] : a.n;
  uint8_t* col = s.base + blockIdx.z * s.layer_pitch + head * s.head_pitch + at;
  Vec kept;
#pragma unroll
  for (int e = 0; e < 8; ++e) kept.w[e] = 0u;
  for (int m = GROUPS ? a.group.first[group] : 0; m < end; m += kBatch) {
    Vec v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (m + u >= end) break;
      const MoveOp& op = a.op[m + u];
      const bool again = u > 0 && op.src >= 0 && op.src == a.op[m + u - 1].src;
      if (again) v[u] = v[u > 0 ? u - 1 : 0];
      else if (op.src >= 0 && at < (long long)op.load[s.count] * s.unit) v[u] = load32(col + op.src * s.seq_pitch);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (m + u >= end) break;
      const MoveOp& op = a.op[m + u];
      if (op.dst == kMoveKept) kept = v[u];
      else if (at < (long long)op.n[s.count] * s.unit) store32(col + op.dst * s.seq_pitch, op.src == kMoveKept ? kept : v[u]);
    }
  }
}

// Page table rows and device lengths under the same list of moves: column c is block c of the table,
// then layer c - nblk_max of the lengths.  Entries past a sequence's blocks become -1.
__global__ void __launch_bounds__(128) move_ints_kernel(const __grid_constant__ MoveInts a) {
  const int c = blockIdx.x * 128 + threadIdx.x;
  const bool table = c < a.nblk_max;
  if (c >= a.nblk_max + a.layers) return;
  int32_t* base = table ? a.table + c : a.lens + (size_t)(c - a.nblk_max) * a.B;
  if (table ? !a.table : !a.lens) return;
  const size_t pitch = table ? a.nblk_max : 1;
  int32_t kept = table ? -1 : 0;
  constexpr int kTogether = 8;                                 // loads in flight; no move reads what an earlier one wrote
  const int end = a.group.first[blockIdx.y + 1];
  for (int m = a.group.first[blockIdx.y]; m < end; m += kTogether) {
    int32_t v[kTogether];
#pragma unroll
    for (int u = 0; u < kTogether; ++u)
      if (m + u < end && a.op[m + u].src >= 0) v[u] = base[a.op[m + u].src * pitch];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      if (m + u >= end) break;
      const MoveOp& op = a.op[m + u];
      const int32_t x = op.src >= 0 ? v[u] : op.src == kMoveKept ? kept : table ? -1 : 0;
      if (op.dst == kMoveKept) kept = x;
      else base[op.dst * pitch] = table ? (c < op.blocks ? x : -1) : min(x, op.cap);
    }
  }
}

// Pages that get copies of their own: page src[y] of every layer to page dst[y], and the table's entry.
__global__ void __launch_bounds__(kRowThreads) copy_pages_kernel(const __grid_constant__ CopyPages a) {
  const long long at = ((long long)blockIdx.x * kRowThreads + threadIdx.x) * 32;
  const int k = blockIdx.y;
  uint8_t* layer = a.blocks + blockIdx.z * a.layer_pitch;
  if (at < a.page_bytes && a.src[k] >= 0) store32(layer + a.dst[k] * a.page_bytes + at, load32(layer + a.src[k] * a.page_bytes + at));
  if (at == 0 && blockIdx.z == 0) a.table[a.idx[k]] = a.dst[k];
}

}  // namespace

cudaError_t launch_move_rows(MoveRows& a, int layers, int heads, cudaStream_t st) {
  unsigned blocks = 0;
  for (int k = 0; k < a.n_streams; ++k) {
    a.s[k].block0 = blocks;
    int most = 0;
    for (int m = 0; m < a.n; ++m) most = a.op[m].n[a.s[k].count] > most ? a.op[m].n[a.s[k].count] : most;
    blocks += (unsigned)(((long long)most * a.s[k].unit / 32 + kRowThreads - 1) / kRowThreads);
  }
  if (blocks == 0) return cudaSuccess;
  if ((long long)blocks * heads * layers < kManyBlocks && (long long)heads * a.group.n <= 65535)
    move_rows_kernel<true><<<dim3(blocks, heads * a.group.n, layers), kRowThreads, 0, st>>>(a);
  else
    move_rows_kernel<false><<<dim3(blocks, heads, layers), kRowThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_move_ints(const MoveInts& a, cudaStream_t st) {
  if (a.n == 0) return cudaSuccess;
  move_ints_kernel<<<dim3((a.nblk_max + a.layers + 127) / 128, a.group.n), 128, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_copy_pages(const CopyPages& a, int layers, cudaStream_t st) {
  if (a.n == 0) return cudaSuccess;
  const unsigned x = (unsigned)((a.page_bytes / 32 + kRowThreads - 1) / kRowThreads);
  copy_pages_kernel<<<dim3(x, a.n, layers), kRowThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace witcert
