// Beam search: the best continuations of each request, and the token sequences of its beams.
//
// Selection.  A live row (request, beam) of logits x and score c offers s_v = c + x_v - lse, lse = log sum
// exp x.  Two launches:
//
//   scan   one pass over the logits: for every chunk of kChunk tokens its maximum, for every warp's run of
//          chunks the maximum m and sum exp(x - m).  Bound by HBM; five lane operations an element.
//   pick   one CTA a request.  The n best candidates lie in the n chunks with the best maxima (ordered as
//          candidates are: a candidate in any other chunk is beaten by n chunk maxima), so it ranks the
//          chunks' maxima, reads those n chunks again and ranks their elements.  Bound by latency.
//
// Ranking goes by a key in 64 bits, (s, lower row, lower token).  Most of the work is a filter in 32 bits:
// a lower bound of the n-th best key comes from the threads' own maxima, every key that its rounding
// does not put below that bound is listed, and only the list is formed in 64 bits and ranked by counting.
#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace witcert {

namespace {

constexpr int kChunk = kBeamChunk;
constexpr int kLane = kChunk / 32;               // elements of a chunk a lane holds: 16
constexpr int kScanWarps = 8;
constexpr int kPickThreads = 1024;
constexpr int kList = 1024;                      // candidates that are ranked exactly
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float redux_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Row {
  const T* x;
  int lead;                  // elements between the 32-byte boundary before the row and the row
  int vocab;
  __device__ Row(const BeamArgs& a, int r, int w) {
    x = static_cast<const T*>(a.logits) + r * a.request_stride + w * a.beam_stride;
    lead = (int)((reinterpret_cast<uintptr_t>(x) & 31) / sizeof(T));
    vocab = a.vocab;
  }
  // First token of lane `lane`'s part of chunk c (may lie outside the row at either end).
  __device__ int first(int c, int lane) const { return c * kChunk + lane * kLane - lead; }
  // The lane's sixteen elements; -inf outside the row.
  __device__ void load(int c, int lane, float (&v)[kLane]) const {
    const int e0 = first(c, lane);
    if (e0 >= 0 && e0 <= vocab - kLane) {
      if constexpr (sizeof(T) == 2) {
        uint32_t w[8];
        load8(x + e0, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[2 * k] = __uint_as_float(w[k] << 16);
          v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[8];
          load8(x + e0 + 8 * h, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[8 * h + k] = __uint_as_float(w[k]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < kLane; ++k) {
        const int e = e0 + k;
        v[k] = e >= 0 && e < vocab ? to_f32(x[e]) : -INFINITY;
      }
    }
  }
  static __device__ __forceinline__ void load8(const T* p, uint32_t (&w)[8]) {
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p));
  }
};

// A row takes part while its score is finite; a finished one offers only itself.
__device__ __forceinline__ bool live(float score) { return fabsf(score) <= FLT_MAX; }

template <typename T>
__global__ void __launch_bounds__(kScanWarps * 32) beam_scan_kernel(const __grid_constant__ BeamArgs a) {
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long wid = (long long)blockIdx.x * kScanWarps + (threadIdx.x >> 5);
  const long long row = wid / a.parts;
  if (row >= (long long)a.requests * a.beams) return;
  const int part = (int)(wid - row * a.parts), r = (int)(row / a.beams), w = (int)(row % a.beams);
  if (!live(a.scores[row]) || (a.finished && a.finished[row])) return;
  const Row<T> x(a, r, w);
  float* maxima = a.maxima + row * a.chunks;
  float m = -INFINITY, sum = 0.f, lost = 0.f;                  // of this lane: sum + lost = sum exp(x - m)
  const int c1 = min(a.chunks, (part + 1) * a.chunks_per_part);
  for (int c = part * a.chunks_per_part; c < c1; ++c) {
    float v[kLane];
    x.load(c, lane, v);
    float top = v[0];
#pragma unroll
    for (int k = 1; k < kLane; ++k) top = fmaxf(top, v[k]);
    const float most = redux_max(top);
    if (lane == 0) maxima[c] = most;
    if (top > m) {
      const float f = ex2((m - top) * kLog2e);                 // 0 for the first
      sum *= f; lost *= f;
      m = top;
    }
    // exponents relative to the lane's maximum: differences of logits, which lose nothing next to it; a
    // lane that has seen only -inf adds zeros, and +inf or NaN anywhere makes the row's sum NaN
    const float ref = m == -INFINITY ? 0.f : m;
    float e[kLane];
#pragma unroll
    for (int k = 0; k < kLane; ++k) e[k] = ex2((v[k] - ref) * kLog2e);
#pragma unroll
    for (int h = kLane / 2; h > 0; h /= 2)
#pragma unroll
      for (int k = 0; k < h; ++k) e[k] += e[k + h];
    const float s = sum + e[0], back = s - sum;                // two-sum: the running sum keeps its rounding
    lost += (sum - (s - back)) + (e[0] - back);
    sum = s;
  }
  const float top = redux_max(m), ref = top == -INFINITY ? 0.f : top;
  sum = (sum + lost) * (m == -INFINITY ? (sum == 0.f ? 0.f : NAN) : ex2((m - ref) * kLog2e));
#pragma unroll
  for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) a.records[wid] = make_float2(top, sum);
}

// ------------------------------------------------------------------ pick
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long ordered(double x) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(x + 0.0);   // one zero
  return b >> 63 ? ~b : b | 1ull << 63;
}

struct Key {                 // larger s first, then lower place (row << 32 | token, or chunk)
  unsigned long long s, place;
};
__device__ __forceinline__ bool before(const Key& x, const Key& y) { return x.s != y.s ? x.s > y.s : x.place < y.place; }

struct PickShared {
  Key key[kList];
  uint32_t id[kList];
  uint32_t best[kBeamMaxOut];          // chosen ids, in order
  Key best_key[kBeamMaxOut];
  double lse[kBeamMaxBeams];
  float score[kBeamMaxBeams];
  uint8_t state[kBeamMaxBeams];        // 0 no candidates, 1 live, 2 finished
  int count, got;
  uint32_t top;
  float size;                          // bound of |score| + |lse| over the rows
};

// The n first of the keys that Keys::each(visit) gives this thread as visit(s, id), s within Keys' rounding
// of the key's score; Keys::exact(id) is the key.  They end up in sh.best in order; returns how many there
// are.  Called by the whole CTA.
template <class Keys>
__device__ int pick_best(PickShared& sh, const Keys& keys, int n) {
  const int tid = threadIdx.x, lane = tid & 31;
  float mine = -INFINITY;
  keys.each([&](float s, uint32_t) { mine = fmaxf(mine, s); });
  const uint32_t my = mine == -INFINITY ? 0u : ordered(mine);
  if (tid == 0) { sh.count = 0; sh.top = 0u; }
  __syncthreads();
  const uint32_t wtop = __reduce_max_sync(0xffffffffu, my);
  if (lane == 0 && wtop) atomicMax(&sh.top, wtop);
  // the largest bound that n threads' maxima reach (all keys, if fewer threads have one), by halving
  uint32_t lo = 1u;
  if (__syncthreads_count(my != 0u) > n) {
    uint32_t hi = sh.top;                                      // count(>= lo) >= n, sought in [lo, hi]
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      const int c = __syncthreads_count(my >= mid);
      if (c >= n) lo = mid; else hi = mid - 1;
      if (c == n) break;
    }
  }
  // keys within twice the rounding of the bound may still be first
  const float bound = lo == 1u ? -INFINITY : __uint_as_float(lo & 0x80000000u ? lo & 0x7FFFFFFFu : ~lo);
  const float off = 0x1p-20f * (fabsf(bound) + 2.f * sh.size);
  const float from = bound - off > -INFINITY ? bound - off : -FLT_MAX;     // also where that is no number
  keys.each([&](float s, uint32_t id) {
    if (s >= from) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kList) sh.id[at] = id;
    }
  });
  __syncthreads();
  int listed = sh.count;
  if (listed > kList) {
    // Very many equal or nearly equal keys: halve the space of the keys themselves, which are distinct.
    unsigned __int128 low = 0, high = ~(unsigned __int128)0;   // count(>= low) > kList, count(> high) < n
    for (;;) {
      const unsigned __int128 mid = low + (high - low) / 2 + 1;
      __syncthreads();
      if (tid == 0) sh.count = 0;
      __syncthreads();
      int c = 0;
      keys.each([&](float s, uint32_t id) {
        if (s < from) return;
        const Key k = keys.exact(id);
        c += ((unsigned __int128)k.s << 64 | ~k.place) >= mid;
      });
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0 && c) atomicAdd(&sh.count, c);
      __syncthreads();
      c = sh.count;
      if (c < n) high = mid - 1; else low = mid;
      if (c >= n && c <= kList) break;
    }
    __syncthreads();
    if (tid == 0) sh.count = 0;
    __syncthreads();
    keys.each([&](float s, uint32_t id) {
      if (s < from) return;
      const Key k = keys.exact(id);
      if (((unsigned __int128)k.s << 64 | ~k.place) >= low) sh.id[atomicAdd(&sh.count, 1)] = id;
    });
    __syncthreads();
    listed = sh.count;
  }
  for (int i = tid; i < listed; i += kPickThreads) sh.key[i] = keys.exact(sh.id[i]);
  __syncthreads();
  // a key's rank is the number of keys before it: a warp counts for one key at a time
  for (int i = tid >> 5; i < listed; i += kPickThreads / 32) {
    const Key k = sh.key[i];
    int rank = 0;
    for (int j = lane; j < listed; j += 32) rank += before(sh.key[j], k);
    rank = __reduce_add_sync(0xffffffffu, rank);
    if (lane == 0 && rank < n) {
      sh.best[rank] = sh.id[i];
      sh.best_key[rank] = k;
    }
  }
  __syncthreads();
  return min(listed, n);
}

// Chunk maxima of a request: id = beam * chunks + chunk.
struct ChunkKeys {
  const BeamArgs& a;
  const PickShared& sh;
  const float* maxima;
  __device__ float value(int w, int c) const { return sh.state[w] == 2 ? (c == 0 ? 0.f : -INFINITY) : maxima[(size_t)w * a.chunks + c]; }
  template <class V> __device__ void each(V&& visit) const {
    for (int w = 0; w < a.beams; ++w) {
      if (sh.state[w] == 0) continue;
      const float score = sh.score[w], lse = (float)sh.lse[w];
      const int end = sh.state[w] == 2 ? 1 : a.chunks;
      // rows start at different threads, so that the threads' shares are alike
      for (int c = (threadIdx.x + w * 416) % kPickThreads; c < end; c += kPickThreads) {
        const float x = value(w, c);
        if (x > -INFINITY) visit(fmaxf(score + (x - lse), -FLT_MAX), (uint32_t)w * a.chunks + c);
      }
    }
  }
  __device__ Key exact(uint32_t id) const {
    const int w = id / a.chunks, c = id % a.chunks;
    return {ordered((double)sh.score[w] + ((double)value(w, c) - sh.lse[w])), id};
  }
};

// Elements of the chosen chunks: id = place among the chosen * kChunk + element.
template <typename T>
struct TokenKeys {
  const BeamArgs& a;
  const PickShared& sh;
  const uint32_t* chunk;               // the chosen chunks' ids
  int n, r;
  template <class V> __device__ void each(V&& visit) const {
    const int lane = threadIdx.x & 31;
    for (int k = threadIdx.x >> 5; k < n; k += kPickThreads / 32) {
      const int w = chunk[k] / a.chunks, c = chunk[k] % a.chunks;
      const float score = sh.score[w], lse = (float)sh.lse[w];
      if (sh.state[w] == 2) {
        if (lane == 0) visit(score, (uint32_t)k * kChunk);
        continue;
      }
      float v[kLane];
      Row<T>(a, r, w).load(c, lane, v);
#pragma unroll
      for (int e = 0; e < kLane; ++e)
        if (v[e] > -INFINITY) visit(fmaxf(score + (v[e] - lse), -FLT_MAX), (uint32_t)k * kChunk + lane * kLane + e);
    }
  }
  __device__ Key exact(uint32_t id) const {
    const int k = id / kChunk, w = chunk[k] / a.chunks, c = chunk[k] % a.chunks;
    if (sh.state[w] == 2) return {ordered((double)sh.score[w]), (unsigned long long)w << 32 | (uint32_t)a.eos};
    const Row<T> x(a, r, w);
    const int token = x.first(c, 0) + (int)(id % kChunk);
    return {ordered((double)sh.score[w] + ((double)to_f32(x.x[token]) - sh.lse[w])), (unsigned long long)w << 32 | (uint32_t)token};
  }
};

template <typename T>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const __grid_constant__ BeamArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  PickShared& sh = *reinterpret_cast<PickShared*>(smem);
  uint32_t* chunk = reinterpret_cast<uint32_t*>(smem + sizeof(PickShared));
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) sh.size = 0.f;
  __syncthreads();
  pdl_wait();
  // the rows' sums: a warp a row
  for (int w = tid >> 5; w < a.beams; w += kPickThreads / 32) {
    const long long row = (long long)r * a.beams + w;
    const float score = a.scores[row];
    int state = !live(score) ? 0 : a.finished && a.finished[row] ? 2 : 1;
    double lse = 0.0;
    if (state == 1) {
      const float2* rec = a.records + row * a.parts;
      float top = -INFINITY;
      for (int p = lane; p < a.parts; p += 32) top = fmaxf(top, rec[p].x);
      top = redux_max(top);
      double sum = 0.0;
      for (int p = lane; p < a.parts; p += 32)
        sum += (double)(rec[p].x > -INFINITY ? rec[p].y * ex2((rec[p].x - top) * kLog2e) : rec[p].y);
#pragma unroll
      for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      // no softmax: nothing but -inf, or +inf or NaN among the logits
      if (!(sum > 0.0) || !(fabsf(top) <= FLT_MAX)) state = 0;
      else lse = (double)top + log(sum);
    }
    if (lane == 0) {
      sh.score[w] = score;
      sh.lse[w] = lse;
      sh.state[w] = (uint8_t)state;
      // non-negative floats order like their bits
      if (state) atomicMax(reinterpret_cast<int*>(&sh.size), __float_as_int(fminf(fabsf(score) + (float)fabs(lse), FLT_MAX)));
    }
  }
  __syncthreads();
  const int n_chunks = pick_best(sh, ChunkKeys{a, sh, a.maxima + (size_t)r * a.beams * a.chunks}, a.n_out);
  if (tid < n_chunks) chunk[tid] = sh.best[tid];
  __syncthreads();
  const TokenKeys<T> tokens{a, sh, chunk, n_chunks, r};
  const int n = pick_best(sh, tokens, a.n_out);
  if (tid >= a.n_out) return;
  const long long at = (long long)r * a.n_out + tid;
  float score = -INFINITY;
  int row = -1, token = -1;
  bool ended = false;
  if (tid < n) {
    const Key k = sh.best_key[tid];
    const int w = (int)(k.place >> 32);
    token = (int)(uint32_t)k.place;
    row = r * a.beams + w;
    score = (float)__longlong_as_double((long long)(k.s >> 63 ? k.s & ~(1ull << 63) : ~k.s));
    ended = sh.state[w] == 2 || token == a.eos;
  }
  a.out_scores[at] = score;
  a.rows[at] = row;
  a.tokens[at] = token;
  if (a.out_finished) a.out_finished[at] = ended;
}

// ------------------------------------------------------------------ paths
// The beam that step t's choice for the last beam w came from is a chain of maps, which are put together in
// any grouping: a CTA a request takes a tile of steps from the end, each warp forms the map of its share of
// the tile (a walk for every beam), takes over the maps after its own, and walks its share again, writing
// for each step which entry the last beams chose.  The tile's entries and tokens lie in shared memory, so
// that a step of a walk is one shared-memory load, and the sequences go out along time.
constexpr int kPathThreads = 1024, kPathWarps = kPathThreads / 32;
constexpr int kPathPerLane = (kBeamMaxBeams + 31) / 32;
constexpr int kPathShared = 160 * 1024;

__global__ void __launch_bounds__(kPathThreads) beam_paths_kernel(const __grid_constant__ PathArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint8_t map[kPathWarps][kBeamMaxBeams + 1];
  __shared__ uint8_t carry[kBeamMaxBeams];
  const int W = a.beams, r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* tok = reinterpret_cast<int32_t*>(smem);             // [tile][W]
  uint8_t* rel = smem + (size_t)a.tile * W * 4;                // [tile][W]: the parent beam, W for none
  int n = a.steps;
  if (a.n_steps) n = min(max(a.n_steps[r], 0), a.steps);
  const size_t step = (size_t)a.requests * W;
  int32_t* out = a.out + (size_t)r * W * a.steps;
  for (int w = 0; w < W; ++w)
    for (int t = n + tid; t < a.steps; t += kPathThreads) out[(size_t)w * a.steps + t] = a.pad;
  if (tid < W) carry[tid] = (uint8_t)tid;
  for (int t1 = n; t1 > 0; t1 -= a.tile) {
    const int t0 = max(0, t1 - a.tile), len = t1 - t0;
    __syncthreads();
    for (int i = tid; i < len * W; i += kPathThreads) {
      const size_t at = (t0 + i / W) * step + (size_t)r * W + i % W;
      const long long p = (long long)a.rows[at] - (long long)r * W;
      rel[i] = p >= 0 && p < W ? (uint8_t)p : (uint8_t)W;
      tok[i] = a.tokens[at];
    }
    __syncthreads();
    const int share = (len + kPathWarps - 1) / kPathWarps, b = min(len, warp * share), e = min(len, b + share);
    int at[kPathPerLane];
#pragma unroll
    for (int k = 0; k < kPathPerLane; ++k) at[k] = min(lane + 32 * k, W);
    for (int t = e - 1; t >= b; --t)
#pragma unroll
      for (int k = 0; k < kPathPerLane; ++k)
        if (at[k] < W) at[k] = rel[t * W + at[k]];
#pragma unroll
    for (int k = 0; k < kPathPerLane; ++k)
      if (lane + 32 * k < W) map[warp][lane + 32 * k] = (uint8_t)at[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPathPerLane; ++k) at[k] = lane + 32 * k < W ? carry[lane + 32 * k] : W;
    for (int j = kPathWarps - 1; j > warp; --j)
#pragma unroll
      for (int k = 0; k < kPathPerLane; ++k)
        if (at[k] < W) at[k] = map[j][at[k]];
    for (int t = e - 1; t >= b; --t) {
      int to[kPathPerLane];
#pragma unroll
      for (int k = 0; k < kPathPerLane; ++k) to[k] = at[k] < W ? rel[t * W + at[k]] : W;
      __syncwarp();                                            // the step's parents are read: its choices replace them
#pragma unroll
      for (int k = 0; k < kPathPerLane; ++k) {
        if (lane + 32 * k < W) rel[t * W + lane + 32 * k] = (uint8_t)(to[k] < W ? at[k] : W);
        at[k] = to[k];
      }
      __syncwarp();
    }
    __syncthreads();                                           // every warp has read the carry
    if (warp == 0)
#pragma unroll
      for (int k = 0; k < kPathPerLane; ++k)
        if (lane + 32 * k < W) carry[lane + 32 * k] = (uint8_t)at[k];
    for (int w = 0; w < W; ++w)
      for (int t = tid; t < len; t += kPathThreads) {
        const int c = rel[t * W + w];
        out[(size_t)w * a.steps + t0 + t] = c < W ? tok[t * W + c] : a.pad;
      }
  }
}

template <typename T>
cudaError_t select_t(const BeamArgs& a, cudaStream_t st) {
  const long long warps = (long long)a.requests * a.beams * a.parts;
  beam_scan_kernel<T><<<(unsigned)((warps + kScanWarps - 1) / kScanWarps), kScanWarps * 32, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.requests);
  cfg.blockDim = dim3(kPickThreads);
  cfg.dynamicSmemBytes = sizeof(PickShared) + kBeamMaxOut * sizeof(uint32_t);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_pick_kernel<T>, a);
}

}  // namespace

cudaError_t launch_beam_select(const BeamArgs& a, cudaStream_t st) {
  return a.is_bf16 ? select_t<__nv_bfloat16>(a, st) : select_t<float>(a, st);
}

cudaError_t launch_beam_paths(PathArgs& a, cudaStream_t st) {
  a.tile = kPathShared / (a.beams * 5);
  if (a.tile > a.steps) a.tile = a.steps;
  const int bytes = a.tile * a.beams * 5;
  if (bytes > 47 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(beam_paths_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPathShared);
    if (e != cudaSuccess) return e;
  }
  beam_paths_kernel<<<a.requests, kPathThreads, bytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace witcert
