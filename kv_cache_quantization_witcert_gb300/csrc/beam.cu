// Beam search: the best continuations of each request, and the token sequences of its beams.
//
// Selection.  A live row (request, beam) of logits x and score c offers s_v = c + x_v - log sum exp x, formed
// as (c - log sum exp(x - m)) + (x_v - m) with the row's maximum m.  Two steps, a launch each, or for few small
// requests one launch of clusters:
//
//   scan   one pass over the logits: for every chunk of kChunk tokens its maximum, for every warp's chunks the
//          maximum m and sum exp(x - m).  Bound by HBM and, at both ends of the launch, by latency: 64 x 8 rows of
//          131072 bf16 tokens, 462 of them live (121 MB), 26.2 us in a loop of launches, 4.6 TB/s (a bare read 20.5).
//   pick   one CTA a request.  The n best candidates lie in the n chunks with the best maxima (ordered as
//          candidates are: a candidate in any other chunk is beaten by n chunk maxima), so it ranks the
//          chunks' maxima, reads those n chunks again and ranks their elements.  Bound by the latency of
//          its phases: about 5 us for 4 beams and 8 out, 6 for 8 and 16, 13 for 32 and 64.
//
// Ranking goes by (s in 64 bits, lower row, larger logit, lower token).  A row's log sum has fp32 terms and is off by
// up to 2^-18 + 2^-23 (log V + 1), the same for all its candidates: their order is exact, that of different rows as
// far as twice that tells them apart.  Most of the work is a filter in 32 bits: a lower bound of the n-th best key
// comes from the largest keys of groups of threads, every key that its rounding does not put below that bound is
// listed, and only the list is formed in 64 bits (whose rate is a 64th of fp32's) and ranked by counting.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace witcert {

namespace {

constexpr int kChunk = kBeamChunk;
constexpr int kLane = kChunk / 32;               // elements of a chunk a lane holds: 16
constexpr int kScanWarps = 4;
constexpr int kPickThreads = 1024;
constexpr int kList = 4096;                      // candidates that are ranked exactly, a power of two
constexpr int kCounted = 256;                    // lists up to this are ranked by counting, longer ones sorted
constexpr int kMaxGroups = 512;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float redux_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
template <typename T>
struct Row {
  static constexpr int kWords = kLane * sizeof(T) / 4;         // registers a lane's part of a chunk takes
  const T* x;
  int lead;                  // elements between the 32-byte boundary before the row and the row
  int vocab;
  __device__ Row(const BeamArgs& a, int r, int w) {
    x = static_cast<const T*>(a.logits) + r * a.request_stride + w * a.beam_stride;
    lead = (int)((reinterpret_cast<uintptr_t>(x) & 31) / sizeof(T));
    vocab = a.vocab;
  }
  // Token of element e of chunk c (may lie outside the row at either end).
  __device__ int token(int c, int e) const { return c * kChunk + e - lead; }
  // N words of elements from token t on, as they lie (t's place is aligned to them); -inf outside the row.
  template <int N>
  static __device__ __forceinline__ void load_at(const T* x, int vocab, int t, uint32_t (&w)[N]) {
    constexpr int n = N * 4 / sizeof(T);
    if (t >= 0 && t <= vocab - n) {
      if constexpr (N == 2)
        asm("ld.global.nc.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(x + t));
      else if constexpr (N == 4)
        asm("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(x + t));
      else
#pragma unroll
        for (int h = 0; h < N; h += 8)
          asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
              : "=r"(w[h]), "=r"(w[h + 1]), "=r"(w[h + 2]), "=r"(w[h + 3]), "=r"(w[h + 4]), "=r"(w[h + 5]), "=r"(w[h + 6]), "=r"(w[h + 7])
              : "l"(x + t + h * 4 / sizeof(T)));
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if constexpr (sizeof(T) == 2) w[k] = bits(x, vocab, t + 2 * k) | bits(x, vocab, t + 2 * k + 1) << 16;
        else w[k] = bits(x, vocab, t + k);
      }
    }
  }
  static __device__ __forceinline__ uint32_t bits(const T* x, int vocab, int t) {
    const bool in = t >= 0 && t < vocab;
    if constexpr (sizeof(T) == 2) return in ? reinterpret_cast<const uint16_t*>(x)[t] : 0xFF80u;
    else return in ? reinterpret_cast<const uint32_t*>(x)[t] : 0xFF800000u;
  }
  // Element k of loaded words.
  template <int N>
  static __device__ __forceinline__ float value(const uint32_t (&w)[N], int k) {
    if constexpr (sizeof(T) == 2) return __uint_as_float(k & 1 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
    else return __uint_as_float(w[k]);
  }
};

// A row takes part while its score is finite; a finished one offers only itself.
__device__ __forceinline__ bool live(float score) { return fabsf(score) <= FLT_MAX; }

// s + x as a rounded sum and what the rounding dropped.
__device__ __forceinline__ void two_sum(float& s, float& lost, float x) {
  const float t = s + x, back = t - s;
  lost += (s - (t - back)) + (x - back);
  s = t;
}

// A warp's chunks on their way: each lane copies its own pieces of a chunk to shared memory and reads them back
// itself, so that a wait for the lane's own copies is all there is to wait for.
// 48 warps of 4 KB, loops of launches, us: 26.2 by 28 parts a row, 26.5 by 9; 32 warps of 6 KB 26.6, 30.0.
constexpr int kRing = 4 * 1024;                  // bytes of a warp's chunks in shared memory
template <typename T>
struct Ring {
  static constexpr int kBytes = kChunk * sizeof(T), kPieces = kBytes / 512, kStages = kRing / kBytes, kPiece = 16 / sizeof(T);
  uint32_t at;               // shared address of the lane's first piece
  int lane;
  // Copies chunk c of the row; from = where the lane's first piece lies in it.
  __device__ __forceinline__ void fetch(const Row<T>& row, const T* from, int c, int stage) const {
    const uint32_t to = at + stage * kBytes;
    if (c > 0 && row.token(c, kChunk) <= row.vocab) {          // all of it in the row
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + k * 512), "l"(from + k * 32 * kPiece) : "memory");
    } else {
#pragma unroll 1
      for (int k = 0; k < kPieces; ++k) {
        uint32_t w[4];
        Row<T>::load_at(row.x, row.vocab, row.token(c, (k * 32 + lane) * kPiece), w);
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to + k * 512), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
      }
    }
  }
  __device__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  __device__ __forceinline__ void take(int stage, uint32_t (&w)[Row<T>::kWords]) const {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[4 * k]), "=r"(w[4 * k + 1]), "=r"(w[4 * k + 2]),
                   "=r"(w[4 * k + 3]) : "r"(at + stage * kBytes + k * 512) : "memory");
  }
};

// Two floats in a register pair.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ float low(f32x2 p) { return __uint_as_float((uint32_t)p); }
__device__ __forceinline__ float high(f32x2 p) { return __uint_as_float((uint32_t)(p >> 32)); }
__device__ __forceinline__ f32x2 fma_pair(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 add_pair(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 ex2_pair(f32x2 a) { return pair(ex2(low(a)), ex2(high(a))); }

// The largest of a lane's words of logits (NaN where there is nothing else).
template <typename T, int N>
__device__ __forceinline__ float largest(const uint32_t (&w)[N]) {
  if constexpr (sizeof(T) == 2) {
    auto bf = [](uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); };
    __nv_bfloat162 m = bf(w[0]);
#pragma unroll
    for (int k = 1; k < N; ++k) m = __hmax2(m, bf(w[k]));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    float m = __uint_as_float(w[0]);
#pragma unroll
    for (int k = 1; k < N; ++k) m = fmaxf(m, __uint_as_float(w[k]));
    return m;
  }
}

// A lane's part of the sum of exp(x - m), m the largest logit its warp has seen.  The exponents are x log2 e - R
// with R = m log2 e rounded once: a fused product loses nothing, and what R lost, below 2^-8 and the same for
// every term, goes back in at the end.  Next to huge logits R would lose more: the exponents are (x - m) log2 e there,
// and a maximum that passes from one kind to the other takes what R lost in or out.
struct LaneSum {
  float m = -INFINITY, R = 0.f, sum = 0.f, lost = 0.f;         // sum + lost = sum 2^(x log2 e - R)
  bool far = false;                                            // a huge maximum: differences instead
  __device__ __forceinline__ void raise(float top) {
    const bool now = !(fabsf(top) < 0x1p16f);
    const float to = now ? 0.f : __fmul_rn(top, kLog2e);       // rounded as stored, not fused into R - to
    float f = 1.f;                                             // before any maximum the sum is 0 (or NaN)
    if (m > -INFINITY) {
      const float out = far ? 0.f : __fmaf_rn(m, kLog2e, -R), in = now ? 0.f : __fmaf_rn(top, kLog2e, -to);
      f = far || now ? ex2(__fmaf_rn(m - top, kLog2e, in - out)) : ex2(R - to);
    }
    sum *= f; lost *= f;
    m = top; R = to; far = now;
  }
  // Pairs of logits at a time: one instruction for two products, and for two sums.
  template <int N>
  __device__ __forceinline__ void add(const f32x2 (&v)[N]) {
    f32x2 e[N];
    const f32x2 scale = pair(kLog2e, kLog2e);
    if (far) {                                                 // inf - inf is NaN, and so is the row's sum
#pragma unroll
      for (int k = 0; k < N; ++k) e[k] = ex2_pair(fma_pair(add_pair(v[k], pair(-m, -m)), scale, pair(0.f, 0.f)));
    } else {                                                   // zeros, or NaN, while there is nothing but -inf
#pragma unroll
      for (int k = 0; k < N; ++k) e[k] = ex2_pair(fma_pair(v[k], scale, pair(-R, -R)));
    }
#pragma unroll
    for (int h = N / 2; h > 0; h /= 2)
#pragma unroll
      for (int k = 0; k < h; ++k) e[k] = add_pair(e[k], e[k + h]);
    two_sum(sum, lost, low(e[0]) + high(e[0]));
  }
  __device__ __forceinline__ float total() const {
    return (sum + lost) * (far || m == -INFINITY ? 1.f : ex2(-__fmaf_rn(m, kLog2e, -R)));
  }
};

// A warp's part of beam w of request r; `held`, kRing bytes of shared memory, is the warp's.  after(): behind the last
// load, before the sums are written.
template <typename T, class After>
__device__ __forceinline__ void scan_part(const BeamArgs& a, uint8_t* held, int r, int w, int part, After&& after) {
  const int lane = threadIdx.x & 31;
  const uint32_t row = (uint32_t)r * a.beams + w;
  const Row<T> x(a, r, w);
  float* maxima = a.maxima + (size_t)row * a.chunks;
  LaneSum l;
  // every parts-th chunk: the row's warps read side by side
  const Ring<T> ring{smem_addr(held) + lane * 16, lane};
  constexpr int kStages = Ring<T>::kStages;
  const T* from = x.x + x.token(part, lane * Ring<T>::kPiece);
  const long long step = (long long)a.parts * kChunk;
  int ahead = part;
  auto fetch = [&](int stage) {
    if (ahead < a.chunks) ring.fetch(x, from, ahead, stage);
    ring.commit();
    ahead += a.parts;
    from += step;
  };
  // the first chunk is on its way while the score is: 64 x 8 rows 28.8 -> 28.0 us with the ranking; first steps, where
  // three of four rows are absent, 9.3 -> 9.5
  fetch(0);
  if (!live(a.scores[row]) || (a.finished && a.finished[row])) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
#pragma unroll
  for (int u = 1; u < kStages - 1; ++u) fetch(u);
  for (int c = part; c < a.chunks;) {
#pragma unroll
    for (int stage = 0; stage < kStages; ++stage) {
      fetch(stage ? stage - 1 : kStages - 1);                  // the stage read last
      uint32_t raw[Row<T>::kWords];
      ring.take(stage, raw);
      const float most = redux_max(largest<T>(raw));
      if (lane == 0) maxima[c] = most;
      if (most > l.m) l.raise(most);
      f32x2 v[kLane / 2];
#pragma unroll
      for (int k = 0; k < kLane / 2; ++k) v[k] = pair(Row<T>::value(raw, 2 * k), Row<T>::value(raw, 2 * k + 1));
      l.add(v);
      c += a.parts;
      if (c >= a.chunks) break;
    }
  }
  after();
  float sum = l.total();
#pragma unroll
  for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) a.records[row * a.parts + part] = make_float2(l.m, sum);
}

template <typename T>
__global__ void __launch_bounds__(kScanWarps * 32, kBeamScanWarps / kScanWarps) beam_scan_kernel(const __grid_constant__ BeamArgs a) {
  __shared__ __align__(16) uint8_t held[kScanWarps * kRing];
  const uint32_t warp = threadIdx.x >> 5, wid = blockIdx.x * kScanWarps + warp, row = wid / (uint32_t)a.parts;
  if (row >= (uint32_t)a.requests * a.beams) return;
  const uint32_t r = row / (uint32_t)a.beams;
  // the next kernel's blocks not before the end: they would take registers that scan blocks still to come need
  scan_part<T>(a, held + warp * kRing, (int)r, (int)(row - r * a.beams), (int)(wid - row * a.parts), [] { pdl_trigger(); });
}

// ------------------------------------------------------------------ pick
__device__ __forceinline__ unsigned long long ordered(double x) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(x);
  return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double unordered(unsigned long long k) {
  return __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k));
}

constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPer = 4;                          // keys a thread looks at together
constexpr int kAhead = 4;                        // such rounds whose loads are in flight together, where there are more

template <typename T>
struct alignas(16) Chosen {  // a chosen chunk
  const T* x;                // its row
  int first;                 // the token of its element 0, which may lie before the row
  float least;               // logits below this are no candidates; +inf: a finished row
};
template <typename T>
struct PickShared {
  unsigned __int128 key[kList];                  // listed: a logit's bits above its place; then its key (Pick::exact)
  Chosen<T> chunk[kBeamMaxOut];
  int row[kBeamMaxOut];                          // the chosen chunks' beams
  double base[kBeamMaxBeams];                    // score - log sum exp(x - top): a logit's key is base + (x - top)
  float mine[kPickThreads + kPickWarps];         // threads' largest keys, a warp's behind the other at 33 words
  float group[kMaxGroups];
  float base32[kBeamMaxBeams], score[kBeamMaxBeams], top[kBeamMaxBeams], log_sum[kBeamMaxBeams];
  int exponent[kBeamMaxBeams], state[kBeamMaxBeams];     // state: 0 no candidates, 1 live, 2 finished
  int count;
  float bound, size;                             // size: the largest |score| + |log sum|
};

template <typename T>
struct Pick {
  const BeamArgs& a;
  PickShared<T>& sh;
  int r, n;
  int tid, warp, lane;

  // The least key in 32 bits that may belong to a key which reaches the bound.  With L = e log 2 + log f the log sum,
  // base is score - L rounded four times: e log 2 by 2^-24 (and its constant by 2^-25) of at most 2.1 |L|, the sum by
  // 2^-24 |L|, the difference by 2^-24 of itself.  That is 2^-24 of 5.2 (|score| + |L|) however far the two cancel, so
  // size is taken before they do: key + size bounds x - top, whose rounding and the last sum's add 2^-24 (2 |key| + size).
  // So a key is off by less than 2^-21 (|key| + size); bound and key together by twice that, and as much is to spare.
  __device__ __forceinline__ float from() const {
    const float f = sh.bound - 0x1p-19f * (fabsf(sh.bound) + sh.size);
    return f > -INFINITY ? f : -FLT_MAX;                       // also where that is no number
  }
  __device__ __forceinline__ static float key32(float base, float top, float x) { return fmaxf(base + (x - top), -FLT_MAX); }
  __device__ __forceinline__ unsigned long long key(float x, int w) const { return ordered(sh.base[w] + ((double)x - (double)sh.top[w])); }

  // A bound that n keys reach, from the threads' largest ones: groups of threads, a third more of them than n,
  // have their largest key each, and the n-th largest of these is the bound (-inf if fewer groups than n have
  // one).  About G log(G / (G - n)) keys reach it when they are spread at random: 9 for n = 8, 89 for n = 64.
  // The threads of a group are of different warps, so that few keys fill many groups.
  __device__ __forceinline__ void bound(float mine) const {
    sh.mine[tid + warp] = mine;
    __syncthreads();
    float g = sh.mine[lane * 33 + warp];
    if (n <= 24) {                                             // 32 groups, one a warp
      g = redux_max(g);
      if (lane == 0) sh.group[warp] = g;
      __syncthreads();
      const float o = sh.group[lane], v = sh.group[warp];
      if (__popc(__ballot_sync(0xffffffffu, o > v || (o == v && lane < warp))) == n - 1 && lane == 0) sh.bound = v;
    } else {
      const int width = n <= 96 ? 8 : 2, groups = kPickThreads / width, k = tid / width;
      for (int o = width / 2; o > 0; o /= 2) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
      if (lane % width == 0) sh.group[k] = g;
      __syncthreads();
      int rank = 0;                                            // the group's own threads count for it
#pragma unroll 4
      for (int j = tid % width; j < groups; j += width) {
        const float o = sh.group[j];
        rank += (int)(o > g) | ((int)(o == g) & (int)(j < k));
      }
      for (int o = width / 2; o > 0; o /= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
      if (rank == n - 1 && lane % width == 0) sh.bound = g;
    }
    __syncthreads();
  }

  // Lists a candidate: its logit x, and place = beam << 32 | chunk's number or token.
  __device__ __forceinline__ void add(float x, unsigned long long place) const {
    const int at = atomicAdd(&sh.count, 1);
    if (at < kList) sh.key[at] = (unsigned __int128)__float_as_uint(x) << 64 | place;
  }
  // Orders like the logits, one zero.
  __device__ __forceinline__ static uint32_t ordered32(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
  }
  // The key of a listed candidate, larger ones first: the score, ~beam (7 bits), the logit (32), ~number (25).
  __device__ __forceinline__ unsigned __int128 exact(unsigned __int128 k) const {
    const unsigned long long w = (unsigned long long)k >> 32, number = (uint32_t)k;
    const float x = __uint_as_float((uint32_t)(k >> 64));
    const unsigned long long place = w << 57 | (unsigned long long)~ordered32(x) << 25 | number;
    return (unsigned __int128)key(x, (int)w) << 64 | ~place;
  }

  // The q first of a warp's candidates of one row, by logit and then in order: value(j), j = 0 .. m - 1, are the
  // lane's logits (-inf: none), those of lower lanes come first.  Calls visit(j, logit) for each.
  template <class Value, class Visit>
  __device__ __forceinline__ void first_of(int m, int q, Value&& value, Visit&& visit) const {
    auto count = [&](uint32_t least) {
      int c = 0;
      for (int j = 0; j < m; ++j) c += ordered32(value(j)) >= least;
      return (int)__reduce_add_sync(0xffffffffu, c);
    };
    uint32_t lo = ordered32(-FLT_MAX), hi = ordered32(FLT_MAX);
    if (count(lo) > q)
      while (lo < hi) {                                        // the largest that q of them reach
        const uint32_t mid = lo + (hi - lo) / 2 + 1;
        if (count(mid) >= q) lo = mid; else hi = mid - 1;
      }
    int same = 0;
    for (int j = 0; j < m; ++j) same += ordered32(value(j)) == lo;
    int before = same;                                         // those equal to it in lower lanes
    for (int o = 1; o < 32; o *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      before += lane >= o ? v : 0;
    }
    before -= same;
    const int room = q - count(lo + 1);
    for (int j = 0; j < m; ++j) {
      const float x = value(j);
      const uint32_t k = ordered32(x);
      if (k > lo || (k == lo && before++ < room)) visit(j, x);
    }
  }

  // Ranks the listed keys and calls put(rank, score, beam, number) on one thread for each of the n first.  If more were listed
  // than fit (very many equal or nearly equal keys), few() lists only those that their row's or chunk's own order
  // leaves, at most `at_most` of them; if these may be too many as well, each(visit) visits all candidates again,
  // and a bound is found by halving the space of the keys, which are distinct.  Returns how many there are.
  template <class Each, class Few, class Put>
  __device__ __forceinline__ int rank(Each&& each, int at_most, Few&& few, Put&& put) const {
    __syncthreads();
    int listed = sh.count;
    if (listed > kList) {
      __syncthreads();
      if (tid == 0) sh.count = 0;
      __syncthreads();
      if (at_most <= kList) {
        few();
        __syncthreads();
        listed = sh.count;
      } else {
        unsigned __int128 low = 0, high = ~(unsigned __int128)0;         // count(>= low) > kList, count(> high) < n
        do {
          const unsigned __int128 mid = low + (high - low) / 2 + 1;
          __syncthreads();
          if (tid == 0) sh.count = 0;
          __syncthreads();
          each([&](float x, unsigned long long place) {
            if (exact((unsigned __int128)__float_as_uint(x) << 64 | place) >= mid) add(x, place);
          });
          __syncthreads();
          listed = sh.count;
          if (listed < n) high = mid - 1; else low = mid;
        } while (listed < n || listed > kList);
      }
    }
    auto put_key = [&](int rank, unsigned __int128 k) {
      const unsigned long long place = ~(unsigned long long)k;
      put(rank, unordered((unsigned long long)(k >> 64)), (int)(place >> 57), (int)(place & 0x1FFFFFF));
    };
    for (int i = tid; i < listed; i += kPickThreads) sh.key[i] = exact(sh.key[i]);
    __syncthreads();
    if (listed <= kCounted) {
      // a key's rank is the number of keys before it: eight lanes count for one key at a time
      for (int i = tid / 8; i - tid % 32 / 8 < listed; i += kPickThreads / 8) {
        const unsigned __int128 k = i < listed ? sh.key[i] : 0;
        int rank = 0;
#pragma unroll 2
        for (int j = tid % 8; j < listed; j += 8) rank += sh.key[j] > k;
#pragma unroll
        for (int o = 4; o > 0; o /= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
        if (tid % 8 == 0 && i < listed && rank < n) put_key(rank, k);
      }
    } else {                                                   // sorted by exchanges, the largest first
      int size = 2 * kCounted;
      while (size < listed) size *= 2;
      for (int i = listed + tid; i < size; i += kPickThreads) sh.key[i] = 0;
      for (int run = 2; run <= size; run *= 2)
        for (int d = run / 2; d > 0; d /= 2) {
          __syncthreads();
          for (int i = tid; i < size / 2; i += kPickThreads) {
            const int x = 2 * i - (i & (d - 1)), y = x + d;    // the i-th pair d apart
            const unsigned __int128 u = sh.key[x], v = sh.key[y];
            if ((u < v) == ((x & run) == 0)) { sh.key[x] = v; sh.key[y] = u; }
          }
        }
      __syncthreads();
      if (tid < min(listed, n)) put_key(tid, sh.key[tid]);
    }
    return min(listed, n);
  }

  // ---- the chunks' maxima: number beam * chunks + chunk, a thread takes every kPickThreads-th
  __device__ __forceinline__ int row_of(uint32_t i) const {    // i / chunks
    const uint32_t q = __umulhi(i, a.chunks_inv);
    return q + (i - q * a.chunks >= (uint32_t)a.chunks);
  }
  __device__ __forceinline__ void load_maxima(const float* maxima, int keys, int i0, float (&x)[kPer]) const {
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] = i0 + e * kPickThreads < keys ? maxima[i0 + e * kPickThreads] : -INFINITY;
  }
  // visit(key32, logit, place) of those among x that count.
  template <class V>
  __device__ __forceinline__ void each_chunk(int keys, int i0, const float (&x)[kPer], V&& visit) const {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int i = i0 + e * kPickThreads;
      if (i >= keys) break;
      const int w = row_of(i), state = sh.state[w];
      float v = x[e];
      if (state == 2) v = i == w * a.chunks ? 0.f : -INFINITY; // a finished row has one candidate: itself
      if (state == 0 || !(v > -INFINITY)) continue;
      visit(key32(sh.base32[w], sh.top[w], v), v, (unsigned long long)w << 32 | (uint32_t)i);
    }
  }

  // ---- elements of the chosen chunks; a thread takes four adjacent ones, a warp a quarter of a chunk
  static constexpr int kWords = kPer * sizeof(T) / 4;
  // visit(raw, i, chunk) for the thread's elements i .. i + 3 of the chosen chunks (i counts through all of them).
  template <class V>
  __device__ __forceinline__ void each_four(int chosen, V&& visit) const {
    for (int i0 = tid * kPer; i0 < chosen * kChunk; i0 += kAhead * kPer * kPickThreads) {
      uint32_t raw[kAhead][kWords];
      Chosen<T> c[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kPer * kPickThreads;
        if (i >= chosen * kChunk) break;
        c[u] = sh.chunk[i / kChunk];
        if (c[u].least < INFINITY) Row<T>::load_at(c[u].x, a.vocab, c[u].first + i % kChunk, raw[u]);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kPer * kPickThreads;
        if (i >= chosen * kChunk) break;
        if (c[u].least < INFINITY) visit(raw[u], i, c[u]);
      }
    }
  }
  // Logits of chunk k below this are below `from` whatever was rounded; next to huge logits none are.
  __device__ __forceinline__ float least(int k, float from) const {
    const int w = sh.row[k];
    const float d = from - sh.base32[w], l = (d + sh.top[w]) - 0x1p-21f * (fabsf(d) + fabsf(sh.top[w]));
    return sh.state[w] == 2 ? INFINITY : l >= -FLT_MAX ? fminf(l, FLT_MAX) : -FLT_MAX;
  }
  // visit(logit, place) of the tokens that reach their chunk's least logit.
  template <class V>
  __device__ __forceinline__ void each_token(int chosen, V&& visit) const {
    each_four(chosen, [&](const uint32_t (&raw)[kWords], int i, const Chosen<T>& c) {
      float v[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[e] = Row<T>::value(raw, e);
      if (!(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) >= c.least)) return;
      const unsigned long long w = (unsigned long long)sh.row[i / kChunk] << 32;
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (v[e] >= c.least) visit(v[e], w | (uint32_t)(c.first + i % kChunk + e));
    });
    if (tid < chosen && sh.state[sh.row[tid]] == 2) visit(0.f, (unsigned long long)sh.row[tid] << 32 | (uint32_t)a.eos);
  }
};

// Ranks request r's candidates, one CTA; scanned(): waits for the scan.
template <typename T, class Scanned>
__device__ __forceinline__ void pick_request(const BeamArgs& a, PickShared<T>& sh, int r, Scanned&& scanned) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = a.n_out;
  const Pick<T> p{a, sh, r, n, tid, warp, lane};
  if (tid == 0) { sh.size = 0.f; sh.bound = -INFINITY; sh.count = 0; }
  if (tid < a.beams) {
    const long long row = (long long)r * a.beams + tid;
    sh.score[tid] = a.scores[row];
    sh.state[tid] = !live(a.scores[row]) ? 0 : a.finished && a.finished[row] ? 2 : 1;
  }
  if (tid < n) {                                               // places that no candidate takes
    const long long to = (long long)r * n + tid;
    a.rows[to] = -1;
    a.tokens[to] = -1;
  }
  __syncthreads();
  scanned();
  const float* maxima = a.maxima + (size_t)r * a.beams * a.chunks;
  const int keys = a.beams * a.chunks;
  float x[kPer];                                               // a thread's first keys stay in registers
  p.load_maxima(maxima, keys, tid, x);
  // the rows' sums, a warp a row
  for (int w = warp; w < a.beams; w += kPickWarps) {
    const float2* rec = a.records + ((long long)r * a.beams + w) * a.parts;
    float2 v = lane < a.parts ? rec[lane] : make_float2(-INFINITY, 0.f);     // not written for rows that do not count
    float top = v.x, sum = 0.f, lost = 0.f;
    for (int k = lane + 32; k < a.parts; k += 32) top = fmaxf(top, rec[k].x);
    top = redux_max(top);
    for (int k = lane;;) {
      two_sum(sum, lost, v.x > -INFINITY ? v.y * ex2((v.x - top) * kLog2e) : v.y);
      k += 32;
      if (k >= a.parts) break;
      v = rec[k];
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
      const float s = __shfl_xor_sync(0xffffffffu, sum, o);
      lost += __shfl_xor_sync(0xffffffffu, lost, o);
      two_sum(sum, lost, s);
    }
    // log sum = exponent log 2 + log of a fraction about 1 (2^-25 off) + the sum's dropped part
    const int e = (int)(__float_as_uint(sum * 1.41421356f) >> 23) - 127;
    const float log_f = logf(__uint_as_float(__float_as_uint(sum) - ((uint32_t)e << 23))) + __fdividef(lost, sum);
    int state = sh.state[w];
    // no softmax: nothing but -inf, or +inf or NaN among the logits
    if (state == 1 && (!(sum > 0.f) || !(fabsf(top) <= FLT_MAX))) state = 0;
    if (lane == 0 && state) {
      const bool done = state == 2;
      const float log_sum = done ? 0.f : (float)e * 0.693147181f + log_f;
      sh.top[w] = done ? 0.f : top;
      sh.exponent[w] = done ? 0 : e;
      sh.log_sum[w] = done ? 0.f : log_f;
      sh.base32[w] = sh.score[w] - log_sum;
      // non-negative floats order like their bits
      atomicMax(reinterpret_cast<int*>(&sh.size), __float_as_int(fminf(fabsf(sh.score[w]) + fabsf(log_sum), FLT_MAX)));
    }
    __syncwarp();
    if (lane == 0) sh.state[w] = state;
  }
  __syncthreads();
  // 64-bit bases, while the others look for the bound
  if (tid >= kPickThreads - kBeamMaxBeams && tid - (kPickThreads - kBeamMaxBeams) < a.beams) {
    const int w = tid - (kPickThreads - kBeamMaxBeams);
    if (sh.state[w]) sh.base[w] = (double)sh.score[w] - ((double)sh.exponent[w] * 0.69314718055994531 + (double)sh.log_sum[w]) + 0.0;   // one zero
  }

  // the n best chunks
  float mine = -INFINITY;
  auto most = [&](float s, float, unsigned long long) { mine = fmaxf(mine, s); };
  p.each_chunk(keys, tid, x, most);
  for (int i0 = tid + kPer * kPickThreads; i0 < keys; i0 += kPer * kPickThreads) {
    float y[kPer];
    p.load_maxima(maxima, keys, i0, y);
    p.each_chunk(keys, i0, y, most);
  }
  p.bound(mine);
  auto chunks = [&](auto&& visit) {
    const float from = p.from();
    auto reach = [&](float s, float v, unsigned long long place) {
      if (s >= from) visit(v, place);
    };
    p.each_chunk(keys, tid, x, reach);
    for (int i0 = tid + kPer * kPickThreads; i0 < keys; i0 += kPer * kPickThreads) {
      float y[kPer];
      p.load_maxima(maxima, keys, i0, y);
      p.each_chunk(keys, i0, y, reach);
    }
  };
  auto add = [&](float v, unsigned long long place) { p.add(v, place); };
  chunks(add);
  auto few_chunks = [&] {                                      // n of a row's chunks at most
    for (int w = warp; w < a.beams; w += kPickWarps) {
      const int state = sh.state[w], m = (a.chunks + 31) / 32, c0 = lane * m;
      const float from = p.from(), base = sh.base32[w], top = sh.top[w];
      p.first_of(state ? m : 0, n, [&](int j) {
        const int c = c0 + j;
        const float v = c >= a.chunks ? -INFINITY : state == 2 ? (c ? -INFINITY : 0.f) : maxima[(size_t)w * a.chunks + c];
        return v > -INFINITY && p.key32(base, top, v) >= from ? v : -INFINITY;
      }, [&](int j, float v) { p.add(v, (unsigned long long)w << 32 | (uint32_t)(w * a.chunks + c0 + j)); });
    }
  };
  const int chosen = p.rank(chunks, a.beams * n, few_chunks, [&](int rank, double s, int w, int i) {
    const Row<T> row(a, r, w);
    sh.chunk[rank] = Chosen<T>{row.x, row.token(i - w * a.chunks, 0), 0.f};
    sh.row[rank] = w;
    if (rank == n - 1) sh.bound = (float)s;                    // n chunks' maxima are n tokens
  });
  __syncthreads();

  // the n best tokens in them
  if (chosen < n) {                                            // fewer chunks than n: another bound
    if (tid < chosen) sh.chunk[tid].least = sh.state[sh.row[tid]] == 2 ? INFINITY : 0.f;
    __syncthreads();
    if (tid == 0) sh.bound = -INFINITY;
    mine = -INFINITY;
    p.each_four(chosen, [&](const uint32_t (&raw)[Pick<T>::kWords], int i, const Chosen<T>&) {
      const int w = sh.row[i / kChunk];
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const float v = Row<T>::value(raw, e);
        if (v > -INFINITY) mine = fmaxf(mine, p.key32(sh.base32[w], sh.top[w], v));
      }
    });
    if (tid < chosen && sh.state[sh.row[tid]] == 2) mine = fmaxf(mine, sh.score[sh.row[tid]]);
    p.bound(mine);
  }
  if (tid == 0) sh.count = 0;
  if (tid < chosen) sh.chunk[tid].least = p.least(tid, p.from());
  __syncthreads();
  auto tokens = [&](auto&& visit) { p.each_token(chosen, visit); };
  tokens(add);
  const long long to = (long long)r * n;
  auto few_tokens = [&] {          // k chunks' maxima are before any token of chunk k: n - k of its tokens at most
    for (int k = warp; k < chosen; k += kPickWarps) {
      const Chosen<T> c = sh.chunk[k];
      const unsigned long long w = (unsigned long long)sh.row[k] << 32;
      if (c.least == INFINITY) {
        if (lane == 0) p.add(0.f, w | (uint32_t)a.eos);
        continue;
      }
      uint32_t part[Row<T>::kWords];
      Row<T>::load_at(c.x, a.vocab, c.first + lane * kLane, part);
      float v[kLane];
#pragma unroll
      for (int e = 0; e < kLane; ++e) v[e] = Row<T>::value(part, e);
      p.first_of(kLane, n - k, [&](int j) {
        float x = -INFINITY;
#pragma unroll
        for (int e = 0; e < kLane; ++e) x = e == j ? v[e] : x;
        return x >= c.least ? x : -INFINITY;
      }, [&](int j, float x) { p.add(x, w | (uint32_t)(c.first + lane * kLane + j)); });
    }
  };
  const int found = p.rank(tokens, chosen * (2 * n - chosen + 1) / 2, few_tokens, [&](int rank, double s, int w, int token) {
    a.out_scores[to + rank] = (float)s;
    a.rows[to + rank] = r * a.beams + w;
    a.tokens[to + rank] = token;
    if (a.out_finished) a.out_finished[to + rank] = sh.state[w] == 2 || token == a.eos;
  });
  if (tid >= found && tid < n) {
    a.out_scores[to + tid] = -INFINITY;
    if (a.out_finished) a.out_finished[to + tid] = 0;
  }
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads, 1) beam_pick_kernel(const __grid_constant__ BeamArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  pick_request<T>(a, *reinterpret_cast<PickShared<T>*>(smem), blockIdx.x, [] { pdl_wait(); });
}

// Both in one launch, a cluster of CTAs a request: all of them scan, the first one ranks.
template <typename T>
__global__ void __launch_bounds__(kPickThreads, 1) beam_step_kernel(const __grid_constant__ BeamArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int r = blockIdx.x / kBeamCluster, cta = blockIdx.x % kBeamCluster, warp = threadIdx.x >> 5;
  const int wid = cta * kPickWarps + warp, w = wid / a.parts;
  auto scan = [&] {
    if (w < a.beams) scan_part<T>(a, smem + sizeof(PickShared<T>) + warp * kRing, r, w, wid - w * a.parts, [] {});
    cluster_sync();
  };
  if (cta == 0) pick_request<T>(a, *reinterpret_cast<PickShared<T>*>(smem), r, scan);
  else scan();
}

// ------------------------------------------------------------------ paths
// The way back from the last beams is a chain of maps, which may be put together in any grouping.  A cluster of
// CTAs a request takes a tile of steps from the end, each of its threads a share of them for one beam: they walk
// through their shares from every beam (a map a share), put the maps of all later shares together in
// log2(shares) rounds within a CTA and one after another across the cluster, and walk again from where the
// last beams come in.  Parents and tokens of the tile lie in shared memory, so that a step is one shared-memory
// load, and the sequences leave along time.  Bound by the latency of that chain: load, two walks, the
// rounds between.
constexpr int kPathThreads = 1024;
constexpr int kPathShared = 200 * 1024;
constexpr int kNoBeam = 255;

// A byte of CTA `rank`'s shared memory, at the same place as p in this one.
__device__ __forceinline__ int of_cta(const uint8_t* p, int rank) {
  uint32_t at, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return (int)v;
}

__global__ void __launch_bounds__(kPathThreads, 1) beam_paths_kernel(const __grid_constant__ PathArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint8_t map[2][kPathThreads];
  __shared__ uint8_t whole[2][kBeamMaxBeams];                  // this CTA's steps as one map, of this tile and the next
  const int W = a.beams, ctas = a.ctas, cta = blockIdx.x % ctas, r = blockIdx.x / ctas, tid = threadIdx.x, lw = a.log_beams;
  const int shares = kPathThreads >> lw, share = tid >> lw, w = tid & ((1 << lw) - 1);
  const bool here = w < W;
  const int pitch = a.tile | 1;                                // of the sequences: odd, beams on different banks
  int32_t* tok = reinterpret_cast<int32_t*>(smem);             // [tile][W]
  int32_t* seq = tok + (size_t)a.tile * W;                     // [W][pitch]
  uint8_t* par = reinterpret_cast<uint8_t*>(seq + (size_t)W * pitch);      // [tile][W]
  int n = a.steps;
  if (a.n_steps) n = min(max(a.n_steps[r], 0), a.steps);
  const size_t step = (size_t)a.requests * W;
  int32_t* out = a.out + (size_t)r * W * a.steps;
  // 32 steps of a beam a warp at a time: fn(beam, step in 0 .. count - 1)
  auto along_time = [&](int count, auto&& fn) {
    const int tasks = (int)((count + 31u) / 32) * W;           // count up to 2^31 - 1
#pragma unroll 4
    for (int k = tid / 32; k < tasks; k += kPathThreads / 32) {
      const int t = k / W * 32 + tid % 32;
      if (t < count) fn(k % W, t);
    }
  };
  if (cta == 0) along_time(a.steps - n, [&](int k, int t) { out[(size_t)k * a.steps + n + t] = a.pad; });
  int carry = here ? w : kNoBeam;                              // where last beam w is when the tile begins (at its end)
  for (int t2 = n, turn = 0; t2 > 0; t2 -= ctas * a.tile, turn ^= 1) {
    // the CTAs take equal parts of the tile, the last one the last steps
    const int all = min(t2, ctas * a.tile), part = (all + ctas - 1) / ctas;
    const int t0 = t2 - all + min(all, cta * part), len = t2 - all + min(all, (cta + 1) * part) - t0;
    __syncthreads();
    if (here) {
      const size_t from = t0 * step + (size_t)r * W + w;
#pragma unroll 8
      for (int t = share; t < len; t += shares) {
        const long long p = (long long)a.rows[from + t * step] - (long long)r * W;
        const int32_t x = a.tokens[from + t * step];
        par[t * W + w] = p >= 0 && p < W ? (uint8_t)p : (uint8_t)kNoBeam;
        tok[t * W + w] = x;
      }
    }
    __syncthreads();
    const int each = (len + shares - 1) >> (10 - lw), b = min(len, share * each), e = min(len, b + each);
    int at = here ? w : kNoBeam;
    for (int t = e - 1; t >= b && at != kNoBeam; --t) at = par[t * W + at];
    map[0][tid] = (uint8_t)at;
    __syncthreads();
    int now = 0;                                               // map[now][share]: through this share and all later ones
    for (int d = 1; d < shares; d *= 2, now ^= 1) {
      int v = w;
      if (share + d < shares) v = map[now][tid + (d << lw)];
      map[now ^ 1][tid] = v == kNoBeam ? kNoBeam : map[now][(share << lw) + v];
      __syncthreads();
    }
    at = carry;
    if (ctas > 1) {
      if (share == 0 && here) whole[turn][w] = map[now][tid];
      cluster_sync();
      for (int c = ctas - 1; c >= 0; --c) {                    // through the later CTAs, and then through the others
        if (c == cta) at = carry;
        if (carry != kNoBeam) carry = of_cta(&whole[turn][carry], c);
      }
    } else if (carry != kNoBeam) {
      carry = map[now][carry];
    }
    if (share + 1 < shares && at != kNoBeam) at = map[now][((share + 1) << lw) + at];
    if (here)
      for (int t = e - 1; t >= b; --t) {
        int x = a.pad;
        if (at != kNoBeam) {
          const int to = par[t * W + at];
          if (to != kNoBeam) x = tok[t * W + at];
          at = to;
        }
        seq[w * pitch + t] = x;
      }
    __syncthreads();
    along_time(len, [&](int k, int t) { out[(size_t)k * a.steps + t0 + t] = seq[k * pitch + t]; });
  }
  if (ctas > 1) cluster_sync();                                // nobody leaves while its maps are read
}

template <typename T>
cudaError_t step_t(const BeamArgs& a, cudaStream_t st) {
  constexpr int kBytes = sizeof(PickShared<T>) + kPickWarps * kRing;
  cudaError_t e = cudaFuncSetAttribute(beam_step_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.requests * kBeamCluster);
  cfg.blockDim = dim3(kPickThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kBeamCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_step_kernel<T>, a);
}

template <typename T>
cudaError_t select_t(const BeamArgs& a, cudaStream_t st) {
  if (a.clustered) return step_t<T>(a, st);
  const long long warps = (long long)a.requests * a.beams * a.parts;
  cudaError_t e = cudaFuncSetAttribute(beam_pick_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(PickShared<T>));
  if (e != cudaSuccess) return e;
  beam_scan_kernel<T><<<(unsigned)((warps + kScanWarps - 1) / kScanWarps), kScanWarps * 32, 0, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.requests);
  cfg.blockDim = dim3(kPickThreads);
  cfg.dynamicSmemBytes = sizeof(PickShared<T>);
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

cudaError_t launch_beam_paths(PathArgs& a, int sm_count, cudaStream_t st) {
  a.log_beams = 0;
  while (1 << a.log_beams < a.beams) ++a.log_beams;
  // CTAs a request while they have an SM each and four steps a share.  By 1, 2, 4 and 8 of them, us: 5 requests
  // of 33 beams and 777 steps (4 a share by 8) 23.2, 13.4, 9.7, 8.4; 64 of 8 beams and 2048 steps (8 by 2) 12.8, 9.2, 14.5
  // by 4 (256 CTAs); 16 of 4 beams and 512 steps (2 by 1) 5.3, 5.6, 5.6, 11.1
  a.ctas = 1;
  while (a.ctas < 8 && 2 * a.ctas * (long long)a.requests <= sm_count && 2 * a.ctas * 4 * (kPathThreads >> a.log_beams) <= a.steps) a.ctas *= 2;
  a.tile = std::min(kPathShared / (a.beams * 9) - 1, (a.steps - 1) / a.ctas + 1);
  const int bytes = a.tile * a.beams * 5 + a.beams * (a.tile | 1) * 4;
  if (bytes > 44 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(beam_paths_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPathShared);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.requests * a.ctas);
  cfg.blockDim = dim3(kPathThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_paths_kernel, (const PathArgs)a);
}

}  // namespace witcert
