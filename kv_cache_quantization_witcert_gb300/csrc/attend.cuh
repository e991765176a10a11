// What the chunk attention kernels share: the walk over a CTA's work, the staging of query rows and
// the softmax of one key tile.
//
// A query row is handled by N threads (two, or four where only few rows are there) of N warps that
// can reach the same tensor-memory lanes, each with 128 / N of the tile's columns: fewer registers,
// and more warps to hide the latency of a tile's chain (tensor memory, maximum, exponentials, tensor
// memory), which is what bounds a step.  They agree on the row's maximum through shared memory.
//
// Softmax: weights 2^(s c - m + off) with the row's reference m in log2 units.  m follows the running
// maximum only when that has grown by more than grow, so O and the sum l are rescaled rarely, by the
// softmax threads themselves.  fp16 weights reach 2^15 at most; off keeps the small ones normal, for a
// key's value can be zero where the weights are large: those below 2^-26 of the reference (2^-36 before
// they vanish) lose bits (off 8, grow 7: 864 us against 882 for 2048 of 32768 tokens, but 2^-22).
// bf16 has fp32's range, so m hardly ever moves.
#pragma once
#include "kernels.h"
#include "tcgen05.cuh"

namespace witcert {

template <bool BF16>
struct WeightRange {
  static constexpr float off = BF16 ? 0.0f : 12.0f, grow = BF16 ? 40.0f : 3.0f;
};
constexpr uint64_t kAttendWaitNs = 2000000000ull;          // 2 s per barrier wait

// A kernel of a call behind the call's earlier ones: it may start while its predecessor ends, and
// waits for it (pdl_wait) before it reads anything.
template <typename K>
cudaError_t launch_after(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, const AttendArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// One stretch of key tiles of one unit.
struct Segment {
  int k, h, r0, rows;        // sequence, KV head, first query row of the unit, rows of the sequence
  int j0, nk;                // key tiles j0 .. j0 + nk - 1
  bool whole;                // all of the unit's key tiles: the output is final
  int slot;                  // otherwise: where its records go
};
__device__ __forceinline__ bool same_unit(const AttendStart& a, const AttendStart& b) {
  return a.k == b.k && a.tile == b.tile && a.h == b.h;
}
// Rows of a unit and its key tiles; row_tiles: the sequence's units a head.
__device__ __forceinline__ int unit_place(const AttendArgs& a, const AttendStart& at, Segment& x, int& row_tiles) {
  const int n = a.n[at.k], len = a.len[at.k];
  x.k = at.k;
  x.h = at.h;
  x.rows = n * a.grp;
  row_tiles = (x.rows + a.unit_rows - 1) / a.unit_rows;
  x.r0 = (row_tiles - 1 - at.tile) * a.unit_rows;          // last rows, which see most keys, first
  const int last = min(x.rows, x.r0 + a.unit_rows) - 1;
  return (len - n + last / a.grp) / kTileTok + 1;
}
// The segments of CTA c in order: f(segment) until it returns false.
template <typename F>
__device__ __forceinline__ void walk(const AttendArgs& a, int c, F f) {
  AttendStart at = a.start[c];
  const AttendStart end = a.start[c + 1];
  while (!(same_unit(at, end) && at.j >= end.j)) {
    Segment x;
    int row_tiles;
    const int nt = unit_place(a, at, x, row_tiles);
    const int to = same_unit(at, end) ? end.j : nt;
    x.j0 = at.j;
    x.nk = to - at.j;
    x.whole = at.j == 0 && to == nt;
    x.slot = 2 * c + (at.j == 0 ? 1 : 0);
    if (!f(x)) return;
    if (to < nt) return;                                   // the CTA ends inside this unit
    at.j = 0;
    if (++at.h == a.s.Hkv) {
      at.h = 0;
      if (++at.tile == row_tiles) { at.tile = 0; ++at.k; }
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return BF16 ? bf2_bits(__floats2bfloat162_rn(a, b)) : h2_bits(__floats2half2_rn(a, b));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Bounded barrier wait.  Each attempt lets the hardware suspend the thread for up to a millisecond
// (it wakes when the phase completes), so waiting warps take no issue slots from working ones.
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  if (bar_try(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!bar_try(bar, parity))
    if (global_ns() - t0 > kAttendWaitNs) return false;
  return true;
}
// One arrival for a warp whose lanes have all come here (their earlier writes included).
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// A wait of a whole warp: its lanes give up together (tensor-memory accesses need all of them).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, bar_try(bar, parity))) return true;      // the usual case, 70 cycles
  return !__any_sync(0xffffffffu, !bar_wait(bar, parity));
}

// A row's N threads: one shared word each, 128 rows a part, and the barrier of their warps (an
// mbarrier of N arrivals, so that the wait has a limit).  A combination may overwrite the words of
// the one before it only when the partners have read them: either something between the two says so
// (stride 0), or combinations alternate between words `stride` apart, whose last use lies before the
// combination in between.
template <int N>
struct RowGroup {
  volatile float* words;       // of this row: part p at words[128 p]
  int part, stride;
  uint32_t bar, phase;
  bool ok;
  __device__ __forceinline__ void sync() {
    warp_arrive(bar);
    ok = ok && warp_wait(bar, phase++ & 1);
  }
  template <typename F> __device__ __forceinline__ float all(float v, F f) {
    volatile float* w = words + (phase & 1 ? stride : 0);
    w[128 * part] = v;
    sync();
#pragma unroll
    for (int p = 1; p < N; ++p) v = f(v, w[128 * ((part + p) % N)]);
    return v;
  }
  __device__ __forceinline__ float top(float v) { return all(v, [](float a, float b) { return fmaxf(a, b); }); }
  __device__ __forceinline__ float sum(float v) { return all(v, [](float a, float b) { return a + b; }); }
};

// 32 bytes a thread: a whole sector, where a warp's threads each have a row of their own.
__device__ __forceinline__ void load32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w) : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
               "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// This thread's 128 / N channels of query row `row` of a segment as operand words in the key images'
// channel order; zero for rows past the sequence's.  Returns log2(e)/sqrt(d) times the power of two
// that the row was divided by: fp16 rows are scaled to a largest element in [1, 2), which keeps bf16's eight
// bits of elements down to 2^-17 of it.
template <bool BF16, int N>
__device__ __forceinline__ float query_words(const AttendArgs& a, const Segment& u, int row, uint32_t (&w)[64 / N],
                                             RowGroup<N>& grp) {
  uint4 v[16 / N];
#pragma unroll
  for (int c = 0; c < 16 / N; ++c) v[c] = make_uint4(0, 0, 0, 0);
  if (row < u.rows) {
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(a.q) +
        ((size_t)(a.row0[u.k] + row / a.grp) * a.Hq + u.h * a.grp + row % a.grp) * kD + (128 / N) * grp.part);
#pragma unroll
    for (int c = 0; c < 16 / N; c += 2) load32(src + c, v[c], v[c + 1]);
  }
  // 16-byte piece 4 jj + t: channels 32 jj + 4t .. + 3 and 32 jj + 16 + 4t .. + 3
#pragma unroll
  for (int jj = 0; jj < 4 / N; ++jj)
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint4& x = v[4 * jj + 2 * m + (t >> 1)];
        w[16 * jj + 4 * t + 2 * m] = t & 1 ? x.z : x.x;
        w[16 * jj + 4 * t + 2 * m + 1] = t & 1 ? x.w : x.y;
      }
  float scale = a.scale_log2;
  if (!BF16) {
    uint32_t top = 0;                                     // largest magnitude's bits, two lanes of bf16
#pragma unroll
    for (int c = 0; c < 64 / N; ++c) top = __vmaxu2(top, w[c] & 0x7FFF7FFFu);
    // as a bf16 value, which orders like its bits; a NaN or infinity counts as the largest exponent
    const float mine = __uint_as_float(min(max(top & 0xFFFFu, top >> 16), 0x7F7Fu) << 16);
    // biased exponent of the row's largest element, kept where 2^-e and 2^e are normal numbers
    const int e = min(max((int)(__float_as_uint(grp.top(mine)) >> 23), 16), 238) - 127;
    const float down = __int_as_float((127 - e) << 23);
    scale *= __int_as_float((127 + e) << 23);
#pragma unroll
    for (int c = 0; c < 64 / N; ++c)
      w[c] = pack2<false>(__uint_as_float(w[c] << 16) * down, __uint_as_float(w[c] & 0xFFFF0000u) * down);
    grp.sync();                                           // all have read before the words are used again
  }
  return scale;
}

// One key tile's softmax for this thread's 128 / N columns of a row: logits at ts, weights to tp (half
// as many columns, over the logits), O at to.  rel: the last token of the tile this row sees (127 or
// more: all, negative: none).  o_wait(): O holds all earlier tiles' products (asked before O is
// rescaled).  The weights of each thread's first and last half of places are announced on p_bar and
// p_bar + 8.
template <bool BF16, int N, typename W>
__device__ __forceinline__ void softmax_tile(uint32_t ts, uint32_t tp, uint32_t to, int rel, bool first, float scale,
                                             float& m, float& l, RowGroup<N>& grp, uint32_t p_bar, W o_wait) {
  constexpr int kCols = 128 / N;
  uint32_t v[kCols / 32][32];
#pragma unroll
  for (int c = 0; c < kCols / 32; ++c) tmem_ld32(ts + 32 * c, v[c]);
  tmem_wait_ld();
  if (__any_sync(0xffffffffu, rel < kTileTok - 1)) {
    const int lim = rel - kCols * grp.part;
#pragma unroll
    for (int c = 0; c < kCols / 32; ++c)
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        // token of place e (see expand.cuh)
        const int tok = 32 * c + 16 * (e & 1) + 2 * (e >> 3) + ((e >> 2) & 1) + 8 * ((e >> 1) & 1);
        if (tok > lim) v[c][e] = 0xFF800000u;
      }
  }
  float mx[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    constexpr int kRun = kCols / 4;
    const uint32_t* x = &v[c * kRun / 32][c * kRun % 32];
    mx[c] = __uint_as_float(x[0]);
#pragma unroll
    for (int e = 1; e + 1 < kRun; e += 2) mx[c] = max3(mx[c], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
    mx[c] = fmaxf(mx[c], __uint_as_float(x[kRun - 1]));
  }
  // the partners' logits have left tensor memory when this returns: weights may overwrite them
  const float top = grp.top(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]));
  const bool grow = (top - m) * scale > WeightRange<BF16>::grow;   // also from -inf; false while nothing is visible
  if (__any_sync(0xffffffffu, grow)) {
    const float mn = grow ? top : m, f = grow ? ex2((m - mn) * scale) : 1.0f;
    l *= f;
    m = mn;
    if (!first) {
      o_wait();
#pragma unroll 1
      for (int c = 0; c < kCols; c += 16) {
        uint32_t o[16];
        tmem_ld16(to + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tmem_st16(to + c, o);
      }
    }
  }
  const float bias = WeightRange<BF16>::off - (m == -INFINITY ? 0.f : m * scale);
  const float2 sc2 = make_float2(scale, scale), b2 = make_float2(bias, bias);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    constexpr int kPairs = kCols / 4;                      // weight pairs of half the columns
    uint32_t pk[kPairs];
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      const uint32_t* y = &v[(c * 2 * kPairs + 2 * e) / 32][(c * 2 * kPairs + 2 * e) % 32];
      const float2 x = __ffma2_rn(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), sc2, b2);
      const float2 p = make_float2(ex2(x.x), ex2(x.y));
      sum[e & 1] = __fadd2_rn(sum[e & 1], p);
      pk[e] = pack2<BF16>(p.x, p.y);
    }
    tmem_st(tp + kPairs * c, pk);
    tmem_wait_st();
    tc_fence_before();
    warp_arrive(p_bar + 8 * c);
  }
  l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// O += P V for one tile: A in tensor memory, the value image at descriptor vd; the first and last half
// of each of the N threads' places as they are announced.  False if a wait ran out.
template <int N>
__device__ __forceinline__ bool issue_pv(uint32_t to, uint32_t tp, uint64_t vd, uint32_t idesc, bool first,
                                         uint32_t p_bar, uint32_t parity) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (!warp_wait(p_bar + 8 * c, parity)) return false;
    tc_fence_after();
    if (elect_one()) {
#pragma unroll
      for (int y = 0; y < 4; ++y) {                        // 16 places a step, 64 a panel
        const int x = N == 2 ? 4 * (y >> 1) + 2 * c + (y & 1) : 2 * y + c;
        mma_ts(to, tp + x * 8, vd + (uint64_t)(x >> 2) * (kD * 128 >> 4) + (x & 3) * 2, idesc, !first || c > 0 || y > 0);
      }
    }
    __syncwarp();
  }
  return true;
}
// S = Q K^T for one tile; done is told when it (and all before it) is complete.
__device__ __forceinline__ void issue_qk(uint32_t ts, uint64_t qd, uint64_t kd, uint32_t idesc, uint32_t done) {
  if (elect_one()) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {                          // 16 channels a step, 64 a panel
      const uint64_t o = (uint64_t)(x >> 2) * (kTileRows * 128 >> 4) + (x & 3) * 2;
      mma_ss(ts, qd + o, kd + o, idesc, x > 0);
    }
    mma_commit(done);
  }
  __syncwarp();
}
__device__ __forceinline__ void warp_commit(uint32_t bar) {
  if (elect_one()) mma_commit(bar);
  __syncwarp();
}
// A place in a ring of N stages and the parity of the visit.
template <int N> struct RingAt {
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == N) { st = 0; ph ^= 1; }
  }
};

// This thread's 128 / N columns of a row of a finished segment: the output itself, or its record.  O's
// columns are in the value images' channel order.
template <int N>
__device__ __forceinline__ void store_row(const AttendArgs& a, const Segment& u, int row, int part, uint32_t to, float m,
                                          float l, float scale, bool ok) {
  constexpr int kCols = 128 / N;
  const bool store = ok && row < u.rows;
  float* rec = nullptr;
  __nv_bfloat16* out = nullptr;
  if (u.whole) {
    out = static_cast<__nv_bfloat16*>(a.out) +
          ((size_t)(a.row0[u.k] + row / a.grp) * a.Hq + u.h * a.grp + row % a.grp) * kD + kCols * part;
  } else {
    rec = a.rec + ((size_t)u.slot * a.unit_rows + (row - u.r0)) * kRecStride;
    if (store && part == 0) *reinterpret_cast<float2*>(rec) = make_float2(m == -INFINITY ? m : m * scale, l);
    rec += 8 + kCols * part;
  }
  const float inv = 1.0f / l;                              // a whole unit's row sees at least one key
#pragma unroll 1
  for (int c = 0; c < kCols; c += 16) {
    uint32_t o[16];
    tmem_ld16(to + c, o);
    tmem_wait_ld();
    float x[16];                                           // by channel
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(o[(e & 8) + 4 * (e & 1) + ((e & 7) >> 1)]);
    uint32_t b[2][8];
    if (store && !u.whole) {
#pragma unroll
      for (int e = 0; e < 16; ++e) b[e >> 3][e & 7] = __float_as_uint(x[e]);
      store32(rec + c, b[0]);
      store32(rec + c + 8, b[1]);
    } else if (store) {
#pragma unroll
      for (int e = 0; e < 8; ++e) b[0][e] = pack2<true>(x[2 * e] * inv, x[2 * e + 1] * inv);
      store32(out + c, b[0]);
    }
    __syncwarp();
  }
}

}  // namespace witcert
