// Rotary positions of queries and keys, in one pass: y = gain R(pos) x on the first `rot` channels
// of every head, a copy of the rest.
//
// Bound by HBM: each element is read once and written once.  A CTA takes TOK tokens; its threads
// first issue their loads of x, then form the (gain cos, gain sin) pairs of those tokens once in
// shared memory (the turns are the same for all heads), and turn what has arrived.  Angles come
// from the 64-bit fixed-point product of rope.cuh, so there is no table to read.
//
// A thread's unit is one vector of VE channels (16 bytes) together with its partners: half layout,
// the vectors at c and c + rot/2; interleaved, one vector that holds VE/2 pairs.  Vectors past
// `rot` are copied.  Pointers, strides or widths that do not allow 16-byte vectors take VE = 1
// (half layout) or 2 (interleaved): one pair a unit, element by element.
#include "rope.cuh"

namespace witcert {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;       // units of a thread in flight

// Narrow vectors promise the element's alignment only (odd strides are allowed).
template <typename T, int VE> struct __align__(sizeof(T) * VE == 16 ? 16 : sizeof(T)) Vec { T v[VE]; };

// Unit u of a token: tensor, head and vector.
template <typename T, int VE, bool INTER>
struct Unit {
  const T* x;
  T* y;
  int p;                         // first pair, or -1: plain copy
  Vec<T, VE> a, b;
  __device__ __forceinline__ void place(const RopeLaunch& r, int tok, int u, int per_head, int turned) {
    int head = u / per_head;
    const int v = u - head * per_head;
    const int k = head >= r.t[0].heads;
    head -= k ? r.t[0].heads : 0;
    const RopeTensor& t = r.t[k];
    // half layout: vectors 0 .. turned - 1 are pairs of vectors, the rest copies from channel rot on
    const int c = INTER || v < turned ? v * VE : r.rot + (v - turned) * VE;
    p = v >= turned ? -1 : INTER ? c / 2 : c;
    x = reinterpret_cast<const T*>(t.x) + (size_t)tok * t.x_tok + (size_t)head * t.x_head + c;
    y = reinterpret_cast<T*>(t.y) + (size_t)tok * t.y_tok + (size_t)head * t.y_head + c;
  }
  __device__ __forceinline__ void load(int half) {
    a = *reinterpret_cast<const Vec<T, VE>*>(x);
    if (!INTER && p >= 0) b = *reinterpret_cast<const Vec<T, VE>*>(x + half);
  }
  __device__ __forceinline__ void finish(const float2* cs, int half) {
    if (p >= 0) {
#pragma unroll
      for (int e = 0; e < (INTER ? VE / 2 : VE); ++e) {
        const float2 w = cs[p + e];
        T& f = INTER ? a.v[2 * e] : a.v[e];
        T& s = INTER ? a.v[2 * e + 1] : b.v[e];
        const float xf = to_f32<T>(f), xs = to_f32<T>(s);
        f = T(rope_first(xf, xs, w.x, w.y));
        s = T(rope_second(xf, xs, w.x, w.y));
      }
      if (!INTER) *reinterpret_cast<Vec<T, VE>*>(y + half) = b;
    }
    *reinterpret_cast<Vec<T, VE>*>(y) = a;
  }
};

template <typename T, int VE, bool INTER, int TOK>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeLaunch r) {
  __shared__ float2 cs[TOK][kRopeMaxPairs];
  const int tok0 = blockIdx.x * TOK, n = min(TOK, r.n_tok - tok0);
  const int pairs = r.rot >> 1, half = r.rot >> 1;
  // vectors of a head: turned ones (one or two vectors each) and copies
  const int turned = INTER ? r.rot / VE : half / VE;
  const int per_head = turned + (r.head_dim - r.rot) / VE;
  const int per_tok = per_head * (r.t[0].heads + r.t[1].heads), total = per_tok * n;
  // units of this CTA: blockIdx.y takes every gridDim.y-th run of kThreads * kUnroll
  bool have = false;
  for (int base = blockIdx.y * kThreads * kUnroll; base < total; base += gridDim.y * kThreads * kUnroll) {
    Unit<T, VE, INTER> w[kUnroll];
    int tok[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int u = base + k * kThreads + threadIdx.x;
      tok[k] = -1;
      if (u < total) {
        tok[k] = u / per_tok;
        w[k].place(r, tok0 + tok[k], u - tok[k] * per_tok, per_head, turned);
        w[k].load(half);
      }
    }
    if (!have) {
      for (int k = threadIdx.x; k < n * pairs; k += kThreads) {
        const int t = k / pairs, p = k - t * pairs;
        float c, s;
        rope_cs(r.turn[p], r.pos[tok0 + t], r.gain, c, s);
        cs[t][p] = make_float2(c, s);
      }
      __syncthreads();
      have = true;
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (tok[k] >= 0) w[k].finish(cs[tok[k]], half);
  }
}

template <typename T, int VE, bool INTER>
cudaError_t launch_t(const RopeLaunch& a, int sm_count, cudaStream_t st) {
  const int turned = INTER ? a.rot / VE : a.rot / 2 / VE;
  const long long per_tok = (long long)(turned + (a.head_dim - a.rot) / VE) * (a.t[0].heads + a.t[1].heads);
  const long long chunk = kThreads * kUnroll;
  // few tokens: one token a CTA, its heads spread over gridDim.y
  if (a.n_tok < 4 * sm_count) {
    long long gy = (per_tok + chunk - 1) / chunk;
    if (gy > 64) gy = 64;
    rope_kernel<T, VE, INTER, 1><<<dim3((unsigned)a.n_tok, (unsigned)gy), kThreads, 0, st>>>(a);
  } else {
    rope_kernel<T, VE, INTER, 4><<<dim3((unsigned)((a.n_tok + 3) / 4)), kThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& a, int sm_count, cudaStream_t st) {
  // 16-byte vectors: every row starts on 16 bytes and every vector lies within its part of the head
  const int e = a.is_bf16 ? 2 : 4, ve = 16 / e;
  bool wide = (a.interleaved ? a.rot : a.rot / 2) % ve == 0 && (a.head_dim - a.rot) % ve == 0;
  for (const RopeTensor& t : a.t)
    if (t.heads)
      wide = wide && ((uintptr_t)t.x | (uintptr_t)t.y) % 16 == 0 &&
             (t.x_tok | t.x_head | t.y_tok | t.y_head) % ve == 0;
  if (a.is_bf16) {
    using T = __nv_bfloat16;
    if (wide) return a.interleaved ? launch_t<T, 8, true>(a, sm_count, st) : launch_t<T, 8, false>(a, sm_count, st);
    return a.interleaved ? launch_t<T, 2, true>(a, sm_count, st) : launch_t<T, 1, false>(a, sm_count, st);
  }
  using T = float;
  if (wide) return a.interleaved ? launch_t<T, 4, true>(a, sm_count, st) : launch_t<T, 4, false>(a, sm_count, st);
  return a.interleaved ? launch_t<T, 2, true>(a, sm_count, st) : launch_t<T, 1, false>(a, sm_count, st);
}

}  // namespace witcert
