// Rotary positions of queries and keys, in one pass: y = gain R(pos) x on the first `rot` channels
// of every head, a copy of the rest.
//
// Bound by HBM: each element is read once and written once.  A CTA takes TOK tokens: its threads form
// the (gain cos, gain sin) pairs of those tokens once in shared memory (the turns are the same for
// all heads), then thread (v, s) turns vector v of heads s, s + blockDim.y, ... of one token after
// the other, two heads at a time.  Angles come from the 64-bit fixed-point product of rope.cuh, so
// there is no table to read.  More units in flight a thread cost more warps than they bring (four:
// 113 registers, 142 us for 16384 tokens of 40 heads).
//
// A unit is one vector of VE channels (16 bytes) together with its partners: half layout, the vectors
// at c and c + rot/2; interleaved, one vector that holds VE/2 pairs.  Vectors past `rot` are copied.
// Pointers, strides or widths that do not allow 16-byte vectors take VE = 1 (half layout) or 2
// (interleaved): one pair a unit, element by element.
#include <algorithm>

#include "rope.cuh"

namespace witcert {

namespace {

constexpr int kMaxThreads = 256;
constexpr int kUnroll = 2;       // units of a thread in flight
// A unit's pairs, and where pair p's (cos, sin) sits in the shared table: pair e of every unit
// together, so that neighbouring units read neighbouring words.
template <int VE, bool INTER> constexpr int kPairs = INTER ? VE / 2 : VE;
template <int VE, bool INTER> __device__ __forceinline__ int cs_at(int p) {
  constexpr int P = kPairs<VE, INTER>;
  return p % P * (kRopeMaxPairs / P) + p / P;
}

// Narrow vectors promise the element's alignment only (odd strides are allowed).
template <typename T, int VE> struct __align__(sizeof(T) * VE == 16 ? 16 : sizeof(T)) Vec { T v[VE]; };

template <typename T, int VE, bool INTER, int TOK>
__global__ void __launch_bounds__(kMaxThreads, 4) rope_kernel(const __grid_constant__ RopeLaunch r, int turned) {
  using V = Vec<T, VE>;
  constexpr int P = kPairs<VE, INTER>;
  __shared__ float2 cs[TOK][kRopeMaxPairs];
  const int tok0 = blockIdx.x * TOK, n = min(TOK, r.n_tok - tok0);
  const int half = r.rot >> 1, v = threadIdx.x, ny = blockDim.y;
  for (int k = threadIdx.y * blockDim.x + threadIdx.x; k < n * half; k += blockDim.x * ny) {
    const int t = TOK == 1 ? 0 : k / half, p = k - t * half;
    float c, s;
    rope_cs(r.turn[p], r.pos[tok0 + t], r.gain, c, s);
    cs[t][cs_at<VE, INTER>(p)] = make_float2(c, s);
  }
  __syncthreads();
  // vectors 0 .. turned - 1 of a head are turned, the rest copies from channel rot on
  const bool turn = v < turned;
  const int c = INTER || turn ? v * VE : r.rot + (v - turned) * VE;
  const int hq = r.t[0].heads, heads = hq + r.t[1].heads;
  // this thread's units: (token, head) pairs in steps of ny (and of all gridDim.y CTAs of a token)
  const int stride = ny * gridDim.y, dt = stride / heads, dh = stride % heads;
  int t = 0, h = blockIdx.y * ny + threadIdx.y;
  if (h >= heads) { t = h / heads; h %= heads; }
  while (t < n) {
    V a[kUnroll], b[kUnroll];
    T* y[kUnroll];
    int tok[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      tok[k] = t;
      if (t < n) {
        const RopeTensor& z = r.t[h >= hq];
        const int hz = h >= hq ? h - hq : h;
        const T* x = static_cast<const T*>(z.x) + (size_t)(tok0 + t) * z.x_tok + (size_t)hz * z.x_head + c;
        y[k] = static_cast<T*>(z.y) + (size_t)(tok0 + t) * z.y_tok + (size_t)hz * z.y_head + c;
        a[k] = *reinterpret_cast<const V*>(x);
        if (!INTER && turn) b[k] = *reinterpret_cast<const V*>(x + half);
      }
      t += dt;
      h += dh;
      if (h >= heads) { h -= heads; ++t; }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (tok[k] >= n) continue;
      if (turn) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 w = cs[tok[k]][e * (kRopeMaxPairs / P) + v];
          T& f = INTER ? a[k].v[2 * e] : a[k].v[e];
          T& s = INTER ? a[k].v[2 * e + 1] : b[k].v[e];
          const float xf = to_f32<T>(f), xs = to_f32<T>(s);
          f = T(rope_first(xf, xs, w.x, w.y));
          s = T(rope_second(xf, xs, w.x, w.y));
        }
        if (!INTER) *reinterpret_cast<V*>(y[k] + half) = b[k];
      }
      *reinterpret_cast<V*>(y[k]) = a[k];
    }
  }
}

template <typename T, int VE, bool INTER>
cudaError_t launch_t(const RopeLaunch& a, int sm_count, cudaStream_t st) {
  const int turned = INTER ? a.rot / VE : a.rot / 2 / VE;
  const int per_head = turned + (a.head_dim - a.rot) / VE, heads = a.t[0].heads + a.t[1].heads;
  // few tokens: one token a CTA, its heads spread over gridDim.y; otherwise four a CTA
  if (a.n_tok < 4 * sm_count) {
    const int ny = std::max(1, std::min(heads, 128 / per_head));
    const unsigned gy = (unsigned)std::min((heads + kUnroll * ny - 1) / (kUnroll * ny), 64);
    rope_kernel<T, VE, INTER, 1><<<dim3((unsigned)a.n_tok, gy), dim3((unsigned)per_head, (unsigned)ny), 0, st>>>(a, turned);
  } else {
    const int ny = std::max(1, kMaxThreads / per_head);
    rope_kernel<T, VE, INTER, 4><<<dim3((unsigned)((a.n_tok + 3) / 4)), dim3((unsigned)per_head, (unsigned)ny), 0, st>>>(a, turned);
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
