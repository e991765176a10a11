// Chunk attention over the operand images of a compressed cache: out = softmax(q K^T / sqrt d) V
// for the newest tokens of every sequence, token at position p over the keys 0 .. p.
//
// A CTA owns 256 query rows (two tiles of 128; a row is one head of one token) of one KV head and
// a run of its key tiles, or, for sequences with at most 128 rows, one row tile whose two softmax
// groups take alternate key tiles (pair).  Twelve warps:
//   warp 0   copies key and value images into a ring of five 32 KB stages, one bulk copy a tile
//   warp 1   issues the MMAs: S_w = Q_w K^T (operands in shared memory, 128 x 128 fp32 in tensor
//            memory), O_w += P_w V (P from tensor memory over S_w's first columns)
//   warp 2   tensor memory: S_0, S_1, O_0, O_1, 128 columns each, all 512
//   warps 4..7, 8..11   softmax of row tile (pair: key-tile parity) w, a query row a thread
// While one group turns S_w into P_w, the tensor cores run the other tile's products.
//
// Softmax: weights 2^(s c - m + kOff) with the row's reference m in log2 units.  m follows the
// running maximum only when that has grown by more than kGrow, so O and the sum l are rescaled
// rarely, by the softmax warp itself (its S_w is complete only after the last O_w += P_w V, which
// was issued before it).  kOff keeps the small weights of fp16 normal: weights reach 2^15 at most,
// and those below 2^-23 of the reference (2^-33 before they vanish) lose bits.  The operands are fp16
// (2^-12) for the quantized stores, with every query row scaled by a power of two to a largest
// element in [1, 2), and bf16 for the black-box store, whose values bf16 holds exactly; weights
// round to the same type.  Sums and products accumulate in fp32.
//
// Rows are independent, so a row tile may mix tokens; keys past a row's position, and image rows
// past the sequence's length (zero), get weight 0 through a logit of -inf.
#include "kernels.h"
#include "tcgen05.cuh"

namespace witcert {

namespace {

constexpr int kThreads = 384;
constexpr int kStages = 5;
constexpr int kSmemQ = 0, kSmemKV = 2 * kTileBytes, kSmemBar = kSmemKV + kStages * kTileBytes;
constexpr int kSmemBytes = kSmemBar + 256 + 1024;          // barriers; slack for the 1024-byte alignment
constexpr float kOff = 8.0f, kGrow = 7.0f;
constexpr uint64_t kWaitNs = 2000000000ull;                // 2 s per barrier wait

// What this CTA does.
struct Unit {
  int k, h, r0, rows, row_tiles, part0, parts, j0, nk;
};
template <bool PAIR>
__device__ __forceinline__ Unit unit_of(const AttendArgs& a, int u) {
  Unit x;
  int lo = 0, hi = a.n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.unit_off[mid] <= u) lo = mid; else hi = mid - 1;
  }
  x.k = lo;
  u -= a.unit_off[lo];
  constexpr int kRows = PAIR ? kTileRows : 2 * kTileRows;
  x.rows = a.n[lo] * a.grp;
  const int tiles = (x.rows + kRows - 1) / kRows, splits = a.splits[lo];
  x.h = u % a.s.Hkv;
  u /= a.s.Hkv;
  const int sp = u % splits;
  x.r0 = (tiles - 1 - u / splits) * kRows;                 // last rows, which see most keys, first
  const int last = min(x.rows, x.r0 + kRows) - 1;
  x.row_tiles = PAIR ? 2 : (last - x.r0) / kTileRows + 1;
  const int nt = (a.len[lo] - a.n[lo] + last / a.grp) / kTileTok + 1;
  x.j0 = (int)((long long)nt * sp / splits);
  x.nk = (int)((long long)nt * (sp + 1) / splits) - x.j0;
  x.parts = splits * (PAIR ? 2 : 1);
  x.part0 = sp * (PAIR ? 2 : 1);
  return x;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return BF16 ? bf2_bits(__floats2bfloat162_rn(a, b)) : h2_bits(__floats2half2_rn(a, b));
}

// One query row into the swizzled operand tile; returns log2(e)/sqrt(d) times the power of two that
// the row was divided by.
template <bool BF16>
__device__ __forceinline__ float stage_query(const AttendArgs& a, const Unit& u, int row, int r, uint8_t* tile) {
  uint4 v[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) v[c] = make_uint4(0, 0, 0, 0);
  if (row < u.rows) {
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(a.q) +
        ((size_t)(a.row0[u.k] + row / a.grp) * a.Hq + u.h * a.grp + row % a.grp) * kD);
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] = src[c];
  }
  float scale = a.scale_log2;
  if (!BF16) {
    uint32_t top = 0;                                     // largest magnitude's bits, two lanes of bf16
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7FFF7FFFu);
    }
    // biased exponent of the row's largest element, kept where 2^-e and 2^e are normal numbers
    const int e = min(max((int)(max(top & 0xFFFFu, top >> 16) >> 7), 16), 238) - 127;
    const float down = __int_as_float((127 - e) << 23);
    scale *= __int_as_float((127 + e) << 23);
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      uint32_t* w = &v[c].x;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = pack2<false>(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xFFFF0000u) * down);
    }
  }
  if (tile) {
#pragma unroll
    for (int c = 0; c < 16; ++c)
      *reinterpret_cast<uint4*>(tile + (c >> 3) * (kTileRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v[c];
  }
  return scale;
}

template <bool BF16, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  const uint32_t sq = smem_addr(sm) + kSmemQ, skv = smem_addr(sm) + kSmemKV, bars = smem_addr(sm) + kSmemBar;
  const uint32_t q_full = bars, full = bars + 8, empty = full + 8 * kStages, s_full = empty + 8 * kStages;
  const uint32_t p_full = s_full + 16, o_full = p_full + 16, drain = o_full + 16, slot = drain + 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Unit u = unit_of<PAIR>(a, blockIdx.x);
  // key tiles of each softmax group
  const int steps[2] = {PAIR ? (u.nk + 1) / 2 : u.nk, PAIR ? u.nk / 2 : u.row_tiles > 1 ? u.nk : 0};
  const int loads = 2 * u.nk;

  if (threadIdx.x == 0) {
    mbar_init(q_full, PAIR ? kTileRows : u.row_tiles * kTileRows);
    for (int s = 0; s < kStages; ++s) { mbar_init(full + 8 * s, 1); mbar_init(empty + 8 * s, 1); }
    for (int w = 0; w < 2; ++w) { mbar_init(s_full + 8 * w, 1); mbar_init(p_full + 8 * w, kTileRows); mbar_init(o_full + 8 * w, 1); }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 2) tmem_alloc<512>(slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *reinterpret_cast<const uint32_t*>(sm + kSmemBar + (slot - bars));
  bool dead = false;                                       // a wait ran out: give up, in order

  if (warp == 0) {
    if (lane == 0) {
      const uint8_t* img = a.images + ((size_t)a.tile_off[u.k] * a.s.Hkv + u.h) * 2 * kTileBytes;
      const size_t stride = (size_t)a.s.Hkv * 2 * kTileBytes;
      int idx = 0;
      auto load = [&](int j, int which) {
        if (dead) return;
        const int st = idx % kStages;
        if (idx >= kStages && !mbar_wait(empty + 8 * st, (idx / kStages - 1) & 1, kWaitNs)) { dead = true; return; }
        mbar_expect_tx(full + 8 * st, kTileBytes);
        bulk_g2s(skv + st * kTileBytes, img + (size_t)(u.j0 + j) * stride + which * kTileBytes, kTileBytes, full + 8 * st);
        ++idx;
      };
      if (PAIR) {
        for (int w = 0; w < 2; ++w) if (steps[w] > 0) load(w, 0);
        for (int s = 0; s < steps[0]; ++s)
          for (int w = 0; w < 2; ++w)
            if (s < steps[w]) {
              load(2 * s + w, 1);
              if (s + 1 < steps[w]) load(2 * s + 2 + w, 0);
            }
      } else {
        if (u.nk > 0) load(0, 0);
        for (int s = 0; s < u.nk; ++s) {
          load(s, 1);
          if (s + 1 < u.nk) load(s + 1, 0);
        }
      }
      // giving up: the copies in flight still land in this CTA's shared memory
      if (dead)
        for (int i = max(0, idx - kStages); i < idx; ++i) mbar_wait(full + 8 * (i % kStages), (i / kStages) & 1, kWaitNs);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = mma_idesc(BF16, kTileRows, kTileTok);
      int idx = 0;
      auto take = [&]() {                                  // the next image, in load order
        const int i = idx++;
        if (!dead && !mbar_wait(full + 8 * (i % kStages), (i / kStages) & 1, kWaitNs)) dead = true;
        return i;
      };
      auto release = [&](int i) { if (i + kStages < loads) mma_commit(empty + 8 * (i % kStages)); };
      auto qk = [&](int w, int i) {
        const uint64_t qd = sw128_desc(sq + (PAIR ? 0 : w) * kTileBytes), kd = sw128_desc(skv + (i % kStages) * kTileBytes);
#pragma unroll
        for (int x = 0; x < 8; ++x) {                      // 16 channels a step, 64 a panel
          const uint64_t o = (uint64_t)(x >> 2) * (kTileRows * 128 >> 4) + (x & 3) * 2;
          mma_ss(tm + w * 128, qd + o, kd + o, idesc, x > 0);
        }
        mma_commit(s_full + 8 * w);
      };
      auto pv = [&](int w, int i, int s) {
        const uint64_t vd = sw128_desc(skv + (i % kStages) * kTileBytes);
        if (!dead && !mbar_wait(p_full + 8 * w, s & 1, kWaitNs)) dead = true;
        if (dead) return;
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 8; ++x) {                      // 16 token places a step
          const uint64_t o = (uint64_t)(x >> 2) * (kD * 128 >> 4) + (x & 3) * 2;
          mma_ts(tm + 256 + w * 128, tm + w * 128 + x * 8, vd + o, idesc, s > 0 || x > 0);
        }
        if (s + 1 == steps[w]) mma_commit(o_full + 8 * w);
      };
      if (u.nk > 0 && !mbar_wait(q_full, 0, kWaitNs)) dead = true;
      tc_fence_after();
      if (PAIR) {
        for (int w = 0; w < 2; ++w)
          if (steps[w] > 0) {
            const int i = take();
            if (!dead) { qk(w, i); release(i); }
          }
        for (int s = 0; s < steps[0] && !dead; ++s)
          for (int w = 0; w < 2 && !dead; ++w)
            if (s < steps[w]) {
              const int i = take();
              pv(w, i, s);
              if (dead) break;
              release(i);
              if (s + 1 < steps[w]) {
                const int n = take();
                if (!dead) { qk(w, n); release(n); }
              }
            }
      } else if (u.nk > 0) {
        int i = take();
        if (!dead) {
          for (int w = 0; w < u.row_tiles; ++w) qk(w, i);
          release(i);
        }
        for (int s = 0; s < u.nk && !dead; ++s) {
          i = take();
          int n = -1;
          for (int w = 0; w < u.row_tiles && !dead; ++w) {
            pv(w, i, s);
            if (s + 1 < u.nk && !dead) {
              if (n < 0) n = take();
              if (!dead) qk(w, n);
            }
          }
          if (!dead) {
            release(i);
            if (n >= 0) release(n);
          }
        }
      }
      if (dead) {                                          // the MMAs in flight still use this CTA's memories
        mma_commit(drain);
        mbar_wait(drain, 0, kWaitNs);
      }
    }
  } else if (warp >= 4) {
    const int w = (warp - 4) >> 2, r = threadIdx.x & 127;
    const int row = u.r0 + (PAIR ? 0 : w * kTileRows) + r;
    const bool mine = PAIR || w < u.row_tiles;
    if (mine) {
      float scale = stage_query<BF16>(a, u, row, r, PAIR && w ? nullptr : sm + kSmemQ + (PAIR ? 0 : w) * kTileBytes);
      if (!(PAIR && w)) {
        fence_proxy_async();
        mbar_arrive(q_full);
      }
      // last key this row sees (-1: a row past the end)
      const int limit = row < u.rows ? a.len[u.k] - a.n[u.k] + row / a.grp : -1;
      const uint32_t ts = tm + ((uint32_t)(warp & 3) << 21) + w * 128, to = ts + 256;
      float m = -INFINITY, l = 0.f;                        // reference in units of s, sum of weights
      for (int s = 0; s < steps[w]; ++s) {
        // the warp gives up together: tensor-memory accesses need all its lanes
        if (__any_sync(0xffffffffu, !mbar_wait(s_full + 8 * w, s & 1, kWaitNs))) { dead = true; break; }
        tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, v[c]);
        tmem_wait_ld();
        const int rel = limit - (u.j0 + (PAIR ? 2 * s + w : s)) * kTileTok;
        if (__any_sync(0xffffffffu, rel < kTileTok - 1)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              // token of place e (see expand.cu)
              const int p = e & 15, tok = 32 * c + (e & 16) + 2 * (p >> 2) + (p & 1) + 8 * ((p >> 1) & 1);
              if (tok > rel) v[c][e] = 0xFF800000u;
            }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = __uint_as_float(v[c][0]);
#pragma unroll
          for (int e = 1; e < 32; ++e) mx[c] = fmaxf(mx[c], __uint_as_float(v[c][e]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const bool grow = (top - m) * scale > kGrow;       // also from -inf; false while nothing is visible
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = grow ? top : m, f = grow ? ex2((m - mn) * scale) : 1.0f;
          l *= f;
          m = mn;
          if (s > 0) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tmem_ld32(to + 32 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(to + 32 * c, o);
            }
          }
        }
        const float bias = kOff - (m == -INFINITY ? 0.f : m * scale);
        const float2 sc2 = make_float2(scale, scale), b2 = make_float2(bias, bias);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[2 * c2 + c][e]), __uint_as_float(v[2 * c2 + c][e + 1])), sc2, b2);
              const float2 p = make_float2(ex2(x.x), ex2(x.y));
              sum = __fadd2_rn(sum, p);
              pk[16 * c + e / 2] = pack2<BF16>(p.x, p.y);
            }
          tmem_st32(ts + 32 * c2, pk);
        }
        l += sum.x + sum.y;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full + 8 * w);
      }
      if (!dead && steps[w] > 0 && __any_sync(0xffffffffu, !mbar_wait(o_full + 8 * w, 0, kWaitNs))) dead = true;
      tc_fence_after();
      const bool store = row < u.rows && !dead;
      const int tokr = row / a.grp;
      float* rec = nullptr;
      __nv_bfloat16* out = nullptr;
      if (u.parts > 1) {
        rec = a.rec + (a.rec_off[u.k] + ((long long)u.h * u.rows + row) * u.parts + u.part0 + (PAIR ? w : 0)) * kRecStride;
        if (store) *reinterpret_cast<float2*>(rec) = make_float2(m == -INFINITY ? m : m * scale, l);
      } else {
        out = static_cast<__nv_bfloat16*>(a.out) + ((size_t)(a.row0[u.k] + tokr) * a.Hq + u.h * a.grp + row % a.grp) * kD;
      }
      const float inv = l > 0.f ? 1.0f / l : l;            // l is 0 only in a part without keys; NaN stays
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (steps[w] > 0) {
          tmem_ld32(to + 32 * c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (store && rec) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(rec + 4 + 32 * c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        } else if (store) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t b[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              b[x] = pack2<true>(__uint_as_float(o[e + 2 * x]) * inv, __uint_as_float(o[e + 2 * x + 1]) * inv);
            *reinterpret_cast<uint4*>(out + 32 * c + e) = make_uint4(b[0], b[1], b[2], b[3]);
          }
        }
        __syncwarp();
      }
    }
  }
  if (dead) atomicAdd(a.err, 1);
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_free<512>(tm);
  }
}

// Records of a row's parts joined: out = sum 2^(m - M) O / sum 2^(m - M) l.  One warp a row.
__global__ void __launch_bounds__(256) attend_merge_kernel(const __grid_constant__ AttendArgs a, int per_split) {
  const int k = blockIdx.y, lane = threadIdx.x & 31;
  const int rows = a.n[k] * a.grp, parts = a.splits[k] * per_split;
  const long long rh = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (parts == 1 || rh >= (long long)rows * a.s.Hkv) return;
  const float* rec = a.rec + (a.rec_off[k] + rh * parts) * kRecStride;
  float top = -INFINITY;
  for (int p = 0; p < parts; ++p) top = fmaxf(top, rec[(size_t)p * kRecStride]);
  if (top == -INFINITY) top = 0.f;
  float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < parts; ++p) {
    const float* r = rec + (size_t)p * kRecStride;
    const float2 ml = *reinterpret_cast<const float2*>(r);
    const float4 v = *reinterpret_cast<const float4*>(r + 4 + 4 * lane);
    const float f = ex2(ml.x - top);
    l = fmaf(f, ml.y, l);
    o[0] = fmaf(f, v.x, o[0]); o[1] = fmaf(f, v.y, o[1]); o[2] = fmaf(f, v.z, o[2]); o[3] = fmaf(f, v.w, o[3]);
  }
  const float inv = 1.0f / l;
  const int h = (int)(rh / rows), row = (int)(rh % rows);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) +
                            ((size_t)(a.row0[k] + row / a.grp) * a.Hq + h * a.grp + row % a.grp) * kD + 4 * lane) =
      make_uint2(pack2<true>(o[0] * inv, o[1] * inv), pack2<true>(o[2] * inv, o[3] * inv));
}

template <bool BF16, bool PAIR>
cudaError_t launch_t(const AttendArgs& a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<BF16, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  attend_kernel<BF16, PAIR><<<(unsigned)a.unit_off[a.n_seq], kThreads, kSmemBytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend(int scheme, const AttendArgs& a, bool pair, cudaStream_t st) {
  if (scheme == kBbox) return pair ? launch_t<true, true>(a, st) : launch_t<true, false>(a, st);
  return pair ? launch_t<false, true>(a, st) : launch_t<false, false>(a, st);
}

cudaError_t launch_attend_merge(const AttendArgs& a, bool pair, cudaStream_t st) {
  long long most = 0;
  for (int k = 0; k < a.n_seq; ++k)
    if (a.splits[k] * (pair ? 2 : 1) > 1) most = most > (long long)a.n[k] * a.grp * a.s.Hkv ? most : (long long)a.n[k] * a.grp * a.s.Hkv;
  if (most == 0) return cudaSuccess;
  attend_merge_kernel<<<dim3((unsigned)((most + 7) / 8), (unsigned)a.n_seq), 256, 0, st>>>(a, pair ? 2 : 1);
  return cudaGetLastError();
}

}  // namespace witcert
