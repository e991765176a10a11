// Chunk attention over the operand images of a compressed cache (expand.cu): out = softmax(q K^T /
// sqrt d) V for the newest tokens of every sequence, token at position p over the keys 0 .. p.
//
// A unit is 256 query rows (two tiles of 128; a row is one head of one token) of one KV head.  One
// CTA an SM works through its share of all units' key tiles (see AttendArgs::start).  Twenty warps:
//   warp 0   copies key and value images into a ring of five 32 KB stages, one bulk copy a tile
//   warp 1   issues the MMAs: S_w = Q_w K^T (operands in shared memory, 128 x 128 fp32 in tensor
//            memory), O_w += P_w V (P from tensor memory over S_w's first columns)
//   warp 2   tensor memory: S_0, S_1, O_0, O_1, 128 columns each, all 512
//   warps 4..11, 12..19   softmax of row tile w (attend.cuh)
// While one group turns S_w into P_w, the tensor cores run the other tile's products.  S_w(j + 1) is
// issued after O_w += P_w V(j), so a softmax group that holds S_w(j + 1) may rescale O_w, and a
// group that holds its last S_w may overwrite Q_w; and every softmax thread's P_w(j) was announced,
// so its partner has read what they swapped for tile j.
//
// The operands are fp16 for the quantized stores (2^-11 rounding of the decoded values; query rows
// are scaled by powers of two) and bf16 for the black-box store, whose values bf16 holds exactly;
// weights round to the same type.  Sums and products accumulate in fp32.  Rows are independent, so a
// row tile may mix tokens; keys past a row's position, and image rows past the sequence's length
// (zero), get weight 0 through a logit of -inf.
#include "attend.cuh"

namespace witcert {

namespace {

constexpr int kThreads = 640;
constexpr int kStages = 5;
constexpr int kSmemQ = 0, kSmemKV = 2 * kTileBytes, kSmemSwap = kSmemKV + kStages * kTileBytes;
constexpr int kSmemBar = kSmemSwap + 2 * 2 * kTileRows * 4, kSmemBytes = kSmemBar + 256;

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t base = smem_addr(sm), sq = base + kSmemQ, skv = base + kSmemKV, bars = base + kSmemBar;
  const uint32_t q_full = bars, full = bars + 8, empty = full + 8 * kStages, s_full = empty + 8 * kStages;
  const uint32_t p_full = s_full + 16, o_full = p_full + 32, pairs = o_full + 16, drain = pairs + 64, slot = drain + 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  // row tiles of a segment
  auto row_tiles = [&](const Segment& u) { return u.rows - u.r0 > kTileRows ? 2 : 1; };

  if (threadIdx.x == 0) {
    mbar_init(q_full, 16);
    for (int s = 0; s < kStages; ++s) { mbar_init(full + 8 * s, 1); mbar_init(empty + 8 * s, 1); }
    for (int w = 0; w < 2; ++w) {
      mbar_init(s_full + 8 * w, 1);
      mbar_init(p_full + 16 * w, 8);
      mbar_init(p_full + 16 * w + 8, 8);
      mbar_init(o_full + 8 * w, 1);
    }
    for (int x = 0; x < 8; ++x) mbar_init(pairs + 8 * x, 2);
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 2) tmem_alloc<512>(slot);
  pdl_wait();                                              // the images
  if (a.cut) pdl_trigger();                                // a call's last kernel lets nothing start early
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *reinterpret_cast<const uint32_t*>(sm + kSmemBar + (slot - bars));
  bool dead = (base & 1023u) != 0;                         // a wait ran out (or no aligned tiles): give up, in order

  if (warp == 0) {
    if (lane == 0 && !dead) {
      const size_t stride = (size_t)a.s.Hkv * 2 * kTileBytes;
      int idx = 0;
      walk(a, cta, [&](const Segment& u) {
        const uint8_t* img = a.images + ((size_t)(a.tile_off[u.k] + u.j0) * a.s.Hkv + u.h) * 2 * kTileBytes;
        // keys and values of a tile in turn
        for (int t = 0; t < 2 * u.nk && !dead; ++t, ++idx) {
          const int st = idx % kStages;
          if (idx >= kStages && !bar_wait(empty + 8 * st, (idx / kStages - 1) & 1)) { dead = true; break; }
          mbar_expect_tx(full + 8 * st, kTileBytes);
          bulk_g2s(skv + st * kTileBytes, img + (size_t)(t >> 1) * stride + (t & 1) * kTileBytes, kTileBytes, full + 8 * st);
        }
        return !dead;
      });
      // giving up: the copies in flight still land in this CTA's shared memory
      if (dead)
        for (int i = max(0, idx - kStages); i < idx; ++i) bar_wait(full + 8 * (i % kStages), (i / kStages) & 1);
    }
  } else if (warp == 1) {
    if (!dead) {
      constexpr uint32_t idesc = mma_idesc(BF16, kTileRows, kTileTok);
      int left = 0;                                        // images not taken yet
      uint32_t seg = 0, steps[2] = {0, 0};
      RingAt<kStages> at;
      walk(a, cta, [&](const Segment& u) { left += 2 * u.nk; return true; });
      auto take = [&](uint32_t& st) {                      // the next image's stage, in load order
        st = at.st;
        const bool ok = warp_wait(full + 8 * at.st, at.ph);
        at.next();
        --left;
        return ok;
      };
      // stage st is free when the MMAs so far are done; `after` images were taken since (the
      // producer waits only for stages that it fills again)
      auto release = [&](uint32_t st, int after) { if (left + after >= kStages) warp_commit(empty + 8 * st); };
      auto qk = [&](int w, uint32_t st) {
        issue_qk(tm + w * 128, sw128_desc(sq + w * kTileBytes), sw128_desc(skv + st * kTileBytes), idesc, s_full + 8 * w);
      };
      auto pv = [&](int w, uint32_t st, bool first) {
        return issue_pv<2>(tm + 256 + w * 128, tm + w * 128, sw128_desc(skv + st * kTileBytes), idesc, first,
                        p_full + 16 * w, steps[w]++ & 1);
      };
      walk(a, cta, [&](const Segment& u) {
        const bool two = row_tiles(u) == 2;
        uint32_t vs, ks;
        dead = !warp_wait(q_full, seg++ & 1) || !take(ks);
        if (dead) return false;
        tc_fence_after();
        qk(0, ks);
        if (two) qk(1, ks);
        release(ks, 0);
        for (int s = 0; s < u.nk; ++s) {
          const bool more = s + 1 < u.nk;
          dead = !take(vs) || !pv(0, vs, s == 0);
          if (dead) return false;
          if (more) {
            dead = !take(ks);
            if (dead) return false;
            qk(0, ks);
          } else {
            warp_commit(o_full);
          }
          if (two) {
            dead = !pv(1, vs, s == 0);
            if (dead) return false;
            if (more) qk(1, ks);
            else warp_commit(o_full + 8);
          }
          release(vs, more ? 1 : 0);
          if (more) release(ks, 0);
        }
        return true;
      });
      if (dead) {                                          // the MMAs in flight still use this CTA's memories
        warp_commit(drain);
        bar_wait(drain, 0);
      }
    }
  } else if (warp >= 4 && !dead) {
    const int w = (warp - 4) >> 3, hf = ((warp - 4) >> 2) & 1, r = (warp & 3) * 32 + lane;
    RowGroup<2> pair{reinterpret_cast<float*>(sm + kSmemSwap) + w * 2 * kTileRows + r, hf, 0,
                     pairs + 8 * (w * 4 + (warp & 3)), 0, true};
    const uint32_t lanes = tm + ((uint32_t)(warp & 3) << 21) + w * 128;
    const uint32_t ts = lanes + 64 * hf, tp = lanes + 32 * hf, to = lanes + 256 + 64 * hf;
    uint32_t seg = 0, step = 0, done = 0;
    walk(a, cta, [&](const Segment& u) {
      const bool mine = w < row_tiles(u);
      const int row = u.r0 + w * kTileRows + r;
      float scale = 0.f;
      if (mine) {
        uint32_t qw[32];
        scale = query_words<BF16, 2>(a, u, row, qw, pair);
        uint8_t* q = sm + kSmemQ + w * kTileBytes + hf * (kTileRows * 128) + r * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(q + ((c ^ (r & 7)) << 4)) = make_uint4(qw[4 * c], qw[4 * c + 1], qw[4 * c + 2], qw[4 * c + 3]);
        fence_proxy_async();
      }
      warp_arrive(q_full);
      // a group without rows must not run ahead into the next segment's phase
      if (!mine) {
        dead = !warp_wait(q_full, seg++ & 1);
        return !dead;
      }
      ++seg;
      // last key this row sees (-1: a row past the end)
      const int limit = row < u.rows ? a.len[u.k] - a.n[u.k] + row / a.grp : -1;
      float m = -INFINITY, l = 0.f;                        // reference in units of s, sum of weights
      for (int s = 0; s < u.nk; ++s) {
        if (!pair.ok || !warp_wait(s_full + 8 * w, step++ & 1)) { dead = true; return false; }
        tc_fence_after();
        softmax_tile<BF16, 2>(ts, tp, to, limit - (u.j0 + s) * kTileTok, s == 0, scale, m, l, pair, p_full + 16 * w,
                           [] {});                         // S_w(s) is complete, so O_w += P_w V(s - 1) is
      }
      if (!warp_wait(o_full + 8 * w, done++ & 1)) { dead = true; return false; }
      tc_fence_after();
      l = pair.sum(l);
      store_row<2>(a, u, row, hf, to, m, l, scale, pair.ok);
      pair.sync();                                         // the partner has read l
      dead = !pair.ok;
      return !dead;
    });
  }
  if (dead) atomicAdd(a.err, 1);
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_free<512>(tm);
  }
}

// Records of the units that cross CTAs joined: out = sum 2^(m - M) O / sum 2^(m - M) l.  Block row
// blockIdx.y takes the unit that CTA c = blockIdx.y starts without finishing (its slot 2c + 1, then
// the slots 2c' of the CTAs that go on).  Bound by latency: a warp joins R rows of two parts at once,
// all their loads in flight together (units of 256 rows mostly have two parts: 35 us with one row a
// warp), or, where units have few rows and many parts, the block's eight warps share a row's parts
// (R = 0).
template <int R>
__global__ void __launch_bounds__(256) attend_merge_kernel(const __grid_constant__ AttendArgs a) {
  pdl_wait();
  const int c0 = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const AttendStart here = a.start[c0], next = a.start[c0 + 1];
  if (next.j == 0) return;                                 // the CTA ends on a unit's end
  if (same_unit(here, next) && here.j > 0) return;         // a part in the middle
  Segment u;
  int row_tiles;
  unit_place(a, next, u, row_tiles);
  const int r0 = blockIdx.x * (R ? 8 * R : 1) + (R ? warp * R : 0);          // of the unit
  if (u.r0 + r0 >= u.rows) return;
  int n = 2;                                               // parts: consecutive CTAs', two at least
  while (c0 + n < a.n_ctas && same_unit(a.start[c0 + n], next)) ++n;
  const size_t step = (size_t)2 * a.unit_rows * kRecStride;                  // to the next CTA's slot
  auto part = [&](int r, int p) {
    return a.rec + ((size_t)2 * c0 * a.unit_rows + r0 + r) * kRecStride + p * step + (p == 0 ? step / 2 : 0);
  };
  struct Sum {
    float m, l;
    float4 o;
    __device__ __forceinline__ void join(float2 ml, float4 v) {
      const float t = fmaxf(m, ml.x), f = t == -INFINITY ? 0.f : ex2(m - t), g = t == -INFINITY ? 0.f : ex2(ml.x - t);
      l = f * l + g * ml.y;
      o.x = f * o.x + g * v.x; o.y = f * o.y + g * v.y; o.z = f * o.z + g * v.z; o.w = f * o.w + g * v.w;
      m = t;
    }
  };
  auto ml = [&](int r, int p) { return *reinterpret_cast<const float2*>(part(r, p)); };
  auto sums = [&](int r, int p) { return *reinterpret_cast<const float4*>(part(r, p) + 8 + 4 * lane); };
  auto store = [&](int r, const Sum& x) {
    const int row = u.r0 + r0 + r;
    const float inv = 1.0f / x.l;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) +
                              ((size_t)(a.row0[u.k] + row / a.grp) * a.Hq + u.h * a.grp + row % a.grp) * kD + 4 * lane) =
        make_uint2(pack2<true>(x.o.x * inv, x.o.y * inv), pack2<true>(x.o.z * inv, x.o.w * inv));
  };
  if constexpr (R > 0) {
    const int rows = min(R, u.rows - u.r0 - r0);
    float2 m[R][2];
    float4 v[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (r < rows) { m[r][p] = ml(r, p); v[r][p] = sums(r, p); }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r < rows) {
        Sum x{m[r][0].x, m[r][0].y, v[r][0]};
        x.join(m[r][1], v[r][1]);
        for (int p = 2; p < n; ++p) x.join(ml(r, p), sums(r, p));
        store(r, x);
      }
  } else {
    __shared__ float sm[8][kRecStride];
    Sum x{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 4
    for (int p = warp; p < n; p += 8) x.join(ml(0, p), sums(0, p));
    if (lane == 0) { sm[warp][0] = x.m; sm[warp][1] = x.l; }
    *reinterpret_cast<float4*>(&sm[warp][8 + 4 * lane]) = x.o;
    __syncthreads();
    if (warp) return;
    for (int w = 1; w < 8; ++w)
      x.join(make_float2(sm[w][0], sm[w][1]), *reinterpret_cast<const float4*>(&sm[w][8 + 4 * lane]));
    store(0, x);
  }
}

template <bool BF16>
cudaError_t launch_t(const AttendArgs& a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_after(attend_kernel<BF16>, dim3((unsigned)a.n_ctas), kThreads, kSmemBytes, st, a);
}

}  // namespace

cudaError_t launch_attend(int scheme, const AttendArgs& a, cudaStream_t st) {
  return scheme == kBbox ? launch_t<true>(a, st) : launch_t<false>(a, st);
}

cudaError_t launch_attend_merge(const AttendArgs& a, cudaStream_t st) {
  if (!a.cut) return cudaSuccess;
  const unsigned cuts = (unsigned)(a.n_ctas - 1);
  return a.unit_rows > kTinyRows ? launch_after(attend_merge_kernel<4>, dim3((unsigned)(a.unit_rows / 32), cuts), 256, 0, st, a)
                                 : launch_after(attend_merge_kernel<0>, dim3((unsigned)a.unit_rows, cuts), 256, 0, st, a);
}

}  // namespace witcert
