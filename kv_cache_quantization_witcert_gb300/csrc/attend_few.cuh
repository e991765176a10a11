// Chunk attention for few query rows, straight from the compressed store: the tiles' operand images
// are made in shared memory, read once and never stored.  Templates; each scheme instantiates them
// in its own translation unit (attend_few_<scheme>.cu), so the build compiles them in parallel.
//
// A unit is 128 query rows of one KV head, or 32 where no sequence has more (TINY); the CTAs' shares
// and records are those of attend.cuh.  Bound by HBM as far as the stages around the MMAs keep up:
// the codes of a tile, about 37 KB, arrive in 830 ns at an SM's share of HBM.
//   warp 0    one bulk copy per 16-token block into a ring of half tiles (codes as they lie)
//   warp 1    MMAs: S = Q K^T with Q in tensor memory, O += P V with P in tensor memory: only the
//             images are read from shared memory
//   warp 2    tensor memory: S twice (even and odd tiles), O, Q
//   softmax   (attend.cuh) general: warps 4..11, two threads a row, warps whose rows are all past the
//             end only keep the barriers going; TINY: warps 4, 8, 12, 16, four threads a row
//   images    sixteen warps, eight for the keys and eight for the values, each with two of a tile's
//             blocks and half of their channels (expand.cuh).  General: warps 12..27; TINY: the other
//             warps of 5..23
// The rows of TINY lie in the first 32 lanes of tensor memory, which only warps 0 mod 4 reach: all
// its softmax runs on one scheduler of the SM, whose other warps would slow its chain down (general
// kernel with 32 rows: 3100 cycles a tile, all of them the softmax's), so the images are made on
// the other three (one warp but).  The general softmax needs more registers than an even split gives, and its
// warpgroups trade them: launched with 72 a thread, 504 a lane of the seven groups; 40 + 2 x 96 +
// 4 x 64 = 488.
// Two S buffers let S(j + 1) be formed while P(j) is; O += P V(j) follows S(j + 1), so a softmax warp
// that must rescale O waits for it, and a row's threads swap through alternate words (S(j + 1) says
// nothing about the partners' P(j)).  Images live in 32 KB stages, two for keys and one or two for
// values: what is left of shared memory is the ring of codes, whose size bounds the bytes in flight
// (FP8: four half tiles 4.9 TB/s).
#pragma once
#include "attend.cuh"
#include "expand.cuh"

namespace witcert {

namespace {

constexpr int kHalfBlocks = kTileTok / kBlk / 2;           // blocks of a half tile
template <int SCH, bool TINY> struct FewSmem {
  static constexpr int kThreads = TINY ? 768 : 896;
  static constexpr int kN = TINY ? 4 : 2;                  // threads a row
  static constexpr int kSoftWarps = TINY ? 4 : 8;
  static constexpr int kHalf = kHalfBlocks * block_bytes(SCH);
  // a second value stage costs the one-byte stores a third of their ring
  static constexpr int kVStages = SCH == kKivi || SCH == kBbox ? 2 : 1, kImages = 2 + kVStages;
  // half tiles of codes in flight: what fits beside the images, at most eight
  static constexpr int kScratch = SCH == kInt8 ? 8 * kXwWords * 4 : 0;
  static constexpr int kRoom = 232448 - kImages * kTileBytes - kScratch - 2 * kN * kTileRows * 4 - 512;
  // (an even number, so that a stage always holds the same half and the same warps see its every use)
  static constexpr int kRing = kRoom / kHalf < 8 ? kRoom / kHalf / 2 * 2 : 8;
  static constexpr int kRaw = kImages * kTileBytes;
  static constexpr int kXs = kRaw + kRing * kHalf;
  static constexpr int kSwap = kXs + kScratch;
  static constexpr int kBar = kSwap + 2 * kN * kTileRows * 4;
  static constexpr int kBytes = kBar + 512;
  static_assert(kRing >= 2 && kHalf % 16 == 0, "two half tiles at least");
};

template <int SCH, bool TINY>
__global__ void __launch_bounds__(FewSmem<SCH, TINY>::kThreads, 1) attend_few_kernel(const __grid_constant__ AttendArgs a) {
  using L = FewSmem<SCH, TINY>;
  constexpr int N = L::kN;
  constexpr bool BF16 = SCH == kBbox;
  constexpr int kRing = L::kRing;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t base = smem_addr(sm), bars = base + L::kBar;
  const uint32_t q_full = bars, raw_full = bars + 8, raw_empty = raw_full + 8 * kRing, img_full = raw_empty + 8 * kRing;
  const uint32_t img_empty = img_full + 8 * L::kImages, s_full = img_empty + 8 * L::kImages, p_full = s_full + 16;
  const uint32_t pv_done = p_full + 32, o_full = pv_done + 8, pairs = o_full + 8, drain = pairs + 32, slot = drain + 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    mbar_init(q_full, L::kSoftWarps);
    for (int s = 0; s < kRing; ++s) { mbar_init(raw_full + 8 * s, 1); mbar_init(raw_empty + 8 * s, 8); }
    for (int s = 0; s < L::kImages; ++s) { mbar_init(img_full + 8 * s, 8); mbar_init(img_empty + 8 * s, 1); }
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full + 8 * b, 1);
      mbar_init(p_full + 16 * b, L::kSoftWarps);
      mbar_init(p_full + 16 * b + 8, L::kSoftWarps);
    }
    mbar_init(pv_done, 1);
    mbar_init(o_full, 1);
    for (int x = 0; x < 4; ++x) mbar_init(pairs + 8 * x, N);
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 2) tmem_alloc<512>(slot);
  pdl_wait();                                              // the dither, or whatever came before the call
  if (a.cut) pdl_trigger();                                // a call's last kernel lets nothing start early
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *reinterpret_cast<const uint32_t*>(sm + L::kBar + (slot - bars));
  const uint32_t tmem_o = tm + 256, tmem_q = tm + 384;
  bool dead = (base & 1023u) != 0;                         // a wait ran out (or no aligned tiles): give up, in order

  auto produce = [&]() {
    // lane b < 4 copies block b of the half tile
    RingAt<kRing> at;
    int filled = 0;
    walk(a, cta, [&](const Segment& u) {
      const int i = a.seq[u.k], nblk = (a.len[u.k] + kBlk - 1) / kBlk;
      for (int hb = 2 * u.j0; hb < 2 * (u.j0 + u.nk); ++hb) {
        if (filled >= kRing && !warp_wait(raw_empty + 8 * at.st, at.ph ^ 1)) { dead = true; return false; }
        const int blk0 = hb * kHalfBlocks, n = min(max(nblk - blk0, 0), kHalfBlocks);
        if (lane == 0) mbar_expect_tx(raw_full + 8 * at.st, n * block_bytes(SCH));
        __syncwarp();
        if (lane < n)
          bulk_g2s(base + L::kRaw + at.st * L::kHalf + lane * block_bytes(SCH),
                   a.s.blocks + block_index(a.s.table, a.s.Hkv, a.s.nblk_max, i, u.h, blk0 + lane) * block_bytes(SCH),
                   block_bytes(SCH), raw_full + 8 * at.st);
        at.next();
        ++filled;
      }
      return true;
    });
    // giving up: the copies in flight still land in this CTA's shared memory
    if (dead)
      for (int f = max(0, filled - kRing); f < filled; ++f) bar_wait(raw_full + 8 * (f % kRing), (f / kRing) & 1);
  };
  auto multiply = [&]() {
    constexpr uint32_t idesc = mma_idesc(BF16, kTileRows, kTileTok);
    int tiles = 0, done = 0;                               // of this CTA; tiles whose keys were taken
    uint32_t seg = 0;
    walk(a, cta, [&](const Segment& u) { tiles += u.nk; return true; });
    // tile j's keys are in stage j mod 2, its values in stage 2 + j mod kVStages; the barriers tell
    // visits apart by parity, and a stage that is not filled again needs no release
    auto k_stage = [&](int j) { return j & 1; };
    auto v_stage = [&](int j) { return 2 + j % L::kVStages; };
    auto image = [&](int st) { return base + st * kTileBytes; };
    auto release = [&](int st, int next) { if (next < tiles) warp_commit(img_empty + 8 * st); };
    auto qk = [&](int j) {                                 // tile j of this CTA
      if (!warp_wait(img_full + 8 * k_stage(j), (j >> 1) & 1)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t kd = sw128_desc(image(k_stage(j)));
#pragma unroll
        for (int x = 0; x < 8; ++x)
          mma_ts(tm + (j & 1) * 128, tmem_q + x * 8, kd + (uint64_t)(x >> 2) * (kTileRows * 128 >> 4) + (x & 3) * 2, idesc, x > 0);
        mma_commit(s_full + 8 * (j & 1));
      }
      __syncwarp();
      release(k_stage(j), j + 2);
      return true;
    };
    walk(a, cta, [&](const Segment& u) {
      dead = !warp_wait(q_full, seg++ & 1);
      if (dead) return false;
      tc_fence_after();
      dead = !qk(done);
      if (dead) return false;
      for (int s = 0; s < u.nk; ++s) {
        const int j = done + s;
        if (s + 1 < u.nk) dead = !qk(j + 1);
        dead = dead || !warp_wait(img_full + 8 * v_stage(j), (j / L::kVStages) & 1) ||
               !issue_pv<N>(tmem_o, tm + (j & 1) * 128, sw128_desc(image(v_stage(j))), idesc, s == 0, p_full + 16 * (j & 1), (j >> 1) & 1);
        if (dead) return false;
        warp_commit(s + 1 < u.nk ? pv_done : o_full);
        release(v_stage(j), j + L::kVStages);
      }
      done += u.nk;
      return true;
    });
    if (dead) {                                            // the MMAs in flight still use this CTA's memories
      warp_commit(drain);
      bar_wait(drain, 0);
    }
  };
  auto softmax = [&](int part) {
    constexpr int kCols = 128 / N;
    const int r = (warp & 3) * 32 + lane;
    RowGroup<N> grp{reinterpret_cast<float*>(sm + L::kSwap) + r, part, N * kTileRows, pairs + 8 * (warp & 3), 0, true};
    const uint32_t lanes = (uint32_t)(warp & 3) << 21, to = tmem_o + lanes + kCols * part;
    int j = 0;                                             // tiles of this CTA so far
    uint32_t seg = 0, sums = 0;                            // segments so far; their products that were not the last
    walk(a, cta, [&](const Segment& u) {
      const int row = u.r0 + r;
      const bool busy = u.r0 + (warp & 3) * 32 < u.rows;   // some row of the warp is a query
      float scale = 0.f, m = -INFINITY, l = 0.f;
      if (busy) {
        uint32_t qw[64 / N];
        scale = query_words<BF16, N>(a, u, row, qw, grp);
#pragma unroll
        for (int c = 0; c < 64 / N; c += 16)
          tmem_st16(tmem_q + lanes + (64 / N) * part + c, *reinterpret_cast<uint32_t(*)[16]>(qw + c));
        tmem_wait_st();
      }
      tc_fence_before();
      warp_arrive(q_full);
      // last key this row sees (-1: a row past the end)
      const int limit = row < u.rows ? a.len[u.k] - a.n[u.k] + row / a.grp : -1;
      for (int s = 0; s < u.nk; ++s, ++j) {
        const uint32_t ts = tm + (j & 1) * 128 + lanes, pb = p_full + 16 * (j & 1);
        if (!grp.ok || !warp_wait(s_full + 8 * (j & 1), (j >> 1) & 1)) { dead = true; return false; }
        tc_fence_after();
        if (busy) {
          softmax_tile<BF16, N>(ts + kCols * part, ts + kCols / 2 * part, to, limit - (u.j0 + s) * kTileTok, s == 0, scale, m, l,
                                grp, pb, [&] { grp.ok = grp.ok && warp_wait(pv_done, (sums - 1) & 1); tc_fence_after(); });
        } else {
          warp_arrive(pb);
          warp_arrive(pb + 8);
        }
        sums += s + 1 < u.nk;
      }
      // a barrier of its own: the products before the last may be two phases behind, which a parity
      // does not tell
      if (!warp_wait(o_full, seg++ & 1)) { dead = true; return false; }
      tc_fence_after();
      if (busy) {
        l = grp.sum(l);
        store_row<N>(a, u, row, part, to, m, l, scale, grp.ok);
        tc_fence_before();
      }
      dead = !grp.ok;
      return !dead;
    });
  };
  // One of the sixteen warps that make images.
  auto expand = [&](int e) {
    const int values = e >> 3, half = (e >> 2) & 1, j0 = 2 * (e & 1);
    BlockPair x;
    x.lane = lane;
    x.pr = (e >> 1) & 3;
    [[maybe_unused]] uint32_t* xs = reinterpret_cast<uint32_t*>(sm + L::kXs) + (e & 7) * kXwWords;
    RingAt<kRing / 2> at;                                  // the tile's halves: stages 2 at.st and + 1
    const int stages = values ? L::kVStages : 2;
    int made = 0, in = 0;                                  // tiles so far; this tile's stage among them
    uint32_t ph = 0;
    walk(a, cta, [&](const Segment& u) {
      x.h = u.h;
      x.len = a.len[u.k];
      for (int j = u.j0; j < u.j0 + u.nk; ++j, ++made) {
        const int raw_st = 2 * at.st + half, st = 2 * values + in;
        x.tb = j * kTileTok + x.pr * 2 * kBlk;
        x.bp[0] = sm + L::kRaw + raw_st * L::kHalf + (x.pr & 1) * 2 * block_bytes(SCH);
        x.bp[1] = x.bp[0] + block_bytes(SCH);
        // the codes leave the ring as soon as they are in registers, before this tile's stage is free
        auto got = [&] { warp_arrive(raw_empty + 8 * raw_st); };
        auto ready = [&] { return made < stages || warp_wait(img_empty + 8 * st, ph ^ 1); };
        dead = !warp_wait(raw_full + 8 * raw_st, at.ph);
        if (dead) return false;
        if (values) {
          dead = !expand_values<SCH>(a.s, x, j0, xs, sm + st * kTileBytes, got, ready);
        } else {
          find_exact<SCH>(a.s, a.seq[u.k], x);
          dead = !expand_keys<SCH>(a.s, x, j0, sm + st * kTileBytes, got, ready);
        }
        if (dead) return false;
        fence_proxy_async();
        warp_arrive(img_full + 8 * st);
        at.next();
        if (++in == stages) { in = 0; ph ^= 1; }
      }
      return true;
    });
  };

  if (dead) {
  } else if (TINY) {
    if (warp == 0) produce();
    else if (warp == 1) multiply();
    else if (warp >= 4 && warp < 20 && (warp & 3) == 0) softmax((warp - 4) >> 2);
    else if (warp >= 4) expand(warp < 20 ? 3 * ((warp - 4) >> 2) + (warp & 3) - 1 : warp - 8);
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
    if (warp == 0) produce();
    else if (warp == 1) multiply();
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 96;\n");
    softmax((warp - 4) >> 2);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    expand(warp - 12);
  }
  if (dead) atomicAdd(a.err, 1);
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_free<512>(tm);
  }
}

}  // namespace

template <int SCH, bool TINY>
cudaError_t launch_few(const AttendArgs& a, cudaStream_t st) {
  using L = FewSmem<SCH, TINY>;
  cudaError_t e = cudaFuncSetAttribute(attend_few_kernel<SCH, TINY>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  return launch_after(attend_few_kernel<SCH, TINY>, dim3((unsigned)a.n_ctas), L::kThreads, L::kBytes, st, a);
}

template <int SCH>
cudaError_t launch_attend_few(const AttendArgs& a, cudaStream_t st) {
  return a.unit_rows == kTinyRows ? launch_few<SCH, true>(a, st) : launch_few<SCH, false>(a, st);
}

}  // namespace witcert
