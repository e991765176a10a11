// Chunk attention for few query rows, straight from the compressed store: the tiles' operand images
// are made in shared memory, read once and never stored.  Templates; each scheme instantiates them
// in its own translation unit (attend_few_<scheme>.cu), so the build compiles them in parallel.
//
// A unit is 128 query rows of one KV head; the CTAs' shares and records are those of attend.cuh.
// Bound by HBM: the codes of every tile are read once per row tile, so the stages around the MMAs
// only have to keep up with about 37 KB a tile (830 ns at an SM's share of HBM).  Twenty warps:
//   warp 0       one bulk copy per 16-token block into a ring of half tiles (codes as they lie)
//   warp 1       MMAs: S = Q K^T with Q in tensor memory, O += P V with P in tensor memory: only
//                the images are read from shared memory
//   warp 2       tensor memory: S twice (even and odd tiles), O, Q
//   warps 4..11  softmax, two threads a row (attend.cuh); warps whose rows are all past the end only
//                keep the barriers going
//   warps 12..19 images: warp e takes blocks 2 (e / 2), + 1 and half of their channels (expand.cuh)
// Two S buffers let S(j + 1) be formed while P(j) is; O += P V(j) follows S(j + 1), so a softmax warp
// that must rescale O waits for it.  Images live in a ring of four 32 KB stages, keys and values of a
// tile in turn.
#pragma once
#include "attend.cuh"
#include "expand.cuh"

namespace witcert {

namespace {

constexpr int kFewThreads = 640;
constexpr int kFewImages = 4;
constexpr int kHalfBlocks = kTileTok / kBlk / 2;           // blocks of a half tile
template <int SCH> struct FewSmem {
  static constexpr int kHalf = kHalfBlocks * block_bytes(SCH);
  // half tiles of codes in flight: what fits beside the images, at most eight
  static constexpr int kScratch = SCH == kInt8 ? 8 * kXsFloats * 4 : 0;
  static constexpr int kRoom = 232448 - kFewImages * kTileBytes - kScratch - 2 * kTileRows * 4 - 512;
  static constexpr int kRing = kRoom / kHalf < 8 ? kRoom / kHalf : 8;
  static constexpr int kRaw = kFewImages * kTileBytes;
  static constexpr int kXs = kRaw + kRing * kHalf;
  static constexpr int kSwap = kXs + kScratch;
  static constexpr int kBar = kSwap + 2 * kTileRows * 4;
  static constexpr int kBytes = kBar + 512;
  static_assert(kRing >= 2 && kHalf % 16 == 0, "two half tiles at least");
};

template <int SCH>
__global__ void __launch_bounds__(kFewThreads, 1) attend_few_kernel(const __grid_constant__ AttendArgs a) {
  using L = FewSmem<SCH>;
  constexpr bool BF16 = SCH == kBbox;
  constexpr int kRing = L::kRing;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t base = smem_addr(sm), bars = base + L::kBar;
  const uint32_t q_full = bars, raw_full = bars + 8, raw_empty = raw_full + 8 * kRing, img_full = raw_empty + 8 * kRing;
  const uint32_t img_empty = img_full + 8 * kFewImages, s_full = img_empty + 8 * kFewImages, p_full = s_full + 16;
  const uint32_t pv_done = p_full + 32, pairs = pv_done + 8, drain = pairs + 32, slot = drain + 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 8);
    for (int s = 0; s < kRing; ++s) { mbar_init(raw_full + 8 * s, 1); mbar_init(raw_empty + 8 * s, 4); }
    for (int s = 0; s < kFewImages; ++s) { mbar_init(img_full + 8 * s, 8); mbar_init(img_empty + 8 * s, 1); }
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full + 8 * b, 1);
      mbar_init(p_full + 16 * b, 8);
      mbar_init(p_full + 16 * b + 8, 8);
    }
    mbar_init(pv_done, 1);
    for (int x = 0; x < 4; ++x) mbar_init(pairs + 8 * x, 2);
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 2) tmem_alloc<512>(slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *reinterpret_cast<const uint32_t*>(sm + L::kBar + (slot - bars));
  const uint32_t tmem_o = tm + 256, tmem_q = tm + 384;
  bool dead = (base & 1023u) != 0;                         // a wait ran out (or no aligned tiles): give up, in order

  if (warp == 0 && !dead) {
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
      for (int f = max(0, filled - kRing); f < filled; ++f) mbar_wait(raw_full + 8 * (f % kRing), (f / kRing) & 1, kAttendWaitNs);
  } else if (warp == 1 && !dead) {
    constexpr uint32_t idesc = mma_idesc(BF16, kTileRows, kTileTok);
    int tiles = 0, done = 0;                               // of this CTA; tiles whose keys were taken
    uint32_t seg = 0;
    walk(a, cta, [&](const Segment& u) { tiles += u.nk; return true; });
    auto image = [&](int x) { return base + (x % kFewImages) * kTileBytes; };     // image x: keys 2j, values 2j + 1
    auto wait_image = [&](int x) { return warp_wait(img_full + 8 * (x % kFewImages), (x / kFewImages) & 1); };
    // nobody waits for a stage that is not filled again
    auto release = [&](int x) { if (x + kFewImages < 2 * tiles) warp_commit(img_empty + 8 * (x % kFewImages)); };
    auto qk = [&](int j) {                                 // tile j of this CTA
      if (!wait_image(2 * j)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t kd = sw128_desc(image(2 * j));
#pragma unroll
        for (int x = 0; x < 8; ++x)
          mma_ts(tm + (j & 1) * 128, tmem_q + x * 8, kd + (uint64_t)(x >> 2) * (kTileRows * 128 >> 4) + (x & 3) * 2, idesc, x > 0);
        mma_commit(s_full + 8 * (j & 1));
      }
      __syncwarp();
      release(2 * j);
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
        dead = dead || !wait_image(2 * j + 1) ||
               !issue_pv(tmem_o, tm + (j & 1) * 128, sw128_desc(image(2 * j + 1)), idesc, s == 0, p_full + 16 * (j & 1), (j >> 1) & 1);
        if (dead) return false;
        warp_commit(pv_done);
        release(2 * j + 1);
      }
      done += u.nk;
      return true;
    });
    if (dead) {                                            // the MMAs in flight still use this CTA's memories
      warp_commit(drain);
      mbar_wait(drain, 0, kAttendWaitNs);
    }
  } else if (warp >= 4 && warp < 12 && !dead) {
    const int hf = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
    float* swap = reinterpret_cast<float*>(sm + L::kSwap);
    RowPair pair{swap + hf * kTileRows + r, swap + (1 - hf) * kTileRows + r, pairs + 8 * (warp & 3), 0, true};
    const uint32_t lanes = (uint32_t)(warp & 3) << 21, to = tmem_o + lanes + 64 * hf;
    int j = 0;                                             // tiles of this CTA so far
    walk(a, cta, [&](const Segment& u) {
      const int row = u.r0 + r;
      const bool busy = u.r0 + (warp & 3) * 32 < u.rows;   // some row of the warp is a query
      float scale = 0.f, m = -INFINITY, l = 0.f;
      if (busy) {
        uint32_t qw[32];
        scale = query_words<BF16>(a, u, row, hf, qw, pair);
        tmem_st16(tmem_q + lanes + 32 * hf, *reinterpret_cast<uint32_t(*)[16]>(qw));
        tmem_st16(tmem_q + lanes + 32 * hf + 16, *reinterpret_cast<uint32_t(*)[16]>(qw + 16));
        tmem_wait_st();
      }
      tc_fence_before();
      warp_arrive(q_full);
      // last key this row sees (-1: a row past the end)
      const int limit = row < u.rows ? a.len[u.k] - a.n[u.k] + row / a.grp : -1;
      for (int s = 0; s < u.nk; ++s, ++j) {
        const uint32_t ts = tm + (j & 1) * 128 + lanes, pb = p_full + 16 * (j & 1);
        if (!pair.ok || !warp_wait(s_full + 8 * (j & 1), (j >> 1) & 1)) { dead = true; return false; }
        tc_fence_after();
        if (busy) {
          softmax_tile<BF16>(ts + 64 * hf, ts + 32 * hf, to, hf, limit - (u.j0 + s) * kTileTok, s == 0, scale, m, l, pair, pb,
                             [&] { pair.ok = pair.ok && warp_wait(pv_done, (j - 1) & 1); tc_fence_after(); });
        } else {
          warp_arrive(pb);
          warp_arrive(pb + 8);
        }
      }
      if (!warp_wait(pv_done, (j - 1) & 1)) { dead = true; return false; }
      tc_fence_after();
      if (busy) {
        l += pair.swap(l);
        store_row(a, u, row, hf, to, m, l, scale, pair.ok);
        tc_fence_before();
        pair.sync();                                       // the partner has read l
      }
      dead = !pair.ok;
      return !dead;
    });
  } else if (warp >= 12 && !dead) {
    BlockPair x;
    x.pr = (warp - 12) >> 1; x.jh = warp & 1; x.lane = lane;
    float* xs = SCH == kInt8 ? reinterpret_cast<float*>(sm + L::kXs) + (warp - 12) * kXsFloats : nullptr;
    RingAt<kRing> at;                                      // half tiles: this warp reads every second one
    if (x.pr >> 1) at.next();
    RingAt<kFewImages> img;
    int made = 0;
    walk(a, cta, [&](const Segment& u) {
      x.h = u.h;
      x.len = a.len[u.k];
      for (int j = u.j0; j < u.j0 + u.nk; ++j) {
        x.tb = j * kTileTok + x.pr * 2 * kBlk;
        const uint8_t* raw = sm + L::kRaw + at.st * L::kHalf + (x.pr & 1) * 2 * block_bytes(SCH);
        x.bp[0] = raw;
        x.bp[1] = raw + block_bytes(SCH);
        find_exact<SCH>(a.s, a.seq[u.k], x);
        if (!warp_wait(raw_full + 8 * at.st, at.ph)) { dead = true; return false; }
        for (int v = 0; v < 2; ++v) {
          if (made >= kFewImages && !warp_wait(img_empty + 8 * img.st, img.ph ^ 1)) { dead = true; return false; }
          if (v == 0) expand_keys<SCH>(a.s, x, sm + img.st * kTileBytes);
          else expand_values<SCH>(a.s, x, xs, sm + img.st * kTileBytes);
          fence_proxy_async();
          warp_arrive(img_full + 8 * img.st);
          img.next();
          ++made;
        }
        warp_arrive(raw_empty + 8 * at.st);
        at.next();
        at.next();
      }
      return true;
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

}  // namespace

template <int SCH>
cudaError_t launch_attend_few(const AttendArgs& a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(attend_few_kernel<SCH>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewSmem<SCH>::kBytes);
  if (e != cudaSuccess) return e;
  attend_few_kernel<SCH><<<(unsigned)a.n_ctas, kFewThreads, FewSmem<SCH>::kBytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace witcert
