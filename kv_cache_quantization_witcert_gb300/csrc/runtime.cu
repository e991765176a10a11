// Host runtime behind the C ABI in include/witcert.h: owns the cache's device
// pools, the pinned backing store, the side stream of the gate and the events
// that order it against writes and decodes; validates every argument and maps
// failures to status codes with a thread-local message.
#include <algorithm>
#include <atomic>
#include <chrono>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>
#include <memory>
#include <new>
#include <numeric>
#include <thread>
#include <vector>

#include "../../include/witcert.h"
#include "common.cuh"
#include "kernels.h"

using namespace witcert;

namespace {

thread_local char g_err[512];          // no string: a message is also left when host memory ran out

witcert_status fail(witcert_status s, const char* fmt, ...) {
  char buf[sizeof g_err];              // an argument may be the present message
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  memcpy(g_err, buf, sizeof buf);
  return s;
}
witcert_status cuda_fail(cudaError_t e, const char* where) {
  cudaGetLastError();                  // reported here: the next launch that asks must not find it
  return fail(e == cudaErrorMemoryAllocation ? WITCERT_ENOMEM : WITCERT_ECUDA, "%s: %s", where, cudaGetErrorString(e));
}
void ok() { g_err[0] = 0; }

// Ends a C entry whose body allocates host memory: nothing throws across the ABI.
#define WITCERT_NO_THROW                                                                        \
  catch (const std::bad_alloc&) { return fail(WITCERT_ENOMEM, "host allocation failed"); }      \
  catch (const std::exception& e) { return fail(WITCERT_EINVAL, "%s", e.what()); }

struct ProfPair { cudaEvent_t a, b; };

// What the last call on the cache's stream left to the next one's launches.
struct Recent {
  bool lengths_last = false;        // the most recent launch set dlen
  bool apart = false;               // the next launch starts after its predecessor's end: a fork, or a call that failed
  int write_layer = -1, write_blk = 0;   // of the most recent launch when it was a write: its layer and first block
};

}  // namespace

struct witcert_cache {
  witcert_config cfg{};
  int device = 0, sm_count = 0, scheme = 0, bblk = 0, nblk_max = 0, elem = 0, max_splits = 1;
  size_t layer_blocks = 0;          // bytes of one layer's block store
  uint8_t* blocks = nullptr;
  float* kivi_tail = nullptr;       // [L][B][Hkv][16][128]
  __half* vwit = nullptr;           // [L][B][Hkv][nblk_max][16] value witnesses (v_witness caches)
  int32_t* slots = nullptr;         // [L][B][Hkv][nblk_max]
  void* pool = nullptr;             // [cap][16][128] kv dtype
  void* backing_host = nullptr;     // [L][B][Hkv][max_tokens][128] kv dtype, pinned + mapped
  void* backing_dev = nullptr;
  float2* risk_raw = nullptr;       // [B][Hq][nblk_max]
  float* risk = nullptr;            // [L][B][Hq][nblk_max]
  float* part = nullptr;            // [B][Hq][max_splits][kPartStride]
  uint32_t* selmask = nullptr;
  int4* todo = nullptr;
  unsigned int* todo_count = nullptr;
  unsigned int* pool_next = nullptr;
  unsigned long long* gstats = nullptr;   // [6]
  unsigned long long* clamps = nullptr;
  int* err = nullptr;
  int* dlen = nullptr;              // [L][B] per-sequence lengths on the device (ragged batches)
  int32_t* table = nullptr;         // paged store: [B][nblk_max] page of each block (all layers), -1 = none
  std::vector<int32_t> table_host;  // host copy of the page table
  std::vector<int32_t> free_pages;  // paged store: pages no sequence holds
  std::vector<int> page_refs;       // paged store: how many sequences hold each page (forks share them)
  std::vector<int> len;             // per layer: the longest sequence
  std::vector<std::vector<int>> slen;   // per layer and sequence
  std::vector<uint64_t> write_gen, risk_gen;   // per layer: writes / resets so far; at the last metered decode
  bool ragged = false;              // sequence lengths may differ: kernels read dlen
  bool lengths_held = false;        // a captured decode reads dlen: it follows every change, also while lengths are equal
  Recent recent;                    // of the calls in `capture`, or launched (0)
  Recent launched;                  // during a capture: of the calls launched before it
  unsigned long long capture = 0, last_capture = 0;   // the capture that the last call was part of; the last one of all
  std::vector<cudaEvent_t> gate_done;
  std::vector<char> gate_pending;
  std::vector<char> backing_lost;   // per layer: the backing store misses exact keys (gate -> EPAGEIN)
  cudaStream_t side = nullptr;
  bool profiling = false;
  std::vector<ProfPair> prof_pending, prof_free;
  double prof_ms = 0.0;
  uint64_t prof_n = 0, tokens_written = 0, decode_calls = 0, gate_calls = 0;
  int last_n_splits = 0;
  bool overlap = true;       // programmatic dependent launch between the cache's kernels
};

namespace {

// Writes of at least this many tokens copy their exact keys to the backing store with the
// copy engines rather than with the write kernels' stores.
constexpr int kBulkBackingTokens = 64;

size_t layer_rows(const witcert_cache* c) { return (size_t)c->cfg.batch * c->cfg.n_kv_heads; }
// Backing-store rows per (sequence, KV head): capacity rounded up to whole 16-token blocks,
// so page-in can always copy a full block.
size_t backing_rows(const witcert_cache* c) { return (size_t)c->nblk_max * kBlk; }
// Value witnesses of one layer: [B][Hkv][nblk_max][16].
size_t vwit_layer(const witcert_cache* c) { return layer_rows(c) * c->nblk_max * kBlk; }

witcert_status check_layer(const witcert_cache* c, int layer) {
  if (!c) return fail(WITCERT_EINVAL, "cache is NULL");
  if (layer < 0 || layer >= c->cfg.n_layers) return fail(WITCERT_EINVAL, "layer %d out of range [0, %d)", layer, c->cfg.n_layers);
  return WITCERT_OK;
}

void free_all(witcert_cache* c) {
  cudaFree(c->blocks); cudaFree(c->kivi_tail); cudaFree(c->vwit); cudaFree(c->slots); cudaFree(c->pool);
  if (c->backing_host) cudaFreeHost(c->backing_host);
  cudaFree(c->risk_raw); cudaFree(c->risk); cudaFree(c->part); cudaFree(c->selmask); cudaFree(c->todo);
  cudaFree(c->todo_count); cudaFree(c->pool_next); cudaFree(c->gstats); cudaFree(c->clamps); cudaFree(c->err);
  cudaFree(c->dlen); cudaFree(c->table);
  for (auto e : c->gate_done) if (e) cudaEventDestroy(e);
  for (auto& p : c->prof_pending) { cudaEventDestroy(p.a); cudaEventDestroy(p.b); }
  for (auto& p : c->prof_free) { cudaEventDestroy(p.a); cudaEventDestroy(p.b); }
  if (c->side) cudaStreamDestroy(c->side);
}

template <typename T>
cudaError_t dalloc(T** p, size_t bytes) {
  cudaError_t e = cudaMalloc(reinterpret_cast<void**>(p), bytes ? bytes : 16);
  if (e == cudaSuccess) e = cudaMemset(*p, 0, bytes ? bytes : 16);
  return e;
}

// Wait for the gate of `layer` (device-side) before touching that layer again.
// Returns true when it inserted an event wait (the next launch then goes without PDL).
bool order_after_gate(witcert_cache* c, int layer, cudaStream_t st) {
  if (!c->gate_pending[layer]) return false;
  cudaStreamWaitEvent(st, c->gate_done[layer], 0);
  return true;
}

// Begins a call's launches on st.  A captured call launches nothing: what it leaves holds within its capture, for
// the calls behind it there, and a call outside goes by the last one that was launched.  The first of those behind a
// capture starts after its predecessor's end, as graphs may have been launched since, and so does the first call
// that goes on with a capture after others outside.
void follow(witcert_cache* c, cudaStream_t st) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  if (cudaStreamGetCaptureInfo(st, &status, &id) != cudaSuccess) cudaGetLastError();
  if (status == cudaStreamCaptureStatusNone) id = 0;
  else if (status != cudaStreamCaptureStatusActive) id = ~0ull;       // one that has failed
  if (id == c->capture) return;
  if (c->capture == 0) c->launched = c->recent; else c->recent = c->launched;
  if (id == 0 || id == c->last_capture) c->recent.apart = true;
  c->capture = id;
  if (id) c->last_capture = id;
}

// Behind a call on st whose kernels start after their predecessor's end, the next launch has no append or lengths of the
// call before to mind.
void launched_apart(witcert_cache* c, cudaStream_t st) {
  if (c->recent.write_layer < 0 && !c->recent.lengths_last) return;
  follow(c, st);
  c->recent.write_layer = -1;
  c->recent.lengths_last = false;
}

// Whether the next launch may start before its predecessor's end.  The kernels that overlap read older
// blocks, lengths and pages before they wait; a fork writes all of those.  What the call launches has not
// succeeded yet: the call says so with recent.apart = false.
bool may_overlap(witcert_cache* c, bool waited) {
  const bool apart = c->recent.apart;
  c->recent.apart = true;
  return c->overlap && !waited && !apart;
}

// Turns per position of a frequency (see rope.cuh): f / (2 pi) mod 1 in units of 2^-64, to the nearest.
// 1 / (2 pi) is the sum of two doubles, and the products that are split further are fma results, which no
// compiler fuses with what follows.
uint64_t turns_of(double f) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  const double a = std::fabs(f), hi = std::fma(a, kHi, 0.0);
  double lo = std::fma(a, kLo, std::fma(a, kHi, -hi));       // hi + lo = |f| / (2 pi) to 2^-105 of it
  lo -= std::nearbyint(lo);                                  // whole turns (only of enormous frequencies)
  const double up = (hi - std::floor(hi)) * 0x1p64;          // exact, below 2^64: hi >= 0
  const uint64_t whole = (uint64_t)up;
  double rest = std::nearbyint((up - (double)whole) + lo * 0x1p64);
  if (rest >= 0x1p63) rest -= 0x1p64;
  const uint64_t t = whole + (uint64_t)(int64_t)rest;
  return f < 0.0 ? 0 - t : t;
}

// Checks a rotation and converts its frequencies to turns (see rope.cuh).
witcert_status rope_turns(const witcert_rope_config* rope, int head_dim, uint64_t* turn, float* gain) {
  if (!rope) return fail(WITCERT_EINVAL, "rope must not be NULL");
  if (rope->rotary_dim < 8 || rope->rotary_dim % 8 || rope->rotary_dim > head_dim)
    return fail(WITCERT_EINVAL, "rotary_dim must be a multiple of 8 in [8, %d] (got %d)", head_dim, rope->rotary_dim);
  if (!std::isfinite((float)rope->scale)) return fail(WITCERT_EINVAL, "the rotation's scale must be finite in fp32");
  for (int p = 0; p < rope->rotary_dim / 2; ++p) {
    const double f = rope->freq[p];
    if (!std::isfinite(f)) return fail(WITCERT_EINVAL, "frequency %d of the rotation is not finite", p);
    turn[p] = turns_of(f);
  }
  *gain = (float)rope->scale;
  return WITCERT_OK;
}

// SM count of the current device (asked once per device).
int sm_count_now() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 1;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

void collect_profile(witcert_cache* c) {
  for (auto& p : c->prof_pending) {
    float ms = 0.f;
    if (cudaEventElapsedTime(&ms, p.a, p.b) == cudaSuccess) { c->prof_ms += ms; ++c->prof_n; }
    c->prof_free.push_back(p);
  }
  c->prof_pending.clear();
}

}  // namespace

extern "C" {

const char* witcert_last_error(void) { return g_err; }

static int auto_splits(const witcert_cache* c, int nblk, bool meter, int cap);

witcert_status witcert_create(const witcert_config* cfg, witcert_cache** out) try {
  if (!cfg || !out) return fail(WITCERT_EINVAL, "NULL argument");
  *out = nullptr;
  const witcert_config& f = *cfg;
  if (f.head_dim != 128) return fail(WITCERT_EINVAL, "head_dim must be 128 (got %d)", f.head_dim);
  if (f.n_layers <= 0 || f.n_layers > 65535) return fail(WITCERT_EINVAL, "n_layers must be in [1, 65535]");
  if (f.n_kv_heads <= 0 || f.n_kv_heads > 65535 || f.n_q_heads <= 0 || f.n_q_heads % f.n_kv_heads)
    return fail(WITCERT_EINVAL, "n_q_heads must be a positive multiple of n_kv_heads");
  if (f.n_q_heads / f.n_kv_heads > kMaxGroupHeads) return fail(WITCERT_EINVAL, "at most %d query heads per KV head", kMaxGroupHeads);
  if (f.batch <= 0 || f.max_tokens <= 0) return fail(WITCERT_EINVAL, "batch and max_tokens must be positive");
  if (f.scheme < WITCERT_INT8_DITHER || f.scheme > WITCERT_BLACKBOX) return fail(WITCERT_EINVAL, "unknown scheme %d", (int)f.scheme);
  if (f.kv_dtype != WITCERT_F32 && f.kv_dtype != WITCERT_BF16) return fail(WITCERT_EINVAL, "unknown dtype %d", (int)f.kv_dtype);
  if (f.total_steps <= 0) return fail(WITCERT_EINVAL, "total_steps must be positive");
  if (f.n_splits < 0 || f.max_repair_blocks < 0) return fail(WITCERT_EINVAL, "n_splits and max_repair_blocks must be >= 0");
  if (f.pos_offset < 0) return fail(WITCERT_EINVAL, "pos_offset must be >= 0");
  if (f.max_pages < 0) return fail(WITCERT_EINVAL, "max_pages must be >= 0");
  if (f.max_pages > 0 && f.kv_dtype != WITCERT_BF16) return fail(WITCERT_EINVAL, "a paged cache holds bf16 keys and values");
  if (f.max_repair_blocks > 0 && (f.max_tokens + kBlk - 1) / kBlk > gate_max_blocks())
    return fail(WITCERT_EINVAL, "with the gate enabled max_tokens must be at most %d (the gate ranks up to %d blocks)",
                gate_max_blocks() * kBlk, gate_max_blocks());

  // sizes that 64 bits do not hold would wrap to an allocation too small (the other arrays are smaller
  // than the store)
  const double nblk = (f.max_tokens + (double)kBlk - 1) / kBlk, pages = f.max_pages > 0 ? f.max_pages : f.batch * nblk;
  if ((double)f.n_layers * pages * f.n_kv_heads * block_bytes((int)f.scheme) > 0x1p62 ||
      (double)f.batch * f.n_q_heads * std::max(nblk, (double)f.n_splits) * kPartStride * sizeof(float) > 0x1p62)
    return fail(WITCERT_ENOMEM, "a cache of this size cannot be addressed");
  std::unique_ptr<witcert_cache, void (*)(witcert_cache*)> owner(new witcert_cache(), [](witcert_cache* x) { free_all(x); delete x; });
  witcert_cache* c = owner.get();
  c->cfg = f;
  c->len.assign(f.n_layers, 0);
  c->slen.assign(f.n_layers, std::vector<int>(f.batch, 0));
  c->write_gen.assign(f.n_layers, 0);
  c->risk_gen.assign(f.n_layers, ~uint64_t(0));
  c->gate_done.assign(f.n_layers, nullptr);
  c->gate_pending.assign(f.n_layers, 0);
  c->backing_lost.assign(f.n_layers, 0);
  cudaError_t e = cudaGetDevice(&c->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, c->device);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  c->scheme = (int)f.scheme;
  c->bblk = block_bytes(c->scheme);
  c->nblk_max = (f.max_tokens - 1) / kBlk + 1;                 // no sum that could pass 31 bits
  c->elem = f.kv_dtype == WITCERT_BF16 ? 2 : 4;
  c->layer_blocks = f.max_pages > 0 ? (size_t)f.max_pages * f.n_kv_heads * c->bblk : layer_rows(c) * c->nblk_max * c->bblk;
  const int auto_on = auto_splits(c, c->nblk_max, true, 0), auto_off = auto_splits(c, c->nblk_max, false, 0);
  const int auto_max = auto_on > auto_off ? auto_on : auto_off;
  c->max_splits = f.n_splits > auto_max ? f.n_splits : auto_max;
  const size_t L = f.n_layers, cells = (size_t)f.batch * f.n_q_heads;
  const bool gate = f.max_repair_blocks > 0;

#define TRY(x, what) do { e = (x); if (e != cudaSuccess) return cuda_fail(e, what); } while (0)
  TRY(dalloc(&c->blocks, L * c->layer_blocks), "allocating the block store");
  if (c->scheme == kKivi) TRY(dalloc(&c->kivi_tail, L * layer_rows(c) * kBlk * kD * sizeof(float)), "allocating the KIVI tail");
  if (f.v_witness) TRY(dalloc(&c->vwit, L * vwit_layer(c) * sizeof(__half)), "allocating value witnesses");
  TRY(dalloc(&c->part, cells * c->max_splits * kPartStride * sizeof(float)), "allocating split scratch");
  TRY(dalloc(&c->clamps, sizeof(unsigned long long)), "allocating counters");
  TRY(dalloc(&c->err, sizeof(int)), "allocating the error word");
  TRY(dalloc(&c->dlen, L * f.batch * sizeof(int)), "allocating sequence lengths");
  if (f.max_pages > 0) {
    const size_t entries = (size_t)f.batch * c->nblk_max;
    TRY(dalloc(&c->table, entries * sizeof(int32_t)), "allocating the page table");
    TRY(cudaMemset(c->table, 0xFF, entries * sizeof(int32_t)), "clearing the page table");
    c->table_host.assign(entries, -1);
    for (int pg = f.max_pages - 1; pg >= 0; --pg) c->free_pages.push_back(pg);
    c->page_refs.assign(f.max_pages, 0);
  }
  if (gate) {
    TRY(dalloc(&c->slots, L * layer_rows(c) * c->nblk_max * sizeof(int32_t)), "allocating repair slots");
    TRY(cudaMemset(c->slots, 0xFF, L * layer_rows(c) * c->nblk_max * sizeof(int32_t)), "clearing repair slots");
    TRY(dalloc(&c->pool, (size_t)f.max_repair_blocks * kBlk * kD * c->elem), "allocating the exact-key pool");
    const size_t bbytes = L * layer_rows(c) * (size_t)c->nblk_max * kBlk * kD * c->elem;
    TRY(cudaHostAlloc(&c->backing_host, bbytes, cudaHostAllocMapped), "allocating the pinned backing store");
    memset(c->backing_host, 0, bbytes);
    TRY(cudaHostGetDevicePointer(&c->backing_dev, c->backing_host, 0), "mapping the backing store");
    TRY(dalloc(&c->risk_raw, cells * c->nblk_max * sizeof(float2)), "allocating block-risk scratch");
    TRY(dalloc(&c->risk, L * cells * c->nblk_max * sizeof(float)), "allocating block risks");
    TRY(dalloc(&c->selmask, layer_rows(c) * (c->nblk_max / 32 + 1) * sizeof(uint32_t)), "allocating gate masks");
    TRY(dalloc(&c->todo, layer_rows(c) * c->nblk_max * sizeof(int4)), "allocating the gate todo list");
    TRY(dalloc(&c->todo_count, sizeof(unsigned int)), "allocating gate counters");
    TRY(dalloc(&c->pool_next, sizeof(unsigned int)), "allocating gate counters");
    TRY(dalloc(&c->gstats, 6 * sizeof(unsigned long long)), "allocating gate counters");
    TRY(cudaStreamCreateWithFlags(&c->side, cudaStreamNonBlocking), "creating the gate stream");
    for (auto& ev : c->gate_done) TRY(cudaEventCreateWithFlags(&ev, cudaEventDisableTiming), "creating gate events");
  }
#undef TRY
  e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "create");
  *out = owner.release();
  ok();
  return WITCERT_OK;
} WITCERT_NO_THROW

witcert_status witcert_destroy(witcert_cache* c) {
  if (!c) return fail(WITCERT_EINVAL, "cache is NULL");
  cudaDeviceSynchronize();
  free_all(c);
  delete c;
  ok();
  return WITCERT_OK;
}

// Write arguments of `layer` for all sequences: appends of n_tok tokens at t0.
static WriteArgs layer_write_args(const witcert_cache* c, int layer, const void* K, const void* V, const void* Kh,
                                  const void* Vh, int n_tok, int t0) {
  WriteArgs a{};
  a.blocks = c->blocks + layer * c->layer_blocks;
  a.table = c->table;
  a.nblk_max = c->nblk_max;
  a.K = K; a.V = V; a.Kh = Kh; a.Vh = Vh;
  if (c->vwit) a.vwit = c->vwit + layer * vwit_layer(c);
  a.B = c->cfg.batch; a.Hkv = c->cfg.n_kv_heads; a.n_tok = n_tok; a.t0 = t0; a.layer = layer;
  a.backing_rows = (int)backing_rows(c);
  a.is_bf16 = c->cfg.kv_dtype == WITCERT_BF16;
  a.seed = c->cfg.seed;
  philox_round_keys(a.seed, a.rk0, a.rk1);
  a.pos0 = c->cfg.pos_offset;
  if (c->backing_dev)
    a.backing = static_cast<uint8_t*>(c->backing_dev) + layer * layer_rows(c) * backing_rows(c) * kD * c->elem;
  if (c->slots) a.slots = c->slots + layer * layer_rows(c) * c->nblk_max;
  a.pool = c->pool;
  if (c->kivi_tail) a.kivi_tail = c->kivi_tail + layer * layer_rows(c) * kBlk * kD;
  a.clamps = c->clamps;
  return a;
}

// The same arguments narrowed to sequence i alone (B = 1): its n tokens sit at packed input
// row in_row (tokens, each n_kv_heads x 128 elements) and are appended at position t0.
static WriteArgs seq_write_args(const witcert_cache* c, const WriteArgs& all, int i, size_t in_row, int n, int t0) {
  WriteArgs a = all;
  const size_t rows = (size_t)i * c->cfg.n_kv_heads;          // (sequence, KV head) rows before i
  const size_t in_bytes = in_row * c->cfg.n_kv_heads * kD * c->elem;
  if (a.table) a.table += (size_t)i * c->nblk_max;            // paged: the sequence's row of the table
  else a.blocks += rows * c->nblk_max * c->bblk;
  if (a.vwit) a.vwit += rows * c->nblk_max * kBlk;
  if (a.backing) a.backing = static_cast<uint8_t*>(a.backing) + rows * backing_rows(c) * kD * c->elem;
  if (a.slots) a.slots += rows * c->nblk_max;
  if (a.kivi_tail) a.kivi_tail += rows * kBlk * kD;
  a.K = static_cast<const uint8_t*>(all.K) + in_bytes;
  a.V = static_cast<const uint8_t*>(all.V) + in_bytes;
  if (all.Kh) a.Kh = static_cast<const uint8_t*>(all.Kh) + in_bytes;
  if (all.Vh) a.Vh = static_cast<const uint8_t*>(all.Vh) + in_bytes;
  a.B = 1; a.n_tok = n; a.t0 = t0;
  return a;
}

// Device copies of per-sequence lengths: entries (layer * batch + sequence, length), sent as
// kernel parameters (no host buffer outlives the call).
static cudaError_t push_ints(int* dst, const std::vector<std::pair<int, int>>& upd, cudaStream_t st, bool& pdl) {
  for (size_t k0 = 0; k0 < upd.size(); k0 += kRaggedPerLaunch) {
    LengthArgs u{};
    u.dst = dst;
    for (size_t k = k0; k < upd.size() && k < k0 + kRaggedPerLaunch; ++k) {
      u.idx[u.n] = upd[k].first;
      u.len[u.n] = upd[k].second;
      ++u.n;
    }
    cudaError_t e = launch_set_lengths(u, st, pdl);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
static cudaError_t push_lengths(witcert_cache* c, const std::vector<std::pair<int, int>>& upd, cudaStream_t st,
                                bool& pdl) {
  return push_ints(c->dlen, upd, st, pdl);
}

// A page that an append gives its sequence: entry idx of the table changes from `was` (-1: none) to `now`.
// A page that other sequences hold too is left to them, and what the sequence keeps of it is copied.
struct PageTaken { int idx, was, now; bool copy; };

// Paged store: pages of its own for every block the appends of n touch (the table is shared by the
// layers, so the first layer to reach a block takes its page).  Fails, taking back what it took, when
// the pool runs out.
static witcert_status take_pages(witcert_cache* c, int layer, const std::vector<int>& n, std::vector<PageTaken>& taken) {
  if (!c->table) return WITCERT_OK;
  size_t most = 0;
  for (int i = 0; i < c->cfg.batch; ++i) most += n[i] > 0 ? n[i] / kBlk + 2 : 0;
  taken.reserve(std::min(most, c->free_pages.size()));         // no allocation once pages are being taken
  for (int i = 0; i < c->cfg.batch; ++i) {
    if (n[i] == 0) continue;
    const int t0 = c->slen[layer][i];
    // whether some layer of the sequence holds tokens of block b (asked of shared pages alone: for all of them an append
    // to 256 sequences of 80 layers took the host 15.6 us, now 6.5)
    auto held = [&](int b) {
      for (int l = 0; l < c->cfg.n_layers; ++l)
        if (b * kBlk < c->slen[l][i]) return true;
      return false;
    };
    for (int b = t0 / kBlk; b <= (t0 + n[i] - 1) / kBlk; ++b) {
      int32_t& e = c->table_host[(size_t)i * c->nblk_max + b];
      if (e >= 0 && c->page_refs[e] == 1) continue;
      if (c->free_pages.empty()) {
        for (const PageTaken& u : taken) {
          c->free_pages.push_back(u.now);
          c->page_refs[u.now] = 0;
          c->table_host[u.idx] = u.was;
          if (u.was >= 0) ++c->page_refs[u.was];
        }
        taken.clear();
        return fail(WITCERT_ENOMEM, "the page pool (%d pages) is exhausted", c->cfg.max_pages);
      }
      const PageTaken u{(int)((size_t)i * c->nblk_max + b), e, c->free_pages.back(), e >= 0 && held(b)};
      taken.push_back(u);
      c->free_pages.pop_back();
      c->page_refs[u.now] = 1;
      if (u.was >= 0) --c->page_refs[u.was];
      e = u.now;
    }
  }
  return WITCERT_OK;
}

// The device's side of take_pages: copies and table entries.  Copies end before what follows starts.
static cudaError_t push_pages(witcert_cache* c, const std::vector<PageTaken>& taken, cudaStream_t st, bool& pdl) {
  if (taken.empty()) return cudaSuccess;
  CopyPages a{};
  a.blocks = c->blocks;
  a.layer_pitch = (long long)c->layer_blocks;
  a.page_bytes = (long long)c->cfg.n_kv_heads * c->bblk;
  a.table = c->table;
  cudaError_t e = cudaSuccess;
  for (const PageTaken& u : taken) {
    if (!u.copy) continue;
    a.src[a.n] = u.was; a.dst[a.n] = u.now; a.idx[a.n] = u.idx;
    pdl = false;
    if (++a.n == kRaggedPerLaunch) {
      if ((e = launch_copy_pages(a, c->cfg.n_layers, st)) != cudaSuccess) return e;
      a.n = 0;
    }
  }
  if ((e = launch_copy_pages(a, c->cfg.n_layers, st)) != cudaSuccess) return e;
  LengthArgs t{};                                              // no host allocation: the pages are taken
  t.dst = c->table;
  for (const PageTaken& u : taken) {
    if (u.copy) continue;
    t.idx[t.n] = u.idx; t.len[t.n] = u.now;
    if (++t.n == kRaggedPerLaunch) {
      if ((e = launch_set_lengths(t, st, pdl)) != cudaSuccess) return e;
      t.n = 0;
    }
  }
  return launch_set_lengths(t, st, pdl);
}

// From now on the sequences' lengths may differ: the device gets every layer's lengths.
static cudaError_t enter_ragged(witcert_cache* c, cudaStream_t st, bool& pdl) {
  if (c->ragged || c->lengths_held) { c->ragged = true; return cudaSuccess; }
  std::vector<std::pair<int, int>> upd;
  for (int l = 0; l < c->cfg.n_layers; ++l)
    for (int i = 0; i < c->cfg.batch; ++i) upd.emplace_back(l * c->cfg.batch + i, c->slen[l][i]);
  cudaError_t e = push_lengths(c, upd, st, pdl);
  if (e == cudaSuccess) c->ragged = true;
  return e;
}

// Exact keys of n tokens of sequence i (packed input row in_row) to the pinned backing store
// at position t0, one strided copy-engine transfer per KV head.
static cudaError_t backing_copy(witcert_cache* c, int layer, const void* K, int i, size_t in_row, int n, int t0,
                                cudaStream_t st) {
  const size_t row = (size_t)kD * c->elem;
  const int Hkv = c->cfg.n_kv_heads;
  uint8_t* host = static_cast<uint8_t*>(c->backing_host) + layer * layer_rows(c) * backing_rows(c) * row;
  cudaError_t e = cudaSuccess;
  for (int h = 0; h < Hkv && e == cudaSuccess; ++h)
    e = cudaMemcpy2DAsync(host + (((size_t)i * Hkv + h) * backing_rows(c) + t0) * row, row,
                          static_cast<const uint8_t*>(K) + (in_row * Hkv + h) * row, Hkv * row, row, n,
                          cudaMemcpyDeviceToHost, st);
  return e;
}

// Appends counts[i] tokens (n_uniform each when counts is NULL) to every sequence of `layer`;
// inputs are packed sequence-major.  Equal appends to equal lengths take the batched writers;
// anything else marks the cache ragged and writes each sequence at its own position.
static witcert_status write_impl(witcert_cache* c, int layer, const void* K, const void* V, const void* Kh,
                                 const void* Vh, const int32_t* counts, int n_uniform,
                                 const witcert_rope_config* rope, void* stream) {
  if (witcert_status s = check_layer(c, layer)) return s;
  const int B = c->cfg.batch;
  RopeArgs rp{};
  if (rope) {
    if (witcert_status s = rope_turns(rope, kD, rp.turn, &rp.gain)) return s;
    rp.rot = rope->rotary_dim;
    rp.interleaved = rope->interleaved != 0;
  }
  std::vector<int> n(B, n_uniform);
  long long total = 0;
  for (int i = 0; i < B; ++i) {
    if (counts) n[i] = counts[i];
    if (n[i] < 0) return fail(WITCERT_EINVAL, "token counts must be >= 0 (sequence %d: %d)", i, n[i]);
    if ((long long)c->slen[layer][i] + n[i] > c->cfg.max_tokens)
      return fail(WITCERT_EINVAL, "layer %d sequence %d would hold %lld tokens, capacity %d", layer, i,
                  (long long)c->slen[layer][i] + n[i], c->cfg.max_tokens);
    total += n[i];
  }
  if (total > 0 && (!K || !V)) return fail(WITCERT_EINVAL, "K and V must not be NULL");
  if (total > 0 && c->scheme == kBbox && (!Kh || !Vh)) return fail(WITCERT_EINVAL, "K_hat and V_hat must not be NULL");
  if (total == 0) { ok(); return WITCERT_OK; }
  // the writers load four elements at a time
  if (((uintptr_t)K | (uintptr_t)V | (uintptr_t)Kh | (uintptr_t)Vh) % (4 * c->elem))
    return fail(WITCERT_EINVAL, "K, V, K_hat and V_hat must be %d-byte aligned", 4 * c->elem);
  bool uniform = !c->ragged;
  for (int i = 1; i < B && uniform; ++i) uniform = n[i] == n[0];
  std::vector<PageTaken> pages;
  if (witcert_status ps = take_pages(c, layer, n, pages)) return ps;
  auto st = static_cast<cudaStream_t>(stream);
  follow(c, st);
  const bool waited = order_after_gate(c, layer, st);
  bool pdl = may_overlap(c, waited);
  cudaError_t e = push_pages(c, pages, st, pdl);
  if (e != cudaSuccess) return cuda_fail(e, "page table");
  int first_blk = INT_MAX;
  if (uniform) {
    const int n_tok = n[0], t0 = c->len[layer];
    WriteArgs a = layer_write_args(c, layer, K, V, Kh, Vh, n_tok, t0);
    // a page-table update launched just before must be complete before the writers read it
    // (and a write right after another one waits for it first: a decode that follows takes only
    // the last write's blocks for unfinished, and a truncation between them makes their rows meet)
    a.late_wait = pages.empty() && c->recent.write_layer < 0 && !c->lengths_held;
    // rotated keys exist only in the writers' registers: the writers store their exact copies
    if (c->backing_host && n_tok >= kBulkBackingTokens && !rope) {
      // bulk writes copy their exact keys to the pinned backing store with the copy engines
      // instead of the kernels' stores over C2C
      for (int i = 0; i < B && e == cudaSuccess; ++i) e = backing_copy(c, layer, K, i, (size_t)i * n_tok, n_tok, t0, st);
      if (e != cudaSuccess) {
        c->backing_lost[layer] = 1;
        return cuda_fail(e, "backing-store copy");
      }
      a.backing = nullptr;
      pdl = false;                     // the copies sit between this write and its predecessor
    }
    if (c->lengths_held) {
      std::vector<std::pair<int, int>> upd;
      for (int i = 0; i < B; ++i) upd.emplace_back(layer * B + i, t0 + n_tok);
      if ((e = push_lengths(c, upd, st, pdl)) != cudaSuccess) return cuda_fail(e, "sequence lengths");
    }
    e = rope ? launch_write_rope(c->scheme, a, rp, st, pdl) : launch_write(c->scheme, a, st, pdl);
    if (e != cudaSuccess) return cuda_fail(e, "write launch");
    first_blk = t0 / kBlk;
  } else {
    if ((e = enter_ragged(c, st, pdl)) != cudaSuccess) return cuda_fail(e, "sequence lengths");
    std::vector<std::pair<int, int>> upd;
    for (int i = 0; i < B; ++i)
      if (n[i] > 0) upd.emplace_back(layer * B + i, c->slen[layer][i] + n[i]);
    if ((e = push_lengths(c, upd, st, pdl)) != cudaSuccess) return cuda_fail(e, "sequence lengths");
    const WriteArgs all = layer_write_args(c, layer, K, V, Kh, Vh, 0, 0);
    // ragged launches of up to kRaggedPerLaunch sequences; with a backing store, bulk appends go
    // sequence by sequence (their exact keys by the copy engines)
    RaggedArgs g{};
    auto flush = [&]() -> cudaError_t {
      if (g.n_seq == 0) return cudaSuccess;
      cudaError_t r = rope ? launch_write_ragged_rope(c->scheme, all, rp, g, st, pdl)
                           : launch_write_ragged(c->scheme, all, g, st, pdl);
      // KIVI keys close per 16-token block: each sequence's blocks by its own launch
      for (int k = 0; k < g.n_seq && r == cudaSuccess && c->scheme == kKivi; ++k) {
        const WriteArgs ka = seq_write_args(c, all, g.seq[k], (size_t)g.row0[k], g.off[k + 1] - g.off[k], g.t0[k]);
        r = rope ? launch_kivi_keys_rope(ka, rp, st, pdl) : launch_kivi_keys(ka, st, pdl);
      }
      g = RaggedArgs{};
      return r;
    };
    size_t row = 0;
    for (int i = 0; i < B && e == cudaSuccess; ++i) {
      if (n[i] == 0) continue;
      const int t0 = c->slen[layer][i];
      first_blk = t0 / kBlk < first_blk ? t0 / kBlk : first_blk;
      if (c->backing_host && n[i] >= kBulkBackingTokens && !rope) {
        WriteArgs a = seq_write_args(c, all, i, row, n[i], t0);
        e = backing_copy(c, layer, K, i, row, n[i], t0, st);
        if (e != cudaSuccess) {
          c->backing_lost[layer] = 1;
          return cuda_fail(e, "backing-store copy");
        }
        a.backing = nullptr;
        pdl = false;
        e = launch_write(c->scheme, a, st, pdl);
      } else {
        g.seq[g.n_seq] = i;
        g.t0[g.n_seq] = t0;
        g.row0[g.n_seq] = (int)row;
        g.off[g.n_seq + 1] = g.off[g.n_seq] + n[i];
        if (++g.n_seq == kRaggedPerLaunch) e = flush();
      }
      row += n[i];
    }
    if (e == cudaSuccess) e = flush();
    if (e != cudaSuccess) return cuda_fail(e, "ragged write launch");
  }
  c->recent = Recent{};
  c->recent.write_layer = layer;
  c->recent.write_blk = first_blk;
  for (int i = 0; i < B; ++i) c->slen[layer][i] += n[i];
  int mx = 0;
  for (int i = 0; i < B; ++i) mx = c->slen[layer][i] > mx ? c->slen[layer][i] : mx;
  c->len[layer] = mx;
  ++c->write_gen[layer];
  c->tokens_written += (uint64_t)total * c->cfg.n_kv_heads;
  ok();
  return WITCERT_OK;
}

witcert_status witcert_write(witcert_cache* c, int layer, const void* K, const void* V, int n_tok, void* stream) try {
  if (c && c->scheme == kBbox) return fail(WITCERT_EINVAL, "a black-box cache is written with witcert_write_hat");
  if (n_tok < 0) return fail(WITCERT_EINVAL, "n_tok must be >= 0");
  return write_impl(c, layer, K, V, nullptr, nullptr, nullptr, n_tok, nullptr, stream);
} WITCERT_NO_THROW

witcert_status witcert_write_hat(witcert_cache* c, int layer, const void* K, const void* V, const void* K_hat,
                                 const void* V_hat, int n_tok, void* stream) try {
  if (c && c->scheme != kBbox) return fail(WITCERT_EINVAL, "witcert_write_hat needs a WITCERT_BLACKBOX cache");
  if (n_tok < 0) return fail(WITCERT_EINVAL, "n_tok must be >= 0");
  return write_impl(c, layer, K, V, K_hat, V_hat, nullptr, n_tok, nullptr, stream);
} WITCERT_NO_THROW

witcert_status witcert_write_ragged(witcert_cache* c, int layer, const void* K, const void* V, const void* K_hat,
                                    const void* V_hat, const int32_t* n_tok, void* stream) try {
  if (!c || !n_tok) return fail(WITCERT_EINVAL, "cache and n_tok must not be NULL");
  if (c->scheme != kBbox && (K_hat || V_hat)) return fail(WITCERT_EINVAL, "K_hat and V_hat belong to black-box caches");
  return write_impl(c, layer, K, V, K_hat, V_hat, n_tok, 0, nullptr, stream);
} WITCERT_NO_THROW

witcert_status witcert_write_rope(witcert_cache* c, int layer, const void* K, const void* V, const void* K_hat,
                                  const void* V_hat, int n_tok, const witcert_rope_config* rope, void* stream) try {
  if (!c || !rope) return fail(WITCERT_EINVAL, "cache and rope must not be NULL");
  if (n_tok < 0) return fail(WITCERT_EINVAL, "n_tok must be >= 0");
  if (c->scheme != kBbox && (K_hat || V_hat)) return fail(WITCERT_EINVAL, "K_hat and V_hat belong to black-box caches");
  return write_impl(c, layer, K, V, K_hat, V_hat, nullptr, n_tok, rope, stream);
} WITCERT_NO_THROW

witcert_status witcert_write_rope_ragged(witcert_cache* c, int layer, const void* K, const void* V, const void* K_hat,
                                         const void* V_hat, const int32_t* n_tok, const witcert_rope_config* rope,
                                         void* stream) try {
  if (!c || !n_tok || !rope) return fail(WITCERT_EINVAL, "cache, n_tok and rope must not be NULL");
  if (c->scheme != kBbox && (K_hat || V_hat)) return fail(WITCERT_EINVAL, "K_hat and V_hat belong to black-box caches");
  return write_impl(c, layer, K, V, K_hat, V_hat, n_tok, 0, rope, stream);
} WITCERT_NO_THROW

witcert_status witcert_rope(const witcert_rope_config* rope, witcert_dtype dtype, int head_dim, int n_tok,
                            const int64_t* positions, const witcert_rope_tensor* q, const witcert_rope_tensor* k,
                            int inverse, void* stream) {
  if (dtype != WITCERT_F32 && dtype != WITCERT_BF16) return fail(WITCERT_EINVAL, "unknown dtype %d", (int)dtype);
  if (head_dim < 8 || head_dim % 2 || head_dim > 2 * kRopeMaxPairs)
    return fail(WITCERT_EINVAL, "head_dim must be even and in [8, %d] (got %d)", 2 * kRopeMaxPairs, head_dim);
  if (n_tok < 0) return fail(WITCERT_EINVAL, "n_tok must be >= 0");
  RopeLaunch a{};
  if (witcert_status s = rope_turns(rope, head_dim, a.turn, &a.gain)) return s;
  if (!q) return fail(WITCERT_EINVAL, "q must not be NULL");
  const witcert_rope_tensor* in[2] = {q, k};
  for (int i = 0; i < 2; ++i) {
    if (!in[i]) continue;
    const witcert_rope_tensor& t = *in[i];
    if (t.n_heads < 1 || t.n_heads > 65535) return fail(WITCERT_EINVAL, "n_heads must be in [1, 65535]");
    if (n_tok > 0 && (!t.x || !t.y)) return fail(WITCERT_EINVAL, "x and y must not be NULL");
    if (((uintptr_t)t.x | (uintptr_t)t.y) % (dtype == WITCERT_BF16 ? 2 : 4)) return fail(WITCERT_EINVAL, "x and y must be aligned to their elements");
    if ((n_tok > 1 && t.y_token_stride == 0) || (t.n_heads > 1 && t.y_head_stride == 0))
      return fail(WITCERT_EINVAL, "outputs must not share their elements (stride 0)");
    a.t[i] = RopeTensor{t.x, t.y, t.x_token_stride, t.x_head_stride, t.y_token_stride, t.y_head_stride, t.n_heads};
  }
  if (n_tok == 0) { ok(); return WITCERT_OK; }
  if (!positions) return fail(WITCERT_EINVAL, "positions must not be NULL");
  a.pos = positions;
  a.n_tok = n_tok; a.head_dim = head_dim; a.rot = rope->rotary_dim; a.interleaved = rope->interleaved != 0;
  a.is_bf16 = dtype == WITCERT_BF16;
  if (inverse)
    for (uint64_t& t : a.turn) t = 0 - t;
  cudaError_t e = launch_rope(a, sm_count_now(), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope launch");
  ok();
  return WITCERT_OK;
}

witcert_status witcert_reset_sequence(witcert_cache* c, int seq, void* stream) try {
  if (!c) return fail(WITCERT_EINVAL, "cache is NULL");
  if (seq < 0 || seq >= c->cfg.batch) return fail(WITCERT_EINVAL, "sequence %d out of range [0, %d)", seq, c->cfg.batch);
  auto st = static_cast<cudaStream_t>(stream);
  follow(c, st);
  // host memory first: nothing may fail between what the device and what the host is told
  std::vector<std::pair<int, int>> upd, freed;
  for (int l = 0; l < c->cfg.n_layers; ++l) upd.emplace_back(l * c->cfg.batch + seq, 0);
  if (c->table) freed.reserve(c->nblk_max);
  bool waited = false;
  for (int l = 0; l < c->cfg.n_layers; ++l) waited |= order_after_gate(c, l, st);
  bool pdl = may_overlap(c, waited);
  cudaError_t e = enter_ragged(c, st, pdl);
  if (e == cudaSuccess) e = push_lengths(c, upd, st, pdl);
  if (c->table && e == cudaSuccess) {       // its pages go back to the pool
    for (int b = 0; b < c->nblk_max; ++b) {
      int32_t& pg = c->table_host[(size_t)seq * c->nblk_max + b];
      if (pg < 0) continue;
      if (--c->page_refs[pg] == 0) c->free_pages.push_back(pg);
      pg = -1;
      freed.emplace_back((int)((size_t)seq * c->nblk_max + b), -1);
    }
    e = push_ints(c->table, freed, st, pdl);
  }
  // the sequence's repairs go with it (their pool slots are not reused)
  const size_t rows = (size_t)c->cfg.n_kv_heads * c->nblk_max;
  for (int l = 0; l < c->cfg.n_layers && e == cudaSuccess && c->slots; ++l)
    e = cudaMemsetAsync(c->slots + (size_t)l * layer_rows(c) * c->nblk_max + (size_t)seq * rows, 0xFF,
                        rows * sizeof(int32_t), st);
  // an export is as long as the longest sequence: no value witness of the old occupant shows in it
  for (int l = 0; l < c->cfg.n_layers && e == cudaSuccess && c->vwit; ++l)
    e = cudaMemsetAsync(c->vwit + l * vwit_layer(c) + (size_t)seq * rows * kBlk, 0, rows * kBlk * sizeof(__half), st);
  if (e != cudaSuccess) return cuda_fail(e, "reset");
  for (int l = 0; l < c->cfg.n_layers; ++l) {
    c->slen[l][seq] = 0;
    int mx = 0;
    for (int i = 0; i < c->cfg.batch; ++i) mx = c->slen[l][i] > mx ? c->slen[l][i] : mx;
    c->len[l] = mx;
    ++c->write_gen[l];
  }
  c->recent = Recent{};
  c->recent.lengths_last = true;
  ok();
  return WITCERT_OK;
} WITCERT_NO_THROW

witcert_status witcert_truncate(witcert_cache* c, int layer, const int32_t* lengths, void* stream) try {
  if (!c || !lengths) return fail(WITCERT_EINVAL, "cache and lengths must not be NULL");
  if (layer != -1)
    if (witcert_status s = check_layer(c, layer)) return s;
  const int l0 = layer < 0 ? 0 : layer, l1 = layer < 0 ? c->cfg.n_layers : layer + 1, B = c->cfg.batch;
  bool any = false;
  for (int l = l0; l < l1; ++l)
    for (int i = 0; i < B; ++i) {
      const int now = c->slen[l][i], to = lengths[i];
      if (to < 0) return fail(WITCERT_EINVAL, "lengths must be >= 0 (sequence %d: %d)", i, to);
      if (to >= now) continue;
      any = true;
      if (c->scheme == kKivi && to % kBlk && to / kBlk < now / kBlk)
        return fail(WITCERT_EINVAL, "layer %d sequence %d: the exact keys of a finished KIVI block are gone; truncate "
                    "to a multiple of %d or within the unfinished block (at %d)", l, i, kBlk, now / kBlk * kBlk);
    }
  if (!any) { ok(); return WITCERT_OK; }
  auto st = static_cast<cudaStream_t>(stream);
  follow(c, st);
  bool waited = false;
  for (int l = l0; l < l1; ++l) waited |= order_after_gate(c, l, st);
  // lengths that stay equal need no copy on the device
  bool uniform = !c->ragged;
  for (int l = l0; l < l1 && uniform; ++l)
    for (int i = 1; i < B && uniform; ++i)
      uniform = std::min(c->slen[l][i], (int)lengths[i]) == std::min(c->slen[l][0], (int)lengths[0]);
  cudaError_t e = cudaSuccess;
  if (!uniform || c->lengths_held) {
    bool pdl = may_overlap(c, waited);
    if (!uniform) e = enter_ragged(c, st, pdl);
    std::vector<std::pair<int, int>> upd;
    for (int l = l0; l < l1; ++l)
      for (int i = 0; i < B; ++i)
        if (lengths[i] < c->slen[l][i]) upd.emplace_back(l * B + i, lengths[i]);
    if (e == cudaSuccess) e = push_lengths(c, upd, st, pdl);
    if (e != cudaSuccess) return cuda_fail(e, "sequence lengths");
    c->recent.lengths_last = true;
    c->recent.apart = false;
  }
  for (int l = l0; l < l1; ++l) {
    int mx = 0;
    bool moved = false;
    for (int i = 0; i < B; ++i) {
      if (lengths[i] < c->slen[l][i]) { c->slen[l][i] = lengths[i]; moved = true; }
      mx = std::max(mx, c->slen[l][i]);
    }
    c->len[l] = mx;
    if (moved) ++c->write_gen[l];          // block risks of the longer sequence are stale
  }
  ok();
  return WITCERT_OK;
} WITCERT_NO_THROW

// ------------------------------------------------------------------ forks
// What every sequence of a fork becomes: its parent (itself: it stays, or is cut; -1: empty), the most
// tokens it keeps, and how many blocks and KIVI tail rows that is, the longest layer's.
struct ForkPlan {
  std::vector<int> from, cap, blocks, tail;
  std::vector<MoveOp> ops;
  std::vector<size_t> launches;        // first move of each launch, and their end
  std::vector<size_t> groups;          // first move of each set of sequences that have nothing to do with the others
};

static MoveOp fork_move(const ForkPlan& f, int src, int dst, int like, bool rows) {
  MoveOp op{};
  op.src = src; op.dst = dst;
  op.n[0] = op.load[0] = rows ? f.blocks[like] : 0;
  op.n[1] = op.load[1] = rows ? f.tail[like] : 0;
  op.blocks = f.blocks[like];
  op.cap = f.cap[like];
  return op;
}

// The moves of a fork in an order in which none reads what an earlier one wrote, one connected set of
// sequences (a request's beams) after another.  First the sequences that nobody reads any more, source by
// source, which frees their sources in turn; what is left are cycles, each of which saves one row, moves
// the others up and hands the saved one out.  A launch holds kMovesPerLaunch moves; a cycle that crosses
// its end is cut into two that share a sequence, the second of which finds there what the first one saved.
static void fork_moves(ForkPlan& f) {
  const int B = (int)f.from.size();
  std::vector<int> readers(B, 0), first(B + 1, 0), kids, ready;
  std::vector<char> done(B, 0);
  for (int i = 0; i < B; ++i)
    if (f.from[i] >= 0 && f.from[i] != i) ++readers[f.from[i]];
  for (int i = 0; i < B; ++i) first[i + 1] = first[i] + readers[i];
  kids.resize(first[B]);
  std::vector<int> at(first.begin(), first.end() - 1);
  for (int i = 0; i < B; ++i) {
    if (f.from[i] >= 0 && f.from[i] != i) kids[at[f.from[i]]++] = i;
    if (f.from[i] == i) done[i] = 1;
  }
  // connected sets: each sequence points towards its set's representative
  std::vector<int> set(B), member(B), start(B + 1, 0);
  std::iota(set.begin(), set.end(), 0);
  auto find = [&](int i) {
    while (set[i] != i) i = set[i] = set[set[i]];
    return i;
  };
  for (int i = 0; i < B; ++i)
    if (f.from[i] >= 0) set[find(i)] = find(f.from[i]);
  for (int i = 0; i < B; ++i) ++start[find(i) + 1];
  for (int i = 0; i < B; ++i) start[i + 1] += start[i];
  std::vector<int> fill(start.begin(), start.end() - 1);
  for (int i = 0; i < B; ++i) member[fill[find(i)]++] = i;

  f.launches.push_back(0);
  auto room = [&] {
    if (f.ops.size() - f.launches.back() == kMovesPerLaunch) f.launches.push_back(f.ops.size());
    return kMovesPerLaunch - (int)(f.ops.size() - f.launches.back());
  };
  auto emit = [&](int i) {
    room();
    f.ops.push_back(fork_move(f, f.from[i] >= 0 ? f.from[i] : kMoveNone, i, i, f.from[i] >= 0));
    done[i] = 1;
  };
  for (int g = 0; g < B; ++g) {
    f.groups.push_back(f.ops.size());
    for (int m = start[g]; m < start[g + 1]; ++m)
      if (!done[member[m]] && readers[member[m]] == 0) ready.push_back(member[m]);
    while (!ready.empty()) {
      const int i = ready.back(), src = f.from[i];
      ready.pop_back();
      if (done[i]) continue;
      if (src < 0) { emit(i); continue; }
      for (int k = first[src]; k < first[src + 1]; ++k)        // the source's other free children with it
        if (!done[kids[k]] && readers[kids[k]] == 0) { emit(kids[k]); --readers[src]; }
      if (!done[src] && readers[src] == 0) ready.push_back(src);
    }
    for (int m = start[g]; m < start[g + 1]; ++m) {
      const int i = member[m];
      if (done[i]) continue;
      int last = i;                                            // the sequence that takes i's row
      for (int j = f.from[i]; j != i; j = f.from[j]) last = j;
      int to = i;                                              // i <- from(i) <- ... <- last <- i
      while (!done[last]) {
        if (room() < 3) f.launches.push_back(f.ops.size());
        f.ops.push_back(fork_move(f, to, kMoveKept, last, true));
        f.ops.back().cap = INT_MAX;
        while (to != last && room() > 1) {
          emit(to);
          to = f.from[to];
        }
        f.ops.push_back(fork_move(f, kMoveKept, to, last, true));
        if (to == last) done[last] = 1; else f.ops.back().cap = INT_MAX;
      }
    }
    for (int m = start[g]; m < start[g + 1]; ++m)              // sequences that are only cut, after their readers
      if (f.from[member[m]] == member[m] && f.cap[member[m]] >= 0) {
        room();
        f.ops.push_back(fork_move(f, member[m], member[m], member[m], false));
      }
  }
  f.launches.push_back(f.ops.size());
  f.groups.push_back(f.ops.size());
  // a run of moves from one source in one launch loads once what the largest of them takes
  for (size_t l = 0; l + 1 < f.launches.size(); ++l)
    for (size_t m = f.launches[l], to = m; m < f.launches[l + 1]; m = to) {
      MoveOp most = f.ops[m];
      for (to = m; to < f.launches[l + 1] && f.ops[to].src == f.ops[m].src; ++to)
        for (int k = 0; k < 2; ++k) most.load[k] = std::max(most.load[k], f.ops[to].n[k]);
      for (size_t j = m; j < to; ++j)
        for (int k = 0; k < 2; ++k) f.ops[j].load[k] = most.load[k];
    }
}

// The page table under the moves: the host's copy and the pages' holders.
static void fork_table(witcert_cache* c, const ForkPlan& f, std::vector<int32_t>& kept) {
  auto drop = [&](int32_t pg) { if (--c->page_refs[pg] == 0) c->free_pages.push_back(pg); };
  const int nb = c->nblk_max;
  int kept_blocks = 0;
  for (const MoveOp& op : f.ops) {
    const int32_t* src = op.src >= 0 ? c->table_host.data() + (size_t)op.src * nb : kept.data();
    if (op.dst == kMoveKept) {
      for (int b = 0; b < op.blocks; ++b) { kept[b] = src[b]; ++c->page_refs[src[b]]; }
      kept_blocks = op.blocks;
      continue;
    }
    int32_t* dst = c->table_host.data() + (size_t)op.dst * nb;
    constexpr int kSpan = 64;                                  // beams share most of their pages
    for (int b0 = 0; b0 < op.blocks; b0 += kSpan) {
      const int b1 = std::min(op.blocks, b0 + kSpan);
      if (memcmp(dst + b0, src + b0, (b1 - b0) * sizeof *dst) == 0) continue;
      for (int b = b0; b < b1; ++b) {
        if (dst[b] == src[b]) continue;
        ++c->page_refs[src[b]];
        if (dst[b] >= 0) drop(dst[b]);
        dst[b] = src[b];
      }
    }
    for (int b = op.blocks; b < nb && dst[b] >= 0; ++b) {       // a sequence holds its first blocks, without gaps
      drop(dst[b]);
      dst[b] = -1;
    }
    if (op.src == kMoveKept) {
      for (int b = 0; b < kept_blocks; ++b) drop(kept[b]);
      kept_blocks = 0;
    }
  }
}

witcert_status witcert_fork(witcert_cache* c, const int32_t* parents, const int32_t* lengths, void* stream) try {
  if (!c || !parents) return fail(WITCERT_EINVAL, "cache and parents must not be NULL");
  if (c->cfg.max_repair_blocks > 0)
    return fail(WITCERT_EINVAL, "a gated cache cannot fork: repairs and the backing store belong to one sequence");
  const int B = c->cfg.batch, L = c->cfg.n_layers;
  ForkPlan f;
  f.from.resize(B); f.cap.assign(B, -1); f.blocks.assign(B, 0); f.tail.assign(B, 0);
  bool any = false;
  for (int i = 0; i < B; ++i) {
    const int p = parents[i];
    if (p < -1 || p >= B) return fail(WITCERT_EINVAL, "the parent of sequence %d must be in [-1, %d) (got %d)", i, B, p);
    if (lengths && p >= 0 && lengths[i] < 0) return fail(WITCERT_EINVAL, "lengths must be >= 0 (sequence %d: %d)", i, lengths[i]);
    f.from[i] = p;
    if (p < 0) { any = true; f.cap[i] = 0; continue; }
    const int cap = lengths ? lengths[i] : INT_MAX;
    bool cut = false;
    for (int l = 0; l < L; ++l) {
      const int now = c->slen[l][p], to = std::min(now, cap);
      cut |= to < now;
      if (c->scheme == kKivi && to < now && to % kBlk && to / kBlk < now / kBlk)
        return fail(WITCERT_EINVAL, "layer %d sequence %d: the exact keys of a finished KIVI block are gone; keep a "
                    "multiple of %d tokens or end within the unfinished block (at %d)", l, p, kBlk, now / kBlk * kBlk);
      f.blocks[i] = std::max(f.blocks[i], (to + kBlk - 1) / kBlk);
      f.tail[i] = std::max(f.tail[i], to % kBlk);
    }
    // a sequence that stays also gives back the pages past its last token
    const bool spare = lengths && c->table && p == i && f.blocks[i] < c->nblk_max &&
                       c->table_host[(size_t)i * c->nblk_max + f.blocks[i]] >= 0;
    if (p != i || cut || spare) { any = true; f.cap[i] = cap; }
  }
  if (!any) { ok(); return WITCERT_OK; }
  auto st = static_cast<cudaStream_t>(stream);
  follow(c, st);
  if (c->capture)
    return fail(WITCERT_ESTATE, "a fork cannot be captured: the lengths and pages on the host would not follow a replay");
  fork_moves(f);
  // host memory first: nothing may fail between what the device and what the host is told
  std::vector<std::vector<int>> slen(L, std::vector<int>(B));
  bool equal = true;
  for (int l = 0; l < L; ++l)
    for (int i = 0; i < B; ++i) {
      const int p = f.from[i], now = p < 0 ? 0 : c->slen[l][p];
      slen[l][i] = f.cap[i] < 0 ? now : std::min(now, f.cap[i]);
      equal &= slen[l][i] == slen[l][0];
    }
  std::vector<int32_t> kept(c->table ? c->nblk_max : 0);
  cudaError_t e = cudaSuccess;
  bool pdl = false;
  const bool lens = !equal || c->lengths_held;               // lengths that stay equal need no copy on the device
  if (!equal) e = enter_ragged(c, st, pdl);
  MoveRows rows{};
  auto stream_of = [&](void* base, size_t layer_pitch, size_t head_pitch, int unit, int count) {
    MoveStream& s = rows.s[rows.n_streams++];
    s.base = static_cast<uint8_t*>(base);
    s.layer_pitch = (long long)layer_pitch;
    s.head_pitch = (long long)head_pitch;
    s.seq_pitch = (long long)(head_pitch * c->cfg.n_kv_heads);
    s.unit = unit; s.count = count;
  };
  if (!c->table) stream_of(c->blocks, c->layer_blocks, (size_t)c->nblk_max * c->bblk, c->bblk, 0);
  if (c->vwit) stream_of(c->vwit, vwit_layer(c) * sizeof(__half), backing_rows(c) * sizeof(__half), kVwBytes, 0);
  if (c->kivi_tail)
    stream_of(c->kivi_tail, layer_rows(c) * kBlk * kD * sizeof(float), kBlk * kD * sizeof(float), kD * sizeof(float), 1);
  MoveInts ints{};
  ints.table = c->table;
  ints.lens = lens ? c->dlen : nullptr;
  ints.nblk_max = c->table ? c->nblk_max : 0;
  ints.layers = lens ? L : 0;
  ints.B = B;
  for (size_t k = 0; k + 1 < f.launches.size() && e == cudaSuccess; ++k) {
    const size_t m0 = f.launches[k], n = f.launches[k + 1] - m0;
    // up to kMoveGroups groups of about as many moves, each run down by threads of its own
    MoveGroups split{};
    split.first[0] = 0;
    for (size_t g : f.groups) {
      if (g <= m0 || g >= m0 + n || split.n + 1 == kMoveGroups) continue;
      if (g - m0 - split.first[split.n] >= (n + kMoveGroups - 1) / kMoveGroups) split.first[++split.n] = (int)(g - m0);
    }
    split.first[++split.n] = (int)n;
    rows.group = ints.group = split;
    rows.n = ints.n = (int)n;
    std::copy_n(f.ops.data() + m0, n, rows.op);
    std::copy_n(f.ops.data() + m0, n, ints.op);
    if (rows.n_streams) e = launch_move_rows(rows, L, c->cfg.n_kv_heads, st);
    if (e == cudaSuccess && (ints.table || ints.lens)) e = launch_move_ints(ints, st);
  }
  if (e != cudaSuccess) return cuda_fail(e, "fork");
  if (c->table) fork_table(c, f, kept);
  c->slen.swap(slen);
  c->ragged = !equal;
  for (int l = 0; l < L; ++l) {
    c->len[l] = *std::max_element(c->slen[l].begin(), c->slen[l].end());
    ++c->write_gen[l];
  }
  c->recent.write_layer = -1;
  c->recent.lengths_last = c->recent.apart = true;
  ok();
  return WITCERT_OK;
} WITCERT_NO_THROW

// The layer's store as the kernels that expand it read it.
static StoreArgs store_args(const witcert_cache* c, int layer) {
  StoreArgs s{};
  s.blocks = c->blocks + layer * c->layer_blocks;
  s.table = c->table;
  s.nblk_max = c->nblk_max; s.Hkv = c->cfg.n_kv_heads; s.layer = layer; s.pos0 = c->cfg.pos_offset;
  s.is_bf16 = c->cfg.kv_dtype == WITCERT_BF16;
  if (c->slots) s.slots = c->slots + layer * layer_rows(c) * c->nblk_max;
  s.pool = c->pool;
  if (c->kivi_tail) s.kivi_tail = c->kivi_tail + layer * layer_rows(c) * kBlk * kD;
  philox_round_keys(c->cfg.seed, s.rk0, s.rk1);
  return s;
}

witcert_status witcert_read(witcert_cache* c, int layer, const int32_t* t0, const int32_t* n_tok, void* K, void* V,
                            void* stream) {
  if (witcert_status s = check_layer(c, layer)) return s;
  if (!n_tok) return fail(WITCERT_EINVAL, "n_tok must not be NULL");
  const int B = c->cfg.batch;
  long long total = 0;
  for (int i = 0; i < B; ++i) {
    const long long from = t0 ? t0[i] : (long long)c->slen[layer][i] - n_tok[i];
    if (n_tok[i] < 0 || from < 0 || from + n_tok[i] > c->slen[layer][i])
      return fail(WITCERT_EINVAL, "layer %d sequence %d holds %d tokens; cannot read %d from %lld", layer, i,
                  c->slen[layer][i], n_tok[i], from);
    total += n_tok[i];
  }
  if (total == 0) { ok(); return WITCERT_OK; }
  if (!K || !V) return fail(WITCERT_EINVAL, "K and V must not be NULL");
  if (((uintptr_t)K | (uintptr_t)V) % 16) return fail(WITCERT_EINVAL, "K and V must be 16-byte aligned");
  auto st = static_cast<cudaStream_t>(stream);
  order_after_gate(c, layer, st);
  ReadArgs a{};
  a.s = store_args(c, layer);
  a.K = K; a.V = V;
  long long row = 0;
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < B && e == cudaSuccess; ++i) {
    const int n = n_tok[i];
    if (n > 0) {
      const int k = a.n_seq++, from = t0 ? t0[i] : c->slen[layer][i] - n;
      a.seq[k] = i; a.t0[k] = from; a.n[k] = n; a.len[k] = c->slen[layer][i];
      a.row0[k] = row;
      a.blk_off[k + 1] = a.blk_off[k] + (from + n - 1) / kBlk - from / kBlk + 1;
      row += n;
    }
    if (a.n_seq == kRaggedPerLaunch || (i + 1 == B && a.n_seq)) {
      e = launch_read(c->scheme, a, st);
      a.n_seq = 0;
    }
  }
  if (e != cudaSuccess) return cuda_fail(e, "read launch");
  launched_apart(c, st);
  ok();
  return WITCERT_OK;
}

// ------------------------------------------------------------------ chunk attention
// One group of sequences: expanded, attended and merged by one launch each.
// Operand images of a group (64 KB per 128 tokens and KV head) stay below kImageCap, unless a single
// sequence needs more.
constexpr size_t kImageCap = size_t(2) << 30;

// Row tiles of sequence k, and key tiles of its row tile number rt in unit order (last rows first).
static int attend_row_tiles(const AttendArgs& a, int k) { return (int)(((long long)a.n[k] * a.grp + a.unit_rows - 1) / a.unit_rows); }
static int attend_key_tiles(const AttendArgs& a, int k, int rt) {
  const long long rows = (long long)a.n[k] * a.grp, r0 = (long long)(attend_row_tiles(a, k) - 1 - rt) * a.unit_rows;
  const long long last = std::min(rows, r0 + a.unit_rows) - 1;
  return (int)((a.len[k] - a.n[k] + last / a.grp) / kTileTok) + 1;
}

// Shares the units' key tiles out to CTAs, one an SM: the same time to each, units cut where that
// falls, unless whole units do as well.  A unit's time is its key tiles and its start and end (queries
// in, outputs out, the pipeline empty), as long as kStart tiles: with 0, 2, 3, 4 and 6 of them 4096 new
// tokens of 4096 take 318.7, 190.0, 156.3, 147.1, 144.6 us, 700 of 6000 in three sequences 197.8,
// 187.9, 187.6, 187.6, 189.6, and, straight from the store, 4 of 700 in forty sequences 40.5, 39.6,
// 39.6, 41.6, 41.6, 16 of 16384 in two 51.8, 49.8, 47.1, 47.1, 47.7.  A cut costs the records' merge and a second start of the
// pipeline, about kCutTiles key tiles' time, and shares below kMinShare tiles are not worth it: FP8,
// 32 query heads on 8, four tokens a sequence, with (kCutTiles, kMinShare) of (0, 1), (3, 2) and only
// whole units: 16 sequences of 1000 tokens 29.3, 21.2, 21.2 us; 4 of 1024 17.1, 17.1, 19.1; 1 of 512
// 12.9, 14.3, 15.0; 40 of 2000 68.2, 67.2, 76.4.
static void share_units(AttendArgs& a, int sm_count) {
  constexpr int kCutTiles = 3, kMinShare = 2;
  const int kStart = a.unit_rows > kTileRows ? 4 : 3;
  const int Hkv = a.s.Hkv, sms = std::min(sm_count, kAttendCtas);
  long long total = 0, units = 0;
  int most = 1;
  for (int k = 0; k < a.n_seq; ++k)
    for (int rt = 0, rts = attend_row_tiles(a, k); rt < rts; ++rt) {
      const int nt = attend_key_tiles(a, k, rt);
      units += Hkv;
      total += (long long)(nt + kStart) * Hkv;
      most = std::max(most, nt);
    }
  const long long per_cta = (units + sms - 1) / sms;
  const long long even = std::max<long long>((total + sms - 1) / sms, std::min(kMinShare, most) + kStart);
  const bool whole = per_cta * (most + kStart) <= even + kCutTiles;
  // CTA c starts at place c * share, counted in units or in tiles' times (a unit's start first)
  const long long share = whole ? per_cta : even;
  a.n_ctas = (int)(((whole ? units : total) + share - 1) / share);
  int c = 0;
  long long at = 0;                                          // places before the present row tile's units
  for (int k = 0; k < a.n_seq; ++k)
    for (int rt = 0, rts = attend_row_tiles(a, k); rt < rts; ++rt) {
      const int weight = whole ? 1 : attend_key_tiles(a, k, rt) + kStart;
      for (; c < a.n_ctas && c * share < at + (long long)weight * Hkv; ++c) {
        const long long in = c * share - at;
        a.start[c] = {k, rt, (int)(in / weight), whole ? 0 : std::max(0, (int)(in % weight) - kStart)};
        a.cut |= a.start[c].j > 0;
      }
      at += (long long)weight * Hkv;
    }
  a.start[a.n_ctas] = {a.n_seq, 0, 0, 0};
}

// Sequences of at most this many query rows a KV head are attended straight from the store, each
// row tile of 128 reading the codes itself; longer ones share operand images.  Images against store,
// us, 32 query heads on 8: one sequence of 32768 tokens, FP8, 256 rows 109.8 / 74.4, 512 117.4 / 105.1,
// 1024 152.8 / 176.8; two-bit 256 105.7 / 92.8, 384 112.1 / 117.4; eight sequences of 4096, FP8, 256
// 93.4 / 58.0, 512 99.0 / 109.2.  Where every row tile forms the dither itself, one is the limit: 132
// rows 140.8 / 187.0 (with a shared dither, eight sequences, 256 rows: 110.2 / 99.0).
constexpr int kFewRows = 2 * kTileRows, kFewRowsDither = kTileRows;

// What an attend call launches, and the parts of its workspace: the images and the records of the
// largest group, and the dithered store's dither.
struct AttendPlan {
  std::vector<AttendArgs> groups;
  size_t image_bytes = 0, rec_bytes = 0, dither_bytes = 0;
  int dither_tiles = 0;
  size_t bytes() const { return image_bytes + rec_bytes + dither_bytes; }
};
// Sequences that share a dither have it formed once when together they read it at least twice.  Formed
// once against formed by each, us, sequences of 8192 tokens, four new tokens each: 1 sequence 39.6 /
// 39.6, 2 49.8 / 58.0, 4 65.0 / 96.9, 8 98.9 / 174.7; 128 new tokens: 1 75.4 / 70.8, 2 95.4 / 91.4,
// 8 236.2 / 255.2.
constexpr int kDitherShare = 2;

static void plan_attend(const witcert_cache* c, int layer, const int32_t* n_tok, AttendPlan& plan) {
  std::vector<AttendArgs>& groups = plan.groups;
  size_t &image_bytes = plan.image_bytes, &rec_bytes = plan.rec_bytes;
  const int B = c->cfg.batch, Hkv = c->cfg.n_kv_heads, grp = c->cfg.n_q_heads / Hkv;
  const size_t tile = (size_t)Hkv * 2 * kTileBytes;
  long long read_tiles = 0;
  for (int i = 0; i < B && c->scheme == kInt8; ++i)
    if (n_tok[i] > 0) {
      const int tiles = (c->slen[layer][i] + kTileTok - 1) / kTileTok;
      read_tiles += tiles;
      plan.dither_tiles = std::max(plan.dither_tiles, tiles);
    }
  if (read_tiles < (long long)kDitherShare * plan.dither_tiles) plan.dither_tiles = 0;
  plan.dither_bytes = plan.dither_tiles * Hkv * kDitherTile;
  const long long most_few = c->scheme == kInt8 && !plan.dither_tiles ? kFewRowsDither : kFewRows;
  for (const int unit_rows : {kTinyRows, kTileRows, 2 * kTileRows}) {
    const bool few = unit_rows <= kTileRows;
    bool open = false;
    int row0 = 0;
    for (int i = 0; i < B; ++i) {
      const int n = n_tok[i], len = c->slen[layer][i], at = row0;
      row0 += n;
      const long long rows = (long long)n * grp;
      if (n == 0 || unit_rows != (rows <= kTinyRows ? kTinyRows : rows <= most_few ? kTileRows : 2 * kTileRows)) continue;
      const int tiles = (len + kTileTok - 1) / kTileTok;
      if (!open || groups.back().n_seq == kAttendSeqs ||
          (!few && (groups.back().tile_off[groups.back().n_seq] + (size_t)tiles) * tile > kImageCap)) {
        groups.emplace_back();
        AttendArgs& g = groups.back();
        memset(&g, 0, sizeof g);
        g.s = store_args(c, layer);
        g.Hq = c->cfg.n_q_heads; g.grp = grp;
        g.unit_rows = unit_rows;
        g.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)kD));
        g.err = c->err;
        open = true;
      }
      AttendArgs& a = groups.back();
      const int k = a.n_seq++;
      a.seq[k] = i; a.n[k] = n; a.len[k] = len; a.row0[k] = at;
      a.tile_off[k + 1] = a.tile_off[k] + tiles;
    }
  }
  for (AttendArgs& a : groups) {
    share_units(a, c->sm_count);
    if (a.unit_rows > kTileRows) image_bytes = std::max(image_bytes, a.tile_off[a.n_seq] * tile);
    rec_bytes = std::max(rec_bytes, (size_t)2 * a.n_ctas * a.unit_rows * kRecStride * sizeof(float));
  }
}

// The kernels of a call overlap their starts with their predecessors' ends; the first one (after = 0)
// is launched like any other kernel.
static cudaError_t attend_group(int scheme, AttendArgs& a, cudaStream_t st) {
  cudaError_t e;
  if (a.unit_rows <= kTileRows) {
    switch (scheme) {
      case kInt8: e = launch_attend_few<kInt8>(a, st); break;
      case kRtn: e = launch_attend_few<kRtn>(a, st); break;
      case kFp8: e = launch_attend_few<kFp8>(a, st); break;
      case kKivi: e = launch_attend_few<kKivi>(a, st); break;
      default: e = launch_attend_few<kBbox>(a, st); break;
    }
  } else {
    e = launch_expand(scheme, a, st);
    a.after = 1;
    if (e == cudaSuccess) e = launch_attend(scheme, a, st);
  }
  a.after = 1;
  return e == cudaSuccess ? launch_attend_merge(a, st) : e;
}

static witcert_status check_attend(const witcert_cache* c, int layer, const int32_t* n_tok, long long& rows) {
  if (witcert_status s = check_layer(c, layer)) return s;
  if (!n_tok) return fail(WITCERT_EINVAL, "n_tok must not be NULL");
  if (c->cfg.kv_dtype != WITCERT_BF16) return fail(WITCERT_EINVAL, "chunk attention needs a bf16 cache");
  rows = 0;
  for (int i = 0; i < c->cfg.batch; ++i) {
    if (n_tok[i] < 0 || n_tok[i] > c->slen[layer][i])
      return fail(WITCERT_EINVAL, "layer %d sequence %d holds %d tokens; %d queries do not fit", layer, i,
                  c->slen[layer][i], n_tok[i]);
    rows += n_tok[i];
  }
  if (rows * c->cfg.n_q_heads > INT_MAX) return fail(WITCERT_EINVAL, "too many query rows (%lld)", rows);
  return WITCERT_OK;
}

witcert_status witcert_attend_workspace(const witcert_cache* c, int layer, const int32_t* n_tok, size_t* bytes) try {
  long long rows = 0;
  if (witcert_status s = check_attend(c, layer, n_tok, rows)) return s;
  if (!bytes) return fail(WITCERT_EINVAL, "bytes must not be NULL");
  AttendPlan plan;
  plan_attend(c, layer, n_tok, plan);
  *bytes = plan.bytes();
  ok();
  return WITCERT_OK;
} WITCERT_NO_THROW

witcert_status witcert_attend(witcert_cache* c, int layer, const void* q, const int32_t* n_tok, void* out,
                              void* workspace, size_t workspace_bytes, void* stream) try {
  long long rows = 0;
  if (witcert_status s = check_attend(c, layer, n_tok, rows)) return s;
  if (rows == 0) { ok(); return WITCERT_OK; }
  if (!q || !out) return fail(WITCERT_EINVAL, "q and out must not be NULL");
  if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) % 32)
    return fail(WITCERT_EINVAL, "q, out and workspace must be 32-byte aligned");
  AttendPlan plan;
  plan_attend(c, layer, n_tok, plan);
  if (plan.bytes() > workspace_bytes || !workspace)
    return fail(WITCERT_EINVAL, "the workspace needs %zu bytes, got %zu", plan.bytes(), workspace ? workspace_bytes : 0);
  auto st = static_cast<cudaStream_t>(stream);
  order_after_gate(c, layer, st);
  uint8_t* images = static_cast<uint8_t*>(workspace);
  uint4* dither = plan.dither_tiles ? reinterpret_cast<uint4*>(images + plan.image_bytes + plan.rec_bytes) : nullptr;
  if (dither) {
    cudaError_t e = launch_dither_table(store_args(c, layer), dither, plan.dither_tiles, st);
    if (e != cudaSuccess) return cuda_fail(e, "dither launch");
  }
  for (AttendArgs& a : plan.groups) {
    a.q = q; a.out = out;
    a.images = images;
    a.rec = reinterpret_cast<float*>(images + plan.image_bytes);
    a.s.dither = dither;
    a.after = dither || &a != plan.groups.data();
    cudaError_t e = attend_group(c->scheme, a, st);
    if (e != cudaSuccess) return cuda_fail(e, "attend launch");
  }
  launched_apart(c, st);
  ok();
  return WITCERT_OK;
} WITCERT_NO_THROW

// Automatic split count for a decode of nblk blocks: sized by how many split-kernel CTAs of
// this configuration fit on an SM, and never above the scratch sized at create time.
static int auto_splits(const witcert_cache* c, int nblk, bool meter, int cap) {
  DecodeArgs a{};
  a.B = c->cfg.batch;
  a.is_bf16 = c->cfg.kv_dtype == WITCERT_BF16;
  a.meter = meter;
  a.slots = c->slots;
  const int per_sm = decode_ctas_per_sm(c->scheme, a);
  int s = decode_auto_splits(c->scheme, c->cfg.batch, c->cfg.n_kv_heads, nblk > 0 ? nblk : 1, c->sm_count, per_sm);
  if (cap > 0 && s > cap) s = cap;
  return s;
}

// Decode arguments shared by every decode entry point: the layer's store, the query, the
// split count and the Tier B factor kappa = sqrt(2 ln(2 S / delta_loc)) rounded up, with S
// the attended context (s_kappa; the layer's own length when 0).
static void fill_decode(witcert_cache* c, int layer, const void* q, double delta_req, bool meter, long long s_kappa,
                        DecodeArgs& a) {
  const int S = c->len[layer];
  const int nblk = (S + kBlk - 1) / kBlk;
  a.blocks = c->blocks + layer * c->layer_blocks;
  a.nblk_max = c->nblk_max;
  if (c->slots) a.slots = c->slots + layer * layer_rows(c) * c->nblk_max;
  a.pool = c->pool;
  if (c->kivi_tail) a.kivi_tail = c->kivi_tail + layer * layer_rows(c) * kBlk * kD;
  a.q = q;
  a.is_bf16 = c->cfg.kv_dtype == WITCERT_BF16;
  a.B = c->cfg.batch; a.Hq = c->cfg.n_q_heads; a.Hkv = c->cfg.n_kv_heads; a.grp = a.Hq / a.Hkv; a.S = S;
  if (c->ragged) a.seq_len = c->dlen + (size_t)layer * c->cfg.batch;
  a.table = c->table;
  a.n_splits = c->cfg.n_splits > 0 ? c->cfg.n_splits : auto_splits(c, nblk, meter, c->max_splits);
  a.seed = c->cfg.seed;
  philox_round_keys(a.seed, a.rk0, a.rk1);
  a.layer = layer;
  a.pos0 = c->cfg.pos_offset;
  a.dirty_blk = c->recent.write_layer == layer ? c->recent.write_blk : INT_MAX;
  float kappa = 0.f;
  const long long Sk = s_kappa > 0 ? s_kappa : S;
  if (meter && Sk > 0) {
    const double dloc = delta_req / ((double)c->cfg.n_layers * c->cfg.n_q_heads * c->cfg.total_steps);
    const double k = std::sqrt(2.0 * std::log(2.0 * (double)Sk / dloc));
    kappa = (float)k;
    if ((double)kappa < k) kappa = std::nextafter(kappa, INFINITY);
  }
  if (meter) a.log2dl = std::log(2.0 * (double)c->cfg.n_layers * c->cfg.n_q_heads * c->cfg.total_steps / delta_req);
  a.kappa = kappa;
  a.err = c->err;
  if (layer + 1 < c->cfg.n_layers && c->len[layer + 1] > 0) a.next_blocks = c->blocks + (layer + 1) * c->layer_blocks;
  if (c->vwit && meter) a.vwit = c->vwit + layer * vwit_layer(c);
  a.meter = meter;
}

witcert_status witcert_decode(witcert_cache* c, int layer, const void* q, double delta_req, float* out,
                              float* meter_a, float* meter_b, float* raw_a, float* raw_b, float* meter_v,
                              void* stream) try {
  if (witcert_status s = check_layer(c, layer)) return s;
  if (!q || !out) return fail(WITCERT_EINVAL, "q and out must not be NULL");
  if (meter_v && !c->vwit) return fail(WITCERT_EINVAL, "meter_v needs a cache created with v_witness");
  const bool meter = meter_a || meter_b || raw_a || raw_b || meter_v;
  if (meter && !(delta_req > 0.0 && delta_req <= 1.0)) return fail(WITCERT_EINVAL, "delta_req must be in (0, 1]");
  auto st = static_cast<cudaStream_t>(stream);
  follow(c, st);
  const bool waited = order_after_gate(c, layer, st);
  DecodeArgs a{};
  fill_decode(c, layer, q, delta_req, meter, 0, a);
  a.part = c->part;
  const bool gate = c->cfg.max_repair_blocks > 0;
  if (gate && meter) {
    a.risk_raw = c->risk_raw;
    a.risk = c->risk + (size_t)layer * a.B * a.Hq * c->nblk_max;
  }
  a.out = out; a.meter_a = meter_a; a.meter_b = meter_b; a.raw_a = raw_a; a.raw_b = raw_b; a.meter_v = meter_v;
  ProfPair pp{nullptr, nullptr};
  if (c->profiling) {
    if (c->prof_free.empty()) {
      ProfPair n{};
      if (cudaEventCreate(&n.a) != cudaSuccess || cudaEventCreate(&n.b) != cudaSuccess)
        return cuda_fail(cudaGetLastError(), "creating profiling events");
      c->prof_free.push_back(n);
    }
    pp = c->prof_free.back();
    c->prof_free.pop_back();
  }
  // the split kernel reads the sequence lengths before it waits for its predecessor
  cudaError_t e = launch_decode(c->scheme, a, c->sm_count, st, pp.a, pp.b, may_overlap(c, waited) && !c->recent.lengths_last);
  if (pp.a) c->prof_pending.push_back(pp);
  if (e != cudaSuccess) return cuda_fail(e, "decode launch");
  c->recent = Recent{};
  if (c->capture && a.seq_len) c->lengths_held = true;
  if (gate && meter) c->risk_gen[layer] = c->write_gen[layer];
  c->last_n_splits = a.n_splits;
  ++c->decode_calls;
  ok();
  return WITCERT_OK;
} WITCERT_NO_THROW

witcert_status witcert_decode_noalloc(witcert_cache* c, int layer, const void* q, double delta_req, float* out,
                                      float* meter_a, float* meter_b, float* raw_a, float* raw_b, float* meter_v,
                                      void* stream) {
  if (witcert_status s = check_layer(c, layer)) return s;
  if (!q || !out) return fail(WITCERT_EINVAL, "q and out must not be NULL");
  if (meter_v && !c->vwit) return fail(WITCERT_EINVAL, "meter_v needs a cache created with v_witness");
  const bool meter = meter_a || meter_b || raw_a || raw_b || meter_v;
  if (meter && !(delta_req > 0.0 && delta_req <= 1.0)) return fail(WITCERT_EINVAL, "delta_req must be in (0, 1]");
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != c->device)
    return fail(WITCERT_EINVAL, "the cache lives on device %d; make it current before this call", c->device);
  auto st = static_cast<cudaStream_t>(stream);
  follow(c, st);
  DecodeArgs a{};
  fill_decode(c, layer, q, delta_req, meter, 0, a);
  float* scratch = nullptr;
  size_t scratch_bytes = 0;
  cudaError_t e = decode_static_scratch(&scratch, &scratch_bytes);
  if (e != cudaSuccess) return cuda_fail(e, "locating the static split scratch");
  const size_t need = (size_t)a.B * a.Hq * a.n_splits * kPartStride * sizeof(float);
  if (need > scratch_bytes)
    return fail(WITCERT_EINVAL, "batch %d x %d query heads x %d splits needs %zu bytes of split scratch; "
                "the static array holds %zu", a.B, a.Hq, a.n_splits, need, scratch_bytes);
  const bool waited = order_after_gate(c, layer, st);
  a.dirty_blk = c->recent.write_layer == layer ? c->recent.write_blk : INT_MAX;
  a.part = scratch;
  const bool gate = c->cfg.max_repair_blocks > 0;
  if (gate && meter) {
    a.risk_raw = c->risk_raw;
    a.risk = c->risk + (size_t)layer * a.B * a.Hq * c->nblk_max;
  }
  a.out = out; a.meter_a = meter_a; a.meter_b = meter_b; a.raw_a = raw_a; a.raw_b = raw_b; a.meter_v = meter_v;
  e = launch_decode(c->scheme, a, c->sm_count, st, nullptr, nullptr, may_overlap(c, waited) && !c->recent.lengths_last);
  if (e != cudaSuccess) return cuda_fail(e, "decode launch");
  c->recent = Recent{};
  if (c->capture && a.seq_len) c->lengths_held = true;
  if (gate && meter) c->risk_gen[layer] = c->write_gen[layer];
  c->last_n_splits = a.n_splits;
  ++c->decode_calls;
  ok();
  return WITCERT_OK;
}

witcert_status witcert_decode_partial(witcert_cache* c, int layer, const void* q, double delta_req,
                                      long long s_total, float* part, void* stream) {
  if (witcert_status s = check_layer(c, layer)) return s;
  if (!q || !part) return fail(WITCERT_EINVAL, "q and part must not be NULL");
  if (!(delta_req > 0.0 && delta_req <= 1.0)) return fail(WITCERT_EINVAL, "delta_req must be in (0, 1]");
  if (s_total < c->len[layer]) return fail(WITCERT_EINVAL, "s_total %lld is below the slice's own %d tokens",
                                           s_total, c->len[layer]);
  if (c->ragged) return fail(WITCERT_ESTATE, "context-parallel shards hold equal-length sequences");
  auto st = static_cast<cudaStream_t>(stream);
  follow(c, st);
  const bool waited = order_after_gate(c, layer, st);
  DecodeArgs a{};
  fill_decode(c, layer, q, delta_req, true, s_total, a);
  a.part = c->part;
  a.part_out = part;
  a.risk_raw = c->risk_raw;      // a gated cache's split kernel writes block risks; the merge keeps none (no a.risk)
  cudaError_t e = launch_decode(c->scheme, a, c->sm_count, st, nullptr, nullptr, may_overlap(c, waited));
  if (e != cudaSuccess) return cuda_fail(e, "decode launch");
  c->recent.write_layer = -1;
  c->recent.apart = false;
  c->last_n_splits = a.n_splits;
  ++c->decode_calls;
  ok();
  return WITCERT_OK;
}

witcert_status witcert_merge_partials(const float* parts, int n_parts, int batch, int n_q_heads,
                                      witcert_scheme scheme, float* out, float* meter_a, float* meter_b,
                                      float* raw_a, float* raw_b, float* meter_v, void* stream) {
  if (!parts || !out) return fail(WITCERT_EINVAL, "parts and out must not be NULL");
  if (n_parts < 1 || batch < 1 || n_q_heads < 1) return fail(WITCERT_EINVAL, "n_parts, batch and n_q_heads must be >= 1");
  if (scheme < WITCERT_INT8_DITHER || scheme > WITCERT_BLACKBOX) return fail(WITCERT_EINVAL, "unknown scheme %d", (int)scheme);
  DecodeArgs a{};
  a.part = const_cast<float*>(parts);
  a.n_splits = n_parts;
  a.B = batch; a.Hq = n_q_heads;
  a.out = out; a.meter_a = meter_a; a.meter_b = meter_b; a.raw_a = raw_a; a.raw_b = raw_b; a.meter_v = meter_v;
  a.meter = meter_a || meter_b || raw_a || raw_b || meter_v;
  cudaError_t e = launch_merge_records((int)scheme, a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "merge launch");
  ok();
  return WITCERT_OK;
}

witcert_status witcert_gate(witcert_cache* c, int layer, float tau, void* stream) {
  if (witcert_status s = check_layer(c, layer)) return s;
  if (c->cfg.max_repair_blocks <= 0) return fail(WITCERT_ESTATE, "the gate is disabled (max_repair_blocks = 0)");
  if (!(tau >= 0.f) || !std::isfinite(tau)) return fail(WITCERT_EINVAL, "tau must be finite and >= 0");
  if (c->risk_gen[layer] != c->write_gen[layer] || c->len[layer] == 0)
    return fail(WITCERT_ESTATE, "layer %d has no metered decode since its last write", layer);
  if (c->backing_lost[layer])
    return fail(WITCERT_EPAGEIN, "layer %d: the backing store lost exact keys; nothing was paged in", layer);
  auto st = static_cast<cudaStream_t>(stream);
  cudaEvent_t ready = c->gate_done[layer];
  cudaError_t e = cudaEventRecord(ready, st);   // reuse: marks the point the gate must follow
  if (e == cudaSuccess) e = cudaStreamWaitEvent(c->side, ready, 0);
  if (e == cudaSuccess) e = cudaMemsetAsync(c->todo_count, 0, sizeof(unsigned int), c->side);
  if (e != cudaSuccess) return cuda_fail(e, "gate ordering");
  GateArgs a{};
  const size_t cells = (size_t)c->cfg.batch * c->cfg.n_q_heads;
  a.risk = c->risk + (size_t)layer * cells * c->nblk_max;
  a.slots = c->slots + layer * layer_rows(c) * c->nblk_max;
  a.selmask = c->selmask; a.todo = c->todo; a.todo_count = c->todo_count; a.pool_next = c->pool_next;
  a.stats = c->gstats;
  a.blocks = c->blocks + layer * c->layer_blocks;
  a.backing = static_cast<uint8_t*>(c->backing_dev) + layer * layer_rows(c) * backing_rows(c) * kD * c->elem;
  a.pool = c->pool;
  a.nblk_max = c->nblk_max; a.B = c->cfg.batch; a.Hq = c->cfg.n_q_heads; a.Hkv = c->cfg.n_kv_heads;
  a.grp = a.Hq / a.Hkv; a.S = c->len[layer]; a.backing_rows = (int)backing_rows(c);
  if (c->ragged) a.seq_len = c->dlen + (size_t)layer * c->cfg.batch;
  a.table = c->table;
  a.pool_capacity = c->cfg.max_repair_blocks; a.scheme = c->scheme; a.elem_bytes = c->elem;
  a.d_star = std::sqrt(1.0 + 2.0 * (double)tau) - 1.0;
  e = launch_gate(a, c->side);
  if (e == cudaSuccess) e = cudaEventRecord(c->gate_done[layer], c->side);
  if (e != cudaSuccess) return cuda_fail(e, "gate launch");
  c->gate_pending[layer] = 1;
  ++c->gate_calls;
  ok();
  return WITCERT_OK;
}

witcert_status witcert_gate_select(const float* risk, const uint8_t* repaired, int batch, int n_q_heads,
                                   int n_kv_heads, int nblk, float tau, uint32_t* selected, void* stream) {
  if (!risk || !selected) return fail(WITCERT_EINVAL, "risk and selected must not be NULL");
  if (batch < 1 || n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads)
    return fail(WITCERT_EINVAL, "batch >= 1 and n_q_heads a positive multiple of n_kv_heads");
  if (nblk < 1 || nblk > gate_max_blocks()) return fail(WITCERT_EINVAL, "nblk must be in [1, %d]", gate_max_blocks());
  if (!(tau >= 0.f) || !std::isfinite(tau)) return fail(WITCERT_EINVAL, "tau must be finite and >= 0");
  auto st = static_cast<cudaStream_t>(stream);
  GateArgs a{};
  a.risk = risk;
  a.repaired = repaired;
  a.selmask = selected;
  a.nblk_max = nblk; a.B = batch; a.Hq = n_q_heads; a.Hkv = n_kv_heads; a.grp = n_q_heads / n_kv_heads;
  a.S = nblk * kBlk;
  a.d_star = std::sqrt(1.0 + 2.0 * (double)tau) - 1.0;
  cudaError_t e = cudaMemsetAsync(selected, 0, (size_t)batch * n_kv_heads * (nblk / 32 + 1) * sizeof(uint32_t), st);
  if (e == cudaSuccess) e = launch_gate_select(a, st);
  if (e != cudaSuccess) return cuda_fail(e, "gate selection");
  ok();
  return WITCERT_OK;
}

// ------------------------------------------------------------------ beam search
// A step whose requests have a cluster each and whose clusters' warps have this many chunks at most is one launch,
// which costs the host 5.5 us less and the GPU a little more.  One launch / two, us, through the binding and in a
// graph: 1 request of 4 beams, 32000 tokens (1 chunk a warp) 19.1 / 24.7, 7.9 / 7.6; 10 of 8 beams (2) 18.9 / 24.1, 8.9 /
// 8.6; 1 of 4, 152001 tokens (4.6) 18.8 / 24.5, 11.2 / 8.4; 1 of 8, 131072 (8) 18.7 / 24.4, 13.1 / 9.5; 2 of 32, 50001 fp32
// (12) 26.7 / 24.3, 24.8 / 14.5.  Clusters may take two thirds of the SMs: those of 16 requests do not all find their
// place at once (first steps of 4 beams, 131072 tokens: 16.6 / 9.2 in a graph).
constexpr int kClusterChunks = 5;

// Checks a step and lays out its scan.
static witcert_status beam_args(const witcert_beam_step* s, BeamArgs& a, size_t& bytes) {
  if (!s) return fail(WITCERT_EINVAL, "step must not be NULL");
  if (s->dtype != WITCERT_F32 && s->dtype != WITCERT_BF16) return fail(WITCERT_EINVAL, "unknown dtype %d", (int)s->dtype);
  if (s->n_requests < 0) return fail(WITCERT_EINVAL, "n_requests must be >= 0");
  if (s->n_beams < 1 || s->n_beams > kBeamMaxBeams) return fail(WITCERT_EINVAL, "n_beams must be in [1, %d] (got %d)", kBeamMaxBeams, s->n_beams);
  if (s->vocab < 1 || s->vocab > 1 << 25) return fail(WITCERT_EINVAL, "vocab must be in [1, 2^25] (got %d)", s->vocab);
  if (s->n_out < 1 || s->n_out > kBeamMaxOut) return fail(WITCERT_EINVAL, "n_out must be in [1, %d] (got %d)", kBeamMaxOut, s->n_out);
  if (s->eos < -1 || s->eos >= s->vocab) return fail(WITCERT_EINVAL, "eos must be in [-1, %d) (got %d)", s->vocab, s->eos);
  if (s->finished && s->eos < 0) return fail(WITCERT_EINVAL, "finished beams need eos");
  const int elem = s->dtype == WITCERT_BF16 ? 2 : 4;
  const long long rows = (long long)s->n_requests * s->n_beams;
  if (rows > INT_MAX || (long long)s->n_requests * s->n_out > INT_MAX) return fail(WITCERT_EINVAL, "too many rows (%lld)", rows);
  const uintptr_t at = (uintptr_t)s->logits;
  if (at % elem) return fail(WITCERT_EINVAL, "logits must be aligned to their elements");
  // a row's chunks begin at a 32-byte boundary at or before it
  const bool even = at % 32 == 0 && (s->n_requests < 2 || s->request_stride * elem % 32 == 0) &&
                    (s->n_beams < 2 || s->beam_stride * elem % 32 == 0);
  a.chunks = (int)((s->vocab + (even ? 0 : 32 / elem - 1) + (long long)kBeamChunk - 1) / kBeamChunk);
  const int sms = sm_count_now();
  a.clustered = (long long)s->n_requests * kBeamCluster * 3 / 2 <= sms && (long long)s->n_beams * a.chunks <= kClusterChunks * kBeamClusterWarps;
  if (a.clustered) {
    a.parts = std::min(a.chunks, kBeamClusterWarps / s->n_beams);
  } else {
    // a warp a chunk where the rows are few; one wave of warps, then more waves of at most nine chunks a warp
    const long long warps = (long long)sms * kBeamScanWarps;
    a.parts = (int)std::min<long long>(a.chunks, std::max(warps / std::max(rows, 1ll), (a.chunks + 8ll) / 9));
  }
  a.chunks_inv = UINT32_MAX / (uint32_t)a.chunks;
  if (rows * a.parts > INT_MAX) return fail(WITCERT_EINVAL, "too many logits (%lld rows of %d)", rows, s->vocab);
  bytes = (size_t)rows * (a.parts * sizeof(float2) + a.chunks * sizeof(float));
  a.logits = s->logits;
  a.request_stride = s->request_stride; a.beam_stride = s->beam_stride;
  a.scores = s->scores; a.finished = s->finished;
  a.requests = s->n_requests; a.beams = s->n_beams; a.vocab = s->vocab; a.n_out = s->n_out; a.eos = s->eos;
  a.is_bf16 = s->dtype == WITCERT_BF16;
  a.out_scores = s->out_scores; a.rows = s->rows; a.tokens = s->tokens; a.out_finished = s->out_finished;
  return WITCERT_OK;
}

witcert_status witcert_beam_workspace(const witcert_beam_step* step, size_t* bytes) {
  BeamArgs a{};
  size_t need = 0;
  if (witcert_status s = beam_args(step, a, need)) return s;
  if (!bytes) return fail(WITCERT_EINVAL, "bytes must not be NULL");
  *bytes = need;
  ok();
  return WITCERT_OK;
}

witcert_status witcert_beam_select(const witcert_beam_step* step, void* workspace, size_t workspace_bytes, void* stream) {
  BeamArgs a{};
  size_t need = 0;
  if (witcert_status s = beam_args(step, a, need)) return s;
  if (a.requests == 0) { ok(); return WITCERT_OK; }
  if (!a.logits || !a.scores || !a.out_scores || !a.rows || !a.tokens)
    return fail(WITCERT_EINVAL, "logits, scores, out_scores, rows and tokens must not be NULL");
  if (a.n_out != a.beams && a.requests > 1 && (a.out_scores == a.scores || (a.finished && a.out_finished == a.finished)))
    return fail(WITCERT_EINVAL, "outputs may be the inputs only with n_out = n_beams");
  if (!workspace || workspace_bytes < need || (uintptr_t)workspace % 16)
    return fail(WITCERT_EINVAL, "the workspace needs %zu bytes, 16-byte aligned, got %zu", need, workspace ? workspace_bytes : 0);
  a.records = static_cast<float2*>(workspace);
  a.maxima = reinterpret_cast<float*>(a.records + (size_t)a.requests * a.beams * a.parts);
  cudaError_t e = launch_beam_select(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "beam selection launch");
  ok();
  return WITCERT_OK;
}

witcert_status witcert_beam_paths(const int32_t* rows, const int32_t* tokens, int n_steps, int n_requests, int n_beams,
                                  const int32_t* length, int pad, int32_t* out, void* stream) {
  if (n_steps < 0 || n_requests < 0) return fail(WITCERT_EINVAL, "n_steps and n_requests must be >= 0");
  if (n_beams < 1 || n_beams > kBeamMaxBeams) return fail(WITCERT_EINVAL, "n_beams must be in [1, %d] (got %d)", kBeamMaxBeams, n_beams);
  if ((long long)n_requests * n_beams > INT_MAX) return fail(WITCERT_EINVAL, "too many rows");
  if (n_steps == 0 || n_requests == 0) { ok(); return WITCERT_OK; }
  if (!rows || !tokens || !out) return fail(WITCERT_EINVAL, "rows, tokens and out must not be NULL");
  PathArgs a{rows, tokens, length, out, n_steps, n_requests, n_beams, pad, 0, 0, 0};
  cudaError_t e = launch_beam_paths(a, sm_count_now(), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "beam paths launch");
  ok();
  return WITCERT_OK;
}

witcert_status witcert_inject_fault(witcert_cache* c, witcert_fault fault, int layer) {
  if (witcert_status s = check_layer(c, layer)) return s;
  if (fault != WITCERT_FAULT_BACKING_LOST) return fail(WITCERT_EINVAL, "unknown fault %d", (int)fault);
  if (c->cfg.max_repair_blocks <= 0) return fail(WITCERT_ESTATE, "the gate is disabled: there is no backing store");
  c->backing_lost[layer] = 1;
  ok();
  return WITCERT_OK;
}

witcert_status witcert_gate_stats(witcert_cache* c, witcert_gate_counters* out, int timeout_ms) {
  if (!c || !out) return fail(WITCERT_EINVAL, "NULL argument");
  memset(out, 0, sizeof *out);
  out->gate_calls = c->gate_calls;
  if (c->cfg.max_repair_blocks <= 0) { ok(); return WITCERT_OK; }
  const auto deadline = std::chrono::steady_clock::now() + std::chrono::milliseconds(timeout_ms < 0 ? 0 : timeout_ms);
  for (int l = 0; l < c->cfg.n_layers; ++l) {
    if (!c->gate_pending[l]) continue;
    for (;;) {
      cudaError_t q = cudaEventQuery(c->gate_done[l]);
      if (q == cudaSuccess) break;
      if (q != cudaErrorNotReady) return cuda_fail(q, "gate event");
      if (std::chrono::steady_clock::now() > deadline) return fail(WITCERT_ETIMEDOUT, "gate of layer %d still running", l);
      std::this_thread::sleep_for(std::chrono::microseconds(50));
    }
  }
  unsigned long long s[6] = {0, 0, 0, 0, 0, 0};
  cudaError_t e = cudaMemcpy(s, c->gstats, sizeof s, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "reading gate counters");
  out->cells_triggered = s[0]; out->blocks_selected = s[1]; out->blocks_paged_in = s[2];
  out->bytes_paged_in = s[3]; out->blocks_dropped = s[4];
  ok();
  return WITCERT_OK;
}

witcert_status witcert_stats(witcert_cache* c, witcert_stats_t* out) try {
  if (!c || !out) return fail(WITCERT_EINVAL, "NULL argument");
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "stats");
  memset(out, 0, sizeof *out);
  unsigned long long cl = 0;
  int er = 0;
  if ((e = cudaMemcpy(&cl, c->clamps, sizeof cl, cudaMemcpyDeviceToHost)) != cudaSuccess) return cuda_fail(e, "stats");
  if ((e = cudaMemcpy(&er, c->err, sizeof er, cudaMemcpyDeviceToHost)) != cudaSuccess) return cuda_fail(e, "stats");
  collect_profile(c);
  out->tokens_written = c->tokens_written;
  out->decode_calls = c->decode_calls;
  out->int8_clamps = cl;
  out->device_errors = (uint64_t)er;
  out->decode_kernel_ms = c->prof_ms;
  out->decode_kernel_launches = c->prof_n;
  out->last_n_splits = c->last_n_splits;
  out->pages_used = c->table ? (uint64_t)c->cfg.max_pages - c->free_pages.size() : 0;
  ok();
  return WITCERT_OK;
} WITCERT_NO_THROW

witcert_status witcert_set_profiling(witcert_cache* c, int on) try {
  if (!c) return fail(WITCERT_EINVAL, "cache is NULL");
  if (!on && c->profiling) {
    cudaDeviceSynchronize();
    collect_profile(c);
  }
  if (on && !c->profiling) { cudaDeviceSynchronize(); collect_profile(c); c->prof_ms = 0.0; c->prof_n = 0; }
  c->profiling = on != 0;
  ok();
  return WITCERT_OK;
} WITCERT_NO_THROW

witcert_status witcert_set_launch_overlap(witcert_cache* c, int on) {
  if (!c) return fail(WITCERT_EINVAL, "cache is NULL");
  c->overlap = on != 0;
  ok();
  return WITCERT_OK;
}

witcert_status witcert_length(const witcert_cache* c, int layer, int* len) {
  if (witcert_status s = check_layer(c, layer)) return s;
  if (!len) return fail(WITCERT_EINVAL, "len is NULL");
  *len = c->len[layer];
  ok();
  return WITCERT_OK;
}

witcert_status witcert_seq_length(const witcert_cache* c, int layer, int seq, int* len) {
  if (witcert_status s = check_layer(c, layer)) return s;
  if (!len) return fail(WITCERT_EINVAL, "len is NULL");
  if (seq < 0 || seq >= c->cfg.batch) return fail(WITCERT_EINVAL, "sequence %d out of range [0, %d)", seq, c->cfg.batch);
  *len = c->slen[layer][seq];
  ok();
  return WITCERT_OK;
}

witcert_status witcert_export(witcert_cache* c, int layer, witcert_export_kind what, void* dst, size_t bytes,
                              void* stream) {
  if (witcert_status s = check_layer(c, layer)) return s;
  const int S = c->len[layer], nblk = (S + kBlk - 1) / kBlk;
  const size_t B = c->cfg.batch, Hkv = c->cfg.n_kv_heads, Hq = c->cfg.n_q_heads;
  size_t need = 0;
  switch (what) {
    case WITCERT_X_K_CODES: case WITCERT_X_V_CODES: need = B * S * Hkv * kD * (c->scheme == kBbox ? 2 : 1); break;
    case WITCERT_X_K_SCALES: case WITCERT_X_V_SCALES: case WITCERT_X_V_ZEROS: need = B * S * Hkv * 4 * 2; break;
    case WITCERT_X_KIVI_K_SCALE: case WITCERT_X_KIVI_K_ZERO: need = B * nblk * Hkv * kD * 2; break;
    case WITCERT_X_WITNESS: need = B * S * Hkv * kBands * 2; break;
    case WITCERT_X_SLOTS: need = B * Hkv * nblk * 4; break;
    case WITCERT_X_BLOCK_RISK: need = B * Hq * nblk * 4; break;
    case WITCERT_X_V_WITNESS: need = B * S * Hkv * 2; break;
    default: return fail(WITCERT_EINVAL, "unknown export kind %d", (int)what);
  }
  const bool int8 = int8_layout(c->scheme), kivi = c->scheme == kKivi;
  if ((what == WITCERT_X_K_SCALES && !int8) || ((what == WITCERT_X_V_SCALES) && !(int8 || kivi)) ||
      ((what == WITCERT_X_V_ZEROS || what == WITCERT_X_KIVI_K_SCALE || what == WITCERT_X_KIVI_K_ZERO) && !kivi))
    return fail(WITCERT_EINVAL, "export kind %d does not exist for this scheme", (int)what);
  if (what == WITCERT_X_BLOCK_RISK && !c->risk) return fail(WITCERT_ESTATE, "block risks need the gate enabled");
  if (what == WITCERT_X_V_WITNESS && !c->vwit) return fail(WITCERT_EINVAL, "value witnesses need a cache created with v_witness");
  if (!dst || bytes < need) return fail(WITCERT_EINVAL, "export needs %zu bytes, got %zu", need, bytes);
  auto st = static_cast<cudaStream_t>(stream);
  order_after_gate(c, layer, st);
  ExportArgs a{};
  a.blocks = c->blocks + layer * c->layer_blocks;
  a.nblk_max = c->nblk_max; a.B = (int)B; a.Hkv = (int)Hkv; a.Hq = (int)Hq; a.S = S; a.scheme = c->scheme;
  a.slots = c->slots ? c->slots + layer * layer_rows(c) * c->nblk_max : nullptr;
  a.risk = c->risk ? c->risk + (size_t)layer * B * Hq * c->nblk_max : nullptr;
  a.vwit = c->vwit ? c->vwit + layer * vwit_layer(c) : nullptr;
  a.seq_len = c->ragged ? c->dlen + (size_t)layer * B : nullptr;
  a.table = c->table;
  a.dst = dst;
  a.what = (int)what;
  cudaError_t e = launch_export(a, st);
  if (e != cudaSuccess) return cuda_fail(e, "export launch");
  if (need > 0) launched_apart(c, st);                        // nothing was launched for an empty layer
  ok();
  return WITCERT_OK;
}

witcert_status witcert_wait_selftest(int64_t limit_ns, void* stream) {
  if (limit_ns <= 0 || limit_ns > 10000000000ll) return fail(WITCERT_EINVAL, "limit_ns must be in (0, 1e10]");
  int timed_out = -1;
  cudaError_t e = run_wait_selftest((uint64_t)limit_ns, static_cast<cudaStream_t>(stream), &timed_out);
  if (e != cudaSuccess) return cuda_fail(e, "wait self test");
  if (timed_out) return fail(WITCERT_ETIMEDOUT, "device wait gave up after %lld ns", (long long)limit_ns);
  ok();
  return WITCERT_OK;
}

witcert_status witcert_quotient_selftest(int n_f32, uint64_t seed, uint64_t* mismatches, void* stream) {
  if (n_f32 < 0 || n_f32 > (1 << 20) || !mismatches) return fail(WITCERT_EINVAL, "n_f32 in [0, 2^20] and a result pointer");
  unsigned long long m = 0;
  cudaError_t e = run_quotient_selftest(n_f32, seed, &m, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "quotient self test");
  *mismatches = m;
  ok();
  return WITCERT_OK;
}

witcert_status witcert_dither(uint64_t seed, int layer, int kv_head, int t0, int n, int tensor, float* out,
                              void* stream) {
  if (layer < 0 || layer > 65535 || kv_head < 0 || kv_head > 65535 || t0 < 0 || n < 0 || (tensor != 0 && tensor != 1))
    return fail(WITCERT_EINVAL, "bad dither arguments");
  if (n > 0 && !out) return fail(WITCERT_EINVAL, "out is NULL");
  cudaError_t e = launch_dither(seed, layer, kv_head, t0, n, tensor, out, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dither launch");
  ok();
  return WITCERT_OK;
}

}  // extern "C"
