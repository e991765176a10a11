// Plain writers of the cache (kernels in write_kernels.cuh), the device copies of sequence
// lengths and the writers' quotient self test.
#include "write_kernels.cuh"

namespace witcert {

namespace {

// Per-sequence lengths on the device ([B] of one layer), set from the launch's parameters.
__global__ void __launch_bounds__(128) set_lengths_kernel(const LengthArgs u) {
  pdl_wait();
  pdl_trigger();
  for (int k = threadIdx.x; k < u.n; k += blockDim.x) u.dst[u.idx[k]] = u.len[k];
}

}  // namespace

cudaError_t launch_write_ragged(int scheme, const WriteArgs& a, const RaggedArgs& g, cudaStream_t st, bool pdl) {
  return a.is_bf16 ? launch_ragged_t<__nv_bfloat16>(scheme, a, NoRope{}, g, st, pdl)
                   : launch_ragged_t<float>(scheme, a, NoRope{}, g, st, pdl);
}

cudaError_t launch_kivi_keys(const WriteArgs& a, cudaStream_t st, bool pdl) {
  if (a.B == 0 || a.n_tok == 0 || a.Hkv == 0) return cudaSuccess;
  return a.is_bf16 ? kivi_keys_t<__nv_bfloat16>(a, NoRope{}, st, pdl) : kivi_keys_t<float>(a, NoRope{}, st, pdl);
}

cudaError_t launch_set_lengths(const LengthArgs& u, cudaStream_t st, bool pdl) {
  if (u.n <= 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, set_lengths_kernel, u);
}

namespace {

// 32-bit mix of a counter (the xorshift-multiply finalizer of MurmurHash3): test inputs only.
__device__ __forceinline__ uint32_t mix32(uint32_t h) {
  h ^= h >> 16; h *= 0x85ebca6bu; h ^= h >> 13; h *= 0xc2b2ae35u; h ^= h >> 16;
  return h;
}

// One CTA per positive fp16 scale (bits 1 .. 0x7BFF): every bf16 x with |x| <= 127.5 s, then
// n_f32 fp32 x = s * u with u drawn in (-127.5, 127.5).  Two more CTAs divide by the constants
// 127 (the INT8 scale) and 3 (the KIVI scale), every finite bf16 x and n_f32 fp32 x drawn over
// fp32's exponent range.  Counts quotients that differ from the IEEE quotient where a code or a
// scale can depend on them (|x / s| >= 2^-25).
__global__ void __launch_bounds__(256) quotient_selftest_kernel(int n_f32, uint32_t seed, unsigned long long* bad) {
  const bool konst = blockIdx.x >= 0x7BFF;
  const float s = konst ? (blockIdx.x == 0x7BFF ? 127.0f : 3.0f) : __half2float(__ushort_as_half((unsigned short)(blockIdx.x + 1)));
  const float y = konst ? (blockIdx.x == 0x7BFF ? kInv127 : kInv3) : __frcp_rn(s);
  const float range = konst ? FLT_MAX : 127.5f * s;
  unsigned long long cnt = 0;
  for (int b = threadIdx.x; b < 65536 + n_f32; b += blockDim.x) {
    float x;
    if (b < 65536) {
      x = __uint_as_float((uint32_t)b << 16);
    } else {
      const uint32_t h = mix32(seed ^ mix32((uint32_t)(blockIdx.x * 0x9E3779B9u) ^ (uint32_t)b));
      if (konst) x = __uint_as_float(h);                         // any bit pattern; inf and NaN skipped
      else x = __fmul_rn(s, __fmul_rn((float)(int)(h >> 8) - 8388608.0f, 0x1.fep-17f));   // u = 127.5 (m - 2^23) / 2^23
    }
    if (!(fabsf(x) <= range)) continue;
    const float want = __fdiv_rn(x, s);
    if (fabsf(want) >= 0x1p-25f && __float_as_uint(div_rn_by(x, s, y)) != __float_as_uint(want)) ++cnt;
  }
  if (cnt) atomicAdd(bad, cnt);
}

}  // namespace

cudaError_t run_quotient_selftest(int n_f32, uint64_t seed, unsigned long long* mismatches, cudaStream_t st) {
  unsigned long long* d = nullptr;
  cudaError_t e = cudaMalloc(&d, sizeof(unsigned long long));
  if (e != cudaSuccess) return e;
  e = cudaMemsetAsync(d, 0, sizeof(unsigned long long), st);
  if (e == cudaSuccess) {
    quotient_selftest_kernel<<<0x7BFF + 2, 256, 0, st>>>(n_f32, (uint32_t)(seed ^ (seed >> 32)), d);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = cudaMemcpyAsync(mismatches, d, sizeof(unsigned long long), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  cudaFree(d);
  return e;
}

void philox_round_keys(uint64_t seed, uint32_t (&rk0)[10], uint32_t (&rk1)[10]) {
  uint32_t k0 = (uint32_t)(seed & 0xFFFFFFFFull), k1 = (uint32_t)(seed >> 32);
  for (int r = 0; r < 10; ++r) {
    if (r) { k0 += 0x9E3779B9u; k1 += 0xBB67AE85u; }
    rk0[r] = k0;
    rk1[r] = k1;
  }
}

cudaError_t launch_write(int scheme, const WriteArgs& a, cudaStream_t st, bool pdl) {
  if (a.B == 0 || a.n_tok == 0 || a.Hkv == 0) return cudaSuccess;
  return a.is_bf16 ? launch_t<__nv_bfloat16>(scheme, a, NoRope{}, st, pdl) : launch_t<float>(scheme, a, NoRope{}, st, pdl);
}

}  // namespace witcert
