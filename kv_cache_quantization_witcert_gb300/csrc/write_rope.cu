// Writers that rotate the keys on the way (kernels in write_kernels.cuh).
#include "write_kernels.cuh"

namespace witcert {

cudaError_t launch_write_rope(int scheme, const WriteArgs& a, const RopeArgs& rp, cudaStream_t st, bool pdl) {
  if (a.B == 0 || a.n_tok == 0 || a.Hkv == 0) return cudaSuccess;
  return a.is_bf16 ? launch_t<__nv_bfloat16>(scheme, a, rp, st, pdl) : launch_t<float>(scheme, a, rp, st, pdl);
}

cudaError_t launch_write_ragged_rope(int scheme, const WriteArgs& a, const RopeArgs& rp, const RaggedArgs& g,
                                     cudaStream_t st, bool pdl) {
  return a.is_bf16 ? launch_ragged_t<__nv_bfloat16>(scheme, a, rp, g, st, pdl)
                   : launch_ragged_t<float>(scheme, a, rp, g, st, pdl);
}

cudaError_t launch_kivi_keys_rope(const WriteArgs& a, const RopeArgs& rp, cudaStream_t st, bool pdl) {
  if (a.B == 0 || a.n_tok == 0 || a.Hkv == 0) return cudaSuccess;
  return a.is_bf16 ? kivi_keys_t<__nv_bfloat16>(a, rp, st, pdl) : kivi_keys_t<float>(a, rp, st, pdl);
}

}  // namespace witcert
