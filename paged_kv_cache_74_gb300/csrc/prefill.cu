// prefill.cu -- launchers of the chunked-prefill kernel (prefill_kernel.cuh).
#include "prefill_kernel.cuh"

namespace pa {

size_t prefill_partials_bytes(int num_ctas, int head_dim) {
  return static_cast<size_t>(num_ctas) * 2 * 2 * 128 * (2 + head_dim) * sizeof(float);
}

cudaError_t launch_prefill(const PrefillArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, int head_dim, bool kv8, cudaStream_t stream) {
  if (head_dim == 128)
    return kv8 ? launch_prefill_impl<128, true>(a, qmap, kmap, vmap, stream)
               : launch_prefill_impl<128, false>(a, qmap, kmap, vmap, stream);
  if (head_dim == 64)
    return kv8 ? launch_prefill_impl<64, true>(a, qmap, kmap, vmap, stream)
               : launch_prefill_impl<64, false>(a, qmap, kmap, vmap, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
