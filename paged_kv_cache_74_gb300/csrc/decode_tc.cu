// decode_tc.cu -- launchers of the tensor-core paged decode (decode_tc_kernel.cuh).
#include "decode_tc_kernel.cuh"

namespace pa {
namespace {

template <int D, bool KV8>
cudaError_t launch_decode_tc_d(const DecodeArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, cudaStream_t stream) {
  if (a.group <= 4) return launch_decode_tc_impl<D, 4, KV8>(a, qmap, kmap, vmap, stream);
  if (a.group <= 8) return launch_decode_tc_impl<D, 8, KV8>(a, qmap, kmap, vmap, stream);
  if (a.group <= 16) return launch_decode_tc_impl<D, 16, KV8>(a, qmap, kmap, vmap, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_decode_tc(const DecodeArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, int head_dim, bool kv8, cudaStream_t stream) {
  if (head_dim == 128)
    return kv8 ? launch_decode_tc_d<128, true>(a, qmap, kmap, vmap, stream)
               : launch_decode_tc_d<128, false>(a, qmap, kmap, vmap, stream);
  if (head_dim == 64)
    return kv8 ? launch_decode_tc_d<64, true>(a, qmap, kmap, vmap, stream)
               : launch_decode_tc_d<64, false>(a, qmap, kmap, vmap, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
