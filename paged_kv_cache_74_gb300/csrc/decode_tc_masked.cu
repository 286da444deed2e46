// decode_tc_masked.cu -- the tensor-core paged decode with modified scores: launchers
// of the MOD instantiations of decode_tc_kernel.cuh (5 to 16 q heads per kv head).
// Measured on 200 requests of 16 to 4099 keys, 64 q and 8 kv heads of 128, with a
// cap, call after call: bf16 274 us, 6.4 TB/s of visible K/V, 0.94 of the copy
// peak (L2 flushed before each call 312); e4m3 318 us, 2.8 TB/s (the conversion and
// the softmax of a chunk set its rate, not the bytes), without a cap 285.
#include "decode_tc_kernel.cuh"

namespace pa {
namespace {

template <int D, bool KV8>
cudaError_t launch_group(const DecodeArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                         const CUtensorMap& vmap, cudaStream_t stream) {
  const bool cap = a.mods.cap_log2 > 0.f;
  if (a.group <= 8)
    return cap ? launch_decode_tc_impl<D, 8, KV8, kModsCap>(a, qmap, kmap, vmap, stream)
               : launch_decode_tc_impl<D, 8, KV8, kMods>(a, qmap, kmap, vmap, stream);
  if (a.group <= 16)
    return cap ? launch_decode_tc_impl<D, 16, KV8, kModsCap>(a, qmap, kmap, vmap, stream)
               : launch_decode_tc_impl<D, 16, KV8, kMods>(a, qmap, kmap, vmap, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_decode_tc_masked(const DecodeArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                    const CUtensorMap& vmap, int head_dim, bool kv8, cudaStream_t stream) {
  if (head_dim == 128)
    return kv8 ? launch_group<128, true>(a, qmap, kmap, vmap, stream)
               : launch_group<128, false>(a, qmap, kmap, vmap, stream);
  if (head_dim == 64)
    return kv8 ? launch_group<64, true>(a, qmap, kmap, vmap, stream)
               : launch_group<64, false>(a, qmap, kmap, vmap, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
