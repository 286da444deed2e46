// decode_masked.cu -- the streaming paged decode with modified scores (tanh
// cap, distance bias, prefix and first-key masks): launchers of the MOD
// instantiations of decode_kernel.cuh.
//
// The kernel is bound by the K/V bytes of the visible keys, as the plain
// decode is; tiles without a visible key are not loaded.  Measured, call after
// call: 64 requests of 512 to 4096 keys (32 q, 8 kv heads of 128, bf16) with a cap
// 113 us, 5.6 TB/s of visible K/V, 0.83 of the copy peak (without a cap 105); over
// e4m3 72 us, 4.4 TB/s; 8 x 32768 keys of which a window of 4096 and the first 64 are
// seen 37 us (137 MB; the start-up and the merge of the pieces are about 13 us of
// it).
#include "decode_kernel.cuh"

namespace pa {

cudaError_t launch_decode_masked(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                 int head_dim, bool kv8, cudaStream_t stream) {
  const bool mix = a.tile_sms > 0;  // built for head_dim 128 (the host splits the SMs only there)
  // e4m3 units of two kv heads (8 q heads, head_dim 128).
  if (kv8 && a.group == 8 && head_dim == 128)
    return mix ? launch_decode_pair<true, true>(a, kmap, vmap, stream)
               : launch_decode_pair<false, true>(a, kmap, vmap, stream);
  const int gmax = decode_gmax(a.group);
#define PA_DECODE_CASE(DD, GG)                                                                     \
  if (head_dim == DD && gmax == GG)                                                                \
    return kv8 ? (mix ? launch_decode_impl<DD, GG, true, false, DD == 128, true>(a, kmap, vmap, stream)  \
                      : launch_decode_impl<DD, GG, true, false, false, true>(a, kmap, vmap, stream))     \
               : (mix ? launch_decode_impl<DD, GG, false, false, DD == 128, true>(a, kmap, vmap, stream) \
                      : launch_decode_impl<DD, GG, false, false, false, true>(a, kmap, vmap, stream));
  PA_DECODE_CASE(128, 1) PA_DECODE_CASE(128, 2) PA_DECODE_CASE(128, 4)
  PA_DECODE_CASE(64, 1) PA_DECODE_CASE(64, 2) PA_DECODE_CASE(64, 4)
#undef PA_DECODE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace pa
