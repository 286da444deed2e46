// decode.cu -- launchers of the streaming paged decode (decode_kernel.cuh).
#include "decode_kernel.cuh"

namespace pa {

int decode_gmax(int group) {
  if (group <= 1) return 1;
  if (group <= 2) return 2;
  if (group <= 4) return 4;
  return 0;
}

int decode_ctas_per_sm(int head_dim, int group) {
  const int gmax = decode_gmax(group);
#define PA_DECODE_CASE(DD, GG) \
  if (head_dim == DD && gmax == GG) return DecodeCfg<DD, GG>::MINB;
  PA_DECODE_CASE(128, 1) PA_DECODE_CASE(128, 2) PA_DECODE_CASE(128, 4)
  PA_DECODE_CASE(64, 1) PA_DECODE_CASE(64, 2) PA_DECODE_CASE(64, 4)
#undef PA_DECODE_CASE
  return 1;
}

cudaError_t launch_decode(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          int head_dim, bool kv8, bool xsplit, cudaStream_t stream) {
  // e4m3 units of two kv heads (8 q heads, head_dim 128).
  if (kv8 && !xsplit && a.group == 8 && head_dim == 128 && a.tile_sms == 0)
    return launch_decode_pair<false, false>(a, kmap, vmap, stream);
  const int gmax = decode_gmax(a.group);
  const bool mix = a.tile_sms > 0;  // built for head_dim 128 (the host splits the SMs only there)
#define PA_DECODE_CASE(DD, GG)                                                      \
  if (head_dim == DD && gmax == GG)                                                 \
    return kv8 ? (xsplit ? launch_decode_impl<DD, GG, true, true>(a, kmap, vmap, stream)      \
                  : mix    ? launch_decode_impl<DD, GG, true, false, DD == 128>(a, kmap, vmap, stream) \
                           : launch_decode_impl<DD, GG, true, false>(a, kmap, vmap, stream))    \
               : (xsplit ? launch_decode_impl<DD, GG, false, true>(a, kmap, vmap, stream)     \
                  : mix    ? launch_decode_impl<DD, GG, false, false, DD == 128>(a, kmap, vmap, stream) \
                           : launch_decode_impl<DD, GG, false, false>(a, kmap, vmap, stream));
  PA_DECODE_CASE(128, 1) PA_DECODE_CASE(128, 2) PA_DECODE_CASE(128, 4)
  PA_DECODE_CASE(64, 1) PA_DECODE_CASE(64, 2) PA_DECODE_CASE(64, 4)
#undef PA_DECODE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace pa
