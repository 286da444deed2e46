// The streaming decode kernels with the most state per thread, to be compiled
// for their register report (not run).
#include "decode_kernel.cuh"

namespace pa {

cudaError_t decode_registers(const DecodeArgs& a, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
  cudaError_t e = launch_decode_pair<false, false>(a, k, v, s);
  if (e == cudaSuccess) e = launch_decode_pair<true, true>(a, k, v, s);
  if (e == cudaSuccess) e = launch_decode_impl<128, 4, false, false, false, true>(a, k, v, s);
  if (e == cudaSuccess) e = launch_decode_impl<64, 4, true, true>(a, k, v, s);
  return e;
}

}  // namespace pa
