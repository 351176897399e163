// The 8-bit decode for 1 q head a kv head.
#include "decode_fp8.cuh"

namespace bia {

cudaError_t launch_decode_fp8_g1(const DecodeFp8Args &f, cudaStream_t s) {
  return launch_f8_g<1>(f, s);
}

} // namespace bia
