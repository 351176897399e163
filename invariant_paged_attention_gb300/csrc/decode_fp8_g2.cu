// The 8-bit decode for 2 q heads a kv head.
#include "decode_fp8.cuh"

namespace bia {

cudaError_t launch_decode_fp8_g2(const DecodeFp8Args &f, cudaStream_t s) {
  return launch_f8_g<2>(f, s);
}

} // namespace bia
