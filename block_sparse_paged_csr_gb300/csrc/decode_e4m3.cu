// Instances of the decode attention over an e4m3 cache.
#include "decode_split.cuh"

namespace sa {

cudaError_t launch_decode_e4m3(const DecodeArgs& a, int dp, int r, cudaStream_t stream) {
  return dec1::launch_type<SA_DTYPE_E4M3>(a, dp, r, stream);
}

}  // namespace sa
