// Instances of the decode attention over an int8 cache.
#include "decode_split.cuh"

namespace sa {

cudaError_t launch_decode_int8(const DecodeArgs& a, int dp, int r, cudaStream_t stream) {
  return dec1::launch_type<SA_DTYPE_INT8>(a, dp, r, stream);
}

}  // namespace sa
