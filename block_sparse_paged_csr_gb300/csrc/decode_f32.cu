// Instances of the decode attention over an f32 cache.
#include "decode_split.cuh"

namespace sa {

cudaError_t launch_decode_f32(const DecodeArgs& a, int dp, int r, cudaStream_t stream) {
  return dec1::launch_type<SA_DTYPE_F32>(a, dp, r, stream);
}

}  // namespace sa
