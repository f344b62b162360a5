// Instances of the decode attention over a bf16 cache.
#include "decode_split.cuh"

namespace sa {

cudaError_t launch_decode_bf16(const DecodeArgs& a, int dp, int r, cudaStream_t stream) {
  return dec1::launch_type<SA_DTYPE_BF16>(a, dp, r, stream);
}

}  // namespace sa
