// Paged decode of one new token per request: the kernel's instances and their launch (see
// paged_decode.cuh).
#include "paged_decode.cuh"

namespace dsa {

int launch_paged_decode(DecodeArgs& a, bool fp8, int d_rope, int max_tiles, cudaStream_t stream) {
  return decode::launch_decode<false>(a, fp8, d_rope, max_tiles, stream);
}

}  // namespace dsa
