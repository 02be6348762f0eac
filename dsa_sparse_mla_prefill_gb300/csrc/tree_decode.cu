// Attention of a tree of drafted tokens per request over the paged latent cache.
//
//     out[b,i,h,:] = softmax_j(scale q[b,i,h,:] . c_j) . c_j[0:512],   lse likewise,
// over the positions j of request b in front of its drafted tokens, and of those the ones
// that token i's mask word names.  A request's n tokens x H heads are the query rows of the
// paged decode kernel; only the tiles that hold drafted tokens look at the mask.  This form
// takes up to 32 rows (FP8: 64), more go to CTA pairs (tree_pair.cu, where the cache's bytes no
// longer bound the call; the sizes on both sides are at decode_form).  Layout and split are the decode
// kernel's.  32 x 512..16384 keys take 47 us at 16 rows and 52 at 32, where the bytes would take 26 at the copy
// rate: the kernel itself 47, its DRAM at half of its peak over a start and eight tiles of 128 keys a CTA,
// then the join.  FP8 rows at 32 query rows 56 us and at 64, where two CTAs convert every row each for
// itself, 92 (15): the conversion, as in the decode step.
#include "paged_decode.cuh"

namespace dsa {

int launch_tree_decode(DecodeArgs& a, bool fp8, int d_rope, int max_tiles, cudaStream_t stream) {
  return decode::launch_decode<true>(a, fp8, d_rope, max_tiles, stream);
}

}  // namespace dsa
