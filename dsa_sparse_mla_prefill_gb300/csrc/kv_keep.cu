// The accepted path of a tree of drafted tokens takes its place behind the context: the
// row of drafted token keep[b][i] moves to position context + i, in every layer's cache.
//
// keep is ascending, so entry i is never below i, and a place i that is filled is no later
// entry's row (keep[j] > keep[i] >= i for j > i); it may be an earlier one's.  A thread owns
// a 16-byte piece of all rows of one request and cache and moves them in order, eight loads
// ahead of their stores, so nothing is overwritten before it is read.
//
// Bound: launch and four dependent loads (length, path, block ids, rows): 16 requests in one layer
// 3.1 us, 64 requests in 61 layers 7.4 (13.7 MB moved, 2.0 at the copy rate), where every cache's CTAs
// walk the same chain for themselves.
#include "dsa_device.cuh"
#include "dsa_kernels.h"
#include "dsa_launch.cuh"

namespace dsa {
namespace keep {

constexpr int NT = 128;
constexpr int MOST = 64;   // entries of a path
constexpr int AHEAD = 8;

// The row of a position, or -1.
__device__ __forceinline__ int32_t row_of(const KeepArgs& a, int b, int32_t pos) {
  const int32_t page = pos / a.block_size;
  if (pos < 0 || page >= a.max_blocks) return -1;
  const int32_t blk = a.block_table[(int64_t)b * a.max_blocks + page];
  const int64_t row = (int64_t)blk * a.block_size + pos % a.block_size;
  return blk >= 0 && row < a.N ? (int32_t)row : -1;
}

__global__ void __launch_bounds__(NT) keep_kernel(const __grid_constant__ KeepArgs a) {
  __shared__ int32_t src[MOST], dst[MOST];
  __shared__ int entries;
  const int b = (int)blockIdx.x;
  const bool counts = blockIdx.y == 0;   // (one cache's CTAs store the lengths and count bad entries)
  wait_for_previous();
  if (threadIdx.x < 32) {
    const int lane = (int)threadIdx.x;
    const int32_t len = a.kv_lens[b];
    const int drafted = a.num_draft ? a.num_draft[b] : a.n;
    // two entries a lane; one is good if it names a drafted token behind the one before it
    const int32_t e0 = 2 * lane < a.m ? a.keep[(int64_t)b * a.m + 2 * lane] : -1;
    const int32_t e1 = 2 * lane + 1 < a.m ? a.keep[(int64_t)b * a.m + 2 * lane + 1] : -1;
    int32_t before = __shfl_up_sync(0xffffffffu, e1, 1);
    if (lane == 0) before = -1;
    const bool fits = len > 0 && drafted >= 0 && drafted <= a.n && len >= drafted;
    const bool g0 = fits && e0 > before && e0 < drafted, g1 = fits && e1 > e0 && e1 >= 0 && e1 < drafted;
    const uint32_t b0 = ~__ballot_sync(0xffffffffu, g0), b1 = ~__ballot_sync(0xffffffffu, g1);
    const int n0 = b0 ? 2 * (__ffs(b0) - 1) : MOST, n1 = b1 ? 2 * (__ffs(b1) - 1) + 1 : MOST;
    const int n = min(n0, n1);   // entries in front of the first that is not good
    const int32_t context = len - drafted;
    int bad = 0;
    for (int i = 0; i < 2; ++i) {
      const int at = 2 * lane + i;
      const int32_t e = i ? e1 : e0;
      if (at == n && e != -1 && len > 0) ++bad;
      if (at >= n) continue;
      int32_t s = -1, d = -1;
      if (e != at) {
        s = row_of(a, b, context + e);
        d = row_of(a, b, context + at);
        if (s < 0 || d < 0) {
          s = -1;
          ++bad;
        }
      }
      src[at] = s;
      dst[at] = d;
    }
    if (len > 0 && !fits && lane == 0 && e0 == -1) ++bad;   // (a bad length is counted once)
    bad = __reduce_add_sync(0xffffffffu, bad);
    if (lane == 0) {
      entries = n;
      if (counts) {
        a.new_lens[b] = fits ? context + n : len;
        if (bad) atomicAdd(a.err + ERR_BAD_INDEX, (unsigned)bad);
      }
    }
  }
  __syncthreads();
  const int n = entries;
  uint4* rows = static_cast<uint4*>(a.caches[blockIdx.y]);
  for (int p = (int)threadIdx.x; p < a.row_pieces; p += NT) {
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
      uint4 v[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (i0 + i < n && src[i0 + i] >= 0) v[i] = rows[(int64_t)src[i0 + i] * a.row_pieces + p];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (i0 + i < n && src[i0 + i] >= 0) rows[(int64_t)dst[i0 + i] * a.row_pieces + p] = v[i];
    }
  }
}

}  // namespace keep

int launch_kv_keep(const KeepArgs& a, int num_caches, cudaStream_t stream) {
  return launch_after(keep::keep_kernel, dim3((unsigned)a.B, (unsigned)num_caches), keep::NT, 0, stream, a);
}

}  // namespace dsa
