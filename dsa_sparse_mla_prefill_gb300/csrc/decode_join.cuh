// The split of a paged decode call into ranges of key tiles, and the kernel that joins
// the parts of requests that a range border cuts (see paged_decode.cuh).
#pragma once
#include <cstdint>

#include "dsa_device.cuh"
#include "dsa_kernels.h"
#include "dsa_launch.cuh"

namespace dsa {
namespace decode {

// First tile of range g of ng ranges over total tiles: floor(g * total / ng).
__host__ __device__ __forceinline__ uint32_t range_begin(uint32_t g, uint32_t total, uint32_t ng) {
  if (total < (1u << 24)) return g * total / ng;   // (g <= 152)
  return (uint32_t)((uint64_t)g * total / ng);
}
// The range that holds tile t.
__host__ __device__ __forceinline__ uint32_t range_of(uint32_t t, uint32_t total, uint32_t ng) {
  if (total < (1u << 24)) return ((t + 1) * ng - 1) / total;
  return (uint32_t)(((uint64_t)(t + 1) * ng - 1) / total);
}

// A request that the end of a range cuts.
struct Border {
  int request;
  int first;          // range of its first part
  int parts;          // ranges that hold some of it: 2 .. the number of ranges
  bool whole_start;   // it begins where its first range does
};
// The border at the end of range g: head = tiles and ranges of the call, at = the
// request that ends the range, its tiles, and its tiles up to there.  False where no
// request is cut, and for entries that no call can have (a range whose waits ran out
// before its last tile leaves zeros): whatever they hold, a border that is returned
// names a request and ranges of this call.  Where tiles are counted with `gap` blank ones in front
// of every request, a range that begins among them begins with the request.
__host__ __device__ __forceinline__ bool border_of(uint2 head, int4 at, uint32_t g, int B, int groups, Border& cut,
                                                   uint32_t gap = 0) {
  const uint32_t total = head.x, ng = head.y;
  if (ng > (uint32_t)groups || total < ng || total > 0x7fffffffu || g + 1 >= ng) return false;
  if (at.x < 0 || at.x >= B || at.z < 1 || at.z >= at.y) return false;
  const uint32_t end = range_begin(g + 1, total, ng);   // tiles up to here
  if ((uint32_t)at.z > end || (uint32_t)(at.y - at.z) > total - end) return false;
  const uint32_t p0 = end - (uint32_t)at.z;             // tiles before the request
  cut.request = at.x;
  cut.first = (int)range_of(p0, total, ng);
  cut.parts = (int)range_of(p0 + (uint32_t)at.y - 1, total, ng) - cut.first + 1;
  cut.whole_start = p0 - range_begin((uint32_t)cut.first, total, ng) <= gap;
  return true;
}

// --------------------------------------------------------------------------
// Join: out = sum_s 2^(L_s - M) O_s / sum_s 2^(L_s - M) over the parts of a cut
// request (L_s base-2 log-sum-exp, O_s normalised), lse = M + log2 of that sum.
//
// The borders inside one request share its heads' outputs evenly, JOIN_Y CTAs to
// a border and head block, so one long context and a cut batch are both joined by as many CTAs
// as there is work for.  The threads of a CTA stand 128 / G wide over float4
// outputs of a head and G deep over the parts, G = 1, 4 or 16 by their number, so
// that a thread has ten at most.  It loads MOST of them at once, the first ones
// beside the log-sum-exps that weight them: 10 where few requests are cut into
// many parts (a context of 131072 positions: 40 against 44 us with 5), else 5,
// whose registers leave room for more CTAs (64 ragged requests: 72 against 74).  The
// parts are summed in one order, whatever CTA
// stored them first.
// --------------------------------------------------------------------------
constexpr int NT_JOIN = 128;
constexpr int JOIN_Y = 8;          // CTAs per border and head block
constexpr int LSE = 5;             // of a lane
static_assert(kDecodeMaxCtas <= 32 * LSE, "parts of a request");

template <int MOST>
__global__ void __launch_bounds__(NT_JOIN) join_kernel(const __grid_constant__ DecodeArgs a, int heads_padded) {
  __shared__ float4 acc[3][32];
  __shared__ float wgt[4][32 * LSE];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  wait_for_previous();
  Border cut;
  if (!border_of(reinterpret_cast<const uint2*>(a.borders)[0], a.borders[1 + blockIdx.x], blockIdx.x, a.B, a.groups, cut)) return;
  const int64_t b = cut.request;
  const int g0 = cut.first, S = cut.parts, nb = S - 1, rank = (int)blockIdx.x - g0;
  const int first_slot = 2 * g0 + (cut.whole_start ? 0 : 1);
  const int lg = S <= 5 ? 0 : (S <= 20 ? 2 : 4);        // log2 of G
  const int wide = 128 >> lg;                           // float4 outputs of a piece
  const int pieces = a.H << lg;
  const int c0 = pieces * rank / nb, c1 = pieces * (rank + 1) / nb;
  const uint32_t pitch = (uint32_t)heads_padded;        // heads of a slot (all offsets are below 2^23)
  const int deep = (int)threadIdx.x >> (7 - lg);
  const int s0 = (S * deep) >> lg, s1 = (S * (deep + 1)) >> lg;
  auto slot_of = [&](int s) { return (uint32_t)(s == 0 ? first_slot : 2 * (g0 + s)) * pitch; };
#pragma unroll 1
  for (int c = c0 + (int)blockIdx.y; c < c1; c += (int)gridDim.y) {
    const int h = c >> lg;
    const int i = (c & ((1 << lg) - 1)) * wide + ((int)threadIdx.x & (wide - 1));   // float4 of the head
    const float4* src = reinterpret_cast<const float4*>(a.part_o) + h * 128 + i;
    float4 v[MOST];
#pragma unroll
    for (int k = 0; k < MOST; ++k) v[k] = s0 + k < s1 ? src[slot_of(s0 + k) * 128] : make_float4(0.f, 0.f, 0.f, 0.f);
    float l[LSE], m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < LSE; ++k) l[k] = lane + 32 * k < S ? a.part_lse[slot_of(lane + 32 * k) + h] : -INFINITY;
#pragma unroll
    for (int k = 0; k < LSE; ++k) m = fmaxf(m, l[k]);
    m = warp_max(m);
    const float mr = m == -INFINITY ? 0.f : m;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < LSE; ++k) {
      l[k] = exp2f(l[k] - mr);
      sum += l[k];
      wgt[warp][lane + 32 * k] = l[k];
    }
    __syncwarp();
    sum = warp_sum(sum);
    const float inv = sum != 0.f ? 1.0f / sum : 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int s = s0; s < s1; s += MOST) {
#pragma unroll
      for (int k = 0; k < MOST; ++k) {
        if (s + k < s1) {
          const float w = wgt[warp][s + k];
          o.x += w * v[k].x;
          o.y += w * v[k].y;
          o.z += w * v[k].z;
          o.w += w * v[k].w;
          if (s + MOST + k < s1) v[k] = src[slot_of(s + MOST + k) * 128];
        }
      }
    }
    // (the depths that share a warp)
    for (int d = wide; d < 32; d <<= 1) {
      o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
    }
    if (lg > 0) {
      if (warp > 0) acc[warp - 1][lane] = o;
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const float4 y = acc[q][lane];
          o.x += y.x;
          o.y += y.y;
          o.z += y.z;
          o.w += y.w;
        }
      }
    }
    if ((int)threadIdx.x < wide)
      *reinterpret_cast<uint2*>(a.out + (b * a.H + h) * 512 + 4 * i) =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (threadIdx.x == 0 && i == 0)
      a.lse[b * a.H + h] = sum != 0.f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    if (lg > 0) __syncthreads();
  }
}

// The tree form's join, of up to thousands of query rows: a warp takes a row, all parts of it
// DEEP at a time, or where there are more than eight parts the CTA's four warps a fourth of them
// each; the borders inside a request share its rows.  (A warp per 128 columns, with the kernel
// above's way to the weights, was bound by its 540 instructions a piece: 8 requests of 512 rows in
// 19 ranges 17 us, and 21 with that kernel.)
template <int DEEP>
__global__ void __launch_bounds__(NT_JOIN) tree_join_kernel(const __grid_constant__ DecodeArgs a, int rows_padded) {
  __shared__ float4 acc[3][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  wait_for_previous();
  Border cut;
  const int4 head = a.borders[0];
  if (!border_of(make_uint2(head.x, head.y), a.borders[1 + blockIdx.x], blockIdx.x, a.B, a.groups, cut, head.z)) return;
  const int S = cut.parts, nb = S - 1, rank = (int)blockIdx.x - cut.first;
  const uint32_t pitch = (uint32_t)rows_padded;      // (rows of all slots are below 2^23)
  const uint32_t first_slot = (uint32_t)(2 * cut.first + (cut.whole_start ? 0 : 1)) * pitch;
  auto slot_of = [&](int s) { return s == 0 ? first_slot : (uint32_t)(2 * (cut.first + s)) * pitch; };
  const int r0 = (int)((int64_t)a.H * rank / nb), r1 = (int)((int64_t)a.H * (rank + 1) / nb);
  const bool shared = S > 8;                         // a row by the whole CTA
  const int s0 = shared ? S * warp / 4 : 0, s1 = shared ? S * (warp + 1) / 4 : S;
  const int step = (int)gridDim.y * (shared ? 1 : NT_JOIN / 32);
#pragma unroll 1
  for (int row = r0 + (shared ? (int)blockIdx.y : (int)blockIdx.y * (NT_JOIN / 32) + warp); row < r1; row += step) {
    const float4* src = reinterpret_cast<const float4*>(a.part_o) + (uint64_t)row * 128 + lane;
    const float* lse = a.part_lse + row;
    // weights of the parts: lane s has part s's; those from 32 on are worked out as they come
    const float l = lane < S ? lse[slot_of(lane)] : -INFINITY;
    float m = l;
    for (int s = 32 + lane; s < S; s += 32) m = fmaxf(m, lse[slot_of(s)]);
    m = warp_max(m);
    const float mr = m == -INFINITY ? 0.f : m;
    const float w = exp2f(l - mr);
    float sum = w;
    for (int s = 32 + lane; s < S; s += 32) sum += exp2f(lse[slot_of(s)] - mr);
    sum = warp_sum(sum);
    const float inv = sum != 0.f ? 1.0f / sum : 0.f;
    float4 o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int s = s0; s < s1; s += DEEP) {
      float4 v[DEEP][4];
      float ws[DEEP];
#pragma unroll
      for (int k = 0; k < DEEP; ++k) {
        const int at = min(s + k, s1 - 1);
        const float4* from = src + (uint64_t)slot_of(at) * 128;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[k][q] = from[32 * q];
        ws[k] = at < 32 ? __shfl_sync(0xffffffffu, w, at) : exp2f(lse[slot_of(at)] - mr);
        if (s + k >= s1) ws[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < DEEP; ++k) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          fma2(o[q].x, o[q].y, v[k][q].x, v[k][q].y, ws[k], ws[k]);
          fma2(o[q].z, o[q].w, v[k][q].z, v[k][q].w, ws[k], ws[k]);
        }
      }
    }
    if (shared) {   // (the same in the whole CTA)
      if (warp > 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[warp - 1][32 * q + lane] = o[q];
      }
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int p = 0; p < 3; ++p) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 y = acc[p][32 * q + lane];
            o[q].x += y.x;
            o[q].y += y.y;
            o[q].z += y.z;
            o[q].w += y.w;
          }
        }
      }
      __syncthreads();
      if (warp > 0) continue;
    }
    uint2* out = reinterpret_cast<uint2*>(a.out + ((int64_t)cut.request * a.H + row) * 512) + lane;
#pragma unroll
    for (int q = 0; q < 4; ++q) out[32 * q] = make_uint2(pack_bf16x2(o[q].x * inv, o[q].y * inv), pack_bf16x2(o[q].z * inv, o[q].w * inv));
    if (lane == 0) a.lse[(int64_t)cut.request * a.H + row] = sum != 0.f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
  }
}

}  // namespace decode
}  // namespace dsa
