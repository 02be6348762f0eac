// Rotary positions, and new tokens' latent rows into a paged cache.
//
// Rotary positions: pair i of a token at position p is turned by p * f_i,
//     (a, b) -> m * (a cos - b sin, a sin + b cos),
// the pair being elements (2i, 2i+1) (interleaved) or (i, i + d/2) (half);
// the gradient turns back (sin negated) with the same factor m.  The frequency
// table holds f_i / (2 pi) as a 64-bit fraction of a turn, so p * f_i modulo a
// turn is one integer multiplication that drops the whole turns: no angle ever
// grows, and a position of 2^31 loses nothing beyond the table's own 2^-54.
// Taken as a signed number the product is the angle in (-1/2, 1/2] turn; it is
// rounded to float32 there (an error below 2^-24 rad), and sincospif takes half
// turns, so nothing is reduced again.  x, cos and sin are float32 until the
// one rounding of the result.
//
// Bound: HBM (each element read and written once, 3 flops per element); small
// calls are bound by the launch.  A thread holds the cos and sin of the pairs in
// one 16-byte piece of a head (bf16 interleaved: 4 pairs; half layout: 8 pairs,
// from two pieces) and walks over heads with four loads in flight; the heads of
// a token are dealt to as many threads as it takes to fill the GPU, so that one
// token's call is as wide as it can be and a long prompt computes each cos and
// sin once per several heads.  16384 tokens of 32 heads x 64 in bf16: 25.4 us, 5.3
// TB/s; one token 1.9 us, the launch.  Both kernels are launched to start while the
// one before ends (2 to 20 % of back-to-back calls); they let the next one start only
// when they end (earlier, its waiting CTAs cost a ragged append 5.8 against 4.3 us).
#include "dsa_device.cuh"
#include "dsa_kernels.h"
#include "dsa_launch.cuh"

namespace dsa {
namespace rope {

constexpr int NT = 256;
constexpr int UNROLL = 4;   // heads in flight per thread

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// One 16-byte piece of interleaved pairs, or of one half, in float32.
template <typename E>
struct Piece;
template <>
struct Piece<uint16_t> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float* v) {
    v[0] = lo_f32(w.x); v[1] = hi_f32(w.x); v[2] = lo_f32(w.y); v[3] = hi_f32(w.y);
    v[4] = lo_f32(w.z); v[5] = hi_f32(w.z); v[6] = lo_f32(w.w); v[7] = hi_f32(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
  static __device__ __forceinline__ float load(const uint16_t* p) { return bf16_to_f32(*p); }
  static __device__ __forceinline__ void store(uint16_t* p, float v) { *p = f32_to_bf16_rn(v); }
};
template <>
struct Piece<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float* v) {
    v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};

// pairs held by one thread
template <typename E, bool HALF, bool VEC>
constexpr int pairs_per_thread() {
  return !VEC ? 1 : (HALF ? Piece<E>::V : Piece<E>::V / 2);
}

template <typename E, bool HALF, bool VEC>
__global__ void __launch_bounds__(NT) rope_kernel(const __grid_constant__ RopeArgs a) {
  using P = Piece<E>;
  constexpr int PPT = pairs_per_thread<E, HALF, VEC>();
  const uint32_t g = blockIdx.x * NT + threadIdx.x;
  const uint32_t items = (uint32_t)a.d / (2 * PPT);
  const uint32_t item = g % items, rest = g / items;
  const uint32_t hg = rest % (uint32_t)a.head_groups, t = rest / (uint32_t)a.head_groups;
  if (t >= (uint32_t)a.T) return;
  wait_for_previous();
  const int32_t pos = a.positions[t];
  float c[PPT], s[PPT];
#pragma unroll
  for (int i = 0; i < PPT; ++i) {
    rope_cos_sin(a.table.turns[item * PPT + i], pos, a.table.mscale, c[i], s[i]);
    if (a.gradient) s[i] = -s[i];
  }
  const E* x = static_cast<const E*>(a.x) + (int64_t)t * a.x_stride_t;
  E* y = static_cast<E*>(a.y) + (int64_t)t * a.y_stride_t;
  const int lo = HALF ? item * PPT : 2 * item * PPT;   // first element of the thread's pairs
  const int up = HALF ? lo + a.d / 2 : lo + 1;         // the pairs' second elements (scalar and half)
  // (unsigned: a thread's last step looks past the heads, and may pass 2^31)
  const uint32_t step = (uint32_t)a.head_groups, H = (uint32_t)a.H;
  for (uint32_t h0 = hg; h0 < H; h0 += UNROLL * step) {
    if constexpr (VEC) {
      uint4 w[UNROLL], u[UNROLL];
#pragma unroll
      for (int k = 0; k < UNROLL; ++k) {
        const uint32_t h = h0 + k * step;
        if (h < H) {
          const E* src = x + (int64_t)h * a.x_stride_h;
          w[k] = *reinterpret_cast<const uint4*>(src + lo);
          if constexpr (HALF) u[k] = *reinterpret_cast<const uint4*>(src + up);
        }
      }
#pragma unroll
      for (int k = 0; k < UNROLL; ++k) {
        const uint32_t h = h0 + k * step;
        if (h < H) {
          E* dst = y + (int64_t)h * a.y_stride_h;
          float p[P::V], q[P::V];
          P::unpack(w[k], p);
          if constexpr (HALF) {
            float r[P::V];
            P::unpack(u[k], q);
#pragma unroll
            for (int i = 0; i < PPT; ++i) {
              r[i] = p[i] * s[i] + q[i] * c[i];
              p[i] = p[i] * c[i] - q[i] * s[i];
            }
            *reinterpret_cast<uint4*>(dst + lo) = P::pack(p);
            *reinterpret_cast<uint4*>(dst + up) = P::pack(r);
          } else {
#pragma unroll
            for (int i = 0; i < PPT; ++i) {
              q[2 * i] = p[2 * i] * c[i] - p[2 * i + 1] * s[i];
              q[2 * i + 1] = p[2 * i] * s[i] + p[2 * i + 1] * c[i];
            }
            *reinterpret_cast<uint4*>(dst + lo) = P::pack(q);
          }
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < UNROLL; ++k) {
        const uint32_t h = h0 + k * step;
        if (h < H) {
          const E* src = x + (int64_t)h * a.x_stride_h;
          E* dst = y + (int64_t)h * a.y_stride_h;
          const float p = P::load(src + lo), q = P::load(src + up);
          P::store(dst + lo, p * c[0] - q * s[0]);
          P::store(dst + up, p * s[0] + q * c[0]);
        }
      }
    }
  }
}

template <typename E, bool HALF, bool VEC>
static int launch_t(RopeArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int PPT = pairs_per_thread<E, HALF, VEC>();
  const int64_t per_group = (int64_t)a.T * (a.d / (2 * PPT));   // threads of one head group
  a.head_groups = rope_head_groups(a.H, per_group, num_sms);
  const int64_t blocks = (per_group * a.head_groups + NT - 1) / NT;
  if (blocks * NT > 0xffffffffll) return -2;
  return launch_after(rope_kernel<E, HALF, VEC>, dim3((unsigned)blocks), NT, 0, stream, a);
}

// --------------------------------------------------------------------------
// Cache append: token t's latent row (512 NoPE columns as they are, the RoPE
// columns turned) into row table[r][p / block_size] * block_size + p %
// block_size of the cache, r being the token's request and p its position.
// The FP8 row is the one the quantize kernel writes for the same bf16 row
// (the same scale and conversion, e4m3_block_scale and e4m3_quantize2), the RoPE
// columns being rounded to bf16 first.
//
// Bound: HBM; a decode step's handful of tokens by the launch and two
// dependent loads (position, then block id).  One warp per token: lane l holds
// columns 16 l .. 16 l + 15 (eight lanes are a 128-column block of the
// quantization) and pair l of the RoPE columns, all loaded before the row is
// looked up.  128 tokens 1.9 us; 16384 FP8 rows and reading them back as bf16
// 15.9 us; a ragged chunk of 8312 tokens 4.3 us (8.1 with half a CTA per token).
// --------------------------------------------------------------------------
constexpr int NT_APPEND = 64;   // (2 tokens: 16384 of them 4 % faster than 4 or 8 per CTA)

// The physical row of token t, or -1 (a padding token, or a bad entry: *bad).
__device__ __forceinline__ int64_t row_of(const AppendArgs& a, int t, int32_t& pos, bool& bad) {
  bad = false;
  pos = a.positions[t];
  if (pos == -1) return -1;
  const int r = a.token_req ? a.token_req[t] : t;
  bad = true;
  if (pos < 0 || r < 0 || r >= a.num_req || pos / a.block_size >= a.max_blocks) return -1;
  const int32_t blk = a.block_table[(int64_t)r * a.max_blocks + pos / a.block_size];
  const int64_t row = (int64_t)blk * a.block_size + pos % a.block_size;
  if (blk < 0 || row >= a.N) return -1;
  bad = false;
  return row;
}

template <bool F8>
__global__ void __launch_bounds__(NT_APPEND) append_kernel(const __grid_constant__ AppendArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (NT_APPEND / 32) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  wait_for_previous();
  const uint4* src = reinterpret_cast<const uint4*>(a.c_kv + t * a.c_stride) + 2 * lane;
  const uint4 w0 = src[0], w1 = src[1];
  const bool half = a.table.layout == DSA_ROPE_HALF;
  const bool pe = 2 * lane < a.d_rope;
  const int lo = half ? lane : 2 * lane, up = half ? lane + a.d_rope / 2 : lo + 1;
  uint16_t p = 0, q = 0;
  if (pe) {
    p = a.k_pe[t * a.pe_stride + lo];
    q = a.k_pe[t * a.pe_stride + up];
  }
  int32_t pos;
  bool bad;
  const int64_t row = row_of(a, (int)t, pos, bad);
  if (bad && lane == 0) atomicAdd(a.err + ERR_BAD_INDEX, 1u);
  if (row < 0) return;   // (the whole warp)
  uint8_t* dst = static_cast<uint8_t*>(a.cache) + row * (F8 ? 528 + 2 * a.d_rope : 2ll * a.ld_kv);
  if constexpr (F8) {
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    float amax = max_ieee(abs_ieee(lo_f32(w[0])), abs_ieee(hi_f32(w[0])));
#pragma unroll
    for (int i = 1; i < 8; ++i) amax = max_ieee(amax, max_ieee(abs_ieee(lo_f32(w[i])), abs_ieee(hi_f32(w[i]))));
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) amax = max_ieee(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = e4m3_block_scale(amax);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = e4m3_quantize2(w[2 * i], scale) | (uint32_t)e4m3_quantize2(w[2 * i + 1], scale) << 16;
    reinterpret_cast<uint4*>(dst)[lane] = make_uint4(c[0], c[1], c[2], c[3]);
    if ((lane & 7) == 0) *reinterpret_cast<float*>(dst + 512 + (lane >> 1)) = scale;
  } else {
    reinterpret_cast<uint4*>(dst)[2 * lane] = w0;
    reinterpret_cast<uint4*>(dst)[2 * lane + 1] = w1;
  }
  if (pe) {
    if (a.rotate) {
      float c, s;
      rope_cos_sin(a.table.turns[lane], pos, a.table.mscale, c, s);
      const float x = bf16_to_f32(p), y = bf16_to_f32(q);
      p = f32_to_bf16_rn(x * c - y * s);
      q = f32_to_bf16_rn(x * s + y * c);
    }
    uint16_t* d = reinterpret_cast<uint16_t*>(dst + (F8 ? 528 : 1024));
    if (half) {
      d[lo] = p;
      d[up] = q;
    } else {
      reinterpret_cast<uint32_t*>(d)[lane] = (uint32_t)p | (uint32_t)q << 16;
    }
  }
}

}  // namespace rope

int launch_rope(RopeArgs& a, bool f32, bool vec, int num_sms, cudaStream_t stream) {
  using namespace rope;
  const bool half = a.table.layout == DSA_ROPE_HALF;
  if (f32) {
    if (vec) return half ? launch_t<float, true, true>(a, num_sms, stream) : launch_t<float, false, true>(a, num_sms, stream);
    return half ? launch_t<float, true, false>(a, num_sms, stream) : launch_t<float, false, false>(a, num_sms, stream);
  }
  if (vec)
    return half ? launch_t<uint16_t, true, true>(a, num_sms, stream) : launch_t<uint16_t, false, true>(a, num_sms, stream);
  return half ? launch_t<uint16_t, true, false>(a, num_sms, stream) : launch_t<uint16_t, false, false>(a, num_sms, stream);
}

int launch_kv_append(const AppendArgs& a, bool fp8, cudaStream_t stream) {
  using namespace rope;
  const unsigned grid = (unsigned)(((int64_t)a.T + NT_APPEND / 32 - 1) / (NT_APPEND / 32));
  return fp8 ? launch_after(append_kernel<true>, dim3(grid), NT_APPEND, 0, stream, a)
             : launch_after(append_kernel<false>, dim3(grid), NT_APPEND, 0, stream, a);
}

}  // namespace dsa
