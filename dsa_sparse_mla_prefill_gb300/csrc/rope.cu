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
// sin once per several heads.
#include "dsa_device.cuh"
#include "dsa_kernels.h"

namespace dsa {
namespace rope {

constexpr int NT = 256;
constexpr int UNROLL = 4;   // heads in flight per thread

__device__ __forceinline__ void cos_sin(uint64_t turns, int32_t pos, float m, float& c, float& s) {
  const int64_t t = (int64_t)(turns * (uint64_t)(int64_t)pos);
  sincospif(__ll2float_rn(t) * 1.0842021724855044e-19f /* 2^-63: half turns */, &s, &c);
  c *= m;
  s *= m;
}

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
  const int32_t pos = __ldg(a.positions + t);
  float c[PPT], s[PPT];
#pragma unroll
  for (int i = 0; i < PPT; ++i) {
    cos_sin(a.table.turns[item * PPT + i], pos, a.table.mscale, c[i], s[i]);
    if (a.gradient) s[i] = -s[i];
  }
  const E* x = static_cast<const E*>(a.x) + (int64_t)t * a.x_stride_t;
  E* y = static_cast<E*>(a.y) + (int64_t)t * a.y_stride_t;
  const int lo = HALF ? item * PPT : 2 * item * PPT;   // first element of the thread's pairs
  const int up = HALF ? lo + a.d / 2 : lo + 1;         // the pairs' second elements (scalar and half)
  const int step = a.head_groups;
  for (int h0 = hg; h0 < a.H; h0 += UNROLL * step) {
    if constexpr (VEC) {
      uint4 w[UNROLL], u[UNROLL];
#pragma unroll
      for (int k = 0; k < UNROLL; ++k) {
        const int h = h0 + k * step;
        if (h < a.H) {
          const E* src = x + (int64_t)h * a.x_stride_h;
          w[k] = *reinterpret_cast<const uint4*>(src + lo);
          if constexpr (HALF) u[k] = *reinterpret_cast<const uint4*>(src + up);
        }
      }
#pragma unroll
      for (int k = 0; k < UNROLL; ++k) {
        const int h = h0 + k * step;
        if (h < a.H) {
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
        const int h = h0 + k * step;
        if (h < a.H) {
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
  // as many heads per thread, in powers of two, as leave threads for every
  // SM's 2048 slots (16384 tokens of 32 heads: 8 each, 25.7 us; 11 each 27.3,
  // 4 each 27.0, 2 each 36.6, the cos and sin being worked out per thread)
  int each = 1;
  while (2 * each <= a.H && (a.H + 2 * each - 1) / (2 * each) * per_group >= 2048ll * num_sms) each *= 2;
  a.head_groups = (a.H + each - 1) / each;
  const int64_t blocks = (per_group * a.head_groups + NT - 1) / NT;
  if (blocks * NT > 0xffffffffll) return -2;
  rope_kernel<E, HALF, VEC><<<(unsigned)blocks, NT, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

// --------------------------------------------------------------------------
// Cache append: token t's latent row (512 NoPE columns as they are, the RoPE
// columns turned) into row table[r][p / block_size] * block_size + p %
// block_size of the cache, r being the token's request and p its position.
// The FP8 row is the one the quantize kernel writes for the same bf16 row
// (shared e4m3_quantize_block), the RoPE columns being rounded to bf16 first.
//
// Bound: HBM; a decode step's handful of tokens by the launch and two
// dependent loads (position, then block id).  Warps 0-3 take a 128-column
// block of the row each (lane l: columns 4l .. 4l+3, the layout of the block
// quantization), warp 4 the RoPE columns (lane = pair), so that the RoPE
// arithmetic runs beside the copy; ROWS tokens per CTA have their loads in
// flight together (2 for a prompt chunk; 1 while the tokens do not fill the
// GPU, where more CTAs are worth more than more loads per thread).
// --------------------------------------------------------------------------
constexpr int NT_APPEND = 160;
constexpr int ROWS_LONG = 2;

// The physical row of token t, or -1 (a padding token, or a bad entry: *bad).
__device__ __forceinline__ int64_t row_of(const AppendArgs& a, int t, int32_t& pos, bool& bad) {
  bad = false;
  pos = __ldg(a.positions + t);
  if (pos == -1) return -1;
  const int r = a.token_req ? __ldg(a.token_req + t) : t;
  bad = true;
  if (pos < 0 || r < 0 || r >= a.num_req || pos / a.block_size >= a.max_blocks) return -1;
  const int32_t blk = __ldg(a.block_table + (int64_t)r * a.max_blocks + pos / a.block_size);
  const int64_t row = (int64_t)blk * a.block_size + pos % a.block_size;
  if (blk < 0 || row >= a.N) return -1;
  bad = false;
  return row;
}

template <bool F8, int ROWS>
__global__ void __launch_bounds__(NT_APPEND) append_kernel(const __grid_constant__ AppendArgs a) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * ROWS;
  int64_t row[ROWS];
  int32_t pos[ROWS];
  // (called once the token's own data is on its way: the two loads behind each
  // other that find the row then overlap it)
  auto find_rows = [&]() {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      row[r] = -1;
      if (t0 + r < a.T) {
        bool bad;
        row[r] = row_of(a, t0 + r, pos[r], bad);
        if (bad && threadIdx.x == 0) atomicAdd(a.err + ERR_BAD_INDEX, 1u);
      }
    }
  };
  uint8_t* cache = static_cast<uint8_t*>(a.cache);
  const int64_t row_bytes = F8 ? 528 + 2 * a.d_rope : 2ll * a.ld_kv;
  if (w < 4) {
    uint2 raw[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      raw[r] = make_uint2(0, 0);
      if (t0 + r < a.T)
        raw[r] = *reinterpret_cast<const uint2*>(a.c_kv + (int64_t)(t0 + r) * a.c_stride + 128 * w + 4 * lane);
    }
    find_rows();
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (row[r] < 0) continue;   // (uniform over the CTA)
      uint8_t* dst = cache + row[r] * row_bytes;
      if constexpr (F8) {
        float scale;
        const uint32_t codes = e4m3_quantize_block(raw[r], scale);
        *reinterpret_cast<uint32_t*>(dst + 128 * w + 4 * lane) = codes;
        if (lane == 0) *reinterpret_cast<float*>(dst + 512 + 4 * w) = scale;
      } else {
        *reinterpret_cast<uint2*>(dst + 256 * w + 8 * lane) = raw[r];
      }
    }
  } else if (2 * lane < a.d_rope) {
    const bool half = a.table.layout == DSA_ROPE_HALF;
    const int lo = half ? lane : 2 * lane, up = half ? lane + a.d_rope / 2 : lo + 1;
    uint16_t p[ROWS], q[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      p[r] = q[r] = 0;
      if (t0 + r < a.T) {
        const uint16_t* src = a.k_pe + (int64_t)(t0 + r) * a.pe_stride;
        p[r] = src[lo];
        q[r] = src[up];
      }
    }
    find_rows();
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (row[r] < 0) continue;
      if (a.rotate) {
        float c, s;
        cos_sin(a.table.turns[lane], pos[r], a.table.mscale, c, s);
        const float x = bf16_to_f32(p[r]), y = bf16_to_f32(q[r]);
        p[r] = f32_to_bf16_rn(x * c - y * s);
        q[r] = f32_to_bf16_rn(x * s + y * c);
      }
      uint16_t* dst = reinterpret_cast<uint16_t*>(cache + row[r] * row_bytes + (F8 ? 528 : 1024));
      dst[lo] = p[r];
      dst[up] = q[r];
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

int launch_kv_append(const AppendArgs& a, bool fp8, int num_sms, cudaStream_t stream) {
  using namespace rope;
  const int nt = a.d_rope > 0 ? NT_APPEND : 128;
  if ((int64_t)a.T <= 8ll * num_sms) {   // a CTA per token fills the GPU's SMs at most about twice
    if (fp8) append_kernel<true, 1><<<a.T, nt, 0, stream>>>(a);
    else append_kernel<false, 1><<<a.T, nt, 0, stream>>>(a);
  } else {
    const unsigned grid = (unsigned)((a.T + (int64_t)ROWS_LONG - 1) / ROWS_LONG);
    if (fp8) append_kernel<true, ROWS_LONG><<<grid, nt, 0, stream>>>(a);
    else append_kernel<false, ROWS_LONG><<<grid, nt, 0, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace dsa
