// RMS norms of the heads of queries and keys, with the rotation of their RoPE columns in
// the same pass, and the gradients of both.
//
// A row is one head of one token, d columns, of which the first d_norm are normed and the
// last d_rope turned (they may overlap):
//     r = 1 / sqrt(sum_{c < d_norm} x_c^2 / d_norm + eps)
//     n_c = x_c r w_c  (c < d_norm),  x_c  (else);   y = n with its last d_rope columns turned by the position.
// Gradient, g being the result's gradient with its last d_rope columns turned back:
//     dx_c = r (g_c w_c - x_c r^2 S / d_norm),  S = sum_{e < d_norm} g_e w_e x_e   (c < d_norm),   g_c (else)
//     dw_c = sum over all rows of g_c x_c r.
// Everything is float32 between the inputs and the one rounding of each result; dw is
// summed and returned in float32.  The turns are those of the rotary kernel (a 64-bit
// fraction of a turn, see rope.cu).
//
// Bound: HBM, each element read and written once (the gradient reads two).  G lanes share
// a row: a lane holds up to MP 16-byte pieces of the columns in front of the RoPE columns
// and one rotation item, the two pieces that hold its 2 V columns' pairs (interleaved: next
// to each other, half: d_rope / 2 apart), so that a pair lies in one lane in either layout
// and every element is loaded once.  A group of lanes walks over heads of one token, with
// cos, sin and the weights in registers and the next row's loads in flight.
#include "dsa_device.cuh"
#include "dsa_kernels.h"
#include "dsa_launch.cuh"

namespace dsa {
namespace normrope {

constexpr int NT = 256;

// V consecutive elements of a row, as loaded and in float32.
template <typename E, int V>
struct Piece {
  using Raw = uint4;
  static __device__ __forceinline__ Raw load(const E* p) { return *reinterpret_cast<const uint4*>(p); }
  static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ void unpack(const Raw& w, float* v) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(E) == 2) {
        v[2 * i] = __uint_as_float(r[i] << 16);
        v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
      } else {
        v[i] = __uint_as_float(r[i]);
      }
    }
  }
  static __device__ __forceinline__ void store(E* p, const float* v) {
    uint4 w;
    if constexpr (sizeof(E) == 2)
      w = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    else
      w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    *reinterpret_cast<uint4*>(p) = w;
  }
};
template <typename E>
struct Piece<E, 1> {
  using Raw = E;
  static __device__ __forceinline__ Raw load(const E* p) { return *p; }
  static __device__ __forceinline__ Raw zero() { return E(0); }
  static __device__ __forceinline__ void unpack(const Raw& w, float* v) {
    if constexpr (sizeof(E) == 2) v[0] = bf16_to_f32(w);
    else v[0] = w;
  }
  static __device__ __forceinline__ void store(E* p, const float* v) {
    if constexpr (sizeof(E) == 2) *p = f32_to_bf16_rn(v[0]);
    else *p = v[0];
  }
};

// The columns of one lane: piece m starts at col[m] (m < MP in front of the RoPE columns,
// then two per rotation item); a piece that the row does not have is off.
template <typename E, int V, int G, int MP, int RI>
struct Lane {
  static constexpr int NP = MP + 2 * RI;
  int at;         // lane of the row
  int tail, half, step_items, layout;
  int d_norm;

  __device__ __forceinline__ Lane(const NormArgs& a, int lane_of_row) {
    at = lane_of_row;
    tail = a.d - a.d_rope;
    half = a.d_rope / 2;
    layout = a.table.layout;
    d_norm = a.d_norm;
    step_items = a.d_rope / (2 * V);
  }
  __device__ __forceinline__ int item(int i) const { return at + G * i; }
  __device__ __forceinline__ bool on(int m) const {
    if (m < MP) return (at + G * m) * V < tail;
    return item((m - MP) >> 1) < step_items;
  }
  __device__ __forceinline__ int col(int m) const {
    if (m < MP) return (at + G * m) * V;
    const int i = item((m - MP) >> 1), second = (m - MP) & 1;
    return tail + (layout == DSA_ROPE_HALF ? i * V + second * half : (2 * i + second) * V);
  }
  __device__ __forceinline__ bool normed(int m) const { return col(m) < d_norm; }   // (d_norm is a multiple of V)
};

// A rotation item's 2 V columns, in place: pair i is (p[i], q[i]) in halves, elements 2i and
// 2i + 1 of the 2 V interleaved.
template <int V>
__device__ __forceinline__ void turn(float* p, float* q, const float* c, const float* s, bool half, float sign) {
  if (half) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float x = p[i], y = q[i], si = sign * s[i];
      p[i] = x * c[i] - y * si;
      q[i] = x * si + y * c[i];
    }
  } else if constexpr (V == 1) {
    const float x = p[0], y = q[0], si = sign * s[0];
    p[0] = x * c[0] - y * si;
    q[0] = x * si + y * c[0];
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float x = p[2 * i], y = p[2 * i + 1], si = sign * s[i];
      p[2 * i] = x * c[i] - y * si;
      p[2 * i + 1] = x * si + y * c[i];
      const float z = q[2 * i], w = q[2 * i + 1], sj = sign * s[V / 2 + i];
      q[2 * i] = z * c[V / 2 + i] - w * sj;
      q[2 * i + 1] = z * sj + w * c[V / 2 + i];
    }
  }
}

template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cos and sin of a lane's items at one position.
template <int V, int G, int RI>
__device__ __forceinline__ void angles(const NormArgs& a, int lane_of_row, int32_t pos, float (*c)[V], float (*s)[V]) {
  const int items = a.d_rope / (2 * V);
#pragma unroll
  for (int r = 0; r < RI; ++r) {
    const int i = lane_of_row + G * r;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      c[r][e] = 1.f;
      s[r][e] = 0.f;
      if (i < items) rope_cos_sin(a.table.turns[i * V + e], pos, a.table.mscale, c[r][e], s[r][e]);
    }
  }
}

// The weights of a lane's columns (1 where a column is not normed).
template <typename E, int V, int G, int MP, int RI>
__device__ __forceinline__ void weights(const NormArgs& a, const NormSide& sd, const Lane<E, V, G, MP, RI>& ln, float (*w)[V]) {
#pragma unroll
  for (int m = 0; m < MP + 2 * RI; ++m) {
#pragma unroll
    for (int e = 0; e < V; ++e) w[m][e] = 1.f;
    if (ln.on(m) && ln.normed(m)) {
      const int c = ln.col(m);
#pragma unroll
      for (int e = 0; e < V; ++e)
        w[m][e] = a.w_f32 ? static_cast<const float*>(sd.w)[c + e] : bf16_to_f32(static_cast<const uint16_t*>(sd.w)[c + e]);
    }
  }
}

template <typename E, int V, int G, int MP, int RI>
__global__ void __launch_bounds__(NT) norm_rope_kernel(const __grid_constant__ NormArgs a) {
  using P = Piece<E, V>;
  constexpr int NP = MP + 2 * RI;
  const uint32_t g = blockIdx.x * (uint32_t)(NT / G) + threadIdx.x / G;
  const uint32_t per_token = (uint32_t)(a.side[0].groups + a.side[1].groups);
  const uint32_t t = g / per_token;
  uint32_t sub = g - t * per_token;
  const int which = sub < (uint32_t)a.side[0].groups ? 0 : 1;
  const NormSide& sd = a.side[which];
  if (which) sub -= (uint32_t)a.side[0].groups;
  const Lane<E, V, G, MP, RI> ln(a, (int)(threadIdx.x % G));
  const uint32_t H = t < (uint32_t)a.T ? (uint32_t)sd.H : 0u, step = (uint32_t)sd.groups;
  wait_for_previous();
  const E* x = static_cast<const E*>(sd.x) + (int64_t)t * sd.x_stride_t;
  E* y = static_cast<E*>(sd.y) + (int64_t)t * sd.y_stride_t;
  typename P::Raw raw[NP];
  auto load = [&](uint32_t h) {
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      raw[m] = P::zero();
      if (h < H && ln.on(m)) raw[m] = P::load(x + (int64_t)h * sd.x_stride_h + ln.col(m));
    }
  };
  load(sub);
  float c[RI][V], s[RI][V], w[NP][V];
  if (H && a.d_rope) angles<V, G, RI>(a, ln.at, a.positions[t], c, s);
  if (H) weights<E, V, G, MP, RI>(a, sd, ln, w);
  const float inv_n = 1.0f / (float)a.d_norm;
  for (uint32_t h = sub; __any_sync(0xffffffffu, h < H); h += step) {
    float v[NP][V], sum = 0.f;
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      P::unpack(raw[m], v[m]);
      if (ln.normed(m)) {
#pragma unroll
        for (int e = 0; e < V; ++e) sum += v[m][e] * v[m][e];
      }
    }
    load(h + step);   // (the next row, while this one is worked on)
    const float r = rsqrtf(row_sum<G>(sum) * inv_n + a.eps);
    if (h >= H) continue;
    E* dst = y + (int64_t)h * sd.y_stride_h;
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      if (ln.normed(m)) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[m][e] = v[m][e] * r * w[m][e];
      }
      if (m < MP) {
        if (ln.on(m)) P::store(dst + ln.col(m), v[m]);
      } else if ((m - MP) & 1) {
        if (ln.on(m)) {
          turn<V>(v[m - 1], v[m], c[(m - MP) >> 1], s[(m - MP) >> 1], ln.layout == DSA_ROPE_HALF, 1.f);
          P::store(dst + ln.col(m - 1), v[m - 1]);
          P::store(dst + ln.col(m), v[m]);
        }
      }
    }
  }
}

// --------------------------------------------------------------------------
// Gradient.  A CTA works for one side (queries or keys, shared out by their rows), its
// lane groups walk over tasks, `each` heads of a token, and keep their columns' sums for
// dw in registers; the CTA adds them up in shared memory and stores one row of partial
// sums, which a second small kernel adds in a fixed order: no atomics, the same inputs
// give the same bits.
// --------------------------------------------------------------------------
template <typename E, int V, int G, int MP, int RI>
__global__ void __launch_bounds__(NT) norm_rope_gradient_kernel(const __grid_constant__ NormArgs a) {
  using P = Piece<E, V>;
  constexpr int NP = MP + 2 * RI;
  extern __shared__ float dw_sum[];   // [NT / 32][d_norm]
  const int which = (int)blockIdx.x < a.side[0].ctas ? 0 : 1;
  const NormSide& sd = a.side[which];
  const uint32_t cta = blockIdx.x - (which ? (uint32_t)a.side[0].ctas : 0u);
  const uint32_t first = cta * (uint32_t)(NT / G) + threadIdx.x / G, stride = (uint32_t)sd.ctas * (NT / G);
  const Lane<E, V, G, MP, RI> ln(a, (int)(threadIdx.x % G));
  const uint32_t per_token = (uint32_t)sd.groups, H = (uint32_t)sd.H;
  const int64_t tasks = (int64_t)a.T * per_token;
  launch_dependents();
  wait_for_previous();
  float w[NP][V], dw[NP][V];
  weights<E, V, G, MP, RI>(a, sd, ln, w);
#pragma unroll
  for (int m = 0; m < NP; ++m) {
#pragma unroll
    for (int e = 0; e < V; ++e) dw[m][e] = 0.f;
  }
  const float inv_n = 1.0f / (float)a.d_norm;
  for (int64_t task = first; __any_sync(0xffffffffu, task < tasks); task += stride) {
    const bool live = task < tasks;
    const uint32_t t = live ? (uint32_t)(task / per_token) : 0u;
    const uint32_t sub = live ? (uint32_t)(task - (int64_t)t * per_token) : H;
    const E* x = static_cast<const E*>(sd.x) + (int64_t)t * sd.x_stride_t;
    const E* gy = static_cast<const E*>(sd.g) + (int64_t)t * sd.g_stride_t;
    E* y = static_cast<E*>(sd.y) + (int64_t)t * sd.y_stride_t;
    float c[RI][V], s[RI][V];
    if (live && a.d_rope) angles<V, G, RI>(a, ln.at, a.positions[t], c, s);
    for (uint32_t h = sub; __any_sync(0xffffffffu, h < H); h += per_token) {
      float v[NP][V], g[NP][V];
      {
        typename P::Raw rx[NP], rg[NP];
#pragma unroll
        for (int m = 0; m < NP; ++m) {
          rx[m] = rg[m] = P::zero();
          if (h < H && ln.on(m)) {
            rx[m] = P::load(x + (int64_t)h * sd.x_stride_h + ln.col(m));
            rg[m] = P::load(gy + (int64_t)h * sd.g_stride_h + ln.col(m));
          }
        }
#pragma unroll
        for (int m = 0; m < NP; ++m) {
          P::unpack(rx[m], v[m]);
          P::unpack(rg[m], g[m]);
        }
      }
      float sum = 0.f, dot = 0.f;
#pragma unroll
      for (int m = 0; m < NP; ++m) {
        if (m >= MP && ((m - MP) & 1) && h < H && ln.on(m))
          turn<V>(g[m - 1], g[m], c[(m - MP) >> 1], s[(m - MP) >> 1], ln.layout == DSA_ROPE_HALF, -1.f);
      }
#pragma unroll
      for (int m = 0; m < NP; ++m) {
        if (ln.normed(m)) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            sum += v[m][e] * v[m][e];
            dot += g[m][e] * w[m][e] * v[m][e];
          }
        }
      }
      const float r = rsqrtf(row_sum<G>(sum) * inv_n + a.eps);
      const float k = row_sum<G>(dot) * inv_n * r * r;
      if (h >= H) continue;
      E* dst = y + (int64_t)h * sd.y_stride_h;
#pragma unroll
      for (int m = 0; m < NP; ++m) {
        if (!ln.on(m)) continue;
        if (ln.normed(m)) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float gx = g[m][e] * v[m][e];
            g[m][e] = r * (g[m][e] * w[m][e] - v[m][e] * k);
            dw[m][e] += gx * r;
          }
        }
        P::store(dst + ln.col(m), g[m]);
      }
    }
  }
  // the CTA's sums: over the rows of a warp by shuffles, then over the warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int m = 0; m < NP; ++m) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float v = dw[m][e];
#pragma unroll
      for (int o = G; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane < G && ln.on(m) && ln.normed(m)) dw_sum[warp * a.d_norm + ln.col(m) + e] = v;
    }
  }
  __syncthreads();
  float* part = a.part + (int64_t)blockIdx.x * a.d_norm;
  for (int i = threadIdx.x; i < a.d_norm; i += NT) {
    float v = dw_sum[i];
#pragma unroll
    for (int k = 1; k < NT / 32; ++k) v += dw_sum[k * a.d_norm + i];
    part[i] = v;
  }
}

// dw of 32 columns of one side (blockIdx.y) from the CTAs' partial sums.
__global__ void __launch_bounds__(NT) norm_weight_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float acc[NT / 32][32];
  launch_dependents();
  wait_for_previous();
  const int which = a.side[0].H ? (int)blockIdx.y : 1;
  const NormSide& sd = a.side[which];
  const int n = sd.ctas, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = (int)blockIdx.x * 32 + lane;
  const float* part = a.part + (which ? (int64_t)a.side[0].ctas * a.d_norm : 0);
  float v = 0.f;
  if (c < a.d_norm) {
#pragma unroll 4
    for (int i = warp; i < n; i += NT / 32) v += part[(int64_t)i * a.d_norm + c];
  }
  acc[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < a.d_norm) {
#pragma unroll
    for (int k = 1; k < NT / 32; ++k) v += acc[k][lane];
    sd.dw[c] = v;
  }
}

template <typename E, int V, int G, int MP, int RI>
static int launch_t(NormArgs& a, bool gradient, int num_sms, cudaStream_t stream) {
  const int64_t heads = (int64_t)a.side[0].H + a.side[1].H;
  if (!gradient) {
    // heads per group of lanes, as the rotary kernel's
    const int64_t total = rope_head_groups(heads, (int64_t)a.T * G, num_sms);
    const int64_t each = (heads + total - 1) / total;
    for (NormSide& sd : a.side) sd.groups = (int)((sd.H + each - 1) / each);
    const int64_t blocks = ((int64_t)a.T * (a.side[0].groups + a.side[1].groups) * G + NT - 1) / NT;   // (below 2^30)
    return launch_after(norm_rope_kernel<E, V, G, MP, RI>, dim3((unsigned)blocks), NT, 0, stream, a);
  }
  // CTAs: the rows' share of two per SM, at least one a side, no more than rows
  const int64_t most = 2 * (int64_t)num_sms < kNormMaxCtas ? 2 * (int64_t)num_sms : kNormMaxCtas;
  int ctas = 0;
  for (NormSide& sd : a.side) {
    const int64_t need = ((int64_t)a.T * sd.H * G + NT - 1) / NT;
    int64_t share = most * sd.H / heads;
    if (share < 1 && sd.H) share = 1;
    sd.ctas = (int)(need < share ? need : share);
    const int64_t lanes = (int64_t)sd.ctas * NT / G;   // groups of lanes
    int64_t each = 1;                                  // heads of a task
    while (sd.H && each < 8 && 2 * each <= sd.H && (int64_t)a.T * ((sd.H + 2 * each - 1) / (2 * each)) >= 8 * lanes) each *= 2;
    sd.groups = sd.H ? (int)((sd.H + each - 1) / each) : 0;
    ctas += sd.ctas;
  }
  const uint32_t smem = (uint32_t)(NT / 32 * a.d_norm * 4);
  if (ctas > 0) {   // (no tokens: the sums below are of nothing)
    const int r = launch_after(norm_rope_gradient_kernel<E, V, G, MP, RI>, dim3((unsigned)ctas), NT, smem, stream, a);
    if (r != 0) return r;
  }
  const int sides = (a.side[0].H > 0) + (a.side[1].H > 0);
  return launch_after(norm_weight_kernel, dim3((unsigned)((a.d_norm + 31) / 32), (unsigned)sides), NT, 0, stream, a);
}

// The fewest lanes that hold a row in two pieces and one item each, else 32.
template <typename E, int V>
static int launch_v(NormArgs& a, bool gradient, int num_sms, cudaStream_t stream) {
  const int items = a.d_rope / (2 * V), pieces = (a.d - a.d_rope) / V;
  if (items <= 8 && pieces <= 16) return launch_t<E, V, 8, 2, 1>(a, gradient, num_sms, stream);
  if (items <= 16 && pieces <= 32) return launch_t<E, V, 16, 2, 1>(a, gradient, num_sms, stream);
  if (pieces <= 64) return launch_t<E, V, 32, 2, 1>(a, gradient, num_sms, stream);
  if (pieces <= 128) return launch_t<E, V, 32, 4, 1>(a, gradient, num_sms, stream);
  if constexpr (V == 4) return launch_t<E, V, 32, 8, 1>(a, gradient, num_sms, stream);
  return -2;
}

}  // namespace normrope

int launch_norm_rope(NormArgs& a, bool f32, bool vec, bool gradient, int num_sms, cudaStream_t stream) {
  using namespace normrope;
  if (f32)
    return vec ? launch_v<float, 4>(a, gradient, num_sms, stream) : launch_t<float, 1, 32, 32, 4>(a, gradient, num_sms, stream);
  return vec ? launch_v<uint16_t, 8>(a, gradient, num_sms, stream)
             : launch_t<uint16_t, 1, 32, 32, 4>(a, gradient, num_sms, stream);
}

}  // namespace dsa
