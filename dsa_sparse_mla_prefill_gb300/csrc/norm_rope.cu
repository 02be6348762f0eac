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
// Bound: HBM, each element read and written once (the gradient reads two).  A CTA works for
// one side, queries or keys, shared out by their rows; G lanes share a row, each with up to
// NP of its 16-byte pieces, and a warp takes an even run of the side's rows, token by token.
// Every lane copies its pieces of the rows ahead into its own slots in shared memory
// (cp.async, no barrier), so that what is in flight does not cost registers: with the next
// row's loads in registers instead, 16384 tokens of 32 heads of 192 took 75 to 87 us, DRAM at
// half of its peak, the warps waiting for loads.  The weights lie in shared memory.  A
// token's cos and sin are worked out once per run, an even share of the pairs per lane, and
// passed on through shared memory.  The RoPE pieces are a row's last, so they are every lane's
// last RM pieces; in the half layout a pair's other half is a shuffle away, or where the halves
// fill pieces of every lane, in the lane.
//
// Measured on inputs that change from call to call, against the bytes at the copy rate: 16384 tokens of 32
// heads of 192 columns 65.3 us (59.4), 8192 of them in float32 65.2 (59.4), 32767 latent rows of 576 14.4
// (11.1), in float32 27.4 (22.3), the gradient of 4095 x 40 x 128 in float32 45.1 (37.1) and of 8192 x 32 x
// 256 65.4 (59.4), both with the summing kernel; 8 tokens 3.2, the launch.  Further off: heads turned whole,
// whose cos and sin and pieces take more registers than three CTAs leave (8192 x 32 x 256 in bf16, four RoPE pieces
// a lane, 112 bytes of spills: 74.1 in halves, 70.8 interleaved, 39.6 at the copy rate), the gradient of latent rows, 32
// lanes a row with a quarter of their pieces off (32767: 35.3 us, 16.7; in float32 49.0, 33.4), and rows that no
// 16-byte piece fits, element by element (16384 x 32 x 70: 177 us, 21.7; gradient 798, 32.5).
#include "dsa_device.cuh"
#include "dsa_kernels.h"
#include "dsa_launch.cuh"

namespace dsa {
namespace normrope {

constexpr int NT = 256;
constexpr uint32_t kMostSmem = 227u * 1024u;

// A 16-byte piece in float32.
template <typename E>
struct Piece;
template <>
struct Piece<uint16_t> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float* v) {
    v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xffff0000u);
    v[4] = __uint_as_float(w.z << 16); v[5] = __uint_as_float(w.z & 0xffff0000u);
    v[6] = __uint_as_float(w.w << 16); v[7] = __uint_as_float(w.w & 0xffff0000u);
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
  static __device__ __forceinline__ float load(const uint16_t* p) { return bf16_to_f32(*p); }
  static __device__ __forceinline__ void store(uint16_t* p, float v) { *p = f32_to_bf16_rn(v); }
};
template <>
struct Piece<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float* v) {
    v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};

__device__ __forceinline__ float weight_at(const NormArgs& a, const NormSide& sd, int c) {
  return a.w_f32 ? static_cast<const float*>(sd.w)[c] : bf16_to_f32(static_cast<const uint16_t*>(sd.w)[c]);
}

// The side that a CTA works for, and its place among the side's CTAs.
__device__ __forceinline__ const NormSide& side_of(const NormArgs& a, int& cta) {
  const int which = (int)blockIdx.x < a.side[0].ctas ? 0 : 1;
  cta = (int)blockIdx.x - (which ? a.side[0].ctas : 0);
  return a.side[which];
}

// The rows of group of lanes g of K in worker i of n: workers take even, contiguous runs of K
// rows at a time, a group every K-th row of its worker's.  left counts the worker's steps, so it is
// the same in all of a worker's groups; the last step may lack rows (on() false).
struct Rows {
  uint32_t left, t, h, H, dt, dh;
  uint32_t T;
  __device__ __forceinline__ Rows(const NormArgs& a, const NormSide& sd, uint32_t i, uint32_t n, uint32_t g, uint32_t K) {
    H = (uint32_t)sd.H;
    T = (uint32_t)a.T;
    const uint64_t steps = ((uint64_t)T * H + K - 1) / K;
    const uint64_t first = steps * i / n;
    left = (uint32_t)(steps * (i + 1) / n - first);
    const uint64_t row = first * K + g;
    t = (uint32_t)(row / H);
    h = (uint32_t)(row - (uint64_t)t * H);
    dt = K / H;
    dh = K - dt * H;
  }
  __device__ __forceinline__ bool on() const { return left != 0 && t < T; }
  // One step on; true where the heads start anew (it is another token's then, and
  // always where dt is not 0).
  __device__ __forceinline__ bool next() {
    --left;
    h += dh;
    t += dt;
    const bool wraps = h >= H;
    if (wraps) {
      h -= H;
      ++t;
    }
    return wraps;
  }
};
// Where a tensor's row of that run lies: followed step by step.
template <typename E>
struct At {
  E* p;
  E* base;
  int64_t step, wrap;
  At() = default;
  __device__ __forceinline__ At(E* first, const Rows& r, int64_t stride_t, int64_t stride_h, int64_t col) : base(first) {
    p = first + col + (int64_t)r.t * stride_t + (int64_t)r.h * stride_h;
    step = (int64_t)r.dt * stride_t + (int64_t)r.dh * stride_h;
    wrap = stride_t - (int64_t)r.H * stride_h;
  }
  __device__ __forceinline__ void next(bool wraps) {   // (as the run's step did)
    p += step;
    if (wraps) p += wrap;
  }
};

template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The pieces of one lane: piece m is the row's piece m G + lane - pad (off below zero), so
// that a row's last pieces, the RoPE columns', are in every lane's last ones.
template <typename E, int G, int NP, int RM>
struct Lane {
  static constexpr int V = Piece<E>::V;
  int lane, p0, tail, R, hp, normed_pieces;
  bool half;
  __device__ __forceinline__ Lane(const NormArgs& a) {
    lane = (int)threadIdx.x % G;
    p0 = lane - (NP * G - a.d / V);
    R = a.d_rope / V;
    tail = a.d / V - R;
    hp = R / 2;
    half = a.table.layout == DSA_ROPE_HALF;
    normed_pieces = a.d_norm / V;
  }
  __device__ __forceinline__ int piece(int m) const { return p0 + m * G; }
  __device__ __forceinline__ bool on(int m) const { return piece(m) >= 0; }
  __device__ __forceinline__ bool normed(int m) const { return on(m) && piece(m) < normed_pieces; }
  __device__ __forceinline__ bool turned(int m) const { return m >= NP - RM && piece(m) >= tail && R > 0; }

  // A token's cos and sin of the lane's turned pieces.  Half layout: of their columns, for
  // RM > 1 of the first RM / 2 pieces, whose other halves are the last RM / 2; for RM = 1
  // sin has the sign of the column's own half.  Interleaved: piece r's V / 2 pairs at
  // r V / 2.  Called by whole warps; `workers` lanes, this one the `me`-th, share the table.
  static constexpr int CS = RM == 1 ? V : RM * V / 2;
  __device__ __forceinline__ void angles(const NormArgs& a, float2* table, int me, int workers, int32_t pos, float sign,
                                         float* c, float* s) const {
    const int pairs = a.d_rope / 2;
    __syncwarp();
    for (int i = me; i < pairs; i += workers) rope_cos_sin(a.table.turns[i], pos, a.table.mscale, table[i].x, table[i].y);
    __syncwarp();
    if (half) {
#pragma unroll
      for (int r = 0; r < (RM + 1) / 2; ++r) {
        const int j = piece(NP - RM + r) - tail;
        const bool mine = turned(NP - RM + r), second = j >= hp;
        const float si = RM == 1 && !second ? -sign : sign;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 x = mine ? table[(second ? j - hp : j) * V + e] : make_float2(1.f, 0.f);
          c[r * V + e] = x.x;
          s[r * V + e] = si * x.y;
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < RM; ++r) {
        const int j = piece(NP - RM + r) - tail;
        const bool mine = turned(NP - RM + r);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          const float2 x = mine ? table[j * (V / 2) + e] : make_float2(1.f, 0.f);
          c[r * (V / 2) + e] = x.x;
          s[r * (V / 2) + e] = sign * x.y;
        }
      }
    }
  }

  // Turns the lane's pieces v[NP - RM ..] in place.  Called by whole warps.
  __device__ __forceinline__ void turn(float (*v)[V], const float* c, const float* s) const {
    if (!half) {
#pragma unroll
      for (int r = 0; r < RM; ++r) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const float x = v[r][2 * i], y = v[r][2 * i + 1], co = c[r * (V / 2) + i], si = s[r * (V / 2) + i];
          v[r][2 * i] = x * co - y * si;
          v[r][2 * i + 1] = x * si + y * co;
        }
      }
    } else if constexpr (RM > 1) {
#pragma unroll
      for (int r = 0; r < RM / 2; ++r) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float x = v[r][e], y = v[r + RM / 2][e];
          v[r][e] = x * c[r * V + e] - y * s[r * V + e];
          v[r + RM / 2][e] = y * c[r * V + e] + x * s[r * V + e];
        }
      }
    } else {
      const int j = piece(NP - 1) - tail;
      const bool mine = turned(NP - 1);
      const int other = mine ? (j >= hp ? lane - hp : lane + hp) : lane;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float y = __shfl_sync(0xffffffffu, v[0][e], other, G);
        if (mine) v[0][e] = v[0][e] * c[e] + y * s[e];
      }
    }
  }
};

// Weights in shared memory, four columns of every piece together so that lanes read them
// without bank conflicts.
template <int G>
__host__ __device__ __forceinline__ uint32_t staged_bytes(const NormArgs& a) {   // and the tables of cos and sin
  return ((uint32_t)(a.d_norm * 4 + NT / G * (a.d_rope / 2) * 8) + 15u) / 16u * 16u;
}
template <typename E>
__device__ __forceinline__ void stage_weights(const NormArgs& a, const NormSide& sd, float4* w) {
  constexpr int Q = Piece<E>::V / 4;
  const int pieces = a.d_norm / Piece<E>::V;
  for (int i = (int)threadIdx.x; i < Q * pieces; i += NT) {
    const int p = i / Q, q = i - p * Q, c = 4 * i;
    w[q * pieces + p] = make_float4(weight_at(a, sd, c), weight_at(a, sd, c + 1), weight_at(a, sd, c + 2), weight_at(a, sd, c + 3));
  }
}
template <typename E>
__device__ __forceinline__ void read_weights(const float4* w, int pieces, int p, float* v) {
#pragma unroll
  for (int q = 0; q < Piece<E>::V / 4; ++q) {
    const float4 x = w[q * pieces + p];
    v[4 * q] = x.x;
    v[4 * q + 1] = x.y;
    v[4 * q + 2] = x.z;
    v[4 * q + 3] = x.w;
  }
}

// CTAs on an SM, and rows of each lane there (the one in hand and those ahead).  More in
// flight is slower, from 37 KB an SM on (16384 x 32 x 192: 3 CTAs of 2 rows 64.4 us, of 3 rows
// 72.1, 4 of 2 72.7, 2 of 3 70.9; 8192 x 32 x 256: 45.2, 44.8, 48.0, 46.5).
template <int NP>
constexpr int kForwardCtas = NP <= 2 ? 4 : (NP <= 4 ? 3 : 2);
constexpr int kForwardStages = 2;

// A lane's pieces of N tensors' rows, STAGES - 1 rows ahead of the one in hand.
template <typename E, int G, int NP, int RM, int N, int STAGES>
struct Ahead {
  static_assert(STAGES >= 2, "the row in hand and one ahead");
  static constexpr uint32_t STAGE_BYTES = (uint32_t)N * NP * NT * 16u;
  Rows row;
  At<const E> at[N];
  uint32_t slots;   // this thread's first
  int fill = 0, use = 0;
  __device__ __forceinline__ Ahead(const Rows& r, const At<const E> (&from)[N], uint32_t base)
      : row(r), slots(base + threadIdx.x * 16u) {
#pragma unroll
    for (int n = 0; n < N; ++n) at[n] = from[n];
  }
  __device__ __forceinline__ void load(const Lane<E, G, NP, RM>& ln) {
    if (row.left) {
      const bool there = row.on();
#pragma unroll
      for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int m = 0; m < NP; ++m) {
          const bool on = there && ln.on(m);
          cp_async16(slots + (uint32_t)fill * STAGE_BYTES + (uint32_t)((n * NP + m) * NT) * 16u,
                     on ? static_cast<const void*>(at[n].p + m * G * Piece<E>::V) : static_cast<const void*>(at[n].base), on ? 16u : 0u);
        }
      }
      const bool wraps = row.next();
#pragma unroll
      for (int n = 0; n < N; ++n) at[n].next(wraps);
    }
    cp_async_commit();
    if (++fill == STAGES) fill = 0;
  }
  // The next row's pieces of tensor n, once they are there (after wait()).
  __device__ __forceinline__ void wait() const { cp_async_wait<STAGES - 2>(); }
  __device__ __forceinline__ uint4 piece(int n, int m) const {
    return lds128(slots + (uint32_t)use * STAGE_BYTES + (uint32_t)((n * NP + m) * NT) * 16u);
  }
  __device__ __forceinline__ void done() {
    if (++use == STAGES) use = 0;
  }
};

template <typename E, int G, int NP, int RM>
__global__ void __launch_bounds__(NT, kForwardCtas<NP>) norm_rope_kernel(const __grid_constant__ NormArgs a) {
  using P = Piece<E>;
  constexpr int V = P::V, K = 32 / G;
  extern __shared__ float4 smem[];   // weights, then a table of cos and sin per group of lanes
  int cta;
  const NormSide& sd = side_of(a, cta);
  const Lane<E, G, NP, RM> ln(a);
  const int warp = (int)threadIdx.x >> 5, group = ((int)threadIdx.x & 31) / G;
  // the groups of a warp are at one token where its heads are a multiple of them: they then
  // share its table
  const bool together = sd.H % K == 0;
  float2* table = reinterpret_cast<float2*>(smem + a.d_norm / 4) + (warp * K + (together ? 0 : group)) * (a.d_rope / 2);
  const int me = together ? (int)threadIdx.x & 31 : ln.lane, workers = together ? 32 : G;
  Rows row(a, sd, (uint32_t)cta * (NT / 32) + warp, (uint32_t)sd.ctas * (NT / 32), group, K);
  At<E> y(static_cast<E*>(sd.y), row, sd.y_stride_t, sd.y_stride_h, ln.p0 * V);
  const At<const E> x[1] = {{static_cast<const E*>(sd.x), row, sd.x_stride_t, sd.x_stride_h, ln.p0 * V}};
  constexpr int STAGES = kForwardStages;
  Ahead<E, G, NP, RM, 1, STAGES> ahead(row, x, smem_u32(smem) + staged_bytes<G>(a));
  wait_for_previous();
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) ahead.load(ln);
  int32_t pos = a.d_rope && row.on() ? a.positions[row.t] : 0;
  bool fresh = true;
  stage_weights<E>(a, sd, smem);
  __syncthreads();
  const float inv_n = 1.0f / (float)a.d_norm;
  float c[Lane<E, G, NP, RM>::CS], s[Lane<E, G, NP, RM>::CS];
  while (row.left) {   // (the same in the whole warp)
    ahead.wait();
    uint4 now[NP];
#pragma unroll
    for (int m = 0; m < NP; ++m) now[m] = ahead.piece(0, m);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      float v[V];
      P::unpack(now[m], v);
      if (ln.normed(m)) {
#pragma unroll
        for (int e = 0; e < V; e += 2) fma2(s0, s1, v[e], v[e + 1], v[e], v[e + 1]);
      }
    }
    ahead.done();
    ahead.load(ln);   // (into the slots of the row before this one)
    const float r = rsqrtf(row_sum<G>(s0 + s1) * inv_n + a.eps);
    if (a.d_rope && __any_sync(0xffffffffu, fresh)) ln.angles(a, table, me, workers, pos, 1.f, c, s);
    const bool live = row.on();
    E* dst = y.p;
    const bool wraps = row.next();
    y.next(wraps);
    fresh = wraps || row.dt != 0;
    if (a.d_rope && fresh && row.on()) pos = a.positions[row.t];
    auto scaled = [&](int m, float* v) {
      P::unpack(now[m], v);
      if (ln.normed(m)) {
        float w[V];
        read_weights<E>(smem, ln.normed_pieces, ln.piece(m), w);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          mul2(w[e], w[e + 1], w[e], w[e + 1], r, r);
          mul2(v[e], v[e + 1], v[e], v[e + 1], w[e], w[e + 1]);
        }
      }
    };
#pragma unroll
    for (int m = 0; m < NP - RM; ++m) {
      float v[V];
      scaled(m, v);
      if (live && ln.on(m)) *reinterpret_cast<uint4*>(dst + m * G * V) = P::pack(v);
    }
    float v[RM][V];
#pragma unroll
    for (int m = 0; m < RM; ++m) scaled(NP - RM + m, v[m]);
    if (a.d_rope) ln.turn(v, c, s);
#pragma unroll
    for (int m = 0; m < RM; ++m)
      if (live && ln.on(NP - RM + m)) *reinterpret_cast<uint4*>(dst + (NP - RM + m) * G * V) = P::pack(v[m]);
  }
}

// --------------------------------------------------------------------------
// Gradient.  The groups of lanes keep their columns' sums for dw in registers; the CTA adds
// them up in shared memory and stores one row of partial sums, which a second small kernel
// adds in a fixed order: no atomics, the same inputs give the same bits.
// --------------------------------------------------------------------------
// The gradient's, by the registers for dw (8192 x 32 x 256 in bf16, one CTA: of 2 rows 81.2 us, 3
// 65.6, 4 68.7; 4095 x 40 x 128 in float32, two: of 2 46.7, 3 49.3; one of 4: 51.3).
template <int SIZE, int NP>
constexpr int kGradientCtas = NP <= 3 || (SIZE == 4 && NP == 4) ? 2 : 1;
template <int SIZE, int NP>
constexpr int kGradientStages = NP <= 3 || (SIZE == 2 && NP == 4) ? 3 : 2;

template <typename E, int G, int NP, int RM>
__global__ void __launch_bounds__(NT, kGradientCtas<sizeof(E), NP>) norm_rope_gradient_kernel(const __grid_constant__ NormArgs a) {
  using P = Piece<E>;
  constexpr int V = P::V, K = 32 / G;
  extern __shared__ float4 smem[];   // as above; then, over all of it, [NT / 32][d_norm] sums
  int cta;
  const NormSide& sd = side_of(a, cta);
  const Lane<E, G, NP, RM> ln(a);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane / G;
  const bool together = sd.H % K == 0;
  float2* table = reinterpret_cast<float2*>(smem + a.d_norm / 4) + (warp * K + (together ? 0 : group)) * (a.d_rope / 2);
  const int me = together ? lane : ln.lane, workers = together ? 32 : G;
  Rows row(a, sd, (uint32_t)cta * (NT / 32) + warp, (uint32_t)sd.ctas * (NT / 32), group, K);
  At<E> y(static_cast<E*>(sd.y), row, sd.y_stride_t, sd.y_stride_h, ln.p0 * V);
  const At<const E> from[2] = {{static_cast<const E*>(sd.x), row, sd.x_stride_t, sd.x_stride_h, ln.p0 * V},
                               {static_cast<const E*>(sd.g), row, sd.g_stride_t, sd.g_stride_h, ln.p0 * V}};
  constexpr int STAGES = kGradientStages<sizeof(E), NP>;
  Ahead<E, G, NP, RM, 2, STAGES> ahead(row, from, smem_u32(smem) + staged_bytes<G>(a));
  launch_dependents();
  wait_for_previous();
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) ahead.load(ln);
  int32_t pos = a.d_rope && row.on() ? a.positions[row.t] : 0;
  bool fresh = true;
  stage_weights<E>(a, sd, smem);
  __syncthreads();
  const float inv_n = 1.0f / (float)a.d_norm;
  float c[Lane<E, G, NP, RM>::CS], s[Lane<E, G, NP, RM>::CS], dw[NP][V];
#pragma unroll
  for (int m = 0; m < NP; ++m) {
#pragma unroll
    for (int e = 0; e < V; ++e) dw[m][e] = 0.f;
  }
  while (row.left) {   // (the same in the whole warp; a row that is not there is zeros)
    if (a.d_rope && __any_sync(0xffffffffu, fresh)) ln.angles(a, table, me, workers, pos, -1.f, c, s);
    ahead.wait();
    float v[NP][V], g[NP][V];
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      P::unpack(ahead.piece(0, m), v[m]);
      P::unpack(ahead.piece(1, m), g[m]);
    }
    ahead.done();
    if (a.d_rope) ln.turn(g + (NP - RM), c, s);
    const bool live = row.on();
    E* dst = y.p;
    const bool wraps = row.next();
    y.next(wraps);
    fresh = wraps || row.dt != 0;
    if (a.d_rope && fresh && row.on()) pos = a.positions[row.t];
    float s0 = 0.f, s1 = 0.f, d0 = 0.f, d1 = 0.f;
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      if (ln.normed(m)) {
        float w[V];
        read_weights<E>(smem, ln.normed_pieces, ln.piece(m), w);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          fma2(s0, s1, v[m][e], v[m][e + 1], v[m][e], v[m][e + 1]);
          mul2(w[e], w[e + 1], w[e], w[e + 1], g[m][e], g[m][e + 1]);
          fma2(d0, d1, w[e], w[e + 1], v[m][e], v[m][e + 1]);
        }
      }
    }
    // (a row that is not there adds zeros: with eps = 0 its root would be infinite)
    const float rs = row_sum<G>(s0 + s1), r = live ? rsqrtf(rs * inv_n + a.eps) : 0.f;
    const float k = -(row_sum<G>(d0 + d1) * inv_n * r * r);
    ahead.load(ln);   // (into the slots of the row before this one)
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      if (ln.normed(m)) {
        float w[V];
        read_weights<E>(smem, ln.normed_pieces, ln.piece(m), w);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          float gx0, gx1;
          mul2(gx0, gx1, g[m][e], g[m][e + 1], v[m][e], v[m][e + 1]);
          fma2(dw[m][e], dw[m][e + 1], gx0, gx1, r, r);
          mul2(w[e], w[e + 1], w[e], w[e + 1], g[m][e], g[m][e + 1]);
          fma2(w[e], w[e + 1], v[m][e], v[m][e + 1], k, k);
          mul2(g[m][e], g[m][e + 1], w[e], w[e + 1], r, r);
        }
      }
      if (live && ln.on(m)) *reinterpret_cast<uint4*>(dst + m * G * V) = P::pack(g[m]);
    }
  }
  // the CTA's sums: over the rows of a warp by shuffles, then over the warps
  cp_async_wait<0>();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int m = 0; m < NP; ++m) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float x = dw[m][e];
#pragma unroll
      for (int o = G; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane < G && ln.normed(m)) sums[warp * a.d_norm + ln.piece(m) * V + e] = x;
    }
  }
  __syncthreads();
  float* part = a.part + (int64_t)blockIdx.x * a.d_norm;
  for (int i = threadIdx.x; i < a.d_norm; i += NT) {
    float x = sums[i];
#pragma unroll
    for (int k = 1; k < NT / 32; ++k) x += sums[k * a.d_norm + i];
    part[i] = x;
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
#pragma unroll 8
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

// --------------------------------------------------------------------------
// Any columns, strides and alignment: a warp per row, which it holds in shared memory.
// --------------------------------------------------------------------------
constexpr int NT_ANY = 128;

// The last d_rope columns of a row in shared memory, turned in place by one warp.
__device__ __forceinline__ void turn_row(const NormArgs& a, float* row, int32_t pos, float sign) {
  const int pairs = a.d_rope / 2;
  const bool half = a.table.layout == DSA_ROPE_HALF;
  float* v = row + a.d - a.d_rope;
  __syncwarp();
  for (int i = (int)lane_id(); i < pairs; i += 32) {
    const int p = half ? i : 2 * i, q = half ? i + pairs : 2 * i + 1;
    float c, s;
    rope_cos_sin(a.table.turns[i], pos, a.table.mscale, c, s);
    s *= sign;
    const float x = v[p], y = v[q];
    v[p] = x * c - y * s;
    v[q] = x * s + y * c;
  }
  __syncwarp();
}

template <typename E>
__global__ void __launch_bounds__(NT_ANY) norm_rope_any_kernel(const __grid_constant__ NormArgs a) {
  using P = Piece<E>;
  extern __shared__ float4 smem[];
  float* v = reinterpret_cast<float*>(smem) + (threadIdx.x >> 5) * a.d;
  const int lane = (int)lane_id();
  int cta;
  const NormSide& sd = side_of(a, cta);
  wait_for_previous();
  for (Rows row(a, sd, (uint32_t)cta * (NT_ANY / 32) + (threadIdx.x >> 5), (uint32_t)sd.ctas * (NT_ANY / 32), 0, 1); row.left; row.next()) {
    const E* x = static_cast<const E*>(sd.x) + (int64_t)row.t * sd.x_stride_t + (int64_t)row.h * sd.x_stride_h;
    float sum = 0.f;
    for (int c = lane; c < a.d; c += 32) {
      const float e = P::load(x + c);
      v[c] = e;
      if (c < a.d_norm) sum += e * e;
    }
    const float r = rsqrtf(row_sum<32>(sum) / (float)a.d_norm + a.eps);
    for (int c = lane; c < a.d_norm; c += 32) v[c] *= r * weight_at(a, sd, c);
    if (a.d_rope) turn_row(a, v, a.positions[row.t], 1.f);
    E* y = static_cast<E*>(sd.y) + (int64_t)row.t * sd.y_stride_t + (int64_t)row.h * sd.y_stride_h;
    for (int c = lane; c < a.d; c += 32) P::store(y + c, v[c]);
    __syncwarp();
  }
}

template <typename E>
__global__ void __launch_bounds__(NT_ANY) norm_rope_gradient_any_kernel(const __grid_constant__ NormArgs a) {
  using P = Piece<E>;
  extern __shared__ float4 smem[];   // sums of every warp, then its row and gradient row
  constexpr int W = NT_ANY / 32;
  const int lane = (int)lane_id(), warp = (int)threadIdx.x >> 5;
  float* sums = reinterpret_cast<float*>(smem);
  float* dw = sums + warp * a.d_norm;
  float* v = sums + W * a.d_norm + 2 * warp * a.d;
  float* g = v + a.d;
  int cta;
  const NormSide& sd = side_of(a, cta);
  launch_dependents();
  wait_for_previous();
  for (int c = lane; c < a.d_norm; c += 32) dw[c] = 0.f;
  for (Rows row(a, sd, (uint32_t)cta * W + warp, (uint32_t)sd.ctas * W, 0, 1); row.left; row.next()) {
    const E* x = static_cast<const E*>(sd.x) + (int64_t)row.t * sd.x_stride_t + (int64_t)row.h * sd.x_stride_h;
    const E* gy = static_cast<const E*>(sd.g) + (int64_t)row.t * sd.g_stride_t + (int64_t)row.h * sd.g_stride_h;
    float sum = 0.f, dot = 0.f;
    for (int c = lane; c < a.d; c += 32) {
      const float e = P::load(x + c);
      v[c] = e;
      g[c] = P::load(gy + c);
      if (c < a.d_norm) sum += e * e;
    }
    if (a.d_rope) turn_row(a, g, a.positions[row.t], -1.f);
    for (int c = lane; c < a.d_norm; c += 32) dot += g[c] * weight_at(a, sd, c) * v[c];
    const float r = rsqrtf(row_sum<32>(sum) / (float)a.d_norm + a.eps);
    const float k = row_sum<32>(dot) / (float)a.d_norm * r * r;
    E* y = static_cast<E*>(sd.y) + (int64_t)row.t * sd.y_stride_t + (int64_t)row.h * sd.y_stride_h;
    for (int c = lane; c < a.d; c += 32) {
      float e = g[c];
      if (c < a.d_norm) {
        dw[c] += e * v[c] * r;
        e = r * (e * weight_at(a, sd, c) - v[c] * k);
      }
      P::store(y + c, e);
    }
    __syncwarp();
  }
  __syncthreads();
  float* part = a.part + (int64_t)blockIdx.x * a.d_norm;
  for (int c = threadIdx.x; c < a.d_norm; c += NT_ANY) {
    float x = sums[c];
#pragma unroll
    for (int k = 1; k < W; ++k) x += sums[k * a.d_norm + c];
    part[c] = x;
  }
}

// The sides' CTAs: their rows' share of `most`, at least one each, no more than give every
// worker (of `workers` a CTA) a row.  Returns their number.
static int share_ctas(NormArgs& a, int64_t most, int workers) {
  const int64_t heads = (int64_t)a.side[0].H + a.side[1].H;
  int n = 0;
  for (NormSide& sd : a.side) {
    const int64_t need = ((int64_t)a.T * sd.H + workers - 1) / workers;
    int64_t share = most * sd.H / heads;
    if (share < 1 && sd.H) share = 1;
    sd.ctas = (int)(need < share ? need : share);
    n += sd.ctas;
  }
  return n;
}

static int launch_weights(const NormArgs& a, cudaStream_t stream) {
  const int sides = (a.side[0].H > 0) + (a.side[1].H > 0);
  return launch_after(norm_weight_kernel, dim3((unsigned)((a.d_norm + 31) / 32), (unsigned)sides), NT, 0, stream, a);
}

// Rows of many pieces a lane: the gradient has no registers for them.
template <int G, int NP>
constexpr bool kForwardOnly = G == 8 && NP > 4;

template <typename E, int G, int NP, int RM>
static int launch_t(NormArgs& a, bool gradient, int num_sms, cudaStream_t stream) {
  if (!gradient) {
    constexpr int CTAS = kForwardCtas<NP>;
    const uint32_t smem = staged_bytes<G>(a) + kForwardStages * Ahead<E, G, NP, RM, 1, 2>::STAGE_BYTES;
    static PerDevice done;
    if (allow_smem(reinterpret_cast<const void*>(norm_rope_kernel<E, G, NP, RM>), kMostSmem, done) != 0) return -1;
    const int ctas = share_ctas(a, (int64_t)CTAS * num_sms, NT / G);
    return launch_after(norm_rope_kernel<E, G, NP, RM>, dim3((unsigned)ctas), NT, smem, stream, a);
  }
  if constexpr (kForwardOnly<G, NP>) {
    return -2;
  } else {
    constexpr int CTAS = kGradientCtas<sizeof(E), NP>;
    const int64_t most = (int64_t)CTAS * num_sms;
    const int ctas = share_ctas(a, most < kNormMaxCtas ? most : kNormMaxCtas, NT / G);
    const uint32_t ahead = staged_bytes<G>(a) + kGradientStages<sizeof(E), NP> * Ahead<E, G, NP, RM, 2, 2>::STAGE_BYTES;
    const uint32_t sums = (uint32_t)(NT / 32 * a.d_norm * 4);
    if (ctas > 0) {   // (no tokens: the sums below are of nothing)
      static PerDevice done;
      if (allow_smem(reinterpret_cast<const void*>(norm_rope_gradient_kernel<E, G, NP, RM>), kMostSmem, done) != 0) return -1;
      const int r = launch_after(norm_rope_gradient_kernel<E, G, NP, RM>, dim3((unsigned)ctas), NT,
                                 ahead > sums ? ahead : sums, stream, a);
      if (r != 0) return r;
    }
    return launch_weights(a, stream);
  }
}

// RM of G lanes: one piece each holds the RoPE columns, or 2 or 4, in the half layout
// exactly (a pair's other half is then in the lane); 0: none does.
static int rope_pieces(int R, int G, bool half) {
  if (R <= G) return 1;
  if (half ? R == 2 * G : R <= 2 * G) return 2;
  return (half ? R == 4 * G : R <= 4 * G) ? 4 : 0;
}

template <typename E, int G>
static int launch_g(NormArgs& a, int rm, bool gradient, int num_sms, cudaStream_t stream) {
  const int np = (a.d / Piece<E>::V + G - 1) / G;
  if (np == 1 && rm == 1) return launch_t<E, G, 1, 1>(a, gradient, num_sms, stream);
  if (np == 2) return rm == 1 ? launch_t<E, G, 2, 1>(a, gradient, num_sms, stream) : launch_t<E, G, 2, 2>(a, gradient, num_sms, stream);
  if (np == 3 && rm < 4) return rm == 1 ? launch_t<E, G, 3, 1>(a, gradient, num_sms, stream) : launch_t<E, G, 3, 2>(a, gradient, num_sms, stream);
  if (np <= 4) {
    if (rm == 4) return launch_t<E, G, 4, 4>(a, gradient, num_sms, stream);
    return rm == 1 ? launch_t<E, G, 4, 1>(a, gradient, num_sms, stream) : launch_t<E, G, 4, 2>(a, gradient, num_sms, stream);
  }
  if constexpr (G == 8 && Piece<E>::V == 8) {
    if (!gradient && rm == 1) return np <= 6 ? launch_t<E, G, 6, 1>(a, gradient, num_sms, stream) : launch_t<E, G, 9, 1>(a, gradient, num_sms, stream);
  }
  if constexpr (G == 32 && Piece<E>::V == 4)
    return rm == 1 ? launch_t<E, G, 8, 1>(a, gradient, num_sms, stream) : launch_t<E, G, 8, 2>(a, gradient, num_sms, stream);
  return -2;
}

// The fewest lanes that hold a row in four pieces each (32 of float32 rows: eight) and its
// RoPE columns as rope_pieces wants them.
template <typename E>
static int launch_rows(NormArgs& a, bool vec, bool gradient, int num_sms, cudaStream_t stream) {
  constexpr int V = Piece<E>::V;
  const int pieces = a.d / V, R = a.d_rope / V;
  const bool half = a.table.layout == DSA_ROPE_HALF;
  if (vec) {
    int rm = pieces <= 32 || (V == 8 && !gradient && R <= 8 && pieces <= 72) ? rope_pieces(R, 8, half) : 0;
    if (rm) return launch_g<E, 8>(a, rm, gradient, num_sms, stream);
    rm = pieces <= 64 ? rope_pieces(R, 16, half) : 0;
    if (rm) return launch_g<E, 16>(a, rm, gradient, num_sms, stream);
    rm = rope_pieces(R, 32, half);   // (R is 64 at most)
    if (rm) return launch_g<E, 32>(a, rm, gradient, num_sms, stream);
  }
  if (!gradient) {
    const int ctas = share_ctas(a, 8ll * num_sms, NT_ANY / 32);
    return launch_after(norm_rope_any_kernel<E>, dim3((unsigned)ctas), NT_ANY, (uint32_t)(NT_ANY / 32 * a.d * 4), stream, a);
  }
  const int64_t most = 2ll * num_sms;
  const int ctas = share_ctas(a, most < kNormMaxCtas ? most : kNormMaxCtas, NT_ANY / 32);
  if (ctas > 0) {
    const int r = launch_after(norm_rope_gradient_any_kernel<E>, dim3((unsigned)ctas), NT_ANY,
                               (uint32_t)(NT_ANY / 32 * (a.d_norm + 2 * a.d) * 4), stream, a);
    if (r != 0) return r;
  }
  return launch_weights(a, stream);
}

}  // namespace normrope

int launch_norm_rope(NormArgs& a, bool f32, bool vec, bool gradient, int num_sms, cudaStream_t stream) {
  return f32 ? normrope::launch_rows<float>(a, vec, gradient, num_sms, stream)
             : normrope::launch_rows<uint16_t>(a, vec, gradient, num_sms, stream);
}

}  // namespace dsa
