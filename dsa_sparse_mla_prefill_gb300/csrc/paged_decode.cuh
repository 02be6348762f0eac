// Attention of one new token per request, or of a tree of drafted tokens, over a paged
// latent KV cache: the kernel (launched by paged_decode.cu and tree_decode.cu).
//
//     s_hj = scale * q[b,h,:] . c_j          c_j: latent row of position j
//     out[b,h,:] = sum_j softmax_j(s_h) c_j[0:512],   lse[b,h] = ln sum_j exp(s_hj)
// over the positions j < kv_len[b], or over the token's own top-k positions;
// position j lies in row table[b][j / block_size] * block_size + j % block_size.
//
// Bound: every row is read from HBM once for all heads of the request (1152
// bytes, or 656 in FP8, against 2 * 1088 * H flops), so up to 32 heads HBM is the
// bound; at 128 heads the flops come within 15 % of it.
//
// Split over the length: the keys of all requests, in tiles of 128, form one
// line of W tiles, dealt to the CTA groups in equal contiguous ranges
// ([g W / G, (g+1) W / G)), so one long context and a ragged batch alike keep
// every SM busy to within one tile, from the lengths the GPU holds (nothing is
// planned on the host, and a captured graph follows them).  A range ends some
// requests and begins another: a request that lies whole in a range is stored
// at once, the parts of one cut by a range border are stored as normalised fp32
// outputs with their log-sum-exp and joined by a second small kernel (decode_join.cuh), which is
// launched so that its start overlaps the first one's end.
//
// A group is one CTA per 16 heads (H <= 16), 32 (H <= 32, and FP8 rows) or 64, all
// walking the same rows at the same time.  Fewer, wider CTAs per group read fewer
// copies of a row through L2: at 128 heads, 16 x 19456 positions take 193 us as 4
// CTAs of 32 heads and 123 us as 2 of 64 (all pages in L2).  Each CTA loads what its
// own MMAs read, into its own shared memory.
//
// One CTA (24 warps; 28 of the 64-head form, 32 of 16 heads over FP8 rows):
//   softmax     8 warps (16): thread = key (TMEM lane), warpgroup = its share of
//               the heads; online in base 2 with the lazy rescale (only when a
//               head's running max grows by more than 2^8); P to shared memory in
//               bf16; the epilogue (O^T lane = output column).
//   W_QK        S^T = K q^T, keys on the M side (M = 128, N = heads)
//   W_PV        O^T += V^T P^T, one 128-column unit after another
//   W_Q         q per request; the outputs of requests without keys
//   W_SCHED     walks the range, turns 128 positions per tile into rows (a ring of
//               four tiles ahead)
//   W_LOAD ...  TMA loads: row gathers (4 rows x 128 bytes per instruction), or
//               boxes of up to 128 rows where every key of the tile is there and
//               the pages hold them in runs (page sizes that are multiples of 8
//               rows); for FP8 rows the last eight (16) convert.
//
// bf16 rows are loaded twice, from HBM into a ring of 64-column K chunks (QK reads
// them K-major) and from L2 into a ring of 128-column V units (P.V reads them
// MN-major).  Loading them once, into units that QK and P.V share, needs a tile's
// four units from the first QK to the last P.V: the next tile's loads wait for
// this one's softmax, 7000-10000 cycles a tile against 5000 (all pages in L2).
// FP8 rows are loaded once, into a ring of code slots, and converted into such
// shared units, since converting costs more than loading: a tile takes 7500 cycles
// at 16 heads, its four conversions (some 700 cycles apart), the softmax and the
// first P.V one after another.  The conversion is a chain of latencies (two waits,
// load, convert, store, fence), not of arithmetic (none at all: the same time), so
// where registers allow two sets of eight warps take the units in turn: 48 requests
// up to 16384 positions at 16 heads 68 us, 71 with one set (at 32 heads, with 40
// registers a thread, 16 x 19456 would take 96 us instead of 85).
// Rows that are masked (behind kv_len, -1, unmapped pages) are loaded from
// outside the tensor map, which reads as zeros: whatever the cache holds there,
// NaN included, never reaches the sums.
//
// Measured (128-key tiles per CTA of 32 heads): 2.5 us a tile with all pages in
// L2, 3.3 from HBM (5.1 TB/s of 6.8); 64 ragged requests up to 16384 positions
// 73 us against 43.6 for the bytes alone, one request of 131072 42 against 22.3:
// the rest is the start (6 us), the last tile's way through the CTA and the join
// (4-8 us).
//
// Rounding: P is rounded to bf16 for the tensor core.  The outputs are divided
// by the sum of the rounded weights (so that the weights used add up to one);
// the log-sum-exp comes from the unrounded sum, both in fp32.
#pragma once
#include <cfloat>

#include "decode_join.cuh"
#include "dsa_device.cuh"
#include "dsa_kernels.h"
#include "dsa_launch.cuh"

namespace dsa {
namespace decode {

constexpr int BK = 128;          // keys per tile (the MMA's M)
constexpr int NI = 4;            // tiles of rows ahead
constexpr float kTau = 8.0f;     // lazy-rescale threshold (log2 units)

template <int HB, int NC, bool F8>
struct Cfg {
  static constexpr int SWG = HB == 64 ? 4 : 2;           // softmax warpgroups
  static constexpr int HT = HB / SWG;                    // heads per softmax thread
  // warps: the softmax warpgroups, one each for QK, P.V, q and the schedule, then
  // the loaders (and converters)
  static constexpr int W_QK = 4 * SWG, W_PV = W_QK + 1, W_Q = W_QK + 2, W_SCHED = W_QK + 3, W_LOAD = W_QK + 4;
  static constexpr int NCONV = !F8 ? 0 : (HB == 16 ? 16 : 8);   // converting warps, the last ones
  static constexpr int NWARPS = W_LOAD + (HB == 64 ? 8 : (NCONV == 16 ? 20 : 12));
  static constexpr int NTHREADS = 32 * NWARPS;
  // registers: at launch, of the softmax warps and of the others
  static constexpr int REGS_LAUNCH = HB == 64 ? 72 : (NCONV == 16 ? 64 : 80);
  static constexpr int REGS_SOFTMAX = HB == 64 ? 96 : (F8 ? (HB == 16 ? 88 : 128) : 144);
  static constexpr int REGS_REST = HB == 64 ? 40 : (F8 ? 56 : 48);
  static_assert(128 * SWG * REGS_SOFTMAX + (NTHREADS - 128 * SWG) * REGS_REST <= NTHREADS * REGS_LAUNCH, "registers");
  // What shared memory leaves beside q and P.  bf16 rows: a ring of NK 64-column
  // K chunks and one of NV 128-column V units.  FP8 rows: a ring of NK slots for
  // the RoPE columns and the four code blocks (128 rows x 128) of a tile, and NV
  // units of converted columns that QK and P.V both read.
  static constexpr int NK = F8 ? (HB == 16 ? 4 : 3) : (HB == 16 ? 6 : (HB == 32 ? 5 : 4));
  static constexpr int NV = F8 ? 4 : (HB == 64 ? 2 : 3);
  // warps that read the row ring: the loaders, and for FP8 rows the converters
  static constexpr int NPROD = F8 ? NK + NCONV : NK + 2 * NV;
  static_assert(NPROD <= NWARPS - W_LOAD, "warps");
  static_assert(!F8 || NV == 4, "a unit per code block");
  static constexpr uint32_t CHUNK_BYTES = BK * 128u;     // 128 keys x 64 columns
  static constexpr uint32_t UNIT_BYTES = 2u * CHUNK_BYTES;
  static constexpr uint32_t Q_BYTES = NC * HB * 128u;
  static constexpr uint32_t P_BYTES = 2u * HB * 128u;
  static constexpr uint32_t RED_FLOATS = 2u * SWG * 4u * HT;   // [parity][warpgroup][warp][head]
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = OFF_K + NK * CHUNK_BYTES;
  static constexpr uint32_t OFF_Q = OFF_V + NV * UNIT_BYTES;
  static constexpr uint32_t OFF_P = OFF_Q + Q_BYTES;
  static constexpr uint32_t OFF_ROWS = OFF_P + P_BYTES;
  static constexpr uint32_t OFF_META = OFF_ROWS + NI * BK * 4u;
  static constexpr uint32_t OFF_RED = OFF_META + NI * 16u;
  static constexpr uint32_t OFF_BAR = OFF_RED + (2u * RED_FLOATS + HB) * 4u;   // (two sums and a factor per head in the epilogue)
  static constexpr int NBAR = 64;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8u;
  static constexpr uint32_t MISC_BYTES = 256u;
  static constexpr uint32_t SMEM_BYTES = OFF_MISC + MISC_BYTES + 1024u;
  static_assert(SMEM_BYTES <= 227u * 1024u, "shared memory budget");
  // TMEM columns: O^T (4 HB, twice where they fit, so that an epilogue overlaps
  // the next request), S^T double buffer (2 x HB)
  static constexpr int NO = HB == 64 ? 1 : 2;
  static constexpr uint32_t COL_S = NO * 4u * HB;
  static constexpr uint32_t TMEM_COLS = (COL_S + 2u * HB <= 256u) ? 256u : 512u;
};

enum {
  B_IDX_FULL = 0,    // [NI]
  B_IDX_EMPTY = 4,   // [NI]
  B_Q_FULL = 8,
  B_Q_EMPTY = 10,
  B_S_FULL = 12,     // [2]
  B_S_EMPTY = 14,    // [2]
  B_P_FULL = 16,
  B_P_EMPTY = 17,
  B_O_FULL = 18,     // [2]
  B_O_EMPTY = 20,    // [2]
  B_SMX = 60,        // [4] one per softmax warpgroup
  B_PLAN = 9,
  B_DRAIN = 24,      // [2] one per MMA issuer
  B_FULL = 26,       // [16] K slots (FP8: items of a tile) from 0, V units from 8
  B_EMPTY = 42,      // [16]
};

// Drafted tokens of request b (tree form).
__device__ __forceinline__ int drafted_of(const DecodeArgs& a, int b) {
  return a.num_draft == nullptr ? a.n : max(0, min(a.n, a.num_draft[b]));
}

// flags of a tile
constexpr int F_FIRST = 1;    // first tile of its request in this range
constexpr int F_LAST = 2;     // last one
constexpr int F_PART = 4;     // the request is cut: store a partial result
constexpr int F_SLOT1 = 8;    // ... into the range's second slot (it did not begin the range)
constexpr int F_BOX = 16;     // every key there, in runs of box_rows rows: loaded by boxes

// key tiles of a request
__device__ __forceinline__ int tiles_of(const DecodeArgs& a, int len) {
  if (len <= 0) return 0;
  return ((uint32_t)(a.idx != nullptr ? a.k : min(len, a.cap)) + BK - 1) / BK;
}

// TMA loads with an L2 hint.  The rows of a tile are read twice, for K and then
// for V: the first read caches them as usual, the second marks them first to go.
// (Marked on the first read, a sixth to a third of them were gone by the second,
// pushed out by each other while older lines of other tensors stayed.)
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t evict_normal_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void load_2d_hint(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar,
                                             uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// Tensor-core issue by one elected lane of a converged warp: the loops around
// it are warp-uniform, so descriptors and loop state stay in uniform registers
// (issued from inside a one-lane branch, every operand is first moved there,
// about 120 cycles per MMA instead of 45).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ void mma_x4_elected(uint32_t leader, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t da,
                                               uint32_t db, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %11, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %5, %6, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %7, %8, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %9, %10, %3, 1;\n\t}"
      ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "l"(a + da), "l"(b + db), "l"(a + 2ull * da),
      "l"(b + 2ull * db), "l"(a + 3ull * da), "l"(b + 3ull * db), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar)), "r"(leader)
      : "memory");
}

// A tile's 32 row gathers (4 rows x 128 bytes each), issued by one
// elected lane as the MMAs are (a lane per gather: 777 positions 13.9 against 13.4 us).
__device__ __forceinline__ void gather_rows(uint32_t leader, uint32_t dst, const CUtensorMap* map, int x, const int32_t* rows,
                                            uint64_t* bar, uint64_t policy) {
#pragma unroll 4
  for (int n = 0; n < BK / 4; ++n) {
    const int4 r = *reinterpret_cast<const int4*>(rows + 4 * n);
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %9, 0;\n\t"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;\n\t}" ::"r"(dst + n * 512),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(smem_u32(bar)),
        "l"(policy), "r"(leader)
        : "memory");
  }
}

// The row of a page's at-th position, or -1 (counted).
__device__ __forceinline__ int32_t row_at(const DecodeArgs& a, const int32_t* bt, uint32_t page, uint32_t at, int& bad) {
  const int32_t blk = bt[page];
  const int64_t x = (int64_t)blk * a.block_size + at;
  if (blk >= 0 && x < a.N) return (int32_t)x;
  ++bad;
  return -1;
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane_id() >= o) v += up;
  }
  return v;
}

template <int N, bool IS_MAX>
__device__ __forceinline__ float warp_transpose_reduce(float* v) {
  // Every lane holds N values (one per head); afterwards lane L holds the
  // reduction over the 32 lanes of head L mod N.
  const uint32_t lane = lane_id();
  auto op = [](float x, float y) { return IS_MAX ? fmaxf(x, y) : x + y; };
#pragma unroll
  for (int o = 16; o >= N; o >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = op(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
  }
  int n = N;
#pragma unroll
  for (int o = N / 2; o >= 1; o >>= 1) {
    n >>= 1;
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if (i < n) {
        const float send = upper ? v[i] : v[i + n];
        const float keep = upper ? v[i + n] : v[i];
        v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
      }
    }
  }
  return v[0];
}

template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, float* v) {
  if constexpr (N == 8) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
  } else {
    tmem_ld_cols<N>(taddr, v);
  }
}
template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t taddr, const float* v) {
  if constexpr (N == 8) {
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(v[i]);
    tmem_st8_u32(taddr, r);
  } else {
    tmem_st_cols<N>(taddr, v);
  }
}

template <int HB, int NC, bool F8, bool TREE>
__global__ void __launch_bounds__(Cfg<HB, NC, F8>::NTHREADS, 1) decode_kernel(const __grid_constant__ DecodeArgs a) {
  using C = Cfg<HB, NC, F8>;
  constexpr int HT = C::HT;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_u32 + 1023u) & ~1023u) - raw_u32);
  const uint32_t sbase = smem_u32(smem);

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile uint32_t* tmem_base_ptr = misc + 0;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* plan = reinterpret_cast<volatile int*>(misc + 2);   // tiles of this range
  volatile uint32_t* votes = misc + 16;                             // [parity][warpgroup][warp]
  int32_t* rows = reinterpret_cast<int32_t*>(smem + C::OFF_ROWS);   // [NI][BK], -1 = masked
  int4* meta = reinterpret_cast<int4*>(smem + C::OFF_META);         // [NI] request, flags
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
  unsigned int* err = a.err;
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * i; };
  auto poll = [&](int i, uint32_t parity) { return mbar_wait_vote<true>(bar(i), parity, abort_flag, err); };
  auto doze = [&](int i, uint32_t parity) { return mbar_wait_vote<false>(bar(i), parity, abort_flag, err); };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int range = blockIdx.x / a.head_blocks;   // the CTA group
  const int hb = blockIdx.x - range * a.head_blocks;

  if (warp == 0) {
    // a lane per barrier and round: sixty of them one after another by one
    // thread are 700 cycles
    for (int i = lane; i < C::NBAR; i += 32) {
      uint32_t n = 1;
      // 2 MMA warps, the softmax warpgroups, the loading (converting) warps, the q loader
      if (i >= B_IDX_EMPTY && i < B_IDX_EMPTY + NI) n = 2 + C::SWG + C::NPROD + 1;
      if (i == B_S_EMPTY || i == B_S_EMPTY + 1 || i == B_O_EMPTY || i == B_O_EMPTY + 1 || i == B_P_FULL) n = 128 * C::SWG;
      if (i >= B_SMX && i < B_SMX + 4) n = 128;
      // a V unit is two loading warps' work, one of FP8 rows eight converting warps'
      if (i >= B_FULL + 8 && i < B_FULL + 16) n = F8 ? 8 : 2;
      mbar_init(&bars[i], n);
    }
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc(const_cast<uint32_t*>(tmem_base_ptr), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_ptr;
  const int head0 = hb * HB;                                   // this CTA's first head
  const int heads = a.H - head0 < HB ? a.H - head0 : HB;       // the others are padding, never stored
  const int64_t heads_padded = (int64_t)a.head_blocks * HB;

  // the joining kernel may be put on the GPU as soon as there is room
  launch_dependents();

  if (warp >= C::W_QK) {
    regs_dec<C::REGS_REST>();
    // what earlier kernels wrote may be read from here on
    wait_for_previous();
    if (warp == C::W_SCHED) {
      // ------------------------------------------------------------------
      // scheduler
      // ------------------------------------------------------------------
      // The range's tiles: every lane counts those of a run of requests, a scan
      // places the runs, and the lane whose run holds the first tile finds it.
      const int per = (a.B + 31) / 32;
      const int b_lo = min(a.B, lane * per), b_hi = min(a.B, b_lo + per);
      uint32_t mine = 0;
#pragma unroll 4
      for (int i = b_lo; i < b_hi; ++i) mine += tiles_of(a, a.kv_lens[i]);
      const uint32_t incl = warp_scan(mine), total = __shfl_sync(0xffffffffu, incl, 31), before = incl - mine;
      const uint32_t ng = total < (uint32_t)a.groups ? total : (uint32_t)a.groups;   // no range without a tile
      const uint32_t x0 = (uint32_t)range < ng ? range_begin(range, total, ng) : 0;
      const int nt = (uint32_t)range < ng ? (int)(range_begin(range + 1, total, ng) - x0) : 0;
      if (lane == 0) {
        *plan = nt;
        mbar_arrive(&bars[B_PLAN]);
        if (range == 0 && hb == 0) a.borders[0] = make_int4(total, ng, 0, 0);
        // (nothing to join until the range's last tile is reached: a wait may run out before it)
        if (hb == 0) a.borders[1 + range] = make_int4(0, 0, 0, 0);
      }
      int b = 0, j = 0, len = 0, n = 0;
      const bool holds = nt > 0 && before <= x0 && x0 < before + mine;
      if (holds) {
        uint32_t at = before;
        for (b = b_lo;; ++b) {
          len = a.kv_lens[b];
          n = tiles_of(a, len);
          if (x0 < at + n) break;
          at += n;
        }
        j = (int)(x0 - at);
      }
      const int holder = __ffs(__ballot_sync(0xffffffffu, holds)) - 1;
      b = __shfl_sync(0xffffffffu, b, holder & 31);
      j = __shfl_sync(0xffffffffu, j, holder & 31);
      len = __shfl_sync(0xffffffffu, len, holder & 31);
      int bad = 0;
      const bool from_start = j == 0;   // the range's first request begins in it
      int fetch = -1, fetch_next = -1;  // first rows of boxes to fetch
      bool enter = true;                // the next tile is the first of request b here
      int seg = 0;                    // requests begun
      int drafted = 0, context = 0;   // tree form: of request b,
      uint64_t seen = 0;              // the drafted tokens that any of them sees
      for (int it = 0; it < nt; ++it) {
        const int r = it % NI;
        if (enter) {
          // the next request with a tile (one without keys has none; there may be
          // thousands of them in a row, so 32 are looked at at once)
          while (it > 0) {
            len = b + lane < a.B ? a.kv_lens[b + lane] : 0;
            const uint32_t there = __ballot_sync(0xffffffffu, tiles_of(a, len) > 0);
            const int skip = there ? __ffs(there) - 1 : 32;
            b += skip;
            len = __shfl_sync(0xffffffffu, len, skip & 31);
            if (there) break;
            if (b >= a.B) {   // (never with lengths that stay: a tile is left)
              b = a.B - 1;
              break;
            }
          }
          n = tiles_of(a, len);
          if constexpr (TREE) {
            drafted = drafted_of(a, b);
            context = len - drafted;   // (the drafted tokens' first position; below zero where they are more than there is room for)
            uint64_t any = 0;
            for (int i = lane; i < drafted; i += 32) any |= a.tree_mask[(int64_t)b * a.n + i];
            seen = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(any >> 32)) << 32 | __reduce_or_sync(0xffffffffu, (uint32_t)any);
          }
          if (len > a.cap) {
            if (j == 0 && lane == 0) ++bad;
            len = a.cap;
          }
        }
        if (!doze(B_IDX_EMPTY + r, ((it / NI) & 1) ^ 1)) break;
        const int32_t* bt = a.block_table + (int64_t)b * a.max_blocks;
        int32_t row[4];
        const int e0 = j * BK + 4 * lane;   // (as unsigned: the last tile may end past 2^31)
        if (a.idx == nullptr) {
          uint32_t page = (uint32_t)e0 / (uint32_t)a.block_size, at = (uint32_t)e0 - page * (uint32_t)a.block_size;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            bool there = (uint32_t)e0 + e < (uint32_t)len;
            if constexpr (TREE) {
              const int bit = e0 + e - context;
              if (there && bit >= 0) there = seen >> bit & 1;   // (bit < drafted, for the position is below len)
            }
            row[e] = -1;
            if (there) row[e] = row_at(a, bt, page, at, bad);
            if (++at == (uint32_t)a.block_size) { at = 0; ++page; }
          }
        } else {
          int32_t pos[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) pos[e] = (e0 + e < a.k) ? a.idx[(int64_t)b * a.ld + e0 + e] : -1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            row[e] = -1;
            if (pos[e] >= 0 && pos[e] < len) {
              const uint32_t page = (uint32_t)pos[e] / (uint32_t)a.block_size;
              row[e] = row_at(a, bt, page, (uint32_t)pos[e] - page * (uint32_t)a.block_size, bad);
            } else if (pos[e] != -1) {
              ++bad;
            }
          }
        }
        *reinterpret_cast<int4*>(rows + r * BK + 4 * lane) = make_int4(row[0], row[1], row[2], row[3]);
        const bool box = __all_sync(0xffffffffu, (row[0] | row[1] | row[2] | row[3]) >= 0) && a.box_rows > 0;
        // 64 heads: q leaves room for 128 KB of rows in flight, too little for HBM's
        // latency, so the boxes of the tile two back, about a tile ahead of its loads,
        // are fetched to L2, by each of a group's two CTAs its half (64 x 19456 at 64
        // heads 290 -> 265 us; 16 x 19456 at 128: 133).  Not with fewer heads (64 x 256..16384 at
        // 32: 74 -> 79) nor for gathers (96 x 2048 listed at 64 heads: 109 -> 116).
        if constexpr (HB == 64) {
          if (fetch >= 0)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.rows_base + (int64_t)fetch * a.row_bytes),
                         "r"(a.fetch_bytes)
                         : "memory");
          fetch = fetch_next;
          fetch_next = __shfl_sync(0xffffffffu, row[0], (lane * a.box_rows / 4) & 31);   // of box `lane`
          if (!box || a.fetch_bytes == 0 || lane >= BK / a.box_rows || (lane & (a.head_blocks - 1)) != hb)   // (1 or 2 CTAs)
            fetch_next = -1;
        }
        const bool first = enter;
        const bool last = (it == nt - 1) || (j == n - 1);
        if (lane == 0) {
          int flags = (first ? F_FIRST : 0) | (last ? F_LAST : 0) | (box ? F_BOX : 0);
          if (last) {
            // (the range's first request may have begun before it, its last may go on behind it)
            const bool whole = (seg > 0 || from_start) && j == n - 1;
            if (!whole) flags |= F_PART | (seg > 0 ? F_SLOT1 : 0);
          }
          // (tree form: the drafted token at the tile's first position, below zero in the context; drafted tokens)
          meta[r] = make_int4(b, flags, TREE ? j * BK - context : 0, drafted);
          // where the range ends, for the join: the request, its tile count, and its tiles so far
          if (it == nt - 1 && hb == 0) a.borders[1 + range] = make_int4(b, n, j + 1, 0);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_IDX_FULL + r]);
        enter = (j == n - 1);
        if (enter) {
          ++b;
          j = 0;
          ++seg;
        } else {
          ++j;
        }
      }
      bad = __reduce_add_sync(0xffffffffu, bad);
      if (lane == 0 && bad && hb == 0) atomicAdd(err + ERR_BAD_INDEX, (unsigned)bad);
    } else if (const int nt = poll(B_PLAN, 0) ? *plan : 0; warp >= C::W_LOAD) {
      if constexpr (F8) {
        // ----------------------------------------------------------------
        // FP8 rows.  A tile is NC - 4 items: the RoPE columns (bf16, byte 528 of the
        // row), then the four 128-code blocks; they go through the ring's NK slots in
        // turn, warp W_LOAD + s loading every item of slot s.
        // The barriers are by item (0 RoPE, 1 + m block m), a phase per tile, not by
        // slot: a slot's phases would be now QK's, now the converters', and neither
        // may pass over a phase that a parity tells apart.  QK gives an item's slot
        // back: the RoPE columns when it has read them, a code block when the unit
        // made of it is there.
        // The converting warps, in sets of eight that take the units in turn: thread =
        // row and half of the block, by the arithmetic of the dequantize kernel, into
        // the unit as the bf16 rows would have landed.
        // ----------------------------------------------------------------
        constexpr int ITEMS = NC - 4;
        if (warp < C::W_LOAD + C::NK) {
          const int boxes = a.box_rows > 0 ? BK / a.box_rows : 1;
          const int own = warp - C::W_LOAD;
          const uint32_t dst = sbase + C::OFF_K + own * C::CHUNK_BYTES;
          const uint64_t policy = evict_first_policy();
          const uint32_t leader = elect_one();
          int slot = 0;
          int had = -1, had_it = 0;   // the slot's item, its tile
          bool ok = true;
#pragma unroll 1
          for (int it = 0; it < nt && ok; ++it) {
            const int r = it % NI;
            if (!doze(B_IDX_FULL + r, (it / NI) & 1)) break;
            const bool box = (meta[r].y & F_BOX) != 0;
            const int x = rows[r * BK + (lane & (boxes - 1)) * a.box_rows];   // (a box's first row)
#pragma unroll 1
            for (int item = 5 - ITEMS; item < 5; ++item) {
              const bool mine_now = slot == own;
              if (++slot == C::NK) slot = 0;
              if (!mine_now) continue;
              if (had >= 0 && !doze(B_EMPTY + had, had_it & 1)) { ok = false; break; }
              had = item;
              had_it = it;
              uint64_t* full = &bars[B_FULL + item];
              if (leader) {
                mbar_arrive_expect_tx(full, C::CHUNK_BYTES);
                if (item == 1) DSA_TRACE(a.tr, it, 1);
                if (item == 4) DSA_TRACE(a.tr, it, 2);
              }
              const int col = item == 0 ? 528 : 128 * (item - 1);
              __syncwarp();
              if (!box)
                gather_rows(leader, dst, &a.tmap_kv, col, rows + r * BK, full, policy);
              else if (lane < boxes)
                load_2d_hint(dst + lane * a.box_rows * 128, &a.tmap_box, col, x, full, policy);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_IDX_EMPTY + r]);
          }
          if (lane == 0 && had >= 0) mbar_wait_drain(&bars[B_FULL + had], had_it & 1, err);
          __syncwarp();
        } else if (warp >= C::NWARPS - C::NCONV) {
          constexpr int SETS = C::NCONV / 8;
          const int cw = warp - (C::NWARPS - C::NCONV), set = cw >> 3, hf = (cw >> 2) & 1;
          const int row = (warp & 3) * 32 + lane;
          const uint32_t rsw = (uint32_t)(row & 7);   // 128B swizzle phase of this row
          int first = NC - 8;                         // slot of the tile's first code block
          // the four block scales of the row, loaded a tile ahead (zero for a masked row)
          auto scales = [&](int it) {
            const int r = it % NI;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (it < nt && doze(B_IDX_FULL + r, (it / NI) & 1)) {
              const int x = rows[r * BK + row];
              if (x >= 0) s = *reinterpret_cast<const float4*>(a.rows_base + (int64_t)x * a.row_bytes + 512);
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars[B_IDX_EMPTY + r]);
            }
            return s;
          };
          float4 next = scales(0);
          bool ok = true;
#pragma unroll 1
          for (int it = 0; it < nt && ok; ++it) {
            float4 sc = next;
            next = scales(it + 1);
            if (SETS == 2 && set == 1) sc = make_float4(sc.y, sc.z, sc.w, 0.f);
#pragma unroll 1
            for (int m = set; m < 4; m += SETS) {
              if (!poll(B_FULL + 1 + m, it & 1) || !poll(B_EMPTY + 8 + m, (it & 1) ^ 1)) { ok = false; break; }
              const uint32_t src = sbase + C::OFF_K + (first + m) % C::NK * C::CHUNK_BYTES + row * 128;
              const uint32_t dst = sbase + C::OFF_V + m * C::UNIT_BYTES + hf * C::CHUNK_BYTES + row * 128;
              uint4 w[4];
#pragma unroll
              for (int pp = 0; pp < 4; ++pp) w[pp] = lds128(src + ((((uint32_t)(4 * hf + pp)) ^ rsw) << 4));
#pragma unroll
              for (int pp = 0; pp < 4; ++pp) {
                uint32_t v[8];
                e4m3x4_dequant_bf16x4(w[pp].x, sc.x, v[0], v[1]);
                e4m3x4_dequant_bf16x4(w[pp].y, sc.x, v[2], v[3]);
                e4m3x4_dequant_bf16x4(w[pp].z, sc.x, v[4], v[5]);
                e4m3x4_dequant_bf16x4(w[pp].w, sc.x, v[6], v[7]);
                sts128(dst + ((((uint32_t)(2 * pp)) ^ rsw) << 4), v[0], v[1], v[2], v[3]);
                sts128(dst + ((((uint32_t)(2 * pp + 1)) ^ rsw) << 4), v[4], v[5], v[6], v[7]);
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars[B_FULL + 8 + m]);
              sc = SETS == 2 ? make_float4(sc.z, sc.w, 0.f, 0.f) : make_float4(sc.y, sc.z, sc.w, 0.f);
            }
            first = (first + ITEMS) % C::NK;
          }
          __syncwarp();
        }
      } else {
      // ------------------------------------------------------------------
      // row loads: a warp per 64-column chunk in flight, since a warp issues row
      // gathers one after another (about 80 cycles each).  Warp W_LOAD + s owns K
      // slot s, the two warps after those a half of V slot 0, and so on: 32 gathers
      // of four rows, or where the keys lie in runs of box_rows rows 128 / box_rows
      // boxes, one a lane.  Gathers are the slower form: 6.2 us a tile of 32 heads
      // with all rows in L2, 9 with rows all over HBM, boxes 2.5 and 3.3 (16-byte
      // asynchronous copies instead of them: 7.9 and 10).  Each warp opens its
      // chunk's share of every phase of its slot: none can fall behind it, which a
      // wait on parity would not notice.
      // ------------------------------------------------------------------
      const bool ks = warp < C::W_LOAD + C::NK;
      const int vw = warp - C::W_LOAD - C::NK;
      if (ks || vw < 2 * C::NV) {
        const int mine_slot = ks ? warp - C::W_LOAD : vw >> 1, hf = ks ? 0 : vw & 1;
        const int nslots = ks ? C::NK : C::NV, stages = ks ? NC : 4;
        const uint32_t dst = sbase + (ks ? C::OFF_K + mine_slot * C::CHUNK_BYTES
                                         : C::OFF_V + mine_slot * C::UNIT_BYTES + hf * C::CHUNK_BYTES);
        uint64_t* full = &bars[B_FULL + (ks ? 0 : 8) + mine_slot];
        const int empty = B_EMPTY + (ks ? 0 : 8) + mine_slot;
        const int col_step = ks ? 64 : 128;
        const int boxes = a.box_rows > 0 ? BK / a.box_rows : 1;
        const uint32_t leader = elect_one();
        const uint64_t policy = ks ? evict_normal_policy() : evict_first_policy();
        int slot = 0;
        uint32_t used = 0;   // phases of the slot so far
        bool ok = true;
#pragma unroll 1
        for (int it = 0; it < nt && ok; ++it) {
          const int r = it % NI;
          if (!doze(B_IDX_FULL + r, (it / NI) & 1)) break;
          const bool box = (meta[r].y & F_BOX) != 0;
          const int x = rows[r * BK + (lane & (boxes - 1)) * a.box_rows];   // (a box's first row)
          int col = hf * 64;
#pragma unroll 1
          for (int st = 0; st < stages; ++st, col += col_step) {
            const bool mine_now = slot == mine_slot;
            if (++slot == nslots) slot = 0;
            if (!mine_now) continue;
            if (!doze(empty, (used & 1) ^ 1)) { ok = false; break; }
            if (leader) {
              mbar_arrive_expect_tx(full, C::CHUNK_BYTES);
              if (ks && st == 0) DSA_TRACE(a.tr, it, 1);
              if (ks && st == NC - 1) DSA_TRACE(a.tr, it, 2);
            }
            __syncwarp();
            if (!box)
              gather_rows(leader, dst, &a.tmap_kv, col, rows + r * BK, full, policy);
            else if (lane < boxes)
              load_2d_hint(dst + lane * a.box_rows * 128, &a.tmap_box, col, x, full, policy);
            ++used;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_IDX_EMPTY + r]);
        }
        // let the slot's last copies land before the CTA can exit
        if (lane == 0 && used > 0) mbar_wait_drain(full, (used - 1) & 1, err);
        __syncwarp();
      }
      }
    } else if (warp == C::W_Q) {
      // ------------------------------------------------------------------
      // q of every request of the range, one box per swizzle column (rows b*H +
      // head0 ... of q viewed [B*H, D_QK]); then the requests without keys
      // ------------------------------------------------------------------
      int nq = 0;
      for (int it = 0; it < nt; ++it) {
        const int r = it % NI;
        if (!doze(B_IDX_FULL + r, (it / NI) & 1)) break;
        const int4 mt = meta[r];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_IDX_EMPTY + r]);
        if (!(mt.y & F_FIRST)) continue;
        if (!doze(B_Q_EMPTY, (nq & 1) ^ 1)) break;
        if (lane == 0) mbar_arrive_expect_tx(&bars[B_Q_FULL], C::Q_BYTES);
        __syncwarp();
        if (lane < NC)
          tma_load_2d(sbase + C::OFF_Q + lane * (HB * 128), &a.tmap_q, lane * 64, mt.x * a.H + head0, &bars[B_Q_FULL]);
        ++nq;
      }
      if (lane == 0 && nq > 0) mbar_wait_drain(&bars[B_Q_FULL], (nq - 1) & 1, err);
      __syncwarp();
      // requests without keys: out = 0, lse = -inf (dealt over the groups)
      for (int b = range; b < a.B; b += a.groups) {
        if (tiles_of(a, a.kv_lens[b]) > 0) continue;
        uint4* o = reinterpret_cast<uint4*>(a.out + ((int64_t)b * a.H + head0) * 512);
        for (int i = lane; i < heads * 64; i += 32) o[i] = make_uint4(0, 0, 0, 0);
        for (int h = lane; h < heads; h += 32) a.lse[(int64_t)b * a.H + head0 + h] = -INFINITY;
      }
    } else if (warp == C::W_QK) {
      // ------------------------------------------------------------------
      // QK issuer: the chunks as they land
      // ------------------------------------------------------------------
      constexpr uint32_t IDESC = idesc_bf16_f32(128, HB, false, false);
      const uint32_t leader = elect_one();
      const uint64_t k_desc = sdesc_sw128(sbase + C::OFF_K, 16, 1024), q_desc = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);
      int nq = -1;
      uint32_t slot = 0, phase = 0;
      uint32_t cs = 0;   // (FP8 rows: the RoPE columns' slot; slot and phase are the units')
      bool ok = true;
#pragma unroll 1
      for (int it = 0; it < nt && ok; ++it) {
        const int r = it % NI;
        if (!doze(B_IDX_FULL + r, (it / NI) & 1)) break;
        const int flags = __shfl_sync(0xffffffffu, meta[r].y, 0);
        if (leader) mbar_arrive(&bars[B_IDX_EMPTY + r]);
        if (flags & F_FIRST) {
          ++nq;
          if (!poll(B_Q_FULL, nq & 1)) break;
        }
        const int sb = it & 1;
        if (!poll(B_S_EMPTY + sb, ((it >> 1) & 1) ^ 1)) break;
        if constexpr (F8) {
          if constexpr (NC == 9) {
            if (!poll(B_FULL, it & 1)) break;
            tc_fence_after();
            mma_x4_elected(leader, tmem + C::COL_S + sb * HB, k_desc + (uint64_t)(cs * (C::CHUNK_BYTES >> 4)),
                           q_desc + (uint64_t)(8 * (HB * 128) >> 4), 2u, 2u, IDESC, 0u);
            commit_elected(leader, &bars[B_EMPTY]);
            cs = (cs + 5) % C::NK;
          }
          // the units that P.V reads too, which it gives back
#pragma unroll 1
          for (int m = 0; m < 4; ++m) {
            if (!poll(B_FULL + 8 + slot, phase)) { ok = false; break; }
            if (leader) mbar_arrive(&bars[B_EMPTY + 1 + m]);   // (its codes are read)
            tc_fence_after();
            if (leader && m == 0) DSA_TRACE(a.tr, it, 3);
            if (leader && m == 3) DSA_TRACE(a.tr, it, 4);
            const uint64_t u = k_desc + (uint64_t)((C::OFF_V - C::OFF_K + slot * C::UNIT_BYTES) >> 4);
            const uint64_t qd = q_desc + (uint64_t)(2 * m * (HB * 128) >> 4);
            mma_x4_elected(leader, tmem + C::COL_S + sb * HB, u, qd, 2u, 2u, IDESC, (NC == 9 || m > 0) ? 1u : 0u);
            mma_x4_elected(leader, tmem + C::COL_S + sb * HB, u + (C::CHUNK_BYTES >> 4), qd + (uint64_t)(HB * 128 >> 4), 2u,
                           2u, IDESC, 1u);
            if (++slot == C::NV) { slot = 0; phase ^= 1; }
          }
        }
#pragma unroll 1
        for (int c = 0; c < (F8 ? 0 : NC); ++c) {
          if (!poll(B_FULL + slot, phase)) { ok = false; break; }
          tc_fence_after();
          if (leader && c == 0) DSA_TRACE(a.tr, it, 3);
          if (leader && c == NC - 1) DSA_TRACE(a.tr, it, 4);
          mma_x4_elected(leader, tmem + C::COL_S + sb * HB, k_desc + (uint64_t)(slot * (C::CHUNK_BYTES >> 4)),
                         q_desc + (uint64_t)(c * (HB * 128 >> 4)), 2u, 2u, IDESC, c > 0 ? 1u : 0u);
          commit_elected(leader, &bars[B_EMPTY + slot]);
          if (++slot == C::NK) { slot = 0; phase ^= 1; }
        }
        if (!ok) break;
        commit_elected(leader, &bars[B_S_FULL + sb]);
        if (flags & F_LAST) commit_elected(leader, &bars[B_Q_EMPTY]);
      }
      // every MMA issued above has completed
      commit_elected(leader, &bars[B_DRAIN + 0]);
      if (leader) mbar_wait_drain(&bars[B_DRAIN + 0], 0, err);
      __syncwarp();
    } else if (warp == C::W_PV) {
      // ------------------------------------------------------------------
      // PV issuer: the units in order
      // ------------------------------------------------------------------
      constexpr uint32_t IDESC = idesc_bf16_f32(128, HB, true, false);
      const uint32_t leader = elect_one();
      const uint64_t v_desc = sdesc_sw128(sbase + C::OFF_V, C::CHUNK_BYTES, 1024), p_desc = sdesc_sw128(sbase + C::OFF_P, 16, 1024);
      int seg = -1;
      uint32_t slot = 0, phase = 0;
      bool ok = true;
#pragma unroll 1
      for (int it = 0; it < nt && ok; ++it) {
        const int r = it % NI;
        if (!doze(B_IDX_FULL + r, (it / NI) & 1)) break;
        const int flags = __shfl_sync(0xffffffffu, meta[r].y, 0);
        if (leader) mbar_arrive(&bars[B_IDX_EMPTY + r]);
        if (flags & F_FIRST) ++seg;
        const int ob = C::NO == 2 ? seg & 1 : 0, turn = seg / C::NO;   // O buffer and its use
        if (!poll(B_P_FULL, it & 1)) break;
        if (leader) DSA_TRACE(a.tr, it, 0);
        if ((flags & F_FIRST) && !poll(B_O_EMPTY + ob, (turn & 1) ^ 1)) break;
        const uint32_t acc = (flags & F_FIRST) ? 0u : 1u;
#pragma unroll 1
        for (int m = 0; m < 4; ++m) {
          if (!poll(B_FULL + 8 + slot, phase)) { ok = false; break; }
          tc_fence_after();
          const uint64_t v = v_desc + (uint64_t)(slot * (C::UNIT_BYTES >> 4));
          const uint32_t d_o = tmem + ob * (4 * HB) + m * HB;
          // 16 keys (2048 bytes of V^T) per MMA; P^T one 64-key swizzle column per half
          mma_x4_elected(leader, d_o, v, p_desc, 128u, 2u, IDESC, acc);
          mma_x4_elected(leader, d_o, v + 512u, p_desc + (uint64_t)(HB * 128 >> 4), 128u, 2u, IDESC, 1u);
          commit_elected(leader, &bars[B_EMPTY + 8 + slot]);
          if (++slot == C::NV) { slot = 0; phase ^= 1; }
        }
        if (!ok) break;
        if (leader) DSA_TRACE(a.tr, it, 7);
        commit_elected(leader, &bars[B_P_EMPTY]);
        if (flags & F_LAST) commit_elected(leader, &bars[B_O_FULL + ob]);
      }
      commit_elected(leader, &bars[B_DRAIN + 1]);
      if (leader) mbar_wait_drain(&bars[B_DRAIN + 1], 0, err);
      __syncwarp();
    }
  } else {
    regs_inc<C::REGS_SOFTMAX>();
    // --------------------------------------------------------------------
    // softmax and epilogue: thread = key (TMEM lane), warpgroup wg = heads
    // wg*HT .. wg*HT + HT - 1
    // --------------------------------------------------------------------
    const int wg = warp >> 2, w4 = warp & 3;
    const int key = threadIdx.x & 127;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    const uint32_t t_lane = tmem + ((uint32_t)(w4 * 32) << 16) + wg * HT;   // this thread's lane, its heads' columns
    uint8_t* p_key = smem + C::OFF_P + (key >> 6) * (HB * 128) + wg * HT * 128 + (key & 7) * 2;
    uint32_t sync_phase = 0;
    auto group = [&]() {   // the warpgroup's barrier
      mbar_arrive(&bars[B_SMX + wg]);
      const bool ok = poll(B_SMX + wg, sync_phase);
      sync_phase ^= 1u;
      return ok;
    };
    int seg = -1;
    // The running max starts at the lowest finite value, not at -inf, so that no
    // difference of two of them is NaN: a rescale from it gives exactly 0.
    float m_run[HT], l_exact[HT], l_used[HT];
#pragma unroll
    for (int h = 0; h < HT; ++h) { m_run[h] = -FLT_MAX; l_exact[h] = 0.f; l_used[h] = 0.f; }
    wait_for_previous();
    const int nt = poll(B_PLAN, 0) ? *plan : 0;
#pragma unroll 1
    for (int it = 0; it < nt; ++it) {
      const int r = it & (NI - 1);
      const int sb = it & 1;
      if (!poll(B_IDX_FULL + r, (it / NI) & 1)) break;
      const bool valid = rows[r * BK + key] >= 0;
      const int4 mt = meta[r];
      // tree form: the query rows of this thread that see its key, as bits (a drafted
      // token's row i sees drafted key j by bit j of its token's mask word)
      uint32_t sees = valid ? 0xffffffffu : 0u;
      if constexpr (TREE) {
        const int bit = mt.z + key;
        if (valid && bit >= 0) {
          sees = 0u;
          int token = (head0 + wg * HT) / a.heads, left_of = (token + 1) * a.heads - (head0 + wg * HT);
          const uint64_t* word = a.tree_mask + (int64_t)mt.x * a.n;
#pragma unroll 1
          for (int h = 0; h < HT && token < mt.w;) {
            const int upto = min(HT, h + left_of);   // the token's rows
            if (word[token] >> bit & 1) sees |= (0xffffffffu >> (32 - (upto - h))) << h;
            h = upto;
            left_of = a.heads;
            ++token;
          }
        }
      }
      auto on = [&](int h) { return TREE ? (sees >> h & 1u) != 0 : valid; };
      if (!poll(B_S_FULL + sb, (it >> 1) & 1)) break;
      if (threadIdx.x == 0) DSA_TRACE(a.tr, it, 5);
      if (mt.y & F_FIRST) {
        ++seg;
#pragma unroll
        for (int h = 0; h < HT; ++h) { m_run[h] = -FLT_MAX; l_exact[h] = 0.f; l_used[h] = 0.f; }
      }
      const int ob = C::NO == 2 ? seg & 1 : 0;
      tc_fence_after();
      const uint32_t t_s = t_lane + C::COL_S + sb * HB;
      float d[HT];   // scores less the running max, base 2
      tmem_ld_n<HT>(t_s, d);
      tmem_ld_wait();
      float top = -FLT_MAX;
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        d[h] = d[h] * scale_log2 - m_run[h];
        if (!TREE || on(h)) top = fmaxf(top, d[h]);
      }
      // Lazy rescale: a warp with a score above the running max by more than
      // kTau publishes its per-head max; the new reference is the max over
      // those warps, which bounds every score of the tile to within 2^kTau.
      // (One that does not ask publishes the lowest value.)
      // (A masked key's row is zeros, its score 0: it never asks.)
      const bool wneed = __any_sync(0xffffffffu, valid && top > kTau);
      float* redb = red + (sb * C::SWG + wg) * (4 * HT);
      volatile uint32_t* vote = votes + (sb * C::SWG + wg) * 4;
      float wmax = -FLT_MAX;
      if (wneed) {
        float x[HT];
        tmem_ld_n<HT>(t_s, x);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < HT; ++h) x[h] = on(h) ? x[h] * scale_log2 : -FLT_MAX;
        wmax = warp_transpose_reduce<HT, true>(x);
      }
      if (lane < HT) redb[w4 * HT + lane] = wmax;
      if (lane == 0) vote[w4] = wneed ? 1u : 0u;
      if (!group()) break;
      if (key == 0) mbar_arrive(&bars[B_IDX_EMPTY + r]);   // (every thread of the warpgroup has read the tile's rows)
      const uint32_t need = vote[0] | vote[1] | vote[2] | vote[3];
      if (need) {
        float alpha[HT];
#pragma unroll
        for (int h = 0; h < HT; h += 4) {
          float mn[4] = {m_run[h], m_run[h + 1], m_run[h + 2], m_run[h + 3]};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(redb + w * HT + h);
            mn[0] = fmaxf(mn[0], x.x);
            mn[1] = fmaxf(mn[1], x.y);
            mn[2] = fmaxf(mn[2], x.z);
            mn[3] = fmaxf(mn[3], x.w);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            alpha[h + i] = exp2f(m_run[h + i] - mn[i]);
            m_run[h + i] = mn[i];
            l_exact[h + i] *= alpha[h + i];
            l_used[h + i] *= alpha[h + i];
          }
        }
        if (!(mt.y & F_FIRST)) {
          // O in tensor memory, once the previous P.V is done with it
          if (!poll(B_P_EMPTY, sb ^ 1)) break;
          tc_fence_after();
#pragma unroll 1
          for (int m = 0; m < 4; ++m) {
            float o[HT];
            const uint32_t ta = t_lane + ob * (4 * HB) + m * HB;
            tmem_ld_n<HT>(ta, o);
            tmem_ld_wait();
#pragma unroll
            for (int h = 0; h < HT; ++h) o[h] *= alpha[h];
            tmem_st_n<HT>(ta, o);
          }
          tmem_st_wait();
        }
        // (read again rather than kept: the registers are the softmax warps' limit)
        tmem_ld_n<HT>(t_s, d);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < HT; ++h) d[h] = d[h] * scale_log2 - m_run[h];
      }
      tc_fence_before();
      mbar_arrive(&bars[B_S_EMPTY + sb]);
      uint32_t pk[HT / 2];
#pragma unroll
      for (int h = 0; h < HT; h += 2) {
        const float p0 = on(h) ? exp2f(d[h]) : 0.f, p1 = on(h + 1) ? exp2f(d[h + 1]) : 0.f;
        const uint32_t w = pack_bf16x2(p0, p1);
        l_exact[h] += p0;
        l_exact[h + 1] += p1;
        l_used[h] += __uint_as_float(w << 16);
        l_used[h + 1] += __uint_as_float(w & 0xffff0000u);
        pk[h / 2] = w;
      }
      // the previous P.V must be done before P is overwritten
      if (!poll(B_P_EMPTY, sb ^ 1)) break;
      // P^T[h][key], K-major swizzled, two columns of 64 keys: row h at h * 128,
      // 16-byte piece c at (c ^ (h & 7)) * 16
#pragma unroll
      for (int h = 0; h < HT; ++h)
        *reinterpret_cast<uint16_t*>(p_key + h * 128 + ((((key & 63) >> 3) ^ (h & 7)) << 4)) =
            (uint16_t)((h & 1) ? (pk[h / 2] >> 16) : (pk[h / 2] & 0xffffu));
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&bars[B_P_FULL]);
      if (threadIdx.x == 0) DSA_TRACE(a.tr, it, 6);
      if (!(mt.y & F_LAST)) continue;

      // ---- epilogue of the request's part in this range: the warps' sums, then
      // a lane per head for what the outputs are divided by and the log-sum-exp
      // (in the reduction scratch of the other parity: its last readers passed
      // the barrier above)
      const float ex = warp_transpose_reduce<HT, false>(l_exact);
      const float us = warp_transpose_reduce<HT, false>(l_used);
      float* redx = red + ((sb ^ 1) * C::SWG + wg) * (4 * HT);
      float* redu = redx + C::RED_FLOATS;
      float* redi = red + 2 * C::RED_FLOATS + wg * HT;
      // the running max is the same in every thread: lane h keeps head h's
      float mine = 0.f;
#pragma unroll
      for (int h = 0; h < HT; ++h) mine = lane == h ? m_run[h] : mine;
      if (lane < HT) {
        redx[w4 * HT + lane] = ex;
        redu[w4 * HT + lane] = us;
      }
      if (!group()) break;
      const bool part = (mt.y & F_PART) != 0;
      const uint32_t row0 = (uint32_t)(2 * range + ((mt.y & F_SLOT1) ? 1 : 0)) * (uint32_t)heads_padded + head0;   // of the parts
      const int left = heads - wg * HT;                                         // heads to store
      if (lane < HT) {
        float lx = (redx[lane] + redx[HT + lane]) + (redx[2 * HT + lane] + redx[3 * HT + lane]);
        float lu = (redu[lane] + redu[HT + lane]) + (redu[2 * HT + lane] + redu[3 * HT + lane]);
        if (TREE && head0 + wg * HT + lane >= mt.w * a.heads) lx = lu = 0.f;   // (a padding token's row)
        if (w4 == 0) {
          redi[lane] = (lu != 0.f) ? 1.0f / lu : 0.f;
          if (lane < left) {
            const float l2 = (lx != 0.f) ? mine + log2f(lx) : -INFINITY;
            if (part)
              a.part_lse[row0 + wg * HT + lane] = l2;
            else
              a.lse[(int64_t)mt.x * a.H + head0 + wg * HT + lane] = l2 * 0.6931471805599453f;
          }
        }
      }
      // (the next tile's vote and reduction use that scratch again)
      if (!group()) break;
      if (!poll(B_O_FULL + ob, (seg / C::NO) & 1)) break;
      tc_fence_after();
      float inv[HT];
#pragma unroll
      for (int h = 0; h < HT; h += 4) {
        const float4 x = *reinterpret_cast<const float4*>(redi + h);
        inv[h] = x.x;
        inv[h + 1] = x.y;
        inv[h + 2] = x.z;
        inv[h + 3] = x.w;
      }
      uint16_t* out = a.out + ((int64_t)mt.x * a.H + head0 + wg * HT) * 512 + key;
      float* po = a.part_o + (int64_t)(row0 + wg * HT) * 512 + key;
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        float o[HT];
        tmem_ld_n<HT>(t_lane + ob * (4 * HB) + m * HB, o);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          const float v = TREE && inv[h] == 0.f ? 0.f : o[h] * inv[h];
          if (h < left) {
            if (part)
              po[h * 512] = v;
            else
              out[h * 512] = f32_to_bf16_rn(v);
          }
        }
        po += 128;
        out += 128;
      }
      tc_fence_before();
      mbar_arrive(&bars[B_O_EMPTY + ob]);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) tmem_dealloc(tmem, C::TMEM_COLS);
}

template <int HB, int NC, bool F8, bool TREE>
static int launch_t(const DecodeArgs& a, cudaStream_t stream) {
  using C = Cfg<HB, NC, F8>;
  static PerDevice done;
  if (allow_smem(reinterpret_cast<const void*>(decode_kernel<HB, NC, F8, TREE>), C::SMEM_BYTES, done) != 0) return -1;
  // (programmatic: the start, up to griddepcontrol.wait, overlaps the end of the kernel before)
  return launch_after(decode_kernel<HB, NC, F8, TREE>, dim3((unsigned)(a.groups * a.head_blocks)), C::NTHREADS, C::SMEM_BYTES, stream,
                      a);
}

// The join of what range borders cut; padded: rows of a part.
static inline int launch_join(const DecodeArgs& a, int padded, int max_tiles, bool tree, cudaStream_t stream) {
  if (max_tiles <= 1 || a.groups <= 1) return 0;   // no request can be cut
  if (tree) {
    // About a row for each warp, or CTA (see the kernel), where the batch's requests are cut equally
    // often, which is all that the host knows of their lengths; the kernel goes by each request's own
    // parts.  Two against five parts of a row at a time, whole calls in us: 1 x 131072 at 256 rows
    // 65.6 : 63.0, 4 x 30000 at 128 rows 49.8 : 48.6 (more than eight cuts: five); 8 x 4096..32768
    // at 512 rows 96.3 : 97.7, 32 x 512..16384 at 128 rows 58.7 : 58.4 (fewer: two).  A batch whose
    // average misleads loses a little: one request of 131072 among 31 of 500 at 128 rows 60.9 :
    // 58.0, at 512 rows 122.9 : 124.8, 10 x 5000 at 128 rows 34.4 : 33.2.
    const int64_t cuts = (a.groups + a.B - 1) / a.B, y = a.H / (cuts > 8 ? cuts : 4 * cuts) + 1;
    const dim3 grid((unsigned)(a.groups - 1), (unsigned)y);
    return cuts > 8 ? launch_after(tree_join_kernel<5>, grid, NT_JOIN, 0, stream, a, padded)
                    : launch_after(tree_join_kernel<2>, grid, NT_JOIN, 0, stream, a, padded);
  }
  const dim3 grid((unsigned)(a.groups - 1), (unsigned)(JOIN_Y * a.head_blocks));
  return a.groups > 20 * a.B ? launch_after(join_kernel<10>, grid, NT_JOIN, 0, stream, a, padded)
                             : launch_after(join_kernel<5>, grid, NT_JOIN, 0, stream, a, padded);
}

template <bool TREE>
static int launch_decode(DecodeArgs& a, bool fp8, int d_rope, int max_tiles, cudaStream_t stream) {
  const int hb = decode_heads_per_cta(a.H, fp8);
  int r = -2;
  if (hb == 64) {
    // (so many rows of a tree go to CTA pairs)
    if constexpr (!TREE) r = d_rope ? launch_t<64, 9, false, false>(a, stream) : launch_t<64, 8, false, false>(a, stream);
  } else if (hb == 16) {
    if (fp8) r = d_rope ? launch_t<16, 9, true, TREE>(a, stream) : launch_t<16, 8, true, TREE>(a, stream);
    else r = d_rope ? launch_t<16, 9, false, TREE>(a, stream) : launch_t<16, 8, false, TREE>(a, stream);
  } else {
    if (fp8) r = d_rope ? launch_t<32, 9, true, TREE>(a, stream) : launch_t<32, 8, true, TREE>(a, stream);
    else r = d_rope ? launch_t<32, 9, false, TREE>(a, stream) : launch_t<32, 8, false, TREE>(a, stream);
  }
  if (r != 0) return r;
  return launch_join(a, a.head_blocks * hb, max_tiles, TREE, stream);
}

}  // namespace decode
}  // namespace dsa
