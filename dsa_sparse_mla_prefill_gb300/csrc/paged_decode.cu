// Attention of one new token per request over a paged latent KV cache.
//
//     s_hj = scale * q[b,h,:] . c_j          c_j: latent row of position j
//     out[b,h,:] = sum_j softmax_j(s_h) c_j[0:512],   lse[b,h] = ln sum_j exp(s_hj)
// over the positions j < kv_len[b], or over the token's own top-k positions;
// position j lies in row table[b][j / block_size] * block_size + j % block_size.
//
// Bound: every row is read once for all heads of the request (1152 bytes, or
// 656 in FP8, against 2 * 1088 * H flops), so up to 32 heads HBM is the bound;
// at 128 heads the flops come within 15 % of it.
//
// Split over the length: the keys of all requests, in tiles of 128, form one
// line of W tiles, dealt to the CTA groups in equal contiguous ranges
// ([g W / G, (g+1) W / G)), so one long context and a ragged batch alike keep
// every SM busy to within one tile, from the lengths the GPU holds (nothing is
// planned on the host, and a captured graph follows them).  A range ends some
// requests and begins another: a request that lies whole in a range is stored
// at once, the parts of one cut by a range border are stored as normalised fp32
// outputs with their log-sum-exp and joined by a second small kernel, which is
// launched so that its start overlaps the first one's end.  A group is one CTA
// per 32 heads (16 when there are no more), all walking the same rows at the
// same time, so the rows are read from HBM once and from L2 by the others.
//
// One CTA, 24 warps:
//   warps 0-7   softmax: thread = key (TMEM lane), warpgroup = half of the heads;
//               online in base 2 with the lazy rescale (only when a head's
//               running max grows by more than 2^8); P to shared memory in
//               bf16; the epilogue (O^T lane = output column).
//   warp 8      QK issuer: S^T = K q^T, keys on the M side (M = 128, N = heads)
//   warps 9,10  PV issuers: O^T += V^T P^T, alternate 128-column units
//   warp 11     scheduler: walks the range, turns 128 positions per tile into
//               rows (a ring of four tiles ahead), loads q per request
//   warps 12-21 TMA row gathers, two warps per unit slot
//   warp 22     the same for the RoPE columns; warp 23: requests without keys
// Every key row is gathered once: a tile of 128 keys is four 128-column units
// (32 KB, in a ring of five) and one RoPE chunk; QK reads a unit K-major, P.V
// reads the same bytes MN-major, and the unit goes back to the producers when
// its P.V is done.  Rows that are masked (behind kv_len, -1, unmapped pages) are
// gathered from outside the tensor map, which reads as zeros: whatever the
// cache holds there, NaN included, never reaches the sums.
//
// Rounding: P is rounded to bf16 for the tensor core.  The outputs are divided
// by the sum of the rounded weights (so that the weights used add up to one);
// the log-sum-exp comes from the unrounded sum, both in fp32.
#include "dsa_device.cuh"
#include "dsa_kernels.h"

namespace dsa {
namespace decode {

constexpr int BK = 128;          // keys per tile (the MMA's M)
constexpr int NTHREADS = 768;
constexpr int NI = 4;            // tiles of rows ahead
constexpr int NU = 5;            // 128-column unit slots
constexpr float kTau = 8.0f;     // lazy-rescale threshold (log2 units)
// 768 threads launched at 80 registers: 256 * 144 + 512 * 48 = 768 * 80
constexpr int REGS_SOFTMAX = 144;
constexpr int REGS_REST = 48;

template <int HB, int NC>
struct Cfg {
  static constexpr int HT = HB / 2;                      // heads per softmax thread
  static constexpr int NQ = HB == 16 ? 2 : 1;            // q buffers (what shared memory leaves)
  static constexpr uint32_t CHUNK_BYTES = BK * 128u;     // 128 keys x 64 columns
  static constexpr uint32_t UNIT_BYTES = 2u * CHUNK_BYTES;
  static constexpr uint32_t Q_BYTES = NC * HB * 128u;
  static constexpr uint32_t P_BYTES = 2u * HB * 128u;
  static constexpr uint32_t RED_FLOATS = 2u * 2u * 4u * HT;   // [parity][warpgroup][warp][head]
  static constexpr uint32_t OFF_U = 0;
  static constexpr uint32_t OFF_R = NU * UNIT_BYTES;
  static constexpr uint32_t OFF_Q = OFF_R + (NC == 9 ? CHUNK_BYTES : 0u);
  static constexpr uint32_t OFF_P = OFF_Q + NQ * Q_BYTES;
  static constexpr uint32_t OFF_ROWS = OFF_P + P_BYTES;
  static constexpr uint32_t OFF_META = OFF_ROWS + NI * BK * 4u;
  static constexpr uint32_t OFF_RED = OFF_META + NI * 16u;
  static constexpr uint32_t OFF_BAR = OFF_RED + 2u * RED_FLOATS * 4u;   // two sums in the epilogue
  static constexpr int NBAR = 48;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8u;
  static constexpr uint32_t MISC_BYTES = 64u + 2u * 2u * 4u * 4u + 24u * 8u;
  static constexpr uint32_t SMEM_BYTES = OFF_MISC + MISC_BYTES + 1024u;
  static_assert(SMEM_BYTES <= 227u * 1024u, "shared memory budget");
  // TMEM columns: O^T double buffer (2 x 4 HB), S^T double buffer (2 x HB)
  static constexpr uint32_t COL_S = 8u * HB;
  static constexpr uint32_t TMEM_COLS = (10u * HB <= 256u) ? 256u : 512u;
};

enum {
  B_IDX_FULL = 0,    // [NI]
  B_IDX_EMPTY = 4,   // [NI]
  B_Q_FULL = 8,      // [2]
  B_Q_EMPTY = 10,    // [2]
  B_S_FULL = 12,     // [2]
  B_S_EMPTY = 14,    // [2]
  B_P_FULL = 16,
  B_P_EMPTY = 17,
  B_O_FULL = 18,     // [2]
  B_O_EMPTY = 20,    // [2]
  B_SMX = 22,        // [2] one per softmax warpgroup
  B_DRAIN = 24,      // [3]
  B_U_FULL = 28,     // [NU]
  B_U_EMPTY = 34,    // [NU]
  B_R_FULL = 40,
  B_R_EMPTY = 41,
};

// flags of a tile
constexpr int F_FIRST = 1;    // first tile of its request in this range
constexpr int F_LAST = 2;     // last one
constexpr int F_PART = 4;     // the request is cut: store a partial result
constexpr int F_SLOT1 = 8;    // ... into the range's second slot (it did not begin the range)

// key tiles of a request
__device__ __forceinline__ int tiles_of(const DecodeArgs& a, int len) {
  if (len <= 0) return 0;
  if (a.idx != nullptr) return (a.k + BK - 1) / BK;
  const int64_t cap = (int64_t)a.max_blocks * a.block_size;
  const uint32_t n = len < cap ? (uint32_t)len : (uint32_t)cap;
  return (int)((n + BK - 1) / BK);
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

template <int HB, int NC>
__global__ void __launch_bounds__(NTHREADS, 1) decode_kernel(const __grid_constant__ DecodeArgs a) {
  using C = Cfg<HB, NC>;
  constexpr int HT = C::HT;
  constexpr bool ROPE = (NC == 9);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_u32 + 1023u) & ~1023u) - raw_u32);
  const uint32_t sbase = smem_u32(smem);

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile uint32_t* tmem_base_ptr = misc + 0;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  int* sched = reinterpret_cast<int*>(misc + 2);                    // first request, its first tile here
  volatile uint32_t* votes = misc + 16;                             // [parity][warpgroup][warp]
  int64_t* scan = reinterpret_cast<int64_t*>(misc + 32);            // [24] per-warp tile counts
  int32_t* rows = reinterpret_cast<int32_t*>(smem + C::OFF_ROWS);   // [NI][BK], -1 = masked
  int4* meta = reinterpret_cast<int4*>(smem + C::OFF_META);         // [NI] request, flags
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
  unsigned int* err = a.err;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int group = blockIdx.x / a.head_blocks;
  const int hb = blockIdx.x - group * a.head_blocks;

  // the joining kernel may be put on the GPU as soon as there is room
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < NI; ++i) {
      mbar_init(&bars[B_IDX_FULL + i], 1);
      // 3 MMA warps, 2 softmax warpgroups, the unit producers, the RoPE producer
      mbar_init(&bars[B_IDX_EMPTY + i], 3 + 2 + 2 * NU + (ROPE ? 1 : 0));
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[B_Q_FULL + i], 1);
      mbar_init(&bars[B_Q_EMPTY + i], 1);
      mbar_init(&bars[B_S_FULL + i], 1);
      mbar_init(&bars[B_S_EMPTY + i], 256);
      mbar_init(&bars[B_O_FULL + i], 2);    // one commit per PV issuer
      mbar_init(&bars[B_O_EMPTY + i], 256);
      mbar_init(&bars[B_SMX + i], 128);
    }
    mbar_init(&bars[B_P_FULL], 256);
    mbar_init(&bars[B_P_EMPTY], 2);
    for (int i = 0; i < 3; ++i) mbar_init(&bars[B_DRAIN + i], 1);
    for (int i = 0; i < NU; ++i) {
      mbar_init(&bars[B_U_FULL + i], 1);
      mbar_init(&bars[B_U_EMPTY + i], 1);
    }
    mbar_init(&bars[B_R_FULL], 1);
    mbar_init(&bars[B_R_EMPTY], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc(const_cast<uint32_t*>(tmem_base_ptr), C::TMEM_COLS);
    tmem_relinquish();
  }
  // ---- this group's range of tiles: every thread counts the tiles of a run of
  // requests, a block scan places the runs, and the run that holds the range's
  // first tile names it
  const int per = (a.B + NTHREADS - 1) / NTHREADS;
  const int b_lo = min(a.B, (int)threadIdx.x * per), b_hi = min(a.B, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += tiles_of(a, __ldg(a.kv_lens + b));
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) scan[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t before = incl - mine, total = 0;
  for (int w = 0; w < NTHREADS / 32; ++w) {
    const int64_t n = scan[w];
    if (w < warp) before += n;
    total += n;
  }
  const int64_t ng = total < a.groups ? total : a.groups;   // no group without a tile
  const int64_t x0 = group < ng ? group * total / ng : 0;
  const int64_t x1 = group < ng ? (group + 1) * total / ng : 0;
  const int nt = (int)(x1 - x0);
  if (nt > 0 && before <= x0 && x0 < before + mine) {
    int64_t at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const int n = tiles_of(a, __ldg(a.kv_lens + b));
      if (x0 < at + n) {
        sched[0] = b;
        sched[1] = (int)(x0 - at);
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  const uint32_t tmem = *tmem_base_ptr;
  const int head0 = hb * HB;                                   // this CTA's first head
  const int heads = a.H - head0 < HB ? a.H - head0 : HB;       // the others are padding, never stored
  const int64_t heads_padded = (int64_t)a.head_blocks * HB;

  if (warp >= 8) {
    regs_dec<REGS_REST>();
    if (warp == 11) {
      // ------------------------------------------------------------------
      // scheduler
      // ------------------------------------------------------------------
      bool ok = true;
      int bad = 0;
      int b = nt > 0 ? sched[0] : 0, j = nt > 0 ? sched[1] : 0;
      int len = 0, n = 0;
      bool enter = true;              // the next tile is the first of request b here
      int seg = 0;                    // requests begun
      int nq = 0;                     // q loads issued
      const int64_t cap = (int64_t)a.max_blocks * a.block_size;
      for (int it = 0; it < nt; ++it) {
        const int r = it % NI;
        if (enter) {
          // (requests without keys have no tile)
          while (true) {
            len = __ldg(a.kv_lens + b);
            n = tiles_of(a, len);
            if (n > 0) break;
            ++b;
          }
          if (len > cap) {
            if (j == 0 && lane == 0) ++bad;
            len = (int)cap;
          }
        }
        if (!mbar_wait_warp(&bars[B_IDX_EMPTY + r], ((it / NI) & 1) ^ 1, abort_flag, err)) { ok = false; break; }
        const int32_t* bt = a.block_table + (int64_t)b * a.max_blocks;
        int32_t row[4];
        int32_t pos[4];
        const int e0 = j * BK + 4 * lane;   // (as unsigned: the last tile may end past 2^31)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (a.idx != nullptr) {
            pos[e] = (e0 + e < a.k) ? __ldg(a.idx + (int64_t)b * a.ld + e0 + e) : -1;
            if (pos[e] < -1 || pos[e] >= len) {
              ++bad;
              pos[e] = -1;
            }
          } else {
            const uint32_t p = (uint32_t)e0 + e;
            pos[e] = p < (uint32_t)len ? (int32_t)p : -1;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          row[e] = -1;
          if (pos[e] >= 0) {
            const int32_t page = pos[e] / a.block_size;
            const int32_t blk = __ldg(bt + page);
            const int64_t x = (int64_t)blk * a.block_size + (pos[e] - page * a.block_size);
            if (blk < 0 || x >= a.N)
              ++bad;
            else
              row[e] = (int32_t)x;
          }
        }
        *reinterpret_cast<int4*>(rows + r * BK + 4 * lane) = make_int4(row[0], row[1], row[2], row[3]);
        const bool first = enter;
        const bool last = (it == nt - 1) || (j == n - 1);
        if (lane == 0) {
          int flags = (first ? F_FIRST : 0) | (last ? F_LAST : 0);
          if (last) {
            // (the range's first request may have begun before it, its last may go on behind it)
            const bool whole = (seg > 0 || sched[1] == 0) && j == n - 1;
            if (!whole) flags |= F_PART | (seg > 0 ? F_SLOT1 : 0);
          }
          meta[r] = make_int4(b, flags, 0, 0);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_IDX_FULL + r]);
        if (first) {
          // q of request b: rows b*H + head0 ... of q viewed [B*H, D_QK], one box per swizzle column
          const int qb = nq % C::NQ;
          if (!mbar_wait_warp(&bars[B_Q_EMPTY + qb], ((nq / C::NQ) & 1) ^ 1, abort_flag, err)) { ok = false; break; }
          if (lane == 0) {
            mbar_arrive_expect_tx(&bars[B_Q_FULL + qb], C::Q_BYTES);
            for (int c = 0; c < NC; ++c)
              tma_load_2d(sbase + C::OFF_Q + qb * C::Q_BYTES + c * (HB * 128), &a.tmap_q, c * 64, b * a.H + head0,
                          &bars[B_Q_FULL + qb]);
          }
          ++nq;
        }
        enter = (j == n - 1);
        if (enter) {
          ++b;
          j = 0;
          ++seg;
        } else {
          ++j;
        }
      }
      (void)ok;
      bad = __reduce_add_sync(0xffffffffu, bad);
      if (lane == 0) {
        if (bad && hb == 0) atomicAdd(err + ERR_BAD_INDEX, (unsigned)bad);
        // let q copies in flight land before the CTA can exit
        for (int p = nq - 1; p >= 0 && p > nq - 1 - C::NQ; --p)
          mbar_wait_drain(&bars[B_Q_FULL + p % C::NQ], (uint32_t)(p / C::NQ) & 1, err);
      }
      __syncwarp();
    } else if (warp >= 12 && warp < 12 + 2 * NU) {
      // ------------------------------------------------------------------
      // unit producers: warps 12 + 2s and 13 + 2s fill unit slot s, one
      // 64-column chunk of it each (lane l: rows 4l .. 4l+3)
      // ------------------------------------------------------------------
      const int slot = (warp - 12) >> 1, hf = (warp - 12) & 1;
      const uint32_t dst = sbase + C::OFF_U + slot * C::UNIT_BYTES + hf * C::CHUNK_BYTES + lane * 512;
      int64_t armed = -1;
      bool ok = true;
      for (int it = 0; it < nt && ok; ++it) {
        const int r = it % NI;
        if (!mbar_wait_warp(&bars[B_IDX_FULL + r], (it / NI) & 1, abort_flag, err)) break;
        const int4 x = *reinterpret_cast<const int4*>(rows + r * BK + 4 * lane);
        for (int m = 0; m < 4; ++m) {
          const int64_t pos = 4ll * it + m;
          if ((int)(pos % NU) != slot) continue;
          if (!mbar_wait_warp(&bars[B_U_EMPTY + slot], ((uint32_t)(pos / NU) & 1) ^ 1, abort_flag, err)) {
            ok = false;
            break;
          }
          if (lane == 0 && hf == 0) mbar_arrive_expect_tx(&bars[B_U_FULL + slot], C::UNIT_BYTES);
          tma_gather4(dst, &a.tmap_kv, (2 * m + hf) * 64, x.x, x.y, x.z, x.w, &bars[B_U_FULL + slot]);
          armed = pos;
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&bars[B_IDX_EMPTY + r]);
      }
      // let copies in flight land before the CTA can exit
      if (lane == 0 && hf == 0 && armed >= 0)
        mbar_wait_drain(&bars[B_U_FULL + slot], (uint32_t)(armed / NU) & 1, err);
      __syncwarp();
    } else if (warp == 22) {
      if constexpr (ROPE) {
        int armed = -1;
        for (int it = 0; it < nt; ++it) {
          const int r = it % NI;
          if (!mbar_wait_warp(&bars[B_IDX_FULL + r], (it / NI) & 1, abort_flag, err)) break;
          const int4 x = *reinterpret_cast<const int4*>(rows + r * BK + 4 * lane);
          if (!mbar_wait_warp(&bars[B_R_EMPTY], (it & 1) ^ 1, abort_flag, err)) break;
          if (lane == 0) mbar_arrive_expect_tx(&bars[B_R_FULL], C::CHUNK_BYTES);
          __syncwarp();
          tma_gather4(sbase + C::OFF_R + lane * 512, &a.tmap_kv, 512, x.x, x.y, x.z, x.w, &bars[B_R_FULL]);
          armed = it;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_IDX_EMPTY + r]);
        }
        if (lane == 0 && armed >= 0) mbar_wait_drain(&bars[B_R_FULL], armed & 1, err);
        __syncwarp();
      }
    } else if (warp == 23) {
      // requests without keys: out = 0, lse = -inf (dealt over the groups)
      for (int b = group; b < a.B; b += a.groups) {
        if (tiles_of(a, __ldg(a.kv_lens + b)) > 0) continue;
        uint4* o = reinterpret_cast<uint4*>(a.out + ((int64_t)b * a.H + head0) * 512);
        for (int i = lane; i < heads * 64; i += 32) o[i] = make_uint4(0, 0, 0, 0);
        for (int h = lane; h < heads; h += 32) a.lse[(int64_t)b * a.H + head0 + h] = -INFINITY;
      }
    } else if (warp == 8) {
      // ------------------------------------------------------------------
      // QK issuer (one thread): the RoPE chunk, then the units as they land
      // ------------------------------------------------------------------
      if (lane == 0) {
        constexpr uint32_t IDESC = idesc_bf16_f32(128, HB, false, false);
        int nq = -1;
        uint32_t qs = 0;
        bool ok = true;
        for (int it = 0; it < nt && ok; ++it) {
          const int r = it % NI;
          if (!mbar_wait(&bars[B_IDX_FULL + r], (it / NI) & 1, abort_flag, err)) break;
          const int flags = meta[r].y;
          mbar_arrive(&bars[B_IDX_EMPTY + r]);
          if (flags & F_FIRST) {
            ++nq;
            const int qb = nq % C::NQ;
            if (!mbar_wait(&bars[B_Q_FULL + qb], (nq / C::NQ) & 1, abort_flag, err)) break;
            qs = sbase + C::OFF_Q + qb * C::Q_BYTES;
          }
          const int sb = it & 1;
          const uint32_t d_s = tmem + C::COL_S + sb * HB;
          if (!mbar_wait(&bars[B_S_EMPTY + sb], ((it >> 1) & 1) ^ 1, abort_flag, err)) break;
          if constexpr (ROPE) {
            if (!mbar_wait(&bars[B_R_FULL], it & 1, abort_flag, err)) break;
            tc_fence_after();
            mma_bf16_ss_x4(d_s, sdesc_sw128(sbase + C::OFF_R, 16, 1024), sdesc_sw128(qs + 8 * (HB * 128), 16, 1024),
                           2u, 2u, IDESC, 0u);
            mma_commit(&bars[B_R_EMPTY]);
          }
          for (int m = 0; m < 4; ++m) {
            const uint32_t pos = 4u * it + m, slot = pos % NU;
            if (!mbar_wait(&bars[B_U_FULL + slot], (pos / NU) & 1, abort_flag, err)) { ok = false; break; }
            tc_fence_after();
            const uint32_t u = sbase + C::OFF_U + slot * C::UNIT_BYTES;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              mma_bf16_ss_x4(d_s, sdesc_sw128(u + hf * C::CHUNK_BYTES, 16, 1024),
                             sdesc_sw128(qs + (2 * m + hf) * (HB * 128), 16, 1024), 2u, 2u, IDESC,
                             (ROPE || m > 0 || hf > 0) ? 1u : 0u);
          }
          if (!ok) break;
          mma_commit(&bars[B_S_FULL + sb]);
          if (flags & F_LAST) mma_commit(&bars[B_Q_EMPTY + nq % C::NQ]);
        }
        // every MMA issued above has completed
        mma_commit(&bars[B_DRAIN + 0]);
        mbar_wait_drain(&bars[B_DRAIN + 0], 0, err);
      }
      __syncwarp();
    } else if (warp == 9 || warp == 10) {
      // ------------------------------------------------------------------
      // PV issuers (one thread each): units 0, 2 and 1, 3 of every tile
      // ------------------------------------------------------------------
      const int pvi = warp - 9;
      if (lane == 0) {
        constexpr uint32_t IDESC = idesc_bf16_f32(128, HB, true, false);
        const uint32_t p_s = sbase + C::OFF_P;
        int seg = -1;
        bool ok = true;
        for (int it = 0; it < nt && ok; ++it) {
          const int r = it % NI;
          if (!mbar_wait(&bars[B_IDX_FULL + r], (it / NI) & 1, abort_flag, err)) break;
          const int flags = meta[r].y;
          mbar_arrive(&bars[B_IDX_EMPTY + r]);
          if (flags & F_FIRST) ++seg;
          const int ob = seg & 1;
          if (!mbar_wait(&bars[B_P_FULL], it & 1, abort_flag, err)) break;
          if (flags & F_FIRST) {
            if (!mbar_wait(&bars[B_O_EMPTY + ob], ((seg >> 1) & 1) ^ 1, abort_flag, err)) break;
          }
          for (int m = pvi; m < 4; m += 2) {
            const uint32_t pos = 4u * it + m, slot = pos % NU;
            // (landed before QK read it; the wait orders this thread's MMAs after the copy)
            if (!mbar_wait(&bars[B_U_FULL + slot], (pos / NU) & 1, abort_flag, err)) { ok = false; break; }
            tc_fence_after();
            const uint32_t u = sbase + C::OFF_U + slot * C::UNIT_BYTES;
            const uint32_t d_o = tmem + ob * (4 * HB) + m * HB;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              mma_bf16_ss_x4(d_o, sdesc_sw128(u + hf * 4 * 2048, C::CHUNK_BYTES, 1024),
                             sdesc_sw128(p_s + hf * (HB * 128), 16, 1024), 128u, 2u, IDESC,
                             (!(flags & F_FIRST) || hf > 0) ? 1u : 0u);
            mma_commit(&bars[B_U_EMPTY + slot]);
          }
          if (!ok) break;
          mma_commit(&bars[B_P_EMPTY]);
          if (flags & F_LAST) mma_commit(&bars[B_O_FULL + ob]);
        }
        mma_commit(&bars[B_DRAIN + 1 + pvi]);
        mbar_wait_drain(&bars[B_DRAIN + 1 + pvi], 0, err);
      }
      __syncwarp();
    }
  } else {
    regs_inc<REGS_SOFTMAX>();
    // --------------------------------------------------------------------
    // softmax and epilogue: thread = key (TMEM lane), warpgroup wg = heads
    // wg*HT .. wg*HT + HT - 1
    // --------------------------------------------------------------------
    const int wg = warp >> 2, w4 = warp & 3;
    const int key = threadIdx.x & 127;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    const uint32_t lane_off = (uint32_t)(w4 * 32) << 16;
    uint8_t* p_tile = smem + C::OFF_P;
    uint64_t* sync_bar = &bars[B_SMX + wg];
    uint32_t sync_phase = 0;
    int seg = -1;
    float m_run[HT], l_exact[HT], l_used[HT];
    for (int it = 0; it < nt; ++it) {
      const int r = it % NI;
      if (!mbar_wait_warp(&bars[B_IDX_FULL + r], (it / NI) & 1, abort_flag, err)) break;
      const bool valid = rows[r * BK + key] >= 0;
      const int4 mt = meta[r];
      if (mt.y & F_FIRST) {
        ++seg;
#pragma unroll
        for (int h = 0; h < HT; ++h) { m_run[h] = -INFINITY; l_exact[h] = 0.f; l_used[h] = 0.f; }
      }
      const int ob = seg & 1, sb = it & 1;
      if (!mbar_wait_warp(&bars[B_S_FULL + sb], (it >> 1) & 1, abort_flag, err)) break;
      tc_fence_after();
      float s[HT];
      tmem_ld_n<HT>(tmem + lane_off + C::COL_S + sb * HB + wg * HT, s);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(&bars[B_S_EMPTY + sb]);
      bool mine_need = false;
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        s[h] = valid ? s[h] * scale_log2 : -INFINITY;
        mine_need |= (s[h] > m_run[h] + kTau);
      }
      // Lazy rescale: a warp with a score above the running max by more than
      // kTau publishes its per-head max; the new reference is the max over
      // those warps, which bounds every score of the tile to within 2^kTau.
      const bool wneed = __any_sync(0xffffffffu, mine_need);
      float* redb = red + ((it & 1) * 2 + wg) * (4 * HT);
      volatile uint32_t* vote = votes + ((it & 1) * 2 + wg) * 4;
      if (wneed) {
        float x[HT];
#pragma unroll
        for (int h = 0; h < HT; ++h) x[h] = s[h];
        const float wmax = warp_transpose_reduce<HT, true>(x);
        if (lane < HT) redb[w4 * HT + lane] = wmax;
      }
      if (lane == 0) vote[w4] = wneed ? 1u : 0u;
      if (!__all_sync(0xffffffffu, group_sync(sync_bar, sync_phase, abort_flag, err))) break;
      if (key == 0) mbar_arrive(&bars[B_IDX_EMPTY + r]);   // (every thread of the warpgroup has read the tile's rows)
      uint32_t vw[4];
      bool need = false;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        vw[w] = vote[w];
        need |= vw[w] != 0;
      }
      float alpha[HT];
      if (need) {
        float tmax[HT];
#pragma unroll
        for (int h = 0; h < HT; ++h) tmax[h] = m_run[h];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if (vw[w]) {
#pragma unroll
            for (int h = 0; h < HT; h += 4) {
              const float4 x = *reinterpret_cast<const float4*>(redb + w * HT + h);
              tmax[h + 0] = fmaxf(tmax[h + 0], x.x);
              tmax[h + 1] = fmaxf(tmax[h + 1], x.y);
              tmax[h + 2] = fmaxf(tmax[h + 2], x.z);
              tmax[h + 3] = fmaxf(tmax[h + 3], x.w);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          alpha[h] = (m_run[h] == -INFINITY) ? 0.f : exp2f(m_run[h] - tmax[h]);
          m_run[h] = tmax[h];
          l_exact[h] *= alpha[h];
          l_used[h] *= alpha[h];
        }
      }
      uint32_t pk[HT / 2];
#pragma unroll
      for (int h = 0; h < HT; h += 2) {
        const float m0 = (m_run[h] == -INFINITY) ? 0.f : m_run[h];
        const float m1 = (m_run[h + 1] == -INFINITY) ? 0.f : m_run[h + 1];
        const float p0 = exp2f(s[h] - m0), p1 = exp2f(s[h + 1] - m1);
        const uint32_t w = pack_bf16x2(p0, p1);
        l_exact[h] += p0;
        l_exact[h + 1] += p1;
        l_used[h] += __uint_as_float(w << 16);
        l_used[h + 1] += __uint_as_float(w & 0xffff0000u);
        pk[h / 2] = w;
      }
      // the previous P.V must be done before P is overwritten or O rescaled
      if (!mbar_wait_warp(&bars[B_P_EMPTY], (it & 1) ^ 1, abort_flag, err)) break;
      tc_fence_after();
      if (need && !(mt.y & F_FIRST)) {
#pragma unroll 1
        for (int m = 0; m < 4; ++m) {
          float o[HT];
          const uint32_t ta = tmem + lane_off + ob * (4 * HB) + m * HB + wg * HT;
          tmem_ld_n<HT>(ta, o);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < HT; ++h) o[h] *= alpha[h];
          tmem_st_n<HT>(ta, o);
        }
        tmem_st_wait();
      }
      {
        // P^T[h][key] (K-major swizzled, two columns of 64 keys)
        const uint32_t kcol = key & 63;
        uint8_t* pcol = p_tile + (key >> 6) * (HB * 128);
#pragma unroll
        for (int h = 0; h < HT; ++h)
          *reinterpret_cast<uint16_t*>(pcol + sw128_offset(wg * HT + h, kcol)) =
              (uint16_t)((h & 1) ? (pk[h / 2] >> 16) : (pk[h / 2] & 0xffffu));
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&bars[B_P_FULL]);
      if (!(mt.y & F_LAST)) continue;

      // ---- epilogue of the request's part in this range
      const float ex = warp_transpose_reduce<HT, false>(l_exact);
      const float us = warp_transpose_reduce<HT, false>(l_used);
      // (the reduction scratch of the other parity: its last readers passed the group sync above)
      float* redx = red + (((it + 1) & 1) * 2 + wg) * (4 * HT);
      float* redu = redx + C::RED_FLOATS;
      if (lane < HT) {
        redx[w4 * HT + lane] = ex;
        redu[w4 * HT + lane] = us;
      }
      if (!__all_sync(0xffffffffu, group_sync(sync_bar, sync_phase, abort_flag, err))) break;
      float inv[HT];
      const bool part = (mt.y & F_PART) != 0;
      const int64_t slot = 2ll * group + ((mt.y & F_SLOT1) ? 1 : 0);
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        const float lx = (redx[h] + redx[HT + h]) + (redx[2 * HT + h] + redx[3 * HT + h]);
        const float lu = (redu[h] + redu[HT + h]) + (redu[2 * HT + h] + redu[3 * HT + h]);
        inv[h] = (lu != 0.f) ? 1.0f / lu : 0.f;
        const int hh = wg * HT + h;
        if (key == h && hh < heads) {
          const float l2 = (lx != 0.f) ? m_run[h] + log2f(lx) : -INFINITY;
          if (part)
            a.part_lse[slot * heads_padded + head0 + hh] = l2;
          else
            a.lse[(int64_t)mt.x * a.H + head0 + hh] = l2 * 0.6931471805599453f;
        }
      }
      // (the next tile's vote and reduction use that scratch again)
      if (!__all_sync(0xffffffffu, group_sync(sync_bar, sync_phase, abort_flag, err))) break;
      if (!mbar_wait_warp(&bars[B_O_FULL + ob], (seg >> 1) & 1, abort_flag, err)) break;
      tc_fence_after();
      uint16_t* out = a.out + ((int64_t)mt.x * a.H + head0) * 512 + key;
      float* po = a.part_o + (slot * heads_padded + head0) * 512 + key;
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        float o[HT];
        tmem_ld_n<HT>(tmem + lane_off + ob * (4 * HB) + m * HB + wg * HT, o);
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          const int hh = wg * HT + h;
          if (hh < heads) {
            if (part)
              po[hh * 512 + m * 128] = o[h] * inv[h];
            else
              out[hh * 512 + m * 128] = f32_to_bf16_rn(o[h] * inv[h]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bars[B_O_EMPTY + ob]);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) tmem_dealloc(tmem, C::TMEM_COLS);
}

// --------------------------------------------------------------------------
// Join: out = sum_s 2^(L_s - M) O_s / sum_s 2^(L_s - M) over the parts of a cut
// request (L_s base-2 log-sum-exp, O_s normalised), lse = M + log2 of that sum.
//
// One CTA per range border.  The borders inside one request share its H * 512
// outputs evenly, so one long context is joined by all CTAs and a cut batch by
// one CTA per cut, and every CTA reads about as much as its range's CTA wrote.
// The parts are summed in order, whatever CTA stored them first.
// --------------------------------------------------------------------------
constexpr int NT_JOIN = 512;
constexpr int JOIN_ITEMS = 128;   // float4 outputs at a time with four threads each
constexpr int JOIN_W = 1024;

__global__ void __launch_bounds__(NT_JOIN) join_kernel(const __grid_constant__ DecodeArgs a, int heads_padded) {
  __shared__ int64_t scan[NT_JOIN / 32];
  __shared__ int64_t found[2];       // request, tiles before it
  __shared__ int found_n;
  __shared__ float wgt[JOIN_W];
  __shared__ float4 acc[3][JOIN_ITEMS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the lengths were there before the first kernel: this part overlaps its end
  const int per = (a.B + NT_JOIN - 1) / NT_JOIN;
  const int b_lo = min(a.B, (int)threadIdx.x * per), b_hi = min(a.B, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += tiles_of(a, __ldg(a.kv_lens + b));
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) scan[warp] = incl;
  if (threadIdx.x == 0) found_n = 0;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
  for (int w = 0; w < NT_JOIN / 32; ++w) {
    const int64_t n = scan[w];
    if (w < warp) before += n;
    total += n;
  }
  const int64_t ng = total < a.groups ? total : a.groups;
  const int64_t g = blockIdx.x;                       // the border between ranges g and g + 1
  const int64_t x = g + 1 < ng ? (g + 1) * total / ng : 0;
  if (x > 0 && before <= x && x < before + mine) {
    int64_t at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const int n = tiles_of(a, __ldg(a.kv_lens + b));
      if (x < at + n) {
        found[0] = b;
        found[1] = at;
        found_n = n;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  // wait for the first kernel's stores
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (found_n == 0 || found[1] == x) return;          // no border here, or between two requests
  const int64_t p0 = found[1], p1 = p0 + found_n;
  const int64_t b = found[0];
  // the ranges that hold the request's first and last tiles, and this CTA's share
  const int g0 = (int)(((p0 + 1) * ng - 1) / total), g1 = (int)((p1 * ng - 1) / total);
  const int S = g1 - g0 + 1, nb = S - 1, rank = (int)g - g0;
  const int first_slot = 2 * g0 + ((int64_t)g0 * total / ng == p0 ? 0 : 1);
  auto slot_of = [&](int s) { return s == 0 ? (int64_t)first_slot : 2ll * (g0 + s); };
  const int64_t items = (int64_t)a.H * 128;
  const int i0 = (int)(items * rank / nb), i1 = (int)(items * (rank + 1) / nb);
  if (i0 >= i1) return;
  const int ha = i0 >> 7, hz = (i1 - 1) >> 7;
  const int hstep = JOIN_W / S < hz - ha + 1 ? JOIN_W / S : hz - ha + 1;   // heads whose weights fit
  const bool wide = S >= 8;   // four threads per output, a quarter of the parts each
  for (int h0 = ha; h0 <= hz; h0 += hstep) {
    const int h1 = min(h0 + hstep - 1, hz);
    // weights of these heads, one warp per head
    for (int h = h0 + warp; h <= h1; h += NT_JOIN / 32) {
      float m = -INFINITY;
      for (int s = lane; s < S; s += 32) m = fmaxf(m, a.part_lse[slot_of(s) * heads_padded + h]);
      m = warp_max(m);
      const float mr = m == -INFINITY ? 0.f : m;
      float sum = 0.f;
      for (int s = lane; s < S; s += 32) {
        const float w = exp2f(a.part_lse[slot_of(s) * heads_padded + h] - mr);
        wgt[(h - h0) * S + s] = w;
        sum += w;
      }
      sum = warp_sum(sum);
      const float inv = sum != 0.f ? 1.0f / sum : 0.f;
      for (int s = lane; s < S; s += 32) wgt[(h - h0) * S + s] *= inv;
      if (lane == 0 && (h << 7) >= i0 && (h << 7) < i1)
        a.lse[b * a.H + h] = sum != 0.f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
    __syncthreads();
    const int lo = max(i0, h0 << 7), hi = min(i1, (h1 + 1) << 7);
    const int quarter = wide ? (int)threadIdx.x / JOIN_ITEMS : 0;
    const int step = wide ? JOIN_ITEMS : NT_JOIN;
    const int s0 = wide ? S * quarter / 4 : 0, s1 = wide ? S * (quarter + 1) / 4 : S;
    for (int base = lo; base < hi; base += step) {
      const int i = base + (int)threadIdx.x % step;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < hi) {
        const int h = i >> 7;
        const float* src = a.part_o + 4ll * i;
        const float* w = wgt + (h - h0) * S;
#pragma unroll 8
        for (int s = s0; s < s1; ++s) {
          const float4 v = *reinterpret_cast<const float4*>(src + slot_of(s) * heads_padded * 512);
          const float f = w[s];
          o.x += f * v.x;
          o.y += f * v.y;
          o.z += f * v.z;
          o.w += f * v.w;
        }
      }
      if (wide) {
        if (quarter > 0) acc[quarter - 1][threadIdx.x % JOIN_ITEMS] = o;
        __syncthreads();
        if (quarter == 0) {
#pragma unroll
          for (int qd = 0; qd < 3; ++qd) {
            const float4 v = acc[qd][threadIdx.x];
            o.x += v.x;
            o.y += v.y;
            o.z += v.z;
            o.w += v.w;
          }
        }
      }
      if (i < hi && quarter == 0)
        *reinterpret_cast<uint2*>(a.out + b * a.H * 512 + 4ll * i) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
      if (wide) __syncthreads();
    }
    __syncthreads();
  }
}

template <int HB, int NC>
static int launch_t(const DecodeArgs& a, cudaStream_t stream) {
  using C = Cfg<HB, NC>;
  static int attr_set[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !attr_set[dev]) {
    if (cudaFuncSetAttribute(decode_kernel<HB, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) !=
        cudaSuccess)
      return -1;
    attr_set[dev] = 1;
  }
  decode_kernel<HB, NC><<<a.groups * a.head_blocks, NTHREADS, C::SMEM_BYTES, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace decode

int launch_paged_decode(DecodeArgs& a, bool fp8, int d_rope, int max_tiles, cudaStream_t stream) {
  using namespace decode;
  if (fp8) return -2;
  const int hb = decode_heads_per_cta(a.H);
  int r = -2;
  if (hb == 16) r = d_rope ? launch_t<16, 9>(a, stream) : launch_t<16, 8>(a, stream);
  else r = d_rope ? launch_t<32, 9>(a, stream) : launch_t<32, 8>(a, stream);
  if (r != 0) return r;
  if (max_tiles <= 1 || a.groups <= 1) return 0;   // no request can be cut
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.groups - 1));
  cfg.blockDim = dim3(NT_JOIN);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel, a, a.head_blocks * hb) == cudaSuccess ? 0 : -1;
}

}  // namespace dsa
