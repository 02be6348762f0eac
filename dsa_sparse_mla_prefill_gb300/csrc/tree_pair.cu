// Attention of a tree of drafted tokens over the paged latent cache (see tree_decode.cu) for many
// query rows (tokens x heads) per request: CTA pairs with the query rows on the tensor cores' M side.
//
// Bound: from some 120 rows on a key row's flops (2 * 1088 each query row) take longer than its
// 1152 bytes take from HBM, so the tensor cores are the roof, and what feeds them.
//
// A pair (2-CTA cluster, cta_group::2) holds a block of 128 query rows of one request, 64 in
// each CTA, and walks the keys in tiles of 256:
//   S = Q K^T     M = 128, N = 256: CTA r supplies its 64 rows of Q (resident) and 128 keys'
//                 rows of the tile; it gets S of its own 64 query rows, TMEM lanes 0-63 with
//                 the even CTA's keys, lanes 64-127 with the odd one's.
//   softmax       thread = (query row, 64 of the tile's keys): row maxima stay in the CTA
//                 (four threads a row, one exchange through shared memory), P goes to shared
//                 memory as the A operand of the same CTA's rows.
//   O += P V      M = 128, N = 256 for output columns 256 m + ..: CTA r supplies columns 256 m +
//                 128 r .. +127 of all 256 keys.  O takes 2 x 128 TMEM columns, S twice 128.
// With the query rows as M, nothing of P or the maxima crosses the pair, and for 64 query rows
// and a key each CTA's MMAs read 1.6 KB of shared memory and its loads bring 1.1 KB (with the keys
// as M and 64 rows to a CTA, as the decode kernel has it: 3.2 and 2.2).
//
// Loads go through two rings of 16 KB slots: a tile's nine 64-column chunks of 128 keys through
// four, its eight V slots (64 keys x 128 columns) through three, a loading warp per slot (FP8
// rows: two converting ones) and an issuing warp per ring, so that a tile's softmax and P V run
// beside the next tile's QK.  (Five and two slots: 114 against 97 us on 8 x 4096..32768 at 512
// rows, three and four 102; one ring of five with P in two places 111.)  P has one place, whose
// four columns of 64 keys are handed over one by one (with P handed over as a whole the three
// slots less would have cost more than they give).  A request's O leaves through the place of P
// while the next one's first QK runs.  Where several pairs walk the same rows, their scheduling
// warps ask L2 for the boxes of a tile more than a tile ahead of its loads, each for its share (not
// kept: line by line, 96 us against 94 on 8 x 4096..32768; a ring slot's next chunk, 95).
//
// Split over the length, join and the rows of absent keys as in paged_decode.cuh; a range of
// tiles is walked by the pairs of all row blocks at the same time.  A tile takes some 5200 cycles
// (its MMAs 4352), a range 7000 to its first scores, a request's change some 5000, the join 7 us:
// 8 x 4096..32768 at 512 rows 97 us of which 67 at the cuBLAS rate, 32 x 512..16384 at 128 rows
// 58 (27 at the copy rate; 8300 cycles a tile, four slots of K in flight from HBM), 1 x 131072 at
// 256 rows 63 (38); all on inputs that change from call to call.
// FP8 rows: 24 x 1024..16384 at 256 rows 121 us (one CTA per 32 rows 283), 12000 cycles a tile
// for the conversion: see there.
#include <cfloat>

#include "paged_decode.cuh"

namespace dsa {
namespace treepair {

using decode::drafted_of;
using decode::elect_one;
using decode::evict_first_policy;
using decode::evict_normal_policy;
using decode::load_2d_hint;
using decode::range_begin;
using decode::row_at;
using decode::warp_scan;

constexpr int TK = 256;              // keys of a tile
constexpr int ROWS = 64;             // query rows of a CTA
constexpr int NI = 4;                // tiles of rows ahead
constexpr int NK = 4, NV = 3;        // ring slots
constexpr int NSLOT = NK + NV;
constexpr float kTau = 8.0f;         // lazy-rescale threshold (log2 units)
constexpr uint16_t kBoth = 3;
constexpr int W_QK = 8, W_SCHED = 9, W_Q = 10;
template <bool F8>
struct Cfg {
  // a loading warp per ring slot, or two that convert (and one or two without work)
  static constexpr int NTHREADS = F8 ? 896 : 640, REGS = F8 ? 72 : 96;   // registers at launch
  static constexpr int NPROD = F8 ? 2 * NSLOT : NSLOT;
  static constexpr int W_PV = F8 ? 11 : 18, W_LOAD = F8 ? 12 : 11;
  static constexpr int REGS_SOFTMAX = F8 ? 120 : 168, REGS_REST = F8 ? 32 : 48, REGS_PROD = F8 ? 56 : 48;
  static_assert(256 * REGS_SOFTMAX + 128 * REGS_REST + (NTHREADS - 384) * REGS_PROD <= NTHREADS * REGS, "registers");
};

constexpr uint32_t SLOT_BYTES = 16384u, HALF_BYTES = 8192u;
constexpr uint32_t Q_CHUNK = ROWS * 128u;
constexpr uint32_t P_COLUMN = ROWS * 128u;         // 64 rows x 64 keys
constexpr uint32_t OFF_RING = 0;
constexpr uint32_t OFF_Q = OFF_RING + NSLOT * SLOT_BYTES;
constexpr uint32_t OFF_P = OFF_Q + 9 * Q_CHUNK;
constexpr uint32_t OFF_ROWS = OFF_P + 4 * P_COLUMN;
constexpr uint32_t OFF_META = OFF_ROWS + NI * TK * 4u;
constexpr uint32_t OFF_VALID = OFF_META + NI * 16u;
constexpr uint32_t OFF_RED = OFF_VALID + NI * 32u;  // [parity][part][row] maxima, [part][row] sums of each kind
constexpr uint32_t OFF_BAR = OFF_RED + 4u * 4u * ROWS * 4u;
constexpr int NBAR = 61;
constexpr uint32_t OFF_MISC = OFF_BAR + (NBAR + 1) / 2 * 16u;
constexpr uint32_t SMEM_BYTES = OFF_MISC + 64u + 1024u;
static_assert(SMEM_BYTES <= 227u * 1024u, "shared memory budget");
constexpr uint32_t COL_O = 0, COL_S = 256;

enum {
  B_FULL = 0,       // [NK K slots, then NV V slots] even CTA: armed for both CTAs' bytes (FP8: 4 warps)
  B_EMPTY = 8,      // one commit
  B_QF = 16,        // even CTA
  B_QE = 17,
  B_SF = 18,        // [2] one commit
  B_SE = 20,        // [2] even CTA: 16 softmax warps of the pair
  B_PF = 22,        // [4] per 64 keys: this CTA's two softmax warps have stored its rows of P
  B_PE = 26,        // [4] one commit: the MMAs that read these columns of P are done
  B_OF = 30,
  B_OE = 31,        // even CTA: 16 warps of the pair
  B_IDXF = 32,      // [NI]
  B_IDXE = 36,      // [NI] the loaders, Q, softmax and (even CTA) issuing warps
  B_GRP = 40,       // [2] the four warps of 32 query rows
  B_PLAN = 42,
  B_DRAIN = 43,     // [2] one per issuer
  B_RS = 45,        // [2] this CTA's 8 softmax warps: O stands in the tile's reference
  B_RAW = 47,       // [2 NSLOT] FP8: codes and scales of a converting warp have landed
};
constexpr int F_FIRST = 1, F_LAST = 2, F_PART = 4, F_SLOT1 = 8, F_BOX = 16, F_FULL = 32;

__device__ __forceinline__ int tiles_of(const DecodeArgs& a, int len) {
  return len <= 0 ? 0 : (int)(((uint32_t)min(len, a.cap) + TK - 1) / TK);
}

// Hands this CTA's stores to shared memory over to the even CTA, whose issuing warp has the
// tensor cores read them: a release at cluster scope of what was done to this CTA's shared
// memory (by every lane, with its fence to the async proxy and the __syncwarp in front), and a
// bare arrival.  An arrival that releases all memory at cluster scope takes some 2000 cycles in
// a warp that has stored; this one with the waits below, 8 x 4096..32768 at 512 rows 95.7 us
// and 24 x 1024..16384 over FP8 rows 118.7, against 95.1 and 117.4 at CTA scope, which would
// order nothing between two CTAs.
__device__ __forceinline__ void hand_over(uint32_t remote_bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  mbar_arrive_remote_relaxed(remote_bar);
}

// As mbar_wait_vote, for barriers that the other CTA of the pair arrives on too: acquires at
// cluster scope, a poll what was done to shared memory (tensor memory has its own fences; 24 x
// 1024..16384 over FP8 rows 121 us with polls that acquire all memory).
template <bool POLL>
__device__ __forceinline__ bool wait_vote(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
  uint64_t t0 = 0;   // (the clock is first read on the sixteenth turn)
  uint32_t turns = 0;
#pragma unroll 1
  while (true) {
    uint32_t ok;
    if constexpr (POLL)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    else
      ok = mbar_try_wait_cluster_sleep(bar, parity);
    if (__all_sync(0xffffffffu, ok)) {
      if constexpr (POLL) asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
      return true;
    }
    if ((++turns & 15u)) continue;
    const uint64_t now = globaltimer();
    if (t0 == 0) t0 = now;
    const bool raised = *abort_flag != 0, late = now - t0 > kWaitTimeoutNs;
    if (__any_sync(0xffffffffu, raised | late)) {
      mbar_give_up(abort_flag, err);
      return false;
    }
  }
}

__device__ __forceinline__ void mma_pair_x4_elected(uint32_t leader, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t da,
                                                    uint32_t db, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %11, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %5, %6, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %7, %8, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %9, %10, %3, 1;\n\t}"
      ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "l"(a + da), "l"(b + db), "l"(a + 2ull * da),
      "l"(b + 2ull * db), "l"(a + 3ull * da), "l"(b + 3ull * db), "r"(leader)
      : "memory");
}
// (a completion signal to the barriers of both CTAs; no data moves)
__device__ __forceinline__ void commit_pair_elected(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}"
      ::"r"(bar), "r"(leader), "h"(kBoth)
      : "memory");
}

// TMA loads into this CTA that complete on a barrier of the even one.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
// (n gathers of four rows x 128 bytes, issued by one elected lane)
__device__ __forceinline__ void gather(uint32_t leader, uint32_t dst, const CUtensorMap* map, int x, const int32_t* rows,
                                       int count, uint32_t bar, uint64_t policy) {
#pragma unroll 2
  for (int n = 0; n < count; ++n) {
    const int4 r = *reinterpret_cast<const int4*>(rows + 4 * n);
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %9, 0;\n\t"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;\n\t}" ::"r"(dst + n * 512),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar), "l"(policy),
        "r"(leader)
        : "memory");
  }
}

template <int NC, bool F8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<F8>::NTHREADS, 1) tree_pair_kernel(const __grid_constant__ DecodeArgs a) {
  using C = Cfg<F8>;
  constexpr int W_PV = C::W_PV, W_LOAD = C::W_LOAD;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_u32 + 1023u) & ~1023u) - raw_u32);   // (the same offset in both CTAs)
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile uint32_t* tmem_base_ptr = misc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* plan = reinterpret_cast<volatile int*>(misc + 2);
  int32_t* rows = reinterpret_cast<int32_t*>(smem + OFF_ROWS);
  int4* meta = reinterpret_cast<int4*>(smem + OFF_META);
  uint64_t* valid = reinterpret_cast<uint64_t*>(smem + OFF_VALID);
  unsigned int* err = a.err;
  const uint32_t bar0 = sbase + OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * i; };
  auto poll = [&](int i, uint32_t parity) { return wait_vote<true>(bar(i), parity, abort_flag, err); };
  auto doze = [&](int i, uint32_t parity) { return wait_vote<false>(bar(i), parity, abort_flag, err); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const int pair = (int)blockIdx.x >> 1;
  const int range = pair / a.head_blocks, rb = pair - range * a.head_blocks;
  const int row0 = 2 * ROWS * rb + ROWS * rank;   // this CTA's first query row of a request

  if (warp == 0) {
    for (int i = lane; i < NBAR; i += 32) {
      uint32_t n = 1;
      if (i == B_SE || i == B_SE + 1 || i == B_OE) n = 16;
      if (i >= B_PF && i < B_PF + 4) n = 4;
      if (i == B_RS || i == B_RS + 1) n = 16;
      if (i >= B_IDXE && i < B_IDXE + NI) n = C::NPROD + 1 + (rank == 0 ? 2 : 0) + 8;
      if (F8 && i < NSLOT) n = 4;   // (the slot's converting warps of both CTAs)
      if (i == B_GRP || i == B_GRP + 1) n = 4;
      mbar_init(&bars[i], n);
    }
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == W_Q && lane < (F8 ? 1 : 3)) {
    const CUtensorMap* map = lane == 0 ? &a.tmap_q : lane == 1 ? &a.tmap_kv : &a.tmap_box;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  if (warp == W_QK) {
    tmem_alloc_pair(const_cast<uint32_t*>(tmem_base_ptr), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before a copy, commit or arrival reaches them
  tc_fence_after();
  const uint32_t tmem = *tmem_base_ptr;
  launch_dependents();

  if (F8 && warp >= W_LOAD) {
    regs_dec<C::REGS_PROD>();
    wait_for_previous();
    if constexpr (F8) {
      const int nt = warp < W_LOAD + C::NPROD && poll(B_PLAN, 0) ? plan[0] : 0;
      // ----------------------------------------------------------------
      // FP8 rows: two warps per ring slot fill it, each 64 rows x 64 columns of 8 KB.  The codes
      // land in the upper half of that place and the rows' scales at its start, by boxes or, from
      // pages without runs and in tiles with missing keys, by 16-byte copies (eight rows x 64
      // bytes to an instruction).  The warp converts them by the arithmetic of the dequantize
      // kernel and stores them as the bf16 rows would have landed: what a store covers has been
      // read.  The RoPE columns are copied.  Every row is converted twice, for K and for
      // V, whose slots are needed a tile apart.
      //
      // What bounds it: a slot's way from one use to the next, 5000 cycles for 17 uses a tile in
      // seven slots (free 400, asked for 700, landed 1000, converted 2400 beside the other warps,
      // handed over 800), the load-store pipe at half of its peak.  In that time the warps have
      // nothing else to do: codes land in the slot itself, so none can be asked for before it is
      // free.  The 72 registers at launch leave 108 bytes a thread stored to local memory and 404
      // loaded from it.  On 24 x 1024..16384 at 256 rows, 117 us when these were
      // measured: without the loads it would take 103, without
      // the arithmetic no less; all by 16-byte copies 122; half or all of the codes through
      // registers, ahead of the free slot, 137 to 160 (a load's data in flight takes room in 28 KB
      // of L1); one warp a slot 170; four warps on every slot in turn 185.
      // ----------------------------------------------------------------
      const int own = (warp - W_LOAD) >> 1, half = (warp - W_LOAD) & 1;
      const bool is_k = own < NK;
      const int nslots = is_k ? NK : NV, stages = is_k ? NC : 8;
      const int g = lane >> 2, c = lane & 3;   // row of eight, 16 bytes of a row's 64
      const uint32_t base = sbase + OFF_RING + own * SLOT_BYTES + half * HALF_BYTES;
      const uint32_t dst = base + g * 128u, raw = base + HALF_BYTES / 2 + lane * 16u;
      const uint32_t lo = (uint32_t)((2 * c) ^ g) << 4, hi = (uint32_t)((2 * c + 1) ^ g) << 4;
      const uint32_t full0 = map_peer(bar(B_FULL + own), 0);
      auto first_row = [&](int t, int st) { return rows + (t % NI) * TK + (is_k ? 128 * rank + 64 * half : 64 * (st >> 1)); };
      auto byte_of = [&](int32_t x) { return a.rows_base + (int64_t)x * a.row_bytes; };
      auto rope = [&](const int32_t* rr, int b16, int i) {
        const int32_t x = rr[8 * i + g];
        return x >= 0 ? *reinterpret_cast<const uint4*>(byte_of(x) + 528 + 16 * b16) : make_uint4(0, 0, 0, 0);
      };
      const int b_raw = B_RAW + warp - W_LOAD;
      const uint64_t policy = evict_normal_policy();
      int tile = 0, st = is_k ? own : own - NK;
      uint32_t used = 0, landed = 0;
      bool ok = nt > 0 && doze(B_IDXF, 0);
#pragma unroll 1
      while (ok) {
        const int32_t* rr = first_row(tile, st);
        const bool is_rope = is_k && st == 8;
        const bool box = (meta[tile % NI].y & F_BOX) != 0;
        const int block = is_k ? st >> 1 : 2 * (st & 1) + rank;
        const int at = is_k ? 64 * st : 128 * block + 64 * half;
        if (box) {
          const int r = lane * a.box_rows, x = r < 64 ? rr[r] : 0;
          if (!poll(B_EMPTY + own, (used & 1) ^ 1)) break;
          // (whatever has landed before, the phase waits for this arrival)
          if (lane == 0) mbar_arrive_expect_tx(&bars[b_raw], is_rope ? 64 * 128 : 64 * (64 + 16));
          if (r < 64) {
            if (is_rope) {
              load_2d_hint(base + r * 128, &a.tmap_box, 528, x, &bars[b_raw], policy);
            } else {
              load_2d_hint(base + HALF_BYTES / 2 + r * 64, &a.tmap_box8, at, x, &bars[b_raw], policy);
              load_2d_hint(base + r * 16, &a.tmap_kv, 512, x, &bars[b_raw], policy);
            }
          }
          if (!poll(b_raw, landed & 1)) break;
          ++landed;
        }
        if (is_rope) {
          if (!box) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = rope(rr, c, i);
            if (!poll(B_EMPTY + own, (used & 1) ^ 1)) break;
#pragma unroll
            for (int q = 0; q < 4; ++q) {   // rows 0-31, 32-63; their first 64 bytes, their last
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                sts128(dst + (4 * (q >> 1) + i) * 1024u + ((uint32_t)((4 * (q & 1) + c) ^ g) << 4), v[i].x, v[i].y, v[i].z, v[i].w);
                if (q < 3) v[i] = rope(rr, 4 * ((q + 1) & 1) + c, 4 * ((q + 1) >> 1) + i);
              }
            }
          }
        } else {
          float scale[2];   // of rows lane, lane + 32
          if (box) {
#pragma unroll
            for (int i = 0; i < 2; ++i) scale[i] = lds_f32(base + 16u * (lane + 32 * i) + 4u * block);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int32_t x = rr[32 * i + lane];
              scale[i] = x >= 0 ? *reinterpret_cast<const float*>(byte_of(x) + 512 + 4 * block) : 0.f;
            }
            if (!poll(B_EMPTY + own, (used & 1) ^ 1)) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int32_t x = rr[8 * i + g];
              cp_async16(raw + i * 512u, x < 0 ? static_cast<const void*>(a.borders) : byte_of(x) + at + 16 * c, x < 0 ? 0u : 16u);
            }
            cp_async_wait_all();
          }
          uint4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = lds128(raw + i * 512u);
          __syncwarp();   // (all is read)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float s = __shfl_sync(0xffffffffu, scale[i >> 2], 8 * (i & 3) + g);
            uint32_t v[8];
            e4m3x4_dequant_bf16x4(w[i].x, s, v[0], v[1]);
            e4m3x4_dequant_bf16x4(w[i].y, s, v[2], v[3]);
            e4m3x4_dequant_bf16x4(w[i].z, s, v[4], v[5]);
            e4m3x4_dequant_bf16x4(w[i].w, s, v[6], v[7]);
            sts128(dst + i * 1024u + lo, v[0], v[1], v[2], v[3]);
            sts128(dst + i * 1024u + hi, v[4], v[5], v[6], v[7]);
          }
        }
        ++used;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) hand_over(full0);
        st += nslots;
        if (st >= stages) {
          st -= stages;
          if (lane == 0) mbar_arrive(&bars[B_IDXE + tile % NI]);
          if (++tile == nt) break;
          if (!doze(B_IDXF + tile % NI, (tile / NI) & 1)) break;
        }
      }
      cp_async_wait_all();
      if (tile < nt) {
        // a wait ran out: let loads in flight land before this CTA can leave
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 20000ull) {
        }
      }
      __syncwarp();
    }
  } else if (warp >= W_QK) {
    regs_dec<C::REGS_REST>();
    wait_for_previous();
    if (warp == W_SCHED) {
      // ----------------------------------------------------------------
      // scheduler: as the decode kernel's, in each CTA for itself
      // ----------------------------------------------------------------
      const bool counts = rank == 0 && rb == 0;
      const int per = (a.B + 31) / 32;
      const int b_lo = min(a.B, lane * per), b_hi = min(a.B, b_lo + per);
      // Ranges are even in tiles, with a blank one counted in front of every request for what its
      // start costs (128 requests of 100..3000 keys at 128 rows: 65 us without, 57; two blank ones
      // 57, and 24 x 1024..16384 over FP8 rows 122 -> 128) unless a range has less than two.
      uint32_t mine_tiles = 0, mine_requests = 0;
#pragma unroll 4
      for (int i = b_lo; i < b_hi; ++i) {
        const uint32_t n = tiles_of(a, a.kv_lens[i]);
        mine_tiles += n;
        mine_requests += n > 0;
      }
      const uint32_t incl_tiles = warp_scan(mine_tiles), tiles = __shfl_sync(0xffffffffu, incl_tiles, 31);
      const uint32_t ng = tiles < (uint32_t)a.groups ? tiles : (uint32_t)a.groups;
      const uint32_t gap = tiles >= 2 * ng ? 1 : 0;
      // (positions: tiles and blank ones)
      const uint32_t mine = mine_tiles + gap * mine_requests;
      const uint32_t incl = warp_scan(mine), total = __shfl_sync(0xffffffffu, incl, 31), before = incl - mine;
      int b = 0, j = 0, len = 0, n = 0;
      // the first tile at or behind position x, tile j of request b: tiles in front of it
      auto find = [&](uint32_t x) {
        const bool holds = before <= x && x < before + mine;
        uint32_t so_far = 0;
        if (holds) {
          uint32_t at = before;
          so_far = incl_tiles - mine_tiles;
          for (b = b_lo;; ++b) {
            len = a.kv_lens[b];
            n = tiles_of(a, len);
            const uint32_t span = n ? n + gap : 0;
            if (x < at + span) break;
            at += span;
            so_far += n;
          }
          j = x - at < gap ? 0 : (int)(x - at - gap);
          so_far += j;
        }
        const int holder = __ffs(__ballot_sync(0xffffffffu, holds)) - 1;
        b = __shfl_sync(0xffffffffu, b, holder & 31);
        j = __shfl_sync(0xffffffffu, j, holder & 31);
        len = __shfl_sync(0xffffffffu, len, holder & 31);
        return holder < 0 ? tiles : __shfl_sync(0xffffffffu, so_far, holder & 31);
      };
      int nt = 0;
      if ((uint32_t)range < ng) {
        const uint32_t behind = find(range_begin(range + 1, total, ng));
        nt = (int)(behind - find(range_begin(range, total, ng)));
      }
      if (lane == 0) {
        if (range == 0 && counts) a.borders[0] = make_int4(total, ng, gap, 0);
        if (counts) a.borders[1 + range] = make_int4(0, 0, 0, 0);
        plan[0] = nt;
        plan[1] = b;
        mbar_arrive(&bars[B_PLAN]);
      }
      int bad = 0, seg = 0, drafted = 0, context = 0;
      uint64_t seen = 0;   // drafted tokens that any token sees (worked out at the first tile that holds one)
      bool looked = false;
      const bool from_start = j == 0;
      bool enter = true;
      int fetch = -1;   // first row of a box to fetch to L2
      const int sharers = 2 * a.head_blocks, share = 2 * rb + rank;   // CTAs that walk this range
      for (int it = 0; it < nt; ++it) {
        const int r = it % NI;
        if (enter) {
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
          drafted = drafted_of(a, b);
          context = len - drafted;
          looked = false;
          if (len > a.cap) {
            if (j == 0 && lane == 0) ++bad;
            len = a.cap;
          }
        }
        if (!doze(B_IDXE + r, ((it / NI) & 1) ^ 1)) break;
        if (!looked && j * TK > context - TK) {   // (the last tile may end past 2^31)
          uint64_t any = 0;
          for (int i = lane; i < drafted; i += 32) any |= a.tree_mask[(int64_t)b * a.n + i];
          seen = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(any >> 32)) << 32 | __reduce_or_sync(0xffffffffu, (uint32_t)any);
          looked = true;
        }
        const int32_t* bt = a.block_table + (int64_t)b * a.max_blocks;
        int32_t row[8];
        const uint32_t e0 = (uint32_t)j * TK + 8 * lane;
        uint32_t page = e0 / (uint32_t)a.block_size, at = e0 - page * (uint32_t)a.block_size, there8 = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          bool there = e0 + e < (uint32_t)len;
          const int bit = (int)(e0 + e) - context;
          if (there && bit >= 0) there = seen >> bit & 1;   // (bit < drafted, for the position is below len)
          row[e] = -1;
          if (there) row[e] = row_at(a, bt, page, at, bad);
          there8 |= row[e] >= 0 ? 1u << e : 0u;
          if (++at == (uint32_t)a.block_size) { at = 0; ++page; }
        }
        *reinterpret_cast<int4*>(rows + r * TK + 8 * lane) = make_int4(row[0], row[1], row[2], row[3]);
        *reinterpret_cast<int4*>(rows + r * TK + 8 * lane + 4) = make_int4(row[4], row[5], row[6], row[7]);
        reinterpret_cast<uint8_t*>(valid + 4 * r)[lane] = (uint8_t)there8;
        const bool all = __all_sync(0xffffffffu, there8 == 0xffu);
        __syncwarp();
        // the boxes of the tile one back, more than a tile ahead of its loads, to L2: by each CTA its share
        if (!F8 && fetch >= 0)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.rows_base + (int64_t)fetch * a.row_bytes),
                       "r"(a.fetch_bytes)
                       : "memory");
        if (!F8 && a.fetch_bytes) {
          fetch = rows[r * TK + (lane & (TK / a.box_rows - 1)) * a.box_rows];   // of box `lane`
          if (lane >= TK / a.box_rows || lane % sharers != share || fetch > a.N - a.box_rows) fetch = -1;
        }
        const bool first = enter, last = (it == nt - 1) || (j == n - 1);
        if (lane == 0) {
          int flags = (first ? F_FIRST : 0) | (last ? F_LAST : 0) | (all && a.box_rows > 0 ? F_BOX : 0);
          if (all && j * TK <= context - TK) flags |= F_FULL;
          if (last) {
            const bool whole = (seg > 0 || from_start) && j == n - 1;
            if (!whole) flags |= F_PART | (seg > 0 ? F_SLOT1 : 0);
          }
          meta[r] = make_int4(b, flags, j * TK - context, drafted);
          if (it == nt - 1 && counts) a.borders[1 + range] = make_int4(b, n, j + 1, 0);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_IDXF + r]);
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
      if (lane == 0 && bad && counts) atomicAdd(err + ERR_BAD_INDEX, (unsigned)bad);
    } else if (const int nt = poll(B_PLAN, 0) ? plan[0] : 0; !F8 && warp >= W_LOAD && warp < W_LOAD + NSLOT) {
      // ----------------------------------------------------------------
      // loads, a warp per slot of the K and the V ring.  A slot is two halves of 64 rows x 64
      // columns: of K the two halves of this CTA's 128 keys, of V (64 keys) its two 64-column
      // groups.
      // ----------------------------------------------------------------
      const int own = warp - W_LOAD;
      const bool is_k = own < NK;
      const int mine_slot = is_k ? own : own - NK, nslots = is_k ? NK : NV, stages = is_k ? NC : 8;
      const uint32_t dst = sbase + OFF_RING + own * SLOT_BYTES;
      const uint32_t full0 = map_peer(bar(B_FULL + own), 0);
      const uint32_t leader = elect_one();
      const int per_half = a.box_rows > 0 ? ROWS / a.box_rows : 1;   // boxes
      const int h = lane / per_half, at = (lane - h * per_half) * a.box_rows;   // of a lane with a box
      // (the second read of a row, by the only block of query rows, marks it first to go)
      const uint64_t policy = is_k || a.head_blocks > 1 ? evict_normal_policy() : evict_first_policy();
      int slot = 0;
      uint32_t used = 0;
      bool ok = true;
#pragma unroll 1
      for (int it = 0; it < nt && ok; ++it) {
        const int r = it % NI;
        if (!doze(B_IDXF + r, (it / NI) & 1)) { ok = false; break; }
        const bool box = (meta[r].y & F_BOX) != 0;
        const int32_t* tile_rows = rows + r * TK;
#pragma unroll 1
        for (int st = 0; st < stages; ++st) {
          const bool mine_now = slot == mine_slot;
          if (++slot == nslots) slot = 0;
          if (!mine_now) continue;
          if (!doze(B_EMPTY + own, (used & 1) ^ 1)) { ok = false; break; }
          if (rank == 0 && leader) mbar_arrive_expect_tx(&bars[B_FULL + own], 2u * SLOT_BYTES);
          __syncwarp();
          ++used;
          // first row and column of half 0, and how half 1 differs
          const int ra = is_k ? 128 * rank : 64 * (st >> 1), rstep = is_k ? 64 : 0;
          const int ca = is_k ? 64 * st : 256 * (st & 1) + 128 * rank, cstep = is_k ? 0 : 64;
          if (box) {
            if (h < 2)
              load_box(dst + h * HALF_BYTES + at * 128, &a.tmap_box, ca + h * cstep, tile_rows[ra + h * rstep + at], full0, policy);
          } else if (a.box_rows > 0) {
            // where keys are missing: a half that is there, or none of it (read from behind the
            // cache, as zeros), by its boxes; the others by a lane per eight rows, gathered
            // where some of the eight are missing
            const int g = lane >> 3 & 1, i = lane & 7, half_row = ra + g * rstep;
            const uint64_t in64 = valid[4 * r + (half_row >> 6)];
            const uint32_t in = (uint32_t)(in64 >> (8 * i)) & 0xffu;
            const uint32_t half_dst = dst + g * HALF_BYTES;
            const bool whole = in64 == 0 || in64 == ~0ull;
            uint32_t left = __ballot_sync(0xffffffffu, lane < 16 && in != 0 && in != 0xffu);
            if (lane < 16) {
              if (whole) {
                if (i < per_half)
                  load_box(half_dst + i * a.box_rows * 128, &a.tmap_box, ca + g * cstep, in64 ? tile_rows[half_row + i * a.box_rows] : a.N,
                           full0, policy);
              } else if (in == 0 || in == 0xffu) {
                load_box(half_dst + i * 1024, &a.tmap_box8, ca + g * cstep, in ? tile_rows[half_row + 8 * i] : a.N, full0, policy);
              }
            }
            for (; left; left &= left - 1) {
              const int l = __ffs(left) - 1, lg = l >> 3, lat = (l & 7) * 8;
              gather(leader, dst + lg * HALF_BYTES + lat * 128, &a.tmap_kv, ca + lg * cstep, tile_rows + ra + lg * rstep + lat, 2,
                     full0, policy);
            }
          } else {
            gather(leader, dst, &a.tmap_kv, ca, tile_rows + ra, ROWS / 4, full0, policy);
            gather(leader, dst + HALF_BYTES, &a.tmap_kv, ca + cstep, tile_rows + ra + rstep, ROWS / 4, full0, policy);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_IDXE + r]);
      }
      if (!ok) {
        // a wait ran out: let loads in flight land before this CTA can leave
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 20000ull) {
        }
      }
      __syncwarp();
    } else if (warp == W_Q) {
      // ----------------------------------------------------------------
      // Q of every request of the range; then the requests without keys
      // ----------------------------------------------------------------
      const uint32_t full0 = map_peer(bar(B_QF), 0);
      int nq = 0;
      auto load_q = [&](int b) {
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&bars[B_QF], 2u * NC * Q_CHUNK);
        __syncwarp();
        if (lane < NC) tma_load_2d_pair(sbase + OFF_Q + lane * Q_CHUNK, &a.tmap_q, lane * 64, b * a.H + row0, full0);
        ++nq;
      };
      if (nt > 0) load_q(plan[1]);   // (the first request's, while the scheduler looks up its rows)
      for (int it = 0; it < nt; ++it) {
        const int r = it % NI;
        if (!doze(B_IDXF + r, (it / NI) & 1)) break;
        const int4 mt = meta[r];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_IDXE + r]);
        if (it == 0 || !(mt.y & F_FIRST)) continue;
        if (!doze(B_QE, (nq & 1) ^ 1)) break;
        load_q(mt.x);
      }
      const int mine = min(a.H - row0, ROWS);
      for (int b = range; b < a.B; b += a.groups) {
        if (tiles_of(a, a.kv_lens[b]) > 0) continue;
        uint4* o = reinterpret_cast<uint4*>(a.out + ((int64_t)b * a.H + row0) * 512);
        for (int i = lane; i < mine * 64; i += 32) o[i] = make_uint4(0, 0, 0, 0);
        for (int i = lane; i < mine; i += 32) a.lse[(int64_t)b * a.H + row0 + i] = -INFINITY;
      }
    } else if (warp == W_QK) {
      // ----------------------------------------------------------------
      // QK issuer (even CTA)
      // ----------------------------------------------------------------
      const uint32_t leader = elect_one();
      if (rank == 0) {
        constexpr uint32_t IDESC = idesc_bf16_f32(128, 256, false, false);
        const uint64_t k_desc = sdesc_sw128(sbase + OFF_RING, 16, 1024), q_desc = sdesc_sw128(sbase + OFF_Q, 16, 1024);
        uint32_t slot = 0, phase = 0;
        int nq = -1;
        bool ok = true;
#pragma unroll 1
        for (int it = 0; it < nt && ok; ++it) {
          const int r = it % NI, sb = it & 1;
          if (!doze(B_IDXF + r, (it / NI) & 1)) break;
          const int flags = __shfl_sync(0xffffffffu, meta[r].y, 0);
          if (leader) mbar_arrive(&bars[B_IDXE + r]);
          if (flags & F_FIRST) {
            ++nq;
            if (!poll(B_QF, nq & 1)) break;
          }
          if (!poll(B_SE + sb, ((it >> 1) & 1) ^ 1)) break;
          if (leader) DSA_TRACE(a.tr, it, 3);
#pragma unroll 1
          for (int c = 0; c < NC; ++c) {
            if (!poll(B_FULL + slot, phase)) { ok = false; break; }
            tc_fence_after();
            mma_pair_x4_elected(leader, tmem + COL_S + sb * 128, q_desc + (uint64_t)(c * (Q_CHUNK >> 4)),
                                k_desc + (uint64_t)(slot * (SLOT_BYTES >> 4)), 2u, 2u, IDESC, c > 0 ? 1u : 0u);
            commit_pair_elected(leader, bar(B_EMPTY + slot));
            if (++slot == NK) { slot = 0; phase ^= 1; }
          }
          if (!ok) break;
          if (leader) DSA_TRACE(a.tr, it, 4);
          commit_pair_elected(leader, bar(B_SF + sb));
          if (flags & F_LAST) commit_pair_elected(leader, bar(B_QE));
        }
        commit_pair_elected(leader, bar(B_DRAIN));   // every MMA issued above has completed
        if (leader) mbar_wait_drain(&bars[B_DRAIN], 0, err);
      }
      __syncwarp();
    } else if (warp == W_PV && rank == 0) {
      // ----------------------------------------------------------------
      // P.V issuer (even CTA).  (One warp for both products spent 380 cycles on a slot, whose
      // four MMAs take 256: waiting, issuing and committing follow one another.)
      // ----------------------------------------------------------------
      constexpr uint32_t IDESC = idesc_bf16_f32(128, 256, false, true);
      const uint32_t leader = elect_one();
      const uint64_t v_desc = sdesc_sw128(sbase + OFF_RING + NK * SLOT_BYTES, HALF_BYTES, 1024), p_desc = sdesc_sw128(sbase + OFF_P, 16, 1024);
      uint32_t slot = 0, phase = 0;
      int nv = -1;
      bool ok = true;
#pragma unroll 1
      for (int it = 0; it < nt && ok; ++it) {
        const int r = it % NI;
        if (!doze(B_IDXF + r, (it / NI) & 1)) break;
        const int flags = __shfl_sync(0xffffffffu, meta[r].y, 0);
        if (leader) mbar_arrive(&bars[B_IDXE + r]);
        if (flags & F_FIRST) {
          ++nv;
          if (!poll(B_OE, (nv & 1) ^ 1)) break;
        }
        if (!poll(B_RS + (it & 1), (it >> 1) & 1)) break;
        if (leader) DSA_TRACE(a.tr, it, 0);
#pragma unroll 1
        for (int u = 0; u < 8; ++u) {   // (64 keys, then the two blocks of output columns)
          const int c = u >> 1, m = u & 1;
          if (m == 0 && !poll(B_PF + c, it & 1)) { ok = false; break; }
          if (!poll(B_FULL + NK + slot, phase)) { ok = false; break; }
          tc_fence_after();
          mma_pair_x4_elected(leader, tmem + COL_O + m * 128, p_desc + (uint64_t)(c * (P_COLUMN >> 4)),
                              v_desc + (uint64_t)(slot * (SLOT_BYTES >> 4)), 2u, 128u, IDESC, (flags & F_FIRST) && c == 0 ? 0u : 1u);
          commit_pair_elected(leader, bar(B_EMPTY + NK + slot));
          if (m == 1) commit_pair_elected(leader, bar(B_PE + c));
          if (++slot == NV) { slot = 0; phase ^= 1; }
        }
        if (!ok) break;
        if (leader) DSA_TRACE(a.tr, it, 7);
        if (flags & F_LAST) commit_pair_elected(leader, bar(B_OF));
      }
      commit_pair_elected(leader, bar(B_DRAIN + 1));
      if (leader) mbar_wait_drain(&bars[B_DRAIN + 1], 0, err);
      __syncwarp();
    }
  } else {
    regs_inc<C::REGS_SOFTMAX>();
    // --------------------------------------------------------------------
    // softmax and epilogue: warps w, w + 2 (the odd CTA's keys), w + 4 (the second 64 keys
    // of a half) and w + 6 have query rows 32 w .. 32 w + 31, w = 0, 1
    // --------------------------------------------------------------------
    const int wg = warp >> 2, half = (warp >> 1) & 1, rg = warp & 1;
    const int row = 32 * rg + lane;                       // of this CTA
    const int part = 2 * half + wg;                       // 64 keys of the tile: 64 part ..
    const int q_row = row0 + row;                         // of the request
    const int token = q_row / a.heads;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t p_row = sbase + OFF_P + part * P_COLUMN + row * 128;
    const uint32_t sw = (uint32_t)(row & 7);
    float* red = reinterpret_cast<float*>(smem + OFF_RED);
    float* sums = red + 2 * 4 * ROWS;
    const uint32_t se0 = map_peer(bar(B_SE), 0), pf0 = map_peer(bar(B_PF + part), 0), rs0 = map_peer(bar(B_RS), 0), oe0 = map_peer(bar(B_OE), 0);
    uint32_t grp_phase = 0;
    auto group = [&]() {   // the four warps of these rows
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_GRP + rg]);
      const bool ok = poll(B_GRP + rg, grp_phase);
      grp_phase ^= 1u;
      return ok;
    };
    // Sums of the weights as they are, for the log-sum-exp, and as P has them in bf16, which O is
    // divided by: what their rounding adds to O is then in the divisor too.
    float m_run = -FLT_MAX, l_run = 0.f, l_used = 0.f;   // (the lowest finite value, so that no difference of two is NaN)
    uint64_t word = 0;
    // The part of a request that has ended: its last tile's meta, reference and this thread's sums.
    bool pending = false;
    int4 done = make_int4(0, 0, 0, 0);
    float m_done = 0.f, l_done = 0.f, l_used_done = 0.f;
    int seg = 0;
    auto epilogue = [&]() -> bool {
      sums[part * ROWS + row] = l_done;
      sums[(4 + part) * ROWS + row] = l_used_done;
      if (!group()) return false;
      const bool live = token < done.w;   // (a padding token's row is zeros)
      auto sum_of = [&](const float* s) { return live ? (s[row] + s[ROWS + row]) + (s[2 * ROWS + row] + s[3 * ROWS + row]) : 0.f; };
      const float l = sum_of(sums), used = sum_of(sums + 4 * ROWS);
      // (all four warps have read: another part may end right behind this one, and nothing else would
      // keep a warp's sums of that one from this one's readers)
      if (!group()) return false;
      const float inv = used != 0.f ? 1.0f / used : 0.f;
      const bool is_part = (done.y & F_PART) != 0, there = q_row < a.H;
      const int64_t slot_row = (int64_t)(2 * range + ((done.y & F_SLOT1) ? 1 : 0)) * (2 * ROWS * a.head_blocks) + q_row;
      if (part == 0 && there) {
        const float l2 = l != 0.f ? m_done + log2f(l) : -INFINITY;
        if (is_part)
          a.part_lse[slot_row] = l2;
        else
          a.lse[(int64_t)done.x * a.H + q_row] = l2 * 0.6931471805599453f;
      }
      if (!poll(B_OF, seg & 1)) return false;
      ++seg;
      tc_fence_after();
      // Output columns 256 wg + 128 half .. +127 of the warp's 32 rows, 32 at a time, turned in
      // shared memory (the warp's own place in P, which the last P.V has read) so that a store fills
      // whole 128-byte (parts) or 64-byte pieces of rows: a thread storing its own row in 16-byte
      // pieces takes 8000 cycles for it.
      const int col = 256 * wg + 128 * half, first_row = row0 + 32 * rg;
      const uint32_t stage = sbase + OFF_P + part * P_COLUMN + rg * 4096u;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        float o[32];
        tmem_ld_cols<32>(t_lane + COL_O + wg * 128 + c, o);
        tmem_ld_wait();
        if (c == 96) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote_relaxed(oe0);   // (as above: O is read)
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = inv != 0.f ? o[i] * inv : 0.f;
        __syncwarp();   // (the pieces before are read)
        if (is_part) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            sts128(stage + lane * 128u + (((uint32_t)i ^ (lane & 7u)) << 4), __float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]),
                   __float_as_uint(o[4 * i + 2]), __float_as_uint(o[4 * i + 3]));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + (lane >> 3), at = lane & 7;
            const uint4 x = lds128(stage + rr * 128u + (uint32_t)((at ^ (rr & 7)) << 4));
            if (first_row + rr < a.H)
              *reinterpret_cast<uint4*>(a.part_o + (slot_row - q_row + first_row + rr) * 512 + col + c + 4 * at) = x;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sts128(stage + lane * 64u + (((uint32_t)i ^ ((lane >> 1) & 3u)) << 4), pack_bf16x2(o[8 * i], o[8 * i + 1]),
                   pack_bf16x2(o[8 * i + 2], o[8 * i + 3]), pack_bf16x2(o[8 * i + 4], o[8 * i + 5]),
                   pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = 8 * i + (lane >> 2), at = lane & 3;
            const uint4 x = lds128(stage + rr * 64u + (uint32_t)((at ^ ((rr >> 1) & 3)) << 4));
            if (first_row + rr < a.H)
              *reinterpret_cast<uint4*>(a.out + ((int64_t)done.x * a.H + first_row + rr) * 512 + col + c + 8 * at) = x;
          }
        }
      }
      __syncwarp();
      return true;
    };
    wait_for_previous();
    const int nt = poll(B_PLAN, 0) ? plan[0] : 0;
#pragma unroll 1
    for (int it = 0; it < nt; ++it) {
      const int r = it % NI, sb = it & 1;
      if (!doze(B_IDXF + r, (it / NI) & 1)) break;
      const int4 mt = meta[r];
      if (mt.y & F_FIRST) {
        m_run = -FLT_MAX;
        l_run = l_used = 0.f;
        word = token < mt.w ? a.tree_mask[(int64_t)mt.x * a.n + token] : 0ull;
      }
      uint64_t vis = ~0ull;
      if (!(mt.y & F_FULL)) {
        const int first = mt.z + 64 * part;   // drafted token of this thread's first key
        vis = first >= 64 ? 0ull : first >= 0 ? word >> first : first <= -64 ? ~0ull : (word << -first) | (~0ull >> (64 + first));
        vis &= valid[4 * r + part];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_IDXE + r]);
      if (!poll(B_SF + sb, (it >> 1) & 1)) break;
      if (threadIdx.x == 0) DSA_TRACE(a.tr, it, 5);
      tc_fence_after();
      float t[64];
      tmem_ld_cols<64>(t_lane + COL_S + sb * 128 + wg * 64, t);
      tmem_ld_wait();
      tc_fence_before();
      // (a bare "read" signal: nothing of this warp to publish, and a releasing arrival
      // takes 2000 cycles longer to get to the barrier below)
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_relaxed(se0 + 8u * sb);
#pragma unroll
      for (int i = 0; i < 64; i += 2) mul2(t[i], t[i + 1], t[i], t[i + 1], scale_log2, scale_log2);
      if (!(mt.y & F_FULL)) {
        const uint32_t lo = (uint32_t)vis, hi = (uint32_t)(vis >> 32);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          t[i] = lo >> i & 1 ? t[i] : -INFINITY;
          t[32 + i] = hi >> i & 1 ? t[32 + i] : -INFINITY;
        }
      }
      float mx[4] = {t[0], t[1], t[2], t[3]};
#pragma unroll
      for (int i = 4; i < 64; i += 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], t[i + k]);
      }
      float* redb = red + sb * (4 * ROWS);
      redb[part * ROWS + row] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (!group()) break;
      const float top = fmaxf(fmaxf(redb[row], redb[ROWS + row]), fmaxf(redb[2 * ROWS + row], redb[3 * ROWS + row]));
      // lazy rescale: the reference moves only where a score is above it by more than kTau
      float alpha = 1.f;
      if (top > m_run + kTau) {
        alpha = exp2f(m_run - top);
        m_run = top;
        l_run *= alpha;
        l_used *= alpha;
      }
      // O, which holds the P.V of the tile before then, in the new reference
      if (!(mt.y & F_FIRST) && __any_sync(0xffffffffu, alpha != 1.f)) {
        if (!poll(B_PE + 3, (it & 1) ^ 1)) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
          float o[16];
          const uint32_t ta = t_lane + COL_O + wg * 128 + c;
          tmem_ld16(ta, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] *= alpha;
          tmem_st16(ta, o);
        }
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_relaxed(rs0 + 8u * sb);
      const float neg = -m_run;
      float s0 = 0.f, s1 = 0.f;
      uint32_t pk[32];
#pragma unroll
      for (int i = 0; i < 64; i += 2) {
        float x, y;
        add2(x, y, t[i], t[i + 1], neg, neg);
        x = exp2f(x);
        y = exp2f(y);
        add2(s0, s1, s0, s1, x, y);
        pk[i / 2] = pack_bf16x2(x, y);
      }
      l_run += s0 + s1;
      // these columns of P are free once the MMAs of the tile before that read them are done; a
      // request's outputs are stored first, through them
      if (!poll(B_PE + part, (it & 1) ^ 1)) break;
      if (pending) {
        if (!epilogue()) break;
        pending = false;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c)
        sts128(p_row + ((((uint32_t)c) ^ sw) << 4), pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) hand_over(pf0);
      if (threadIdx.x == 0) DSA_TRACE(a.tr, it, 6);
      // (here, where nothing waits for it)
      float u0 = 0.f, u1 = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) add2(u0, u1, u0, u1, __uint_as_float(pk[i] << 16), __uint_as_float(pk[i] & 0xffff0000u));
      l_used += u0 + u1;
      if (mt.y & F_LAST) {
        pending = true;
        done = mt;
        m_done = m_run;
        l_done = l_run;
        l_used_done = l_used;
      }
    }
    if (pending) epilogue();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA leaves or frees tensor memory while the pair may still use it
  tc_fence_after();
  if (warp == W_QK) tmem_dealloc_pair(tmem, 512);
}

template <int NC, bool F8>
static int launch_t(DecodeArgs& a, cudaStream_t stream) {
  static PerDevice done, pairs;
  if (allow_smem(reinterpret_cast<const void*>(tree_pair_kernel<NC, F8>), SMEM_BYTES, done) != 0) return -1;
  // (a range more than the GPU holds at a time would run behind all others)
  const int most = resident_pairs(tree_pair_kernel<NC, F8>, kDecodeMaxCtas, Cfg<F8>::NTHREADS, SMEM_BYTES, pairs) / a.head_blocks;
  if (a.groups > most) a.groups = most > 0 ? most : 1;
  return launch_after(tree_pair_kernel<NC, F8>, dim3((unsigned)(2 * a.groups * a.head_blocks)), Cfg<F8>::NTHREADS, SMEM_BYTES, stream, a);
}

}  // namespace treepair

int launch_tree_pair(DecodeArgs& a, bool fp8, int d_rope, int max_tiles, cudaStream_t stream) {
  using namespace treepair;
  int r;
  if (fp8) r = d_rope ? launch_t<9, true>(a, stream) : launch_t<8, true>(a, stream);
  else r = d_rope ? launch_t<9, false>(a, stream) : launch_t<8, false>(a, stream);
  if (r != 0) return r;
  return decode::launch_join(a, 2 * treepair::ROWS * a.head_blocks, max_tiles, true, stream);
}

}  // namespace dsa
