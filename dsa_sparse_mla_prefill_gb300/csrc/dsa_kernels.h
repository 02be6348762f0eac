// Internal interface between the C-ABI shim (dsa_api.cu) and the kernels.
// Not installed; callers use include/dsa.h.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/dsa.h"

namespace dsa {

// Requests whose host-side sequence offsets travel inside the launch
// parameters (no device copy, no allocation).
constexpr int kMaxReq = 512;

struct ReqTable {
  int num_req;
  int32_t cu_q[kMaxReq + 1];    // query token offsets
  int32_t cu_kv[kMaxReq + 1];   // KV row offsets (masked mode / key mask)
  int32_t cu_g[kMaxReq + 1];    // group (or query tile) offsets
};

// Diagnostic timeline (dsa_debug_trace): when `trace` is set, CTAs 0 and 1
// record clock64() at up to 8 events of each of their first `trace_cap`
// tiles into trace[(cta * trace_cap + tile) * 8 + event].
struct TraceArgs {
  unsigned long long* trace;
  int trace_cap;
};

struct SparseArgs {
  CUtensorMap tmap_kv;  // kv rows, 64-column x 1-row box (row gathers)
  CUtensorMap tmap_q;   // q viewed [T*H, d_qk], 64-column x H-row box
  const uint16_t* q;    // [T, H, d_qk] bf16
  const uint16_t* kv;   // [N, ld_kv] bf16
  const uint8_t* kv8;   // FP8 rows [N, row_bytes] (the FP8 kernel; tmap_kv is then a byte map over them)
  int row_bytes;
  const int32_t* idx;   // [T, ld]
  uint16_t* out;        // [T, H, 512] bf16
  float* lse;           // [T, H]
  unsigned int* err;    // device error counters
  int T, H, d_qk, N, ld_kv, k, ld;
  float scale;
  TraceArgs tr;
  // Streamed from host memory (null otherwise): token t's q and index row may
  // be read once *ready > t (a copy stream raises it after each chunk lands);
  // once token t's out and lse are stored, done[t / done_blk] is incremented
  // (a copy stream waits on those counters before reading a chunk back).  A
  // CTA that gives up still counts its remaining tokens, so every counter
  // reaches its total.
  const uint32_t* ready;
  uint32_t* done;
  int done_blk;
};

struct UnionArgs {
  const int32_t* idx;   // [T, ld]
  int32_t* union_idx;   // [groups, union_pad]
  int32_t* union_len;   // [groups]
  uint8_t* mask;        // [groups, union_pad]
  unsigned int* err;
  int T, k, ld, G, N, union_pad, num_groups;
  ReqTable req;
};

struct Fp8KvArgs {
  const uint16_t* kv;   // quantize: bf16 rows [N, ld_kv]
  uint16_t* kv_out;     // dequantize: bf16 rows [N, ld_kv]
  uint8_t* fp8;         // FP8 rows [N, 528 + 2 d_rope] (quantize writes, dequantize reads)
  int N, ld_kv, d_rope;
};

struct RopeArgs {
  const void* x;              // [T, H, d] by strides (elements), unit last stride
  void* y;                    // may be x
  const int32_t* positions;   // [T]
  int64_t x_stride_t, x_stride_h, y_stride_t, y_stride_h;
  int T, H, d;
  int gradient;               // turn back
  int head_groups;            // threads that share a token's heads (set by the launch)
  dsa_rope_freqs table;
};

// Threads that share a token's heads, per_group threads being one such share of all
// tokens: as many heads per thread, in powers of two, as leave threads for half of
// every SM's 2048 slots (16384 tokens of 32 heads, interleaved bf16: 8 heads each 25.7
// us, 32 each 26.5, 11 each 27.3, 4 each 27.0, 2 each 36.6; 8191 of 16 heads, fp32
// halves: 4 each 13.6 us, 2 each 15.3, the cos and sin being worked out per thread).
inline int rope_head_groups(int64_t H, int64_t per_group, int num_sms) {
  int64_t each = 1;
  while (2 * each <= H && (H + 2 * each - 1) / (2 * each) * per_group >= 1024ll * num_sms) each *= 2;
  return (int)((H + each - 1) / each);
}

// Head norms with rotation (norm_rope.cu): one of queries and keys.
struct NormSide {
  const void* x;              // [T, H, d] by strides (elements), unit last stride
  const void* g;              // gradient: the result's gradient, likewise
  void* y;                    // the result, or x's gradient
  const void* w;              // [d_norm] weights
  float* dw;                  // gradient: [d_norm]
  int64_t x_stride_t, x_stride_h, g_stride_t, g_stride_h, y_stride_t, y_stride_h;
  int H;
  int ctas;                   // CTAs that work for this side (set by the launch)
};
struct NormArgs {
  NormSide side[2];           // queries, keys (H = 0: none)
  const int32_t* positions;   // [T] (unused without RoPE columns)
  float* part;                // gradient: [ctas][d_norm] partial sums of dw
  int T, d, d_norm, d_rope;
  int w_f32;                  // weights are float32, not bf16
  float eps;
  dsa_rope_freqs table;
};
constexpr int kNormMaxCtas = 304;   // of a gradient call; also what its workspace is sized for

struct AppendArgs {
  const uint16_t* c_kv;       // [T, 512] bf16, row stride c_stride
  const uint16_t* k_pe;       // [T, d_rope] bf16, row stride pe_stride
  const int32_t* positions;   // [T], -1 = padding token
  const int32_t* token_req;   // [T] or null: token t is request t's
  const int32_t* block_table; // [num_req, max_blocks]
  void* cache;                // bf16 rows [N, ld_kv] or FP8 rows [N, 528 + 2 d_rope]
  unsigned int* err;
  int64_t c_stride, pe_stride;
  int T, d_rope, num_req, max_blocks, block_size, N, ld_kv;
  int rotate;                 // 0: the RoPE columns are stored as they are
  dsa_rope_freqs table;
};

// Bytes that the 64-head decode form fetches to L2 of a run of `rows` cache rows: from the
// first row to the end of what is read of the last, in one piece, what lies between the
// rows included, so only where that is little (64 x 19456 at 64 heads, rows of 1152
// bytes: a pitch of 1280 278 us, 288 unfetched; of 1408 295 and 289; of 2304 429 and
// 289; row by row 312 at any of them).  0: nothing is fetched.
inline int decode_fetch_bytes(int rows, int64_t row_bytes, int read_bytes) {
  return 8 * (row_bytes - read_bytes) <= read_bytes ? (rows - 1) * (int)row_bytes + read_bytes : 0;
}

struct DecodeArgs {
  CUtensorMap tmap_kv;        // cache rows, 64-column (or 128-byte) x 1-row box (pair form over FP8 rows: 16 bytes x
                              // box_rows, unswizzled, unset when box_rows = 0)
  CUtensorMap tmap_box;       // cache rows, 64-column x box_rows box (unset when box_rows = 0)
  CUtensorMap tmap_box8;      // the same with 8 rows (pair form; over FP8 rows: 64 bytes x box_rows, unswizzled)
  CUtensorMap tmap_q;         // q viewed [B*H, d_qk], 64-column x HB-row box
  const uint8_t* rows_base;   // the cache rows as bytes, and their pitch
  int row_bytes;
  int box_rows;               // rows that a page holds in one run: 8 .. 128, a power of two; 0 = gather rows
  int fetch_bytes;            // fetched to L2 of each run by the 64-head form and by pairs (decode_fetch_bytes)
  const int32_t* block_table; // [B, max_blocks]
  const int32_t* kv_lens;     // [B]
  const int32_t* idx;         // [B, ld] positions, or null: every position < kv_len
  uint16_t* out;              // [B, H, 512] bf16
  float* lse;                 // [B, H]
  int4* borders;              // [1 + groups]: tiles, ranges and blank tiles, then where each range ends
  float* part_o;              // [2 groups][heads padded][512] normalised partial outputs
  float* part_lse;            // [2 groups][heads padded] their log-sum-exp, base 2
  unsigned int* err;
  // tree form: [B, n] mask words, [B] drafted tokens or null (n of every request); H is then
  // the query rows of a request, n * heads
  const uint64_t* tree_mask;
  const int32_t* num_draft;
  int n, heads;
  int B, H, N, k, ld, max_blocks, block_size;
  int cap;                    // positions that the block table has room for
  int groups;                 // CTA groups (each of head_blocks CTAs)
  int head_blocks;            // CTAs of a group, each with its own heads
  float scale;
  TraceArgs tr;
};

struct KeyMaskArgs {
  const int32_t* idx;   // [T, ld] global rows
  uint32_t* key_mask;   // [T, words]
  unsigned int* err;
  int T, k, ld, words;
  ReqTable req;
};

struct ConvertArgs {
  const int32_t* idx_local;    // [T, ld] request-local positions
  int32_t* idx_global;         // [T, ld] physical rows (may alias idx_local)
  const int32_t* block_table;  // [num_req, max_blocks] physical block ids
  unsigned int* err;
  int T, k, ld, max_blocks, block_size, N;
  int vec;                     // 16-byte row accesses (ld % 4 == 0, aligned pointers)
  ReqTable req;                // cu_q: token offsets; cu_kv: cumulative KV lengths
};

struct GroupedArgs {
  CUtensorMap tmap_kv;      // kv rows for tile::gather4 (box 64 columns x 1 row, 128B swizzle)
  CUtensorMap tmap_q;       // q viewed [T*H, d_qk], box 64 columns x 64 rows
  CUtensorMap tmap_kv_blk;  // kv rows, box 64 columns x 64 rows (contiguous runs of the union)
  const uint16_t* q;
  const uint16_t* kv;
  const int32_t* union_idx;
  const int32_t* union_len;
  const uint8_t* mask;
  uint16_t* out;
  float* lse;
  unsigned int* err;
  int T, H, G, d_qk, N, ld_kv, union_pad, num_groups;
  float scale;
  ReqTable req;
  TraceArgs tr;
};

struct MaskedArgs {
  CUtensorMap tmap_q;   // q [T, H, d_qk] (strided): box 64 columns x 1 head x 128 rows
  CUtensorMap tmap_k;   // k [Nk, H, 64 * k_chunks] (strided): same box
  CUtensorMap tmap_v;   // v [Nk, H, d_v] (strided): box 64 columns x 1 head x (128 or 64) rows
  CUtensorMap tmap_kpe; // shared RoPE columns [Nk, d_qk - 64 * k_chunks]: box 64 columns x 128 rows
  int k_chunks;         // 64-column chunks of each key row read from tmap_k (the rest from tmap_kpe)
  const uint32_t* key_mask;  // [T, words]
  uint16_t* out;        // [T, H, d_v]
  float* lse;           // [T, H]
  unsigned int* err;
  int T, H, d_qk, d_v, words, num_qtiles;
  float scale;
  ReqTable req;         // cu_g = query-tile offsets per request
  TraceArgs tr;
};

// Shared memory of the union builder: bitmap and prefix (W words each, W
// rounded up to a multiple of 4 so the mask staging stays 16-byte aligned)
// plus one mask byte per union slot.
inline int union_build_smem_bytes(int N, int union_pad) {
  const int W = (N + 31) / 32;
  const int Wp = (W + 3) & ~3;
  return 8 * Wp + union_pad;
}

// The byte-map variant: one membership byte per KV position (32 Wp bytes),
// the union words and their prefix (Wp words each); used when it needs at
// most kUnionBytemapMaxSmem bytes (two or more CTAs per SM).
constexpr int kUnionBytemapMaxSmem = 96 * 1024;
inline int64_t union_build_bytemap_smem_bytes(int N) {
  const int64_t W = (N + 31) / 32;
  const int64_t Wp = (W + 3) & ~3;
  return 40 * Wp;
}

// Each returns 0 on success, -1 on a CUDA launch error, -2 if the shape has
// no kernel instance.
int launch_sparse_prefill(const SparseArgs& a, int num_sms, cudaStream_t stream);
int launch_sparse_prefill_fp8(const SparseArgs& a, int num_sms, cudaStream_t stream);
int launch_union_build(const UnionArgs& a, cudaStream_t stream);

int launch_topk_to_key_mask(const KeyMaskArgs& a, cudaStream_t stream);
int launch_local_to_global(const ConvertArgs& a, cudaStream_t stream);
int launch_grouped_prefill(const GroupedArgs& a, int num_sms, cudaStream_t stream);
int launch_masked_mha(const MaskedArgs& a, int num_sms, cudaStream_t stream);
int launch_wait_timeout(unsigned int* err, cudaStream_t stream);
int launch_kv_fp8(const Fp8KvArgs& a, bool quantize, int num_sms, cudaStream_t stream);
int launch_rope(RopeArgs& a, bool f32, bool vec, int num_sms, cudaStream_t stream);
int launch_norm_rope(NormArgs& a, bool f32, bool vec, bool gradient, int num_sms, cudaStream_t stream);
int launch_kv_append(const AppendArgs& a, bool fp8, cudaStream_t stream);

// Heads per CTA of the decode kernel and the CTAs its heads take.  (FP8 rows: the
// units they are converted into leave no room for more than 32 heads' q and P.)
inline int decode_heads_per_cta(int H, bool fp8) { return H <= 16 ? 16 : (H <= 32 || fp8 ? 32 : 64); }
constexpr int kDecodeMaxCtas = 152;   // one per SM; also what the workspace is sized for

// How a decode or tree call is cut: query rows of a block (the CTAs that walk the same keys),
// keys of a tile, CTAs of a block.  Many rows of a tree are blocks of 128 to a CTA pair
// (tree_pair.cu), fewer as many heads would be.  In us, one CTA against a pair, for 32 requests of
// 512..16384 keys, one of 777 and one of 131072 (bf16 from 48 rows on: with the CTA of 64 rows
// that trees had before the pairs):
//   bf16  32 rows  52 : 55   17 : 17   51 : 50      FP8  32 rows  56 : 82   16 : 22   56 : 71
//         48       69 : 56   22 : 18                     48       92 : 82   16 : 23   84 : 73
//         64       71 : 57   22 : 19                     64       92 : 82   16 : 24   85 : 74
//         80       92 : 57   24 : 19                     80      128 : 83   18 : 24  114 : 74
//                                                        128     164 : 83   18 : 24  140 : 74
// FP8 calls of 33 to 64 rows are the ones where neither is ahead everywhere: rows alone decide
// because lengths are on the device, where the host cannot look, and the short call, whose time
// is all latency, would lose half of itself where the long ones gain an eighth.
struct DecodeForm {
  int rows, keys, ctas;
};
inline DecodeForm decode_form(int H, bool fp8, bool tree) {
  if (tree && H > (fp8 ? 64 : 32)) return {128, 256, 2};
  return {decode_heads_per_cta(H, fp8), 128, 1};
}
// max_tiles: an upper bound of a request's key tiles (1: nothing is split).
int launch_paged_decode(DecodeArgs& a, bool fp8, int d_rope, int max_tiles, cudaStream_t stream);
int launch_tree_decode(DecodeArgs& a, bool fp8, int d_rope, int max_tiles, cudaStream_t stream);
int launch_tree_pair(DecodeArgs& a, bool fp8, int d_rope, int max_tiles, cudaStream_t stream);

// Rows that move in the caches of one or more layers (kv_keep.cu).
struct KeepArgs {
  void* caches[DSA_MAX_CACHES];
  const int32_t* block_table;   // [B, max_blocks]
  const int32_t* kv_lens;       // [B]
  const int32_t* num_draft;     // [B] or null: n of every request
  const int32_t* keep;          // [B, m], ascending, -1 ends
  int32_t* new_lens;            // [B]
  unsigned int* err;
  int B, m, n, N, max_blocks, block_size;
  int row_pieces;               // 16-byte pieces of a row
};
int launch_kv_keep(const KeepArgs& a, int num_caches, cudaStream_t stream);

// dsa_sparse_prefill with the streamed-call fields of SparseArgs (ready, done,
// done_blk; all null / 0 for an ordinary call).  Same checks and DSA_* status
// as dsa_sparse_prefill.
int sparse_prefill_streamed(const uint16_t* q, const uint16_t* kv, int N, int ld_kv, const int32_t* idx, int T,
                            int H, int d_qk, int d_v, int k, int ld, float scale, uint16_t* out, float* lse,
                            const uint32_t* ready, uint32_t* done, int done_blk, cudaStream_t stream);

}  // namespace dsa
