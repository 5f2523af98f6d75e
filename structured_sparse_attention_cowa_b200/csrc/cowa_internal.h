// cowa_internal.h -- declarations shared by the C-ABI layer and the kernel files.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/cowa.h"
#include "cowa_pattern.h"

namespace cowa {

// Every workspace starts with a 256-byte header whose first word is the device
// status (0 = ok, bit 0 = a bounded wait ran out).  Kernel data follows.
constexpr size_t kWsHeader = 256;
// What the paged calls write to word 3 of the workspace for a bad page.  (A value of its own: the other
// calls never needed that word cleared, and it may hold anything in their workspaces.)
constexpr uint32_t kPageFlag = 0x50414745u;

// A runtime call's result as a status.  A failed call is also kept as the thread's last error, which the check
// after the next launch would take for its own: it is cleared.
inline cowa_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return COWA_OK;
  cudaGetLastError();
  return COWA_ERR_CUDA;
}

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Encode a 4-D bf16 tensor map over (d, t, h, b) with a box of (64, box_rows, 1, 1)
// and 128-byte swizzle.  Returns false if the driver rejects it.
bool make_tmap_bf16(CUtensorMap* map, const void* base, int d, int n_t, int n_h, int n_b, int64_t stride_t,
                    int64_t stride_h, int64_t stride_b, int box_rows);

// ---- decode ----
// Compacted per-head decode cache: only what decode can see, rows of d bf16 per (b, KV head):
//   sink      rows [0, S64)           position p < S at row p
//   band ring rows [S64, S64 + R)     position p at row S64 + (p mod R); R = round64(L) + 64
//   interval  rows [IB, IB + W)       position p of the head's interval [lo, hi) at row
//                                     IB + p - round_down64(lo); IB = S64 + R
// Every 64-aligned block of positions maps to 64 consecutive rows of one region.
struct CompactGeom {
  int S64, R, IB, W, rows;
};
CompactGeom compact_geom(const Pat& p);

struct DecodeArgs {
  Pat pat;
  int B, Hq, Hkv, d, T_cap;
  const void* q_t;
  const int32_t* pos;
  void* o;
  float* lse;        // may be null
  float* partials;   // [B, Hq, n_split, d + 2]
  uint32_t* status;
  int chunk;         // tokens per split
  int n_split;
  float scale_log2;  // softmax scale * log2(e)
  // compacted cache (tm_k / tm_v over [B, H_kv, rows, d]): 0 = full cache indexed by position
  int compact;
  CompactGeom cg;
  // E4M3 cache (tm_k / tm_v over uint8 codes): scale_log2 then includes k_scale, and the
  // partial outputs are multiplied by v_scale
  int kv8;
  float v_scale;
  CUtensorMap tm_k, tm_v;
};
int decode_chunk_tokens(const Pat& p, int B, int Hkv, int T_cap);
int decode_num_splits(const Pat& p, int T_cap, int chunk, bool compact = false);
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_quantize_e4m3(const void* x, void* q, int64_t n, float inv_scale, cudaStream_t s);
cudaError_t launch_compact_append(const Pat& p, int B, int Hkv, int d, const void* k_new, const void* v_new,
                                  const int32_t* pos, void* kc, void* vc, cudaStream_t s);
cudaError_t launch_compact_build(const Pat& p, int B, int N, int Hkv, int d, const void* k, int64_t ksb, int64_t kst,
                                 int64_t ksh, const void* v, int64_t vsb, int64_t vst, int64_t vsh, void* kc, void* vc,
                                 cudaStream_t s);

// ---- paged cache ----
// Entry (b, g, i): the page that holds positions [i * page_size, (i + 1) * page_size) of sequence b
// (and KV head g); per head tables have sh > 0 and pages of one head, shared ones sh = 0.
struct PageTab {
  const int32_t* ptr;
  int64_t sb, sh;
  int max_pages, page_size, n_pages, n_seq;
};
constexpr int kPagedIv = 64;  // heads whose intervals travel with the arguments
struct PagedDecodeArgs {
  Pat pat;
  Range iv[kPagedIv];  // interval_of each KV head (more than kPagedIv heads: worked out on the device)
  int B, Hkv, grp;   // grp: query heads per KV head
  PageTab tab;
  const void* q_t;
  const int32_t* pos;
  void* o;
  float* lse;        // may be null
  uint32_t* status;  // word 3: a visible page's entry was outside the pool
  // [pairs] (by_pair) or [grid], whichever is less: {pair, first CTA, last CTA} of the (b, g), or of the one
  // that begins in the CTA and does not end there; x = -1: nothing to join
  int4* rec;
  int by_pair;
  float* part;       // [2 grid][grp][d + 2] fp32 partials: m, l, o
  float scale_log2, v_scale;
  int grid, cluster; // see paged_decode_plan
  int box_rows;      // rows per TMA box: the largest power of two up to 64 that divides the page size
  int page_shift;    // log2 of the page size, -1 if it is not a power of two
  CUtensorMap tm_k, tm_v;
};
struct PagedPlan {
  int grid, cluster;
};
PagedPlan paged_decode_plan(const Pat& p, int B, int Hq, int Hkv, int d, bool kv8, int max_pages, int page_size);
size_t paged_decode_bytes(int grid, int grp, int d);
cudaError_t launch_paged_decode(const PagedDecodeArgs& a, int d, bool kv8, cudaStream_t s);

// ---- rotary positions, and the write of tokens into a paged cache ----
struct RopeArgs {
  const float* inv_freq;           // [half]
  int half;                        // pairs; 2 * half elements of a head are rotated
  int end0, end1, end2;            // first pair of axes 1, 2, 3
  int interleaved;
  float scale, sin_scale;          // factors of cos and sin (the backward pass negates the second)
  const int32_t* pos;              // position of token t of batch b on an axis; null: t (append: cache_pos)
  int64_t pos_sa, pos_sb;
  long long M;                     // tokens
  int N;                           // per batch element
  int d, Hq, Hk;
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_sb, q_st, q_sh, k_sb, k_st, k_sh, v_st, v_sh;
  __nv_bfloat16 *qo, *ko;
  int64_t qo_sb, qo_st, qo_sh, ko_sb, ko_st, ko_sh;
  // append
  const int32_t* cache_pos;
  const int32_t* seq;              // null: token i belongs to sequence i
  PageTab tab;
  void *kp, *vp;
  int64_t kp_sp, kp_st, kp_sh, vp_sp, vp_st, vp_sh;
  float inv_k, inv_v;              // E4M3: reciprocals of the scales
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);
cudaError_t launch_paged_append(const RopeArgs& a, bool e4m3, cudaStream_t s);

// ---- forward ----
struct FwdArgs {
  Pat pat;
  int B, Hq, Hkv, d;
  int Nq, Nk, q_off;  // query rows q_off .. q_off+Nq-1 (absolute positions) against keys 0 .. Nk-1
  // packed variable-length batch (varlen != 0): sequence s holds rows cu_seqlens[s] ..
  // cu_seqlens[s+1]-1 of q, k, v, o (B = 1) at positions 0..; seq_tab is the sequence table
  // of kernel_common.cuh (tile offsets, first rows, lengths), written first on the device
  int varlen, n_seq, total;
  const int32_t* cu_seqlens;
  int32_t* seq_tab;
  // paged != 0 (a packed batch): keys and values in pages (tm_k, tm_v over the pools), sequence s's
  // query rows at positions q_start[s]..
  int paged, box_rows;
  // parts > 1: each CTA's key tiles are cut into so many parts, whose results go to part_ml (running max
  // in log2 units and sum, [parts][Hq][total]) and part_o ([parts][Hq][total][d])
  int parts;
  int solo;  // != 0: a CTA takes one query head, not two
  float2* part_ml;
  float* part_o;
  PageTab tab;
  Range iv[kPagedIv];  // interval_of each KV head (more than kPagedIv heads: worked out on the device)
  const int32_t* q_start;
  void* o;
  int64_t o_sb, o_st, o_sh;
  float* lse;
  uint32_t* status;
  float scale_log2;
  CUtensorMap tm_q, tm_k, tm_v;
};
cudaError_t launch_fwd(const FwdArgs& a, cudaStream_t s);
struct FwdCut {
  int parts, solo;
};
FwdCut fwd_paged_cut(const Pat& p, int n_seq, int total, int Hq, int Hkv, int d, int max_pages, int page_size);
size_t fwd_paged_bytes(int parts, int total, int Hq, int d);

// ---- packed variable-length batches ----
// Bytes of the sequence table (3 n_seq + 1 int32, 256-aligned) and the kernel that writes it
// from cu_seqlens (device int32 [n_seq + 1]).
inline size_t seq_table_bytes(int n_seq) { return align_up((size_t)(3 * n_seq + 1) * sizeof(int32_t), 256); }
cudaError_t launch_seq_table(const int32_t* cu_seqlens, int n_seq, int total, int32_t* tab, cudaStream_t s);
// upper bound on the 128-row tiles of a packed batch: sum of ceil(len / 128) <= total / 128 + n_seq
__host__ __device__ inline long long packed_tiles_bound(int total, int n_seq) { return (long long)total / 128 + n_seq; }

// ---- backward ----
struct BwdArgs {
  Pat pat;
  int B, N, Hq, Hkv, d;
  // packed variable-length batch (varlen != 0, B = 1): the sequences of seq_tab (see
  // kernel_common.cuh) on a token axis of `total` rows; N is then unused
  int varlen, n_seq, total;
  int32_t* seq_tab;
  int lse_ld;        // row stride of lse: N ([B, Hq, N]) or total (packed: [Hq, total])
  const void* o; int64_t o_sb, o_st, o_sh;
  const void* dO; int64_t do_sb, do_st, do_sh;
  const float* lse;
  void* dq; int64_t dq_sb, dq_st, dq_sh;
  void* dk; int64_t dk_sb, dk_st, dk_sh;
  void* dv; int64_t dv_sb, dv_st, dv_sh;
  float* delta;      // [B, Hq, N_pad] fp32 workspace: rowsum(dO * O), 0 on padded rows
  float* lse2;       // [B, Hq, N_pad] fp32 workspace: lse * log2(e), +inf on padded rows
  int N_pad;         // N rounded up to a whole number of 128-row tiles (packed: 128 x the
                     // tile bound, each sequence's rows starting at its own tile)
  uint32_t* status;
  float scale;       // softmax scale
  float scale_log2;  // softmax scale * log2(e)
  // Query-range split of long dK/dV key tiles (kv_chunk > 0; see kv_split_plan): the grid
  // starts with n_split CTAs, one per chunk kv_tab[e] = {key tile, KV head, batch, chunk} of
  // kv_chunk query tiles; each writes fp32 partial dV, dK ([2][128][d]) to kv_part + e*2*128*d,
  // and a reduction kernel sums a tile's chunks in chunk order.  The unsplit CTA of such a tile
  // leaves at once.  Packed batches do not split (kv_chunk = 0).
  // A packed batch plans its split on the device (the host cannot see the lengths): n_split is
  // then a capacity, unused table slots hold chunk -1, and kv_flag[g * kv_bound + packed tile]
  // says which key tiles were split (a tile that does not fit the capacity stays whole).
  int kv_chunk, n_split;
  int4* kv_tab;
  float* kv_part;
  int32_t* kv_flag;
  int kv_bound;
  CUtensorMap tm_q, tm_k, tm_v, tm_do;
};
struct KvSplit {
  int chunk;             // query tiles per chunk; 0: no key tile is split
  long long n_entries;   // chunks over all split key tiles and batch elements
};
KvSplit kv_split_plan(const Pat& p, int B, int N, int Hq, int Hkv);
// workspace after the header: Delta, lse2, then (split calls) the chunk table and partials
size_t bwd_workspace_bytes(const Pat& p, int B, int N, int Hq, int Hkv, int d);
cudaError_t launch_bwd(const BwdArgs& a, int stages, cudaStream_t s);

// ---- bounded-wait probe ----
cudaError_t launch_wait_timeout_probe(uint32_t* status, unsigned long long limit_ns, cudaStream_t s);

// ---- planner debug kernel ----
cudaError_t launch_plan_debug(const Pat& p, int Hkv, int N, int BM, int BN, int32_t* dev_out, size_t cap,
                              unsigned long long* dev_count, cudaStream_t s);

}  // namespace cowa
