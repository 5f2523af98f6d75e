// cowa_fwd.cu -- CoWA forward on sm_100a: exact softmax attention over the position-defined
// visible set of each KV head ("CoWindow Attention: Full Causal Coverage Is a Collective
// Property", Abstract; skillfed.io news summary, paragraphs 2 and 7).
//
// One CTA = (batch b, KV head g, 128-row query tile i, a pair of query heads of g's GQA
// group).  The two heads share every K/V tile the CTA loads and the same tile plan, because
// the mask depends on g only.  Warp roles (12 warps = 3 warpgroups):
//   warps 0-3  softmax for head slot 0 (thread = query row = TMEM lane)
//   warps 4-7  softmax for head slot 1
//   warp  8    TMA producer: Q once, then K_j, V_j of every visited KV tile into a 5-slot ring
//   warp  9    tcgen05 MMA issuer (the whole warp walks the loop, one elected lane issues):
//              S = Q K^T into TMEM, O += P V into TMEM
//   warps 10-11 idle (they complete the third warpgroup)
// The same kernel serves a block of queries at an offset against keys already written
// (chunked prefill: query rows q_off.., keys 0..Nk-1) and packed variable-length batches (each
// CTA finds its sequence in per-sequence tile offsets and works on that sequence's rows).
// PAGED: a packed batch of query chunks against a paged cache.  The K/V tiles keep their places
// (128 positions each); the producer warp looks up the pages of a tile, one lane per TMA box of 8 to
// 128 rows, and fetches the boxes that some row of the query tile sees.  V rows that are not fetched,
// or lie past the last key, are zeroed (their P is 0, but 0 times what memory holds may be NaN).  The
// CTAs come heaviest first over all sequences (see find_chunk), and those with a single head, of an
// odd group, last.  Where there are too few CTAs for the GPU (a short chunk behind a long prefix), a CTA
// takes one head instead of two (a.solo), or several share the key tiles of one (a.parts) and leave fp32
// results that a second kernel joins.
// Registers: the kernel is compiled for 168 per thread (384 * 168 = 64512 at launch); the two
// softmax warpgroups then raise theirs to 216 and the third lowers to 72
// (2*128*216 + 128*72 = 64512), so a whole 128-column score row stays in registers.  The
// launcher checks the compiled count before the first launch, because a split larger than
// the launch allocation would wait forever.
// The visited KV tiles come from the planner (sink tiles, interval_g tiles, near-diagonal
// band, merged); only tiles that are not entirely visible apply the element mask.
//
// Softmax: online, in the log2 domain, with a lazy rescale of O (only when the running max
// grows by more than 2^8; the final division uses the same stale max, so the result is
// exact).  P is rounded to bf16 and written back into TMEM over the S columns it came from,
// where the P V MMA reads it as its A operand (no shared-memory round trip).  fp32
// accumulation throughout.  Exponentials run on the special-function unit (an FMA-pipe
// polynomial share measured slower on B200 here).  Each tile's exponentials use the running
// max from before the tile while the tile's own max is gathered in the same pass; the tile is
// redone only when that max grows the running one past the rescale threshold, so the common
// path never waits for a row reduction and gives the same bits as max-first.
//
// MMA order per KV tile n: S0(n), PV1(n-1), S1(n), PV0(n).  Softmax 0 works on S0(n) while
// the tensor core runs PV1(n-1) and S1(n), softmax 1 on S1(n) during PV0(n) and S0(n+1).
// tcgen05 MMAs of one thread execute in issue order, so S_k(n+1) overwriting P_k(n) is safe
// once PV_k(n) is issued, and the commit that announces S_k(n) also covers PV_k(n-1).
//
// TMEM (512 columns): S0/P0 [0,128), S1/P1 [128,256), O0 [256, 256+D), O1 [256+D, 256+2D).
#include <cuda_bf16.h>
#include <math.h>

#include "cowa_internal.h"
#include "kernel_common.cuh"
#include "sm100_ptx.cuh"

namespace cowa {
namespace {

constexpr int kBM = kTile, kBN = kTile;
constexpr int kFwdThreads = 384;
constexpr int kRegsLaunch = 168, kRegsSoftmax = 216, kRegsOther = 72;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsOther == kFwdThreads * kRegsLaunch,
              "register split must add up to the launch allocation");
constexpr int kRingMax = 8;
constexpr int kProducerWarp = 8, kMmaWarp = 9;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

template <int D>
struct FwdGeom {
  static constexpr int kQBytes = kBM * D * 2;   // one head's Q tile
  static constexpr int kKVBytes = kBN * D * 2;  // one K or V tile
  // K/V ring depth: a K or V tile takes ~5000 cycles to arrive from L2 under full load, so
  // each slot must be refilled about two tile periods ahead (5 x 32 KB for d = 128)
  static constexpr int kRing = D == 128 ? 5 : kRingMax;
  static constexpr int kOffQ = 0;
  static constexpr int kOffRing = 2 * kQBytes;
  static constexpr int kSmem = kOffRing + kRing * kKVBytes + 1024;  // + alignment slack
  static_assert(kRing <= kRingMax && kSmem <= 227 * 1024, "shared memory budget");
  static constexpr int kColO = 256;
};

// PAGED: what CTA `rank` (of all parts of a tile) works on; one warp.  Pairs of heads come before the single
// heads of odd groups, which are half as much work (a.solo: there are single heads only).
//   * Where all CTAs run at once (148 of them or fewer), or with more than 64 sequences: tile by tile of one
//     sequence after the other.
//   * Up to 64 (KV head, sequence)s: the (head, query tile)s in descending order of their keys, counted in
//     tiles.  A tile that begins at position t has about min(t, L) + clamp(t - L - lo, 0, hi - lo) of them
//     besides the sinks, so those of one head and sequence with x tiles or more are the ones that begin at
//     tile x (x up to the band's width) or x + lo (beyond it).  The x of a rank is found by a binary search,
//     with up to two (head, sequence)s in a lane's registers.  Against the next form: six ragged chunks (40/8
//     heads, L = 2048, interval 4080) 303 -> 264 us, two behind 7K keys (56/8 heads, 1150 rows) 151 -> 121, 4K
//     rows behind 28K keys 503 -> 473; three behind 6K with L = 4096, where positions say as much, 439 -> 444.
//   * Up to 64 sequences: the tiles in descending order of their positions, all heads of a tile together (the
//     same search, with sequences instead).
// The offsets are clamped as in the sequence table of kernel_common.cuh.
struct Chunk {
  int seq, tile, row0, len, start;  // seq -1: there is no work left
  int g, head, two;                 // the first query head within the group, and whether there is a second
};
constexpr int kSorted = 64;
static_assert(kSorted <= kPagedIv, "the search takes the intervals from the arguments");
__device__ __forceinline__ Chunk find_chunk(const FwdArgs& a, int rank) {
  constexpr unsigned kAll = 0xffffffffu;
  const Chunk none{-1, 0, 0, 0, 0, 0, 0, 0};
  const int lane = threadIdx.x & 31, cap = a.tab.max_pages * a.tab.page_size;
  const int grp = a.Hq / a.Hkv, pairs = a.solo ? 0 : grp >> 1, singles = grp - 2 * pairs;
  struct Seq {
    int row0, len, start, tiles;
  };
  int end = imin(imax(a.cu_seqlens[0], 0), a.total);  // of the sequences before
  auto load = [&](int first) {  // sequences first .. first + 31, one per lane
    const int s = first + lane;
    int e = s < a.n_seq ? a.cu_seqlens[s + 1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, e, o);
      if (lane >= o) e = imax(e, y);
    }
    e = imin(imax(e, end), a.total);
    const int before = __shfl_up_sync(kAll, e, 1);
    Seq q;
    q.row0 = lane == 0 ? end : before;
    q.len = e - q.row0;
    q.start = s < a.n_seq ? imax(0, imin(a.q_start[s], cap - q.len)) : 0;
    q.tiles = (q.len + kBM - 1) / kBM;
    end = __shfl_sync(kAll, e, 31);
    return q;
  };
  int g, head;
  bool two;
  auto take_heads = [&](int n) -> bool {  // n: (KV head, tile)s; false: past the last work
    two = rank < n * pairs;
    if (two) {
      head = 2 * (rank % pairs);
      rank /= pairs;
      return true;
    }
    rank -= n * pairs;
    if (rank >= n * singles) return false;
    head = 2 * pairs + rank % singles;
    rank /= singles;
    return true;
  };
  auto sum = [&](int x) { return (int)__reduce_add_sync(kAll, (unsigned)x); };
  // the lane of x's running sum over the lanes that holds place n (n < the sum), n then counting from its own
  auto lane_of = [&](int x, int& n) {
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += y;
    }
    const int l = __ffs(__ballot_sync(kAll, incl > n)) - 1;
    n -= __shfl_sync(kAll, incl - x, l);
    return l;
  };
  auto hand = [&](const Seq& q, int l, int first, int tile) {
    return Chunk{first + l, tile, __shfl_sync(kAll, q.row0, l), __shfl_sync(kAll, q.len, l), __shfl_sync(kAll, q.start, l), g,
                 head, two};
  };
  if (gridDim.x > 148 && a.n_seq <= kSorted) {
    const Seq q0 = load(0);
    Seq q1 = {0, 0, 0, 0};
    if (a.n_seq > 32) q1 = load(32);
    if (!take_heads(a.Hkv * (sum(q0.tiles) + sum(q1.tiles)))) return none;
    const bool by_head = a.n_seq * (int64_t)a.Hkv <= kSorted;
    int band = 1 << 29, wide = 0;  // (all tiles in the band: their positions decide)
    if (by_head) {
      const Range iv = a.iv[0];
      band = (a.pat.L - 1) / kBM + 1;
      wide = (iv.hi - iv.lo) / kBM + 1;
    } else {
      g = rank % a.Hkv;
      rank /= a.Hkv;
    }
    // item i = 32 j + lane: head i / n_seq (by_head) and sequence i % n_seq; its tiles [k, k + n), and the
    // tile its interval begins in
    int k[2], n[2], lo[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = 32 * j + lane, h = i / a.n_seq, s = i - h * a.n_seq;
      const int s0 = __shfl_sync(kAll, q0.start, s & 31), t0 = __shfl_sync(kAll, q0.tiles, s & 31);
      const int s1 = __shfl_sync(kAll, q1.start, s & 31), t1 = __shfl_sync(kAll, q1.tiles, s & 31);
      k[j] = (s < 32 ? s0 : s1) / kBM;
      n[j] = h < (by_head ? a.Hkv : 1) ? (s < 32 ? t0 : t1) : 0;
      lo[j] = by_head && h < a.Hkv ? a.iv[h].lo / kBM : 0;
    }
    // tiles of an item with x tiles of keys or more
    auto with = [&](int j, int x) {
      return x - band > wide ? 0 : imax(0, imin(n[j], k[j] + n[j] - x - (x > band ? lo[j] : 0)));
    };
    auto all_with = [&](int x) { return sum(with(0, x) + with(1, x)); };
    int x = 0, hi = imin(band + wide, (int)__reduce_max_sync(kAll, (unsigned)imax(k[0] + n[0], k[1] + n[1])));
    while (x < hi) {  // the last x with more than `rank` tiles
      const int mid = (x + hi + 1) >> 1;
      if (all_with(mid) > rank) x = mid; else hi = mid - 1;
    }
    int nth = rank - all_with(x + 1);
    const int more0 = with(0, x + 1), more1 = with(1, x + 1), m0 = with(0, x) - more0, m1 = with(1, x) - more1, in0 = sum(m0);
    const bool second = nth >= in0;
    if (second) nth -= in0;
    const int l = lane_of(second ? m1 : m0, nth), i = (second ? 32 : 0) + l, h = i / a.n_seq, s = i - h * a.n_seq;
    if (by_head) g = h;
    const int tile = __shfl_sync(kAll, second ? n[1] - more1 : n[0] - more0, l) - 1 - nth;
    return s < 32 ? hand(q0, s, 0, tile) : hand(q1, s - 32, 32, tile);
  }
  if (!take_heads((int)packed_tiles_bound(a.total, a.n_seq) * a.Hkv)) return none;
  g = rank % a.Hkv;
  rank /= a.Hkv;
  for (int first = 0; first < a.n_seq; first += 32) {
    const Seq q = load(first);
    const int in = sum(q.tiles);
    if (rank < in) {
      const int l = lane_of(q.tiles, rank);
      return hand(q, l, first, __shfl_sync(kAll, q.tiles, l) - 1 - rank);
    }
    rank -= in;
  }
  return none;
}

// Part `part` of `parts` of a tile list, in order (parts differ by at most one tile; some may be empty).
__device__ __forceinline__ Tiles part_of(const Tiles& all, int part, int parts) {
  if (parts == 1) return all;
  const int first = (int)((int64_t)all.count * part / parts), last = (int)((int64_t)all.count * (part + 1) / parts);
  Range r[3];
  int before = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int len = all.r[i].hi - all.r[i].lo;
    const int lo = imax(first - before, 0), hi = imin(last - before, len);
    r[i] = hi > lo ? Range{all.r[i].lo + lo, all.r[i].lo + hi} : Range{0, 0};
    before += len;
  }
  Tiles T;
  T.n = merge3(r[0], r[1], r[2], T.r);
  T.count = (T.r[0].hi - T.r[0].lo) + (T.r[1].hi - T.r[1].lo) + (T.r[2].hi - T.r[2].lo);
  return T;
}

// bits lo .. hi - 1 of a word (either may lie outside it)
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  lo = imax(lo, 0);
  hi = imin(hi, 32);
  return hi > lo ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0u;
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(kFwdThreads, 1) cowa_fwd_kernel(const __grid_constant__ FwdArgs a) {
  using Geo = FwdGeom<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ __align__(8) uint64_t q_full;
  __shared__ __align__(8) uint64_t kv_full[kRingMax], kv_empty[kRingMax];
  __shared__ __align__(8) uint64_t s_full[2], p_ready[2], o_done[2];
  __shared__ __align__(8) uint64_t mma_final;
  // single-head tile (odd GQA group): softmax 1's running max and sum per row for the merge
  __shared__ __align__(8) uint64_t merge_ready;
  __shared__ float merge_m[kBM], merge_l[kBM];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  // PAGED: set when a page with a visible key is not in the pool; and the barrier on which the box
  // of V lands whose last rows still need to be zeroed
  __shared__ int bad_page;
  __shared__ __align__(8) uint64_t landed;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- work item: heaviest (last) query tiles first; all heads/pairs of one tile adjacent
  const int grp = a.Hq / a.Hkv;
  const int npair = (grp + 1) >> 1;
  const int per_i = a.B * a.Hkv * npair;
  int i, row0 = 0, Nq = a.Nq, Nk = a.Nk, q_off = a.q_off;  // row0: first row of the sequence
  int pg_seq = 0, part = 0;
  int head, g, b = 0;  // head: the first of the pair within the group
  bool has1;
  __shared__ Chunk chunk;
  if constexpr (PAGED) {
    // (set up while the kernel before it in the stream ran; waits for that one's results here)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    part = blockIdx.x % a.parts;
    if (warp == 0) {
      const Chunk c = find_chunk(a, blockIdx.x / a.parts);
      if (lane == 0) chunk = c;
    }
    __syncthreads();
    if (chunk.seq < 0) return;  // whole CTA, before any barrier or TMEM use
    pg_seq = chunk.seq;
    g = chunk.g;
    head = chunk.head;
    has1 = chunk.two;
    i = chunk.tile;
    row0 = chunk.row0;
    Nq = chunk.len;
    q_off = chunk.start;
    Nk = imin(q_off + Nq, a.tab.max_pages * a.tab.page_size);
  } else {
    if (!a.varlen) {
      i = (a.Nq + kBM - 1) / kBM - 1 - (int)(blockIdx.x / per_i);
    } else {
      // the grid is an upper bound on the q-tiles of the packed batch: find this CTA's sequence
      const int tiles = a.seq_tab[a.n_seq];
      const int tg = tiles - 1 - (int)(blockIdx.x / per_i);
      if (tg < 0) return;  // whole CTA, before any barrier or TMEM use
      const int sq = seq_of_tile(a.seq_tab, a.n_seq, tg);
      i = tg - a.seq_tab[sq];
      row0 = a.seq_tab[a.n_seq + 1 + sq];
      Nq = Nk = a.seq_tab[2 * a.n_seq + 1 + sq];
      q_off = 0;
    }
    int rem = blockIdx.x % per_i;
    head = 2 * (rem % npair); rem /= npair;
    has1 = head + 1 < grp;
    g = rem % a.Hkv;
    b = rem / a.Hkv;
  }
  int h0 = g * grp + head;
  // query rows of the tile: local q rows [i*BM, ...), absolute positions [t0, t1)
  const int t0 = q_off + i * kBM, t1 = imin(q_off + Nq, t0 + kBM);
  const Range iv = PAGED && a.Hkv <= kPagedIv ? a.iv[g] : interval_of(a.pat, g);
  // (a paged sequence longer than its cache: its last rows see the keys that there are)
  const Tiles T = PAGED ? part_of(plan_tiles(a.pat, iv, t0, imin(t1, Nk)), part, a.parts) : plan_tiles(a.pat, iv, t0, t1);

  uint8_t* sQ = smem + Geo::kOffQ;
  uint8_t* sRing = smem + Geo::kOffRing;

  if (threadIdx.x == 0) {
    ptx::mbar_init(&q_full, 1);
    for (int s = 0; s < Geo::kRing; ++s) {
      ptx::mbar_init(&kv_full[s], PAGED ? kBN / a.box_rows : 1);
      ptx::mbar_init(&kv_empty[s], 1);
    }
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(&s_full[k], 1);
      ptx::mbar_init(&p_ready[k], 4);
      ptx::mbar_init(&o_done[k], 1);
    }
    ptx::mbar_init(&mma_final, 1);
    ptx::mbar_init(&merge_ready, 4);
    if (PAGED) {
      ptx::mbar_init(&landed, 1);
      bad_page = 0;
    }
    abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&tmem_base_sh, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const int ntiles = T.count;
  if (warp >= 8) {
    // warpgroup-wide register reallocation: this warpgroup gives registers to the softmax ones
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  }
  if (warp == kProducerWarp) {
    // ------------------------------------------------------------------ TMA producer
    if constexpr (PAGED) {
      // (debug builds) the work item addresses rows and heads of the call, and a sequence of the table
      const bool q_ok = ptx::dbg_check(i >= 0 && i * kBM < Nq && row0 >= 0 && Nq <= a.total - row0 && q_off >= 0 &&
                                           h0 + (has1 ? 1 : 0) < a.Hq && pg_seq < a.n_seq && part < a.parts,
                                       a.status, &abort_flag, 0x103, i);
      if (q_ok && lane == 0) {
        ptx::tma_prefetch_desc(&a.tm_q);
        ptx::tma_prefetch_desc(&a.tm_k);
        ptx::tma_prefetch_desc(&a.tm_v);
        ptx::mbar_arrive_expect_tx(&q_full, (has1 ? 2 : 1) * Geo::kQBytes);
        for (int u = 0; u < D / 64; ++u) {
          ptx::tma_load_4d(sQ + u * 16384, &a.tm_q, &q_full, u * 64, row0 + i * kBM, h0, 0);
          if (has1) ptx::tma_load_4d(sQ + Geo::kQBytes + u * 16384, &a.tm_q, &q_full, u * 64, row0 + i * kBM, h0 + 1, 0);
        }
      }
      // Each of the first nbox lanes is the producer of one box of every tile: it looks up the box's page
      // (a tile ahead), waits for the slot, announces and issues its own copies, so that no lane waits
      // for another (a slot refilled late stalls the MMAs; with warp-wide steps in between, a 4K chunk
      // of a 32K prompt took 6% longer).  A tile is there when all nbox lanes have arrived.
      const int rows = a.box_rows, nbox = kBN / rows;
      const int32_t* table = a.tab.ptr + pg_seq * a.tab.sb + g * a.tab.sh;
      const int tl = imin(t1, Nk), gp = a.tab.sh ? 0 : g;
      const int box_bytes = rows * 128 * (D / 64);
      int issued = 0;
      if (q_ok && lane < nbox && ntiles > 0) {
        TileCursor cur;
        cur.init(T);
        // (the load is unconditional, at a clamped place: nothing waits for it before its tile's turn)
        auto look = [&](int j) { return table[imin((j * kBN + lane * rows) / a.tab.page_size, a.tab.max_pages - 1)]; };
        int next_page = look(cur.j);
        for (int n = 0; n < ntiles; ++n) {
          const int p = cur.j * kBN + lane * rows, e = imin(p + rows, tl);  // this box's positions
          const int page = next_page;
          cur.next(T);
          if (n + 1 < ntiles) next_page = look(cur.j);
          // some row of the query tile sees a key of the box
          const bool want = p < e && (p < a.pat.S || e > t0 - a.pat.L + 1 || (p < iv.hi && e > iv.lo));
          const int slot = p % a.tab.page_size;
          // (debug builds) the box lies in the cache and in its page
          const bool fits = ptx::dbg_check(!want || (p >= 0 && p / a.tab.page_size < a.tab.max_pages &&
                                                     slot + rows <= a.tab.page_size),
                                           a.status, nullptr, 0x104, p);
          const bool good = want && fits && page >= 0 && page < a.tab.n_pages;
          if (want && !good) {
            a.status[3] = kPageFlag;
            *reinterpret_cast<volatile int*>(&bad_page) = 1;
          }
          bool ok = true;
#pragma unroll
          for (int is_v = 0; is_v < 2; ++is_v) {
            const int idx = 2 * n + is_v, s = idx % Geo::kRing;
            uint8_t* dst = sRing + s * Geo::kKVBytes + lane * rows * 128;
            if (idx >= Geo::kRing &&
                !(ok = ptx::mbar_wait(&kv_empty[s], ((idx / Geo::kRing) - 1) & 1, &abort_flag, a.status)))
              break;
            // rows of V without a key must be zero: not fetched, or behind the last key of the last tile
            const int keys = is_v ? (good ? e - p : 0) : rows;
            if (good) {
              uint64_t* bar = keys < rows ? &landed : &kv_full[s];
              ptx::mbar_arrive_expect_tx(bar, box_bytes);
#pragma unroll
              for (int u = 0; u < D / 64; ++u)
                ptx::tma_load_4d(dst + u * 16384, is_v ? &a.tm_v : &a.tm_k, bar, u * 64, slot, gp, page);
            }
            if (!good || keys < rows) {
              // at most one box of a query tile ends behind its first row (the last key's)
              if (good) ok = ptx::mbar_wait(&landed, 0, nullptr, a.status);
              for (int x = keys * 8; x < rows * 8; ++x)
                for (int u = 0; u < D / 64; ++u) *reinterpret_cast<uint4*>(dst + u * 16384 + x * 16) = make_uint4(0, 0, 0, 0);
              ptx::fence_proxy_async_smem();
              ptx::mbar_arrive(&kv_full[s]);
            }
            issued = idx + 1;
          }
          if (!ok) break;
        }
      }
      __syncwarp();
      // drain: no copy may still be landing in shared memory when the CTA exits
      if (q_ok) ptx::mbar_wait(&q_full, 0, nullptr, a.status);
      for (int idx = (issued > Geo::kRing ? issued - Geo::kRing : 0); idx < issued; ++idx)
        ptx::mbar_wait(&kv_full[idx % Geo::kRing], (idx / Geo::kRing) & 1, nullptr, a.status);
    } else if (lane == 0) {
      ptx::tma_prefetch_desc(&a.tm_q);
      ptx::tma_prefetch_desc(&a.tm_k);
      ptx::tma_prefetch_desc(&a.tm_v);
      // (debug builds) the work item addresses rows and heads of the call
      const bool q_ok = ptx::dbg_check(i >= 0 && i * kBM < Nq && h0 + (has1 ? 1 : 0) < a.Hq && b < a.B, a.status,
                                       &abort_flag, 0x101, i);
      if (q_ok) {
        ptx::mbar_arrive_expect_tx(&q_full, (has1 ? 2 : 1) * Geo::kQBytes);
        for (int u = 0; u < D / 64; ++u) {
          ptx::tma_load_4d(sQ + u * 16384, &a.tm_q, &q_full, u * 64, row0 + i * kBM, h0, b);
          if (has1) ptx::tma_load_4d(sQ + Geo::kQBytes + u * 16384, &a.tm_q, &q_full, u * 64, row0 + i * kBM, h0 + 1, b);
        }
      }
      TileCursor cur;
      cur.init(T);
      int issued = 0;
      for (int idx = 0; q_ok && idx < 2 * ntiles; ++idx) {
        const int s = idx % Geo::kRing;
        if (idx >= Geo::kRing && !ptx::mbar_wait(&kv_empty[s], ((idx / Geo::kRing) - 1) & 1, &abort_flag, a.status)) break;
        // (debug builds) every planned KV tile lies inside the keys of the call
        if (!ptx::dbg_check(cur.j >= 0 && cur.j * kBN < Nk, a.status, &abort_flag, 0x102, cur.j)) break;
        const bool is_v = idx & 1;
        uint8_t* dst = sRing + s * Geo::kKVBytes;
        ptx::mbar_arrive_expect_tx(&kv_full[s], Geo::kKVBytes);
        for (int u = 0; u < D / 64; ++u)
          ptx::tma_load_4d(dst + u * 16384, is_v ? &a.tm_v : &a.tm_k, &kv_full[s], u * 64, row0 + cur.j * kBN, g, b);
        if (is_v) cur.next(T);
        issued = idx + 1;
      }
      // drain: no copy may still be landing in shared memory when the CTA exits
      if (q_ok) ptx::mbar_wait(&q_full, 0, nullptr, a.status);
      for (int idx = (issued > Geo::kRing ? issued - Geo::kRing : 0); idx < issued; ++idx)
        ptx::mbar_wait(&kv_full[idx % Geo::kRing], (idx / Geo::kRing) & 1, nullptr, a.status);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMA issuer
    // The whole warp walks the issue loop (uniform operands); one elected lane issues each
    // MMA and commit.  Descriptors are built once and advanced by constant offsets.
    constexpr uint32_t idesc_s = ptx::idesc_bf16(128, 128, false, false);
    constexpr uint32_t idesc_o = ptx::idesc_bf16(128, D, false, true);
    const uint64_t q_desc = ptx::smem_desc_sw128(ptx::smem_u32(sQ), 16, 1024);
    const uint64_t k_desc = ptx::smem_desc_sw128(ptx::smem_u32(sRing), 16, 1024);
    const uint64_t v_desc = ptx::smem_desc_sw128(ptx::smem_u32(sRing), 16384, 1024);
    const int nslot = has1 ? 2 : 1;

    auto issue_s = [&](int k, int kslot, int qk) {  // S_k = Q_qk K^T
      const uint64_t qd = ptx::desc_advance(q_desc, qk * Geo::kQBytes);
      const uint64_t kd = ptx::desc_advance(k_desc, kslot * Geo::kKVBytes);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
        ptx::mma_bf16_ss_warp(tmem + k * 128, ptx::desc_advance(qd, off), ptx::desc_advance(kd, off), idesc_s,
                              kk > 0 ? 1u : 0u);
      }
    };
    // O_k (+)= P_k V: P_k (bf16, in TMEM over the S_k columns) is the A operand
    auto issue_pv = [&](int k, int vslot, bool accumulate) {
      const uint64_t vd = ptx::desc_advance(v_desc, vslot * Geo::kKVBytes);
#pragma unroll
      for (int kk = 0; kk < kBN / 16; ++kk)
        ptx::mma_bf16_ts_warp(tmem + Geo::kColO + k * D, tmem + k * 128 + kk * 8, ptx::desc_advance(vd, kk * 2048),
                              idesc_o, (accumulate || kk > 0) ? 1u : 0u);
    };

    bool ok = ptx::mbar_wait_warp(&q_full, 0, &abort_flag, a.status);
    ptx::tc_fence_after();
    if (nslot == 1) {
      // One query head (odd group): the two softmax warpgroups take alternate KV tiles of it,
      // slot 0 the even ones and slot 1 the odd ones, each with its own running max, sum and
      // O accumulator (merged at the end), so the tensor core still alternates between two
      // softmaxes.  Iteration j: S0(2j), PV1(2j-1), S1(2j+1), PV0(2j).
      const int n0cnt = (ntiles + 1) / 2, n1cnt = ntiles / 2;
      for (int j = 0; ok && j < n0cnt; ++j) {
        const int ne = 2 * j, no = 2 * j + 1;
        const int kidx0 = 2 * ne, vidx0 = kidx0 + 1, kidx1 = 2 * no;
        if (!(ok = ptx::mbar_wait_warp(&kv_full[kidx0 % Geo::kRing], (kidx0 / Geo::kRing) & 1, &abort_flag,
                                       a.status)))
          break;
        ptx::tc_fence_after();
        issue_s(0, kidx0 % Geo::kRing, 0);
        ptx::mma_commit_warp(&s_full[0]);
        ptx::mma_commit_warp(&kv_empty[kidx0 % Geo::kRing]);
        if (j > 0) {  // PV1 of the previous odd tile 2j-1 (odd-tile index j-1)
          const int pv = 2 * (2 * j - 1) + 1;
          if (!(ok = ptx::mbar_wait_warp(&kv_full[pv % Geo::kRing], (pv / Geo::kRing) & 1, &abort_flag, a.status)))
            break;
          if (!(ok = ptx::mbar_wait_warp(&p_ready[1], (j - 1) & 1, &abort_flag, a.status))) break;
          ptx::tc_fence_after();
          issue_pv(1, pv % Geo::kRing, j - 1 > 0);
          ptx::mma_commit_warp(&kv_empty[pv % Geo::kRing]);
        }
        if (no < ntiles) {
          if (!(ok = ptx::mbar_wait_warp(&kv_full[kidx1 % Geo::kRing], (kidx1 / Geo::kRing) & 1, &abort_flag,
                                         a.status)))
            break;
          ptx::tc_fence_after();
          issue_s(1, kidx1 % Geo::kRing, 0);
          ptx::mma_commit_warp(&s_full[1]);
          ptx::mma_commit_warp(&kv_empty[kidx1 % Geo::kRing]);
        }
        if (!(ok = ptx::mbar_wait_warp(&kv_full[vidx0 % Geo::kRing], (vidx0 / Geo::kRing) & 1, &abort_flag,
                                       a.status)))
          break;
        if (!(ok = ptx::mbar_wait_warp(&p_ready[0], j & 1, &abort_flag, a.status))) break;
        ptx::tc_fence_after();
        issue_pv(0, vidx0 % Geo::kRing, j > 0);
        ptx::mma_commit_warp(&kv_empty[vidx0 % Geo::kRing]);
      }
      if (ok && ntiles > 0) {
        ptx::mma_commit_warp(&o_done[0]);
        if (ntiles % 2 == 0) {  // the last odd tile's PV1 is still to issue
          const int no = ntiles - 1, pv = 2 * no + 1;
          ok = ptx::mbar_wait_warp(&kv_full[pv % Geo::kRing], (pv / Geo::kRing) & 1, &abort_flag, a.status) &&
               ptx::mbar_wait_warp(&p_ready[1], (n1cnt - 1) & 1, &abort_flag, a.status);
          if (ok) {
            ptx::tc_fence_after();
            issue_pv(1, pv % Geo::kRing, n1cnt - 1 > 0);
            ptx::mma_commit_warp(&kv_empty[pv % Geo::kRing]);
          }
        }
        if (ok && n1cnt > 0) ptx::mma_commit_warp(&o_done[1]);
      }
    }
    for (int n = 0; ok && nslot == 2 && n < ntiles; ++n) {
      const int kidx = 2 * n, vidx = 2 * n + 1;
      const int kslot = kidx % Geo::kRing, vslot = vidx % Geo::kRing;
      if (!(ok = ptx::mbar_wait_warp(&kv_full[kslot], (kidx / Geo::kRing) & 1, &abort_flag, a.status))) break;
      ptx::tc_fence_after();
      // S0(n): P0(n-1) was consumed by PV0(n-1), issued earlier
      issue_s(0, kslot, 0);
      ptx::mma_commit_warp(&s_full[0]);
      if (nslot == 2) {
        // PV1(n-1): overlaps with softmax 0 working on S0(n)
        if (n > 0) {
          const int pv = 2 * (n - 1) + 1;
          if (!(ok = ptx::mbar_wait_warp(&p_ready[1], (n - 1) & 1, &abort_flag, a.status))) break;
          ptx::tc_fence_after();
          issue_pv(1, pv % Geo::kRing, n - 1 > 0);
          ptx::mma_commit_warp(&kv_empty[pv % Geo::kRing]);
        }
        issue_s(1, kslot, 1);
        ptx::mma_commit_warp(&s_full[1]);
      }
      ptx::mma_commit_warp(&kv_empty[kslot]);
      // PV0(n)
      if (!(ok = ptx::mbar_wait_warp(&kv_full[vslot], (vidx / Geo::kRing) & 1, &abort_flag, a.status))) break;
      if (!(ok = ptx::mbar_wait_warp(&p_ready[0], n & 1, &abort_flag, a.status))) break;
      ptx::tc_fence_after();
      issue_pv(0, vslot, n > 0);
    }
    if (ok && nslot == 2 && ntiles > 0) {
      ptx::mma_commit_warp(&o_done[0]);
      {
        const int n = ntiles - 1, pv = 2 * n + 1;
        if (ptx::mbar_wait_warp(&p_ready[1], n & 1, &abort_flag, a.status)) {
          ptx::tc_fence_after();
          issue_pv(1, pv % Geo::kRing, n > 0);
          ptx::mma_commit_warp(&kv_empty[pv % Geo::kRing]);
          ptx::mma_commit_warp(&o_done[1]);
        }
      }
    }
    // all issued MMAs complete before TMEM can be released
    ptx::mma_commit_warp(&mma_final);
    ptx::mbar_wait(&mma_final, 0, nullptr, a.status);
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------------ softmax warpgroups
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int k = warp >> 2;  // head slot
    const bool split = !has1;  // one head: the two slots take alternate KV tiles of it
    {
      const int r = (warp & 3) * 32 + lane;  // query row in the tile = TMEM lane
      const int t = t0 + r;
      const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t s_tm = lane_base + k * 128;
      const uint32_t o_tm = lane_base + Geo::kColO + k * D;
      float m_used = -INFINITY;
      const float sl2 = a.scale_log2;
      const uint64_t sl2x2 = ptx::f2_pack(sl2, sl2);
      uint64_t lsum = ptx::f2_pack(0.f, 0.f);
      bool ok = true;
      TileCursor cur;
      cur.init(T);
      int cnt = 0;  // tiles of this slot so far
      for (int n = 0; n < ntiles; ++n, cur.next(T)) {
        if (split && (n & 1) != k) continue;
        const int s0 = cur.j * kBN;
        const bool need_mask = (s0 + kBN > Nk) || !tile_full(a.pat, iv, t0, t1, s0, imin(Nk, s0 + kBN));
        if (!(ok = ptx::mbar_wait_warp(&s_full[k], cnt & 1, &abort_flag, a.status))) break;
        ptx::tc_fence_after();
        // visible key columns of row t within [s0, s0+128), relative to s0 (partial tiles only)
        const int t_end = PAGED ? imin(t + 1, Nk) : t + 1;
        const int sink_end = imin(a.pat.S, t_end) - s0;
        const int band_lo = imax(0, t - a.pat.L + 1) - s0;
        const int diag_end = t_end - s0;
        const int lr_lo = iv.lo - s0, lr_hi = imin(iv.hi, t_end) - s0;
        uint32_t xr[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) ptx::tmem_ld32(s_tm + q * 32, xr + q * 32);
        ptx::tmem_wait_ld();
        if (PAGED && need_mask) {
          // the visible columns as bits (a chunk of a few hundred rows is mostly partial tiles)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int o = 32 * w;
            const uint32_t vis = bit_range(-o, sink_end - o) | bit_range(band_lo - o, diag_end - o) |
                                 bit_range(lr_lo - o, lr_hi - o);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((vis >> c) & 1)) xr[o + c] = 0xff800000u;  // -inf: gives exactly 0
          }
        } else if (need_mask) {
#pragma unroll
          for (int c = 0; c < 128; ++c) {
            const bool vis = (c < sink_end) || (c >= band_lo && c < diag_end) || (c >= lr_lo && c < lr_hi);
            if (!vis) xr[c] = 0xff800000u;  // -inf: gives exactly 0
          }
        }
        // P = 2^(s*scale*log2e - m) with m the running max from before this tile, rounded to
        // bf16 and written back into TMEM over the S columns (the A operand of P V); the tile's
        // row max is gathered in the same pass.  Only when that max grows the running one by
        // more than 2^8 (lazy rescale; rare after the first tiles) is the tile redone with the
        // new max, so the common path never waits for the row reduction.
        uint64_t ts[4];  // this tile's row sum, 4 independent packed accumulators
        float pm[8];     // partial row maxima
        auto pass = [&](float m) {
          const uint64_t negm = ptx::f2_pack(-m, -m);
#pragma unroll
          for (int e = 0; e < 4; ++e) ts[e] = ptx::f2_pack(0.f, 0.f);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pw[32];
#pragma unroll
            for (int c2 = 0; c2 < 32; ++c2) {
              const int c = 64 * h + 2 * c2;
              float e0, e1;
              ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(xr[c]), __uint_as_float(xr[c + 1])), sl2x2, negm),
                             e0, e1);
              const float p0 = ptx::ex2(e0), p1 = ptx::ex2(e1);
              ts[c2 & 3] = ptx::f2_add(ts[c2 & 3], ptx::f2_pack(p0, p1));
              pw[c2] = ptx::pack_bf16(p0, p1);
            }
            ptx::tmem_st32(s_tm + 32 * h, pw);
          }
        };
        pass(m_used == -INFINITY ? 0.f : m_used);
        // row max (independent of the exponentials above, so it overlaps them)
#pragma unroll
        for (int e = 0; e < 8; ++e) pm[e] = fmaxf(__uint_as_float(xr[e]), __uint_as_float(xr[e + 8]));
#pragma unroll
        for (int c = 16; c < 128; c += 16)
#pragma unroll
          for (int e = 0; e < 8; ++e) pm[e] = ptx::fmax3(pm[e], __uint_as_float(xr[c + e]), __uint_as_float(xr[c + 8 + e]));
        const float mx = fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])), fmaxf(fmaxf(pm[4], pm[5]), fmaxf(pm[6], pm[7])));
        const float m_new = fmaxf(m_used, mx * sl2);
        const bool grow = (m_new != -INFINITY) && (m_used == -INFINITY || m_new > m_used + kRescaleThreshold);
        if (__any_sync(0xffffffffu, grow)) {
          float alpha = 1.f;
          if (grow) {
            alpha = ptx::ex2(m_used - m_new);  // 0 when nothing was visible before
            m_used = m_new;
            lsum = ptx::f2_mul(lsum, ptx::f2_pack(alpha, alpha));
          }
          if (cnt > 0) {
            // O row *= alpha, a warp-collective TMEM round trip (alpha = 1 on the other lanes);
            // PV_k(n-1) has completed (the commit of S_k(n) covers it), so O_k is stable here
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ov[32];
              ptx::tmem_ld32(o_tm + c * 32, ov);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              ptx::tmem_st32(o_tm + c * 32, ov);
            }
          }
          // redo the tile from the scores still in registers (lanes whose max did not grow
          // recompute the same values); the stores replace the speculative P
          ptx::tmem_wait_st();
          pass(m_used == -INFINITY ? 0.f : m_used);
        }
        lsum = ptx::f2_add(lsum, ptx::f2_add(ptx::f2_add(ts[0], ts[1]), ptx::f2_add(ts[2], ts[3])));
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&p_ready[k]);
        ++cnt;
      }
      float la, lb;
      ptx::f2_unpack(lsum, la, lb);
      const float l = la + lb;
      // ---- epilogue
      if constexpr (PAGED) {
        // (read again, so that they need no registers in the loop)
        row0 = chunk.row0;
        q_off = chunk.start;
        h0 = chunk.g * grp + chunk.head;
        if (ntiles == 0 && t < t1 && k < (has1 ? 2 : 1)) {  // no keys: an empty part, or past the cache and its band
          const size_t row = (size_t)(h0 + k) * a.total + row0 + t - q_off;
          if (a.parts > 1) {
            a.part_ml[(size_t)part * a.Hq * a.total + row] = make_float2(-INFINITY, 0.f);
          } else {
            __nv_bfloat16* z = reinterpret_cast<__nv_bfloat16*>(a.o) + (size_t)(row0 + t - q_off) * a.o_st + (size_t)(h0 + k) * a.o_sh;
            for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(z)[c] = make_uint4(0, 0, 0, 0);
            a.lse[row] = -INFINITY;
          }
        }
      }
      // (a.parts > 1: the part's running max and sum, the sum -1 for a bad page, and its O as it stands)
      auto part_row = [&](int h) { return ((size_t)part * a.Hq + h) * a.total + row0 + t - q_off; };
      auto put_part = [&](int h, int c, const uint32_t* x) {  // 32 columns of O
        float4* dst = reinterpret_cast<float4*>(a.part_o + part_row(h) * D + c * 32);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dst[e] = make_float4(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1]), __uint_as_float(x[4 * e + 2]),
                               __uint_as_float(x[4 * e + 3]));
      };
      const int rl = t - q_off;  // query row within the call's (or the sequence's) rows
      __nv_bfloat16* orow = reinterpret_cast<__nv_bfloat16*>(a.o) + (size_t)b * a.o_sb + (size_t)(row0 + rl) * a.o_st +
                            (size_t)h0 * a.o_sh;
      // lse: [B, H_q, N_q], or [H_q, total] for a packed batch
      const size_t lse_h0 = a.varlen ? (size_t)h0 * a.total + row0 + rl : ((size_t)b * a.Hq + h0) * a.Nq + rl;
      const size_t lse_step = a.varlen ? (size_t)a.total : (size_t)a.Nq;  // to the next head
      if (!split) {
        if (ok && ntiles > 0 && ptx::mbar_wait_warp(&o_done[k], 0, &abort_flag, a.status)) {
          ptx::tc_fence_after();
          // (a paged row may see nothing, or its query tile a bad page.  The sum tells the first: it is 0 then,
          // and NaN where all scores were, which leave the maximum at -inf too)
          const bool bad = PAGED && *reinterpret_cast<volatile int*>(&bad_page);
          const bool none = PAGED && (l == 0.f || bad);
          const float inv = 1.f / l;
          const bool partial = PAGED && a.parts > 1;
          if (t < t1) {
            if (partial) a.part_ml[part_row(h0 + k)] = make_float2(m_used, bad ? -1.f : l);
            else a.lse[lse_h0 + k * lse_step] = none ? -INFINITY : (m_used + log2f(l)) * 0.69314718055994530942f;
          }
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            ptx::tmem_ld32(o_tm + c * 32, ov);  // warp-collective: every lane loads, valid rows store
            ptx::tmem_wait_ld();
            if (partial) {
              if (t < t1) put_part(h0 + k, c, ov);
            } else if (t < t1) {
#pragma unroll
              for (int c8 = 0; c8 < 4; ++c8) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[e] = ptx::pack_bf16(__uint_as_float(ov[c8 * 8 + 2 * e]) * inv,
                                        __uint_as_float(ov[c8 * 8 + 2 * e + 1]) * inv);
                if (none) w[0] = w[1] = w[2] = w[3] = 0u;
                reinterpret_cast<uint4*>(orow + (size_t)k * a.o_sh)[c * 4 + c8] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        }
      } else if (k == 1) {
        // hand this slot's running max and sum to slot 0, which merges the two halves
        const bool have = ok && cnt > 0 && ptx::mbar_wait_warp(&o_done[1], 0, &abort_flag, a.status);
        ptx::tc_fence_after();
        merge_m[r] = have ? m_used : -INFINITY;
        merge_l[r] = have ? l : 0.f;
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&merge_ready);
      } else if (ok && ntiles > 0 && ptx::mbar_wait_warp(&o_done[0], 0, &abort_flag, a.status) &&
                 ptx::mbar_wait_warp(&merge_ready, 0, &abort_flag, a.status)) {
        // O = (O0 2^(m0-m) + O1 2^(m1-m)) / (l0 2^(m0-m) + l1 2^(m1-m)), m = max(m0, m1)
        ptx::tc_fence_after();
        const float m1 = merge_m[r], l1 = merge_l[r];
        const float m = fmaxf(m_used, m1);
        const float f0 = m_used == -INFINITY ? 0.f : ptx::ex2(m_used - m);
        const float f1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - m);
        const float lt = l * f0 + l1 * f1;
        const bool bad = PAGED && *reinterpret_cast<volatile int*>(&bad_page);
        const bool none = PAGED && (lt == 0.f || bad), partial = PAGED && a.parts > 1;
        const float inv = partial ? 1.f : 1.f / lt, g0 = f0 * inv, g1 = f1 * inv;
        const bool two = ntiles > 1;  // slot 1 has tiles (uniform over the CTA)
        if (t < t1 && partial) a.part_ml[part_row(h0)] = make_float2(m, bad ? -1.f : lt);
        else if (t < t1) a.lse[lse_h0] = none ? -INFINITY : (m + log2f(lt)) * 0.69314718055994530942f;
        const uint32_t o1_tm = lane_base + Geo::kColO + D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32], ow[32];
          ptx::tmem_ld32(o_tm + c * 32, ov);  // warp-collective: every lane loads, valid rows store
          if (two) ptx::tmem_ld32(o1_tm + c * 32, ow);
          ptx::tmem_wait_ld();
          if (partial) {
            if (t < t1) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                ov[e] = __float_as_uint(__uint_as_float(ov[e]) * g0 + (two ? __uint_as_float(ow[e]) * g1 : 0.f));
              put_part(h0, c, ov);
            }
          } else if (t < t1) {
#pragma unroll
            for (int c8 = 0; c8 < 4; ++c8) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int i0 = c8 * 8 + 2 * e;
                float x0 = __uint_as_float(ov[i0]) * g0, x1 = __uint_as_float(ov[i0 + 1]) * g0;
                if (two) {
                  x0 += __uint_as_float(ow[i0]) * g1;
                  x1 += __uint_as_float(ow[i0 + 1]) * g1;
                }
                w[e] = ptx::pack_bf16(x0, x1);
              }
              if (none) w[0] = w[1] = w[2] = w[3] = 0u;
              reinterpret_cast<uint4*>(orow)[c * 4 + c8] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// The sequence table of a packed batch (kernel_common.cuh) from cu_seqlens; one thread: the
// scan is over the sequences of one batch
__global__ void seq_table_kernel(const int32_t* cu, int n_seq, int total, int32_t* tab) {
  if (threadIdx.x != 0) return;
  int off = 0, prev_end = 0;
  for (int s = 0; s < n_seq; ++s) {
    const int st = imin(imax(cu[s], prev_end), total);
    const int en = imin(imax(cu[s + 1], st), total);
    tab[s] = off;
    tab[n_seq + 1 + s] = st;
    tab[2 * n_seq + 1 + s] = en - st;
    off += (en - st + kBM - 1) / kBM;
    prev_end = en;
  }
  tab[n_seq] = off;
}

// Joins the parts of each query row: one warp per (row, head).  Rows outside the sequences stay as they are.
template <int D>
__global__ void __launch_bounds__(256) fwd_join_kernel(const __grid_constant__ FwdArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  // the sequences' rows: from the first offset to the largest (see find_chunk)
  __shared__ int rows_end;
  const int rows_begin = imin(imax(a.cu_seqlens[0], 0), a.total);
  if (threadIdx.x == 0) rows_end = rows_begin;
  __syncthreads();
  int most = rows_begin;
  for (int i = threadIdx.x; i <= a.n_seq; i += blockDim.x) most = imax(most, imin(a.cu_seqlens[i], a.total));
  most = (int)__reduce_max_sync(0xffffffffu, (unsigned)most);
  if (lane == 0) atomicMax(&rows_end, most);
  __syncthreads();
  const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (at >= (int64_t)a.Hq * a.total) return;
  const int h = (int)(at / a.total), row = (int)(at - (int64_t)h * a.total);
  if (row < rows_begin || row >= rows_end) return;
  const size_t step = (size_t)a.Hq * a.total;  // from part to part
  float2 ml = lane < a.parts ? a.part_ml[lane * step + at] : make_float2(-INFINITY, 0.f);
  const bool bad = __any_sync(0xffffffffu, ml.y < 0.f);
  float m = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float f = ml.x == -INFINITY ? 0.f : ptx::ex2(ml.x - m);
  float l = f * ml.y, acc[E] = {};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float* p = a.part_o + at * D + lane * E;
#pragma unroll 4
  for (int i = 0; i < a.parts; ++i) {
    const float w = __shfl_sync(0xffffffffu, f, i);
    if (w == 0.f) continue;  // (an empty part wrote no O)
    float x[E];
    if constexpr (E == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i * step * D);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(p + i * step * D);
      x[0] = v.x; x[1] = v.y;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += w * x[e];
  }
  const bool none = bad || l == 0.f;  // (a part of NaN scores only has the maximum -inf, but the sum NaN)
  uint32_t w[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) w[e] = none ? 0u : ptx::pack_bf16(acc[2 * e] / l, acc[2 * e + 1] / l);
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(a.o) + row * a.o_st + h * a.o_sh + lane * E;
  if constexpr (E == 4) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(o) = w[0];
  if (lane == 0) a.lse[at] = none ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

template <int D, bool PAGED>
cudaError_t launch_fwd_d(const FwdArgs& a, cudaStream_t s) {
  using Geo = FwdGeom<D>;
  auto kern = cowa_fwd_kernel<D, PAGED>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo::kSmem);
  if (e != cudaSuccess) return e;
  const int grp = a.Hq / a.Hkv;
  // packed batch: an upper bound on the q-tiles (sum of ceil(len/BM) <= total/BM + n_seq); the
  // sequence table is computed on the device first
  const long long nq = a.varlen ? packed_tiles_bound(a.total, a.n_seq) : (a.Nq + kBM - 1) / kBM;
  const long long nblk = nq * a.B * a.Hkv * (PAGED && a.solo ? grp : (grp + 1) / 2) * (PAGED ? a.parts : 1);
  if (nblk > 0x7fffffffLL) return cudaErrorInvalidValue;
  // the in-kernel register split assumes the compiled count equals the launch allocation
  static int regs_ok = -1;
  if (regs_ok < 0) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    regs_ok = fa.numRegs == kRegsLaunch ? 1 : 0;
  }
  if (!regs_ok) return cudaErrorInvalidConfiguration;
  if (PAGED) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)nblk);
    cfg.blockDim = dim3(kFwdThreads);
    cfg.dynamicSmemBytes = Geo::kSmem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, kern, a)) != cudaSuccess || a.parts == 1) return e;
    cfg.gridDim = dim3((unsigned)(((int64_t)a.Hq * a.total + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, fwd_join_kernel<D>, a);
  }
  if (a.varlen) {
    if ((e = launch_seq_table(a.cu_seqlens, a.n_seq, a.total, a.seq_tab, s)) != cudaSuccess) return e;
  }
  kern<<<(unsigned)nblk, kFwdThreads, Geo::kSmem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_seq_table(const int32_t* cu_seqlens, int n_seq, int total, int32_t* tab, cudaStream_t s) {
  seq_table_kernel<<<1, 32, 0, s>>>(cu_seqlens, n_seq, total, tab);
  return cudaGetLastError();
}

// How the work of a paged call is cut: the parts of its CTAs' key tiles (1: no cut; at most kPartBytes of
// partial results), and whether a CTA takes one query head instead of two.  A pair of heads is the better use
// of a key tile (4K rows behind 28K keys: 468 us in pairs, 547 with single heads), but fewer CTAs of longer
// work.  The form with the least estimated time is taken, from what the host knows: bounds of the query tiles
// and of the longest list of key tiles.  (kPartBytes: 42 calls that bounds of 0 to 60 MB cut differently took
// 2.9% more than the best of the bounds with 15 MB, 40% with 0, 11% with 4, 4.3% with 8, 5.2% with 12, 5.3 to
// 6.2% with 20 and more, where the estimate lets in cuts that do not pay.)  In us, d = 128 (3/4 of it a tile at
// d = 64):
//   key tiles of a part x (1.65 a pair of heads, 1.2 a single one)
//   + where the CTAs take turns, 4 + a turn beyond the first x (8 + 1/5 of that: the longest come first)
//   + where parts are joined, 3 + their bytes at 3.5 TB/s
// Measured against pairs in as many parts as all run at once: 50 calls 10% less time in the mean (3% more than
// the best of all forms), 52 others 9% less, the worst of them 22 -> 26 us, the most 204 -> 119 (357 rows of 6
// sequences, 32/4 heads: two parts) and 35 -> 23 (339 rows of 5, 20/4 heads: single heads); 16 rows behind 32K
// keys (40/8 heads) 110 -> 32 (parts).
FwdCut fwd_paged_cut(const Pat& p, int n_seq, int total, int Hq, int Hkv, int d, int max_pages, int page_size) {
  constexpr int64_t kPartBytes = 15 << 20;
  constexpr int kMaxParts = 32;  // (a lane each when they are joined)
  const int64_t cap = (int64_t)max_pages * page_size, R = (int64_t)p.T - p.S;
  const int64_t wide = R > 0 ? (R + p.H - 1) / p.H : 0;
  auto tiles = [&](int64_t n) { return n > 0 ? ((n < cap ? n : cap) + kBN - 1) / kBN + 1 : 0; };
  int64_t n = tiles(p.S) + tiles(wide) + tiles((int64_t)p.L + kBM);
  const int64_t all = (cap + kBN - 1) / kBN;
  n = n < all ? n : all;
  const int grp = Hq / Hkv;
  const double work = (double)packed_tiles_bound(total, n_seq) * Hkv, bytes = (double)Hq * total * (d + 2) * sizeof(float);
  FwdCut best{1, 0};
  double least = 1e30;
  for (int solo = 0; solo < (grp > 1 ? 2 : 1); ++solo)
    for (int parts = 1; parts <= kMaxParts && parts <= n && (parts == 1 || parts * bytes <= kPartBytes); ++parts) {
      const double longest = (double)((n + parts - 1) / parts) * (solo ? 1.2 : 1.65) * (d == 128 ? 1.0 : 0.75);
      const double turns = work * (solo ? grp : (grp + 1) / 2) * parts / 148;
      double us = longest;
      if (turns > 1) us += 4 + (turns - 1) * (8 + 0.2 * longest);
      if (parts > 1) us += 3 + parts * bytes / 3.5e6;
      if (us < least) { least = us; best = FwdCut{parts, solo}; }
    }
  return best;
}

size_t fwd_paged_bytes(int parts, int total, int Hq, int d) {
  if (parts == 1) return 0;
  const size_t rows = (size_t)parts * Hq * total;
  return align_up(rows * sizeof(float2), 256) + rows * d * sizeof(float);
}

cudaError_t launch_fwd(const FwdArgs& a, cudaStream_t s) {
  if (a.d == 64) return a.paged ? launch_fwd_d<64, true>(a, s) : launch_fwd_d<64, false>(a, s);
  if (a.d == 128) return a.paged ? launch_fwd_d<128, true>(a, s) : launch_fwd_d<128, false>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace cowa
