// cowa_paged.cu -- decode over a paged K/V cache: one new query token per sequence attends to the
// keys its KV head can see ("CoWindow Attention: Full Causal Coverage Is a Collective Property",
// Abstract: the same position-defined pattern in training and decoding), the rows of position s
// being found in page table[b (, g)][s / page_size] at slot s % page_size.
//
//   o = sum_s p_s v_s / sum_s p_s,   p_s = 2^(scale log2(e) q.k_s - m),   s over the visible set
//
// HBM-bound: each visible K and V row is read once.  What the kernel is built around:
//   * The work is the list of 64-position tiles of all (sequence, KV head) pairs, in that order.
//     Lengths are known on the device only, and differ from 1 to the whole cache, so every CTA adds up
//     the tile counts itself (integer arithmetic on pos) and takes an equal, contiguous share of the
//     list, in which every pair counts a few tiles more than it has (kSegmentOf).  A pair that lies inside one
//     CTA's share is finished there; one that several CTAs share leaves fp32 partials (at most two per CTA),
//     which a second kernel joins in order.
//   * Where no CTA gets more than a few tiles anyway (one user, short caches), latency counts instead:
//     a cluster of CTAs takes one pair, shares its tiles out evenly and joins its results through
//     distributed shared memory, so there is no list to add up and no second kernel.
//   * A producer warp looks up the pages (one lane per box of 8 to 64 rows, two tiles ahead of the
//     copies) and streams K and V tiles into a shared-memory ring with TMA; boxes that hold no
//     visible key are not fetched.
//   * Scores, maxima, sums, O and partials are fp32.  P is rounded to 16 bits, because it is an operand of the
//     second matrix product: to bf16 beside bf16 values (off by at most 2^-8 of sum p |v|), to f16 beside E4M3
//     ones (2^-11), which are exact in f16; the queries become f16 there too (exact unless below f16's range,
//     2^-14, or above it, 65504).  Against 64 bits o is off by 0.0021 to 0.0023 (2-norm) with bf16 pages where a
//     form in 32 bits, which rounds o only, is off by 0.0017.
//   * Short sequences make short segments, so a segment costs little: the intervals of the heads are
//     arguments, each warp works out 32 pairs at once (a lane each) and hands them on by shuffles, and
//     the query rows of the next segment are fetched while the warps of this one are joined.
//   * 4 compute warps each take 16 tokens of a tile.  Tokens are the 16 rows of the warp MMAs
//     (m16n8k16) and the query heads of the group (at most 8) their 8 columns, so no MMA row is
//     wasted: S^T = K Q^T and O^T += V^T P^T, the scores turned into the P^T operand with two 8x8
//     transposes.  Each thread owns two heads, so the running maxima are compared without shuffles;
//     only a growth past 2^8 makes the warp reduce and rescale.
//   * Masked tokens are selected away in the scores and cleared in V, so what stands in unseen rows
//     (infinities, NaN) does not matter.
#include <cuda_bf16.h>
#include <math.h>

#include "cowa_internal.h"
#include "sm100_ptx.cuh"

namespace cowa {
namespace {

constexpr int kWarps = 4;                      // compute warps
constexpr int kThreads = (kWarps + 1) * 32;    // + the producer
constexpr int kTok = 64;                       // positions per tile
constexpr int kBoxBytes = kTok * 128;          // 64 rows x 128 bytes
constexpr float kRescale = 8.0f;               // lazy-rescale threshold, log2 units
// What a segment costs besides its tiles (query rows, join of the warps, a start of the pipeline), in
// tiles: about 2.8 us beside 1.0 us a tile with E4M3 pages, whose tiles are half the bytes (37 sequences
// of 1 to 32K positions: 22.7 us with 3, 24.4 with 2, 36 with 0), and 2 tiles with bf16 (37 of up to 1K:
// 13.3 us with 2, 14.4 with 3).
template <bool KV8>
constexpr int kSegmentOf = KV8 ? 3 : 2;
// Up to how many tiles a CTA may have for the cluster form: with 9.5 (8 sequences of 8K) it took 12.0 us
// against the list's 13.8, with 12.6 (two of 32K) 14.1 against 13.2.
constexpr int kClusterTiles = 10;
constexpr int kMaxCluster = 16;
constexpr int kJoinWarps = 16;  // of a joining block, at most
// E4M3: P is rounded to f16, whose smallest normal number is 2^-14; relative to a running maximum
// lifted by 2^6 (P at most 2^14) it covers P down to 2^-20 of the largest at full precision.
template <bool KV8>
constexpr float kLift = KV8 ? 6.0f : 0.0f;

// BIG: groups of more than 5 query heads, whose join takes more shared memory (with E4M3 pages a stage less
// then keeps three CTAs on an SM)
template <int D, bool KV8, bool BIG>
struct Geo {
  static_assert(!KV8 || D == 128, "E4M3 rows are whole 128-byte rows");
  static constexpr int kBarBytes = 256;  // 3 words per stage, then a few of the block's own
  static constexpr int kUnits = KV8 ? 1 : D / 64;  // 128-byte columns of a row
  static constexpr int kTileBytes = kUnits * kBoxBytes;
  static constexpr int kStages = KV8 ? (BIG ? 3 : 4) : (D == 128 ? 3 : 5);
  static constexpr int kCtas = KV8 ? 3 : 2;        // per SM, what the ring leaves room for
  static constexpr int kOffBar = kStages * 2 * kTileBytes;
  static_assert(3 * kStages <= 16, "the block's own words start at word 16");
  static constexpr int kOffRed = kOffBar + kBarBytes;
  static constexpr int smem(int grp) { return kOffRed + kWarps * grp * (D + 2) * 4; }
  static constexpr int kMostSmem = smem(KV8 && !BIG ? 5 : 8);  // of the largest group
  // of an SM's 228 KB a block takes its shared memory and 1 KB more
  static int ctas(int grp) { return imin(kCtas, (228 * 1024) / (smem(grp) + 1024)); }
};

// A (sequence, KV head) pair: its visible ranges at pos[b] and their 64-position tiles.
struct Pair {
  int b, n;
  int lo0, hi0, lo1, hi1, lo2, hi2;  // visible ranges, sorted and disjoint (empty: 0, 0)
  __device__ __forceinline__ void tile(int i, int& base, int& lo, int& hi) const {
    lo = lo0; hi = hi0;
    int n0 = tiles_of(lo0, hi0);
    if (i >= n0) {
      i -= n0;
      lo = lo1; hi = hi1;
      n0 = tiles_of(lo1, hi1);
      if (i >= n0) { i -= n0; lo = lo2; hi = hi2; }
    }
    base = (lo / kTok + i) * kTok;
    lo = imax(lo, base);
    hi = imin(hi, base + kTok);
  }
  __device__ __forceinline__ static int tiles_of(int lo, int hi) {
    return hi > lo ? (hi + kTok - 1) / kTok - lo / kTok : 0;
  }
};

// pair (b, g) at position t = pos[b]
__device__ __forceinline__ Pair pair_at(const PagedDecodeArgs& a, int b, int g, int t) {
  Pair s;
  s.b = b;
  const int cap = a.tab.max_pages * a.tab.page_size;
  if (t >= cap) t = cap - 1;
  const Range iv = a.Hkv <= kPagedIv ? a.iv[g] : interval_of(a.pat, g);
  Range r[3] = {{0, 0}, {0, 0}, {0, 0}};
  if (t >= 0) {
    const int n = row_ranges(a.pat, iv, t, r);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i >= n) r[i] = Range{0, 0};
  }
  s.lo0 = r[0].lo; s.hi0 = r[0].hi; s.lo1 = r[1].lo; s.hi1 = r[1].hi; s.lo2 = r[2].lo; s.hi2 = r[2].hi;
  s.n = Pair::tiles_of(s.lo0, s.hi0) + Pair::tiles_of(s.lo1, s.hi1) + Pair::tiles_of(s.lo2, s.hi2);
  return s;
}
__device__ __forceinline__ Pair pair_of(const PagedDecodeArgs& a, int item) {
  const int b = item / a.Hkv;
  return pair_at(a, b, item - b * a.Hkv, a.pos[b]);
}

// 32 pairs, one per lane, handed to the whole warp one at a time (all lanes call with the same item,
// items not decreasing): the tile counts alone, or everything.
struct Counts {
  int first, n;
  __device__ __forceinline__ void fill(const PagedDecodeArgs& a, int from, int n_items) {
    first = from;
    const int i = from + (threadIdx.x & 31);
    n = i < n_items ? pair_of(a, i).n : 0;
  }
  __device__ __forceinline__ int get(const PagedDecodeArgs& a, int item, int n_items) {
    if (item - first >= 32) fill(a, item, n_items);
    return __shfl_sync(0xffffffffu, n, item - first);
  }
};
struct Window {
  int first;
  Pair p;
  __device__ __forceinline__ void fill(const PagedDecodeArgs& a, int from, int n_items) {
    first = from;
    const int i = from + (threadIdx.x & 31);
    p = pair_of(a, i < n_items ? i : n_items - 1);
    if (i >= n_items) p.n = 0;
  }
  __device__ __forceinline__ Pair get(const PagedDecodeArgs& a, int item, int n_items) {
    if (item - first >= 32) fill(a, item, n_items);
    const int l = item - first;
    auto sh = [&](int x) { return __shfl_sync(0xffffffffu, x, l); };
    Pair s;
    s.b = sh(p.b); s.n = sh(p.n);
    s.lo0 = sh(p.lo0); s.hi0 = sh(p.hi0); s.lo1 = sh(p.lo1); s.hi1 = sh(p.hi1); s.lo2 = sh(p.lo2); s.hi2 = sh(p.hi2);
    return s;
  }
};

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  return pack_f16(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
// transpose of an 8x8 matrix of 16-bit elements held as an MMA fragment
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// address of 16-byte unit u of row r of a tile whose 128-byte columns are swizzled
__device__ __forceinline__ uint32_t unit_addr(uint32_t tile, int r, int u) {
  return tile + (u >> 3) * kBoxBytes + r * 128 + (((u & 7) ^ (r & 7)) << 4);
}

// Running state of a warp: per thread two heads (2 tq, 2 tq + 1) and D/16 fragments of O^T, whose rows
// are the head dimension: bf16, row r of fragment j is d = 16 j + r; E4M3, rows gr and gr + 8 of
// fragment j are d = 16 gr + 2 j and 16 gr + 2 j + 1 (see below).
template <int D>
struct State {
  float acc[D / 16][4];
  float m0, m1, l0, l1;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < D / 16; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
  }
  // the running maxima grow to cover x0, x1 (this thread's largest scores of its two heads)
  __device__ __forceinline__ void cover(float x0, float x1) {
    if (!__any_sync(0xffffffffu, x0 > m0 + kRescale || x1 > m1 + kRescale)) return;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
    }
    float f0 = 1.f, f1 = 1.f;
    if (x0 > m0 + kRescale) { f0 = m0 == -INFINITY ? 0.f : ptx::ex2(m0 - x0); m0 = x0; }
    if (x1 > m1 + kRescale) { f1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - x1); m1 = x1; }
    l0 *= f0;
    l1 *= f1;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      acc[j][0] *= f0; acc[j][1] *= f1; acc[j][2] *= f0; acc[j][3] *= f1;
    }
  }
};

// W places in G shares: the first `more` shares hold one place more than the `each` of the others.  A
// pair of n > 0 tiles takes kSegmentOf places and then one per tile.
struct Shares {
  int each, more;
  __device__ __forceinline__ int begin(int c) const { return c * each + imin(c, more); }
  __device__ __forceinline__ int of(int w) const {  // the share that holds place w
    const int big = more * (each + 1);
    return w < big ? w / (each + 1) : more + (w - big) / each;
  }
};

// ---- thread-block cluster: barriers of all its threads, and the other CTAs' shared memory
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float cluster_ld(const float* own, int rank) {  // the word at the same place in CTA `rank`
  uint32_t addr;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(ptx::smem_u32(own)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Element d of a row's result, from its maximum, sum and unscaled O.  The sum is 0 only if the row saw nothing
// (o 0, lse -inf); where all scores were NaN the maximum is still -inf, but the sum is NaN, and so is the row.
template <int D>
__device__ __forceinline__ void put_row(const PagedDecodeArgs& a, size_t h, int d, float m, float l, float o) {
  reinterpret_cast<__nv_bfloat16*>(a.o)[h * D + d] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
  if (a.lse && d == 0) a.lse[h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

// CL: CTAs c, c + 1, .. of a cluster of a.cluster share one pair; else every CTA has its share of the list.
template <int D, bool KV8, bool CL, bool BIG>
__global__ void __launch_bounds__(kThreads, Geo<D, KV8, BIG>::kCtas)
    paged_split_kernel(const __grid_constant__ PagedDecodeArgs a) {
  using G_ = Geo<D, KV8, BIG>;
  constexpr int KS = D / 16;
  constexpr int kStages = G_::kStages;
  constexpr int kSegment = kSegmentOf<KV8>;
  auto places = [](int n) { return n > 0 ? n + kSegmentOf<KV8> : 0; };
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + G_::kOffBar);
  uint64_t* empty_bar = full_bar + kStages;
  volatile uint64_t* seen = empty_bar + kStages;  // per stage: the tile's visible positions
  int* warp_sum = reinterpret_cast<int*>(full_bar + 16);  // [5]
  volatile int& abort_flag = *reinterpret_cast<volatile int*>(full_bar + 24);
  int* first_of = reinterpret_cast<int*>(full_bar + 25);  // [2]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  const int n_items = a.B * a.Hkv;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full_bar[s], 1);
      ptx::mbar_init(&empty_bar[s], kWarps);
    }
    abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&a.tm_k);
    ptx::tma_prefetch_desc(&a.tm_v);
  }
  // this kernel was set up while the one before it in the stream ran, and waits for that one's results
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- this CTA's share: places [w0, w1) of the list, the first pair of it and that pair's place
  int w0, w1, first_item, first_place;
  Shares sh{0, 0};
  Pair own;  // (CL) the one pair there is
  if constexpr (CL) {
    first_item = c / a.cluster;
    const int rank = c - first_item * a.cluster;
    own = pair_of(a, first_item);
    // (a.cluster is 4, 8 or 16, and a pair has at most kClusterTiles tiles for each CTA)
    w0 = own.n * rank / a.cluster;
    w1 = own.n * (rank + 1) / a.cluster;
    first_place = -kSegment;  // place w is tile w
    __syncthreads();
  } else {
    // thread i adds up the pairs i0 .. i1 - 1; up to kKept of them stay at hand (more, from 641 pairs on, are
    // walked one by one, and again by the thread that holds the share's start: 640 pairs of up to 4K positions
    // 40.0 us at 1.44 times their bytes at the copy rate, 648 of them 42.3 at 1.47)
    constexpr int kKept = 4;
    const int per = (n_items + kThreads - 1) / kThreads;
    const int i0 = imin(n_items, (int)threadIdx.x * per), i1 = imin(n_items, i0 + per);
    int mine = 0, kept[kKept];
    if (per <= kKept) {
      int b[kKept], g[kKept], t[kKept];
#pragma unroll
      for (int j = 0; j < kKept; ++j) {
        b[j] = (i0 + j) / a.Hkv;
        g[j] = i0 + j - b[j] * a.Hkv;
        t[j] = i0 + j < i1 ? a.pos[b[j]] : -1;
      }
#pragma unroll
      for (int j = 0; j < kKept; ++j) {
        kept[j] = j < per ? places(pair_at(a, b[j], g[j], t[j]).n) : 0;
        mine += kept[j];
      }
    } else {
      for (int i = i0; i < i1; ++i) mine += places(pair_of(a, i).n);
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - mine, W = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      W += warp_sum[w];
    }
    // no share is empty: with fewer places than CTAs the last CTAs have none
    const int G = W < (int)gridDim.x ? W : (int)gridDim.x;
    sh = Shares{G ? W / G : 0, G ? W % G : 0};
    w0 = c < G ? sh.begin(c) : W;
    w1 = c < G ? sh.begin(c + 1) : W;
    if (w0 < w1 && before <= w0 && w0 < before + mine) {
      int p = before;
      if (per <= kKept) {
#pragma unroll
        for (int j = 0; j < kKept; ++j) {
          if (w0 >= p && w0 < p + kept[j]) { first_of[0] = i0 + j; first_of[1] = p; }
          p += kept[j];
        }
      } else {
        for (int i = i0; i < i1; ++i) {
          const int n = places(pair_of(a, i).n);
          if (w0 < p + n) { first_of[0] = i; first_of[1] = p; break; }
          p += n;
        }
      }
    }
    __syncthreads();
    first_item = first_of[0];
    first_place = first_of[1];
  }
  const bool pool_ok = (ptx::smem_u32(smem) & 1023u) == 0;  // the swizzle pattern assumes it

  if (warp == kWarps) {
    // ------------------------------------------------------------------ producer
    if (w0 < w1 && pool_ok) {
      const int nbox = kTok / a.box_rows;
      Window win;
      int item = first_item, place = first_place;
      Pair s = own;
      if constexpr (!CL) {
        win.fill(a, item, n_items);
        s = win.get(a, item, n_items);
      }
      // this CTA's tiles of the pair at hand: [off, lim)
      int off = imax(0, w0 - place - kSegment), lim = imin(s.n, w1 - place - kSegment);
      // Box `lane` of a tile: the page it lies in.  The load is unconditional, at a clamped place, and
      // what it gave is looked at when the tile's turn comes, two tiles later.
      struct Look {
        int base, lo, hi, g, slot, page;
        bool want;
      };
      auto look = [&](Look& k) -> bool {
        while (off >= lim) {
          place += places(s.n);
          if (CL || place >= w1) return false;
          s = win.get(a, ++item, n_items);
          off = 0;
          lim = imin(s.n, w1 - place - kSegment);
        }
        s.tile(off++, k.base, k.lo, k.hi);
        k.g = item - s.b * a.Hkv;
        const int p = k.base + (lane & (nbox - 1)) * a.box_rows;
        k.want = lane < nbox && p < k.hi && p + a.box_rows > k.lo;
        const int i = a.page_shift >= 0 ? p >> a.page_shift : p / a.tab.page_size;
        k.slot = p - i * a.tab.page_size;
        k.page = a.tab.ptr[s.b * a.tab.sb + k.g * a.tab.sh + imin(i, a.tab.max_pages - 1)];
        // (debug builds) the tile's keys lie in the cache and in the tile, the box in its page
        if (!ptx::dbg_check(!k.want || (item < n_items && k.base >= 0 && k.lo >= k.base && k.hi <= k.base + kTok &&
                                        k.hi <= a.tab.max_pages * a.tab.page_size && k.slot >= 0 &&
                                        k.slot + a.box_rows <= a.tab.page_size),
                            a.status, nullptr, 0x402, k.base))
          k.page = -1;  // (not fetched, its keys left out)
        return true;
      };
      int issued = 0;
      auto put = [&](const Look& k, int st) -> bool {
        const int sl = st % kStages;
        const bool good = k.want && k.page >= 0 && k.page < a.tab.n_pages;
        const uint32_t fetch = __ballot_sync(0xffffffffu, good);
        const uint32_t bad = __ballot_sync(0xffffffffu, k.want && !good);
        uint64_t vis = (k.hi - k.base >= kTok ? ~0ull : (1ull << (k.hi - k.base)) - 1) & ~((1ull << (k.lo - k.base)) - 1);
        if (bad) {  // entries outside the pool: reported, their keys left out
          const uint64_t rows = a.box_rows == kTok ? ~0ull : (1ull << a.box_rows) - 1;
          for (int x = 0; x < nbox; ++x)
            if ((bad >> x) & 1) vis &= ~(rows << (x * a.box_rows));
          if (lane == 0) a.status[3] = kPageFlag;
        }
        if (st >= kStages && !ptx::mbar_wait_warp(&empty_bar[sl], ((st / kStages) & 1) ^ 1, &abort_flag, a.status))
          return false;
        uint8_t* ks = smem + sl * 2 * G_::kTileBytes;
        uint8_t* vs = ks + G_::kTileBytes;
        if (lane == 0) {
          seen[sl] = vis;
          ptx::mbar_arrive_expect_tx(&full_bar[sl], 2 * G_::kUnits * __popc(fetch) * a.box_rows * 128);
        }
        __syncwarp();
        if (good) {
          const int at = lane * a.box_rows * 128, g = a.tab.sh ? 0 : k.g;
#pragma unroll
          for (int u = 0; u < G_::kUnits; ++u) {
            ptx::tma_load_4d(ks + u * kBoxBytes + at, &a.tm_k, &full_bar[sl], u * (KV8 ? 128 : 64), k.slot, g, k.page);
            ptx::tma_load_4d(vs + u * kBoxBytes + at, &a.tm_v, &full_bar[sl], u * (KV8 ? 128 : 64), k.slot, g, k.page);
          }
        }
        issued = st + 1;
        return true;
      };
      Look even, odd;
      bool more_even = look(even), more_odd = more_even && look(odd);
      for (int st = 0; more_even; st += 2) {  // by twos, so that nothing has to be moved between the two
        if (!put(even, st)) break;
        more_even = more_odd && look(even);
        if (!more_odd || !put(odd, st + 1)) break;
        more_odd = more_even && look(odd);
      }
      // never leave the CTA with copies in flight
      for (int st = (issued > kStages ? issued - kStages : 0); st < issued; ++st)
        ptx::mbar_wait(&full_bar[st % kStages], (st / kStages) & 1, nullptr, a.status);
    }
    if constexpr (CL) {
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
    return;
  }

  // -------------------------------------------------------------------- compute warps
  const int gr = lane >> 2, tq = lane & 3;
  const int grp = a.grp;
  float* red = reinterpret_cast<float*>(smem + G_::kOffRed);  // [warp][head][D + 2]
  const uint32_t ring = ptx::smem_u32(smem);
  const int row0 = warp * 16;
  bool ok = pool_ok;
  if (!pool_ok && threadIdx.x == 0) atomicOr(a.status, (uint32_t)ptx::kStatusCheck);

  // slots without a sequence see nothing: zeros and -inf, by one CTA each
  for (int i = c; !CL && i < a.B; i += gridDim.x) {
    if (a.pos[i] >= 0) continue;
    const size_t h0 = (size_t)i * a.Hkv * grp;
    for (int x = threadIdx.x; x < a.Hkv * grp * (D / 8); x += kWarps * 32)
      reinterpret_cast<uint4*>(a.o)[h0 * (D / 8) + x] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int x = threadIdx.x; x < a.Hkv * grp; x += kWarps * 32) a.lse[h0 + x] = -INFINITY;
    if (a.by_pair)
      for (int x = threadIdx.x; x < a.Hkv; x += kWarps * 32) a.rec[i * a.Hkv + x].x = -1;
  }

  int4 rec = make_int4(-1, 0, 0, 0);
  int st = 0;
  // Q^T fragments as they stand in memory: columns are the heads of the group
  uint32_t qn[KS][2];
  auto load_q = [&](int it) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(
        reinterpret_cast<const __nv_bfloat16*>(a.q_t) + ((size_t)it * grp + imin(gr, grp - 1)) * D);
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      // E4M3: the head dimension is visited in another order, so that a thread's bytes of a key row are
      // contiguous: chunk kk of thread tq is d = 32 tq + 4 kk .. + 3
      qn[kk][0] = KV8 ? q[16 * tq + 2 * kk] : q[8 * kk + tq];
      qn[kk][1] = KV8 ? q[16 * tq + 2 * kk + 1] : q[8 * kk + 4 + tq];
    }
  };
  Counts counts;
  // the pair at hand: its place, its tiles, and this CTA's share of them [off, lim)
  int item = 0, place = 0, n = 0, off = 0, lim = 0;
  auto step = [&]() -> bool {  // the next pair of which this CTA has tiles
    do {
      place += places(n);
      if (place >= w1) return false;
      n = counts.get(a, ++item, n_items);
      off = 0;
      lim = imin(n, w1 - place - kSegment);
    } while (off >= lim);
    return true;
  };
  // (debug builds) the pair is one of the call's: its query rows, record and outputs lie in their arrays
  auto listed = [&]() { return ptx::dbg_check(item < n_items, a.status, &abort_flag, 0x403, item); };
  bool more = false;
  if (w0 < w1) {
    item = first_item;
    place = first_place;
    if constexpr (CL) {
      n = own.n;
    } else {
      counts.fill(a, item, n_items);
      n = counts.get(a, item, n_items);
    }
    off = imax(0, w0 - place - kSegment);
    lim = imin(n, w1 - place - kSegment);
    more = (off < lim || (!CL && step())) && listed();
    if (more) load_q(item);
  }
  while (more) {
    const int take = lim - off, h0 = item * grp;
    {
      uint32_t qf[KS][2];
#pragma unroll
      for (int kk = 0; kk < KS; ++kk)
#pragma unroll
        for (int h = 0; h < 2; ++h)  // (columns past the group are zero)
          qf[kk][h] = gr < grp ? (KV8 ? bf16x2_to_f16x2(qn[kk][h]) : qn[kk][h]) : 0u;
      State<D> z;
      z.clear();
      for (int i = 0; ok && i < take; ++i, ++st) {
        const int sl = st % kStages;
        if (!ptx::mbar_wait_warp(&full_bar[sl], (st / kStages) & 1, &abort_flag, a.status)) { ok = false; break; }
        const uint32_t bits = (uint32_t)(seen[sl] >> row0) & 0xffffu;  // this warp's 16 tokens
        const uint32_t kt = ring + sl * 2 * G_::kTileBytes, vt = kt + G_::kTileBytes;
        if (bits == 0) {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&empty_bar[sl]);
          continue;
        }
        // ---- scores S^T[token][head]
        float sc[2][4] = {};
        uint4 vr[4];  // E4M3: bytes [16 gr, 16 gr + 16) of value rows 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9
        if constexpr (KV8) {
          uint32_t kw[2][8];  // bytes [32 tq, 32 tq + 32) of key rows gr and gr + 8
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = row0 + 8 * h + gr;
            const uint4 x0 = lds128(kt + r * 128 + (((2 * tq) ^ (r & 7)) << 4));
            const uint4 x1 = lds128(kt + r * 128 + (((2 * tq + 1) ^ (r & 7)) << 4));
            kw[h][0] = x0.x; kw[h][1] = x0.y; kw[h][2] = x0.z; kw[h][3] = x0.w;
            kw[h][4] = x1.x; kw[h][5] = x1.y; kw[h][6] = x1.z; kw[h][7] = x1.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 2 * tq + (e & 1) + 8 * (e >> 1), r = row0 + j;
            vr[e] = lds128(vt + r * 128 + ((gr ^ (r & 7)) << 4));
            if (bits != 0xffffu && !((bits >> j) & 1)) vr[e] = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&empty_bar[sl]);  // the stage's bytes are in registers
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
            const uint32_t f[4] = {e4m3x2_to_f16x2(kw[0][kk] & 0xffffu), e4m3x2_to_f16x2(kw[1][kk] & 0xffffu),
                                   e4m3x2_to_f16x2(kw[0][kk] >> 16), e4m3x2_to_f16x2(kw[1][kk] >> 16)};
            mma_f16(sc[kk & 1], f, qf[kk][0], qf[kk][1]);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
            uint32_t f[4];
            ptx::ldsm_x4(unit_addr(kt, row0 + (lane & 15), 2 * kk + (lane >> 4)), f);
            ptx::mma_16816(sc[kk & 1], f, qf[kk][0], qf[kk][1]);
          }
        }
        // ---- online softmax; tokens gr and gr + 8, heads 2 tq and 2 tq + 1
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = (sc[0][e] + sc[1][e]) * a.scale_log2;
        if (bits != 0xffffu) {
          if (!((bits >> gr) & 1)) x[0] = x[1] = -INFINITY;
          if (!((bits >> (gr + 8)) & 1)) x[2] = x[3] = -INFINITY;
        }
        z.cover(fmaxf(x[0], x[2]), fmaxf(x[1], x[3]));
        const float r0 = z.m0 == -INFINITY ? 0.f : z.m0 - kLift<KV8>, r1 = z.m1 == -INFINITY ? 0.f : z.m1 - kLift<KV8>;
        const float p0 = ptx::ex2(x[0] - r0), p1 = ptx::ex2(x[1] - r1);
        const float p2 = ptx::ex2(x[2] - r0), p3 = ptx::ex2(x[3] - r1);
        z.l0 += p0 + p2;
        z.l1 += p1 + p3;
        // P^T as the second operand: rows are tokens, so transpose the 8x8 halves
        const uint32_t b0 = transpose8(KV8 ? pack_f16(p0, p1) : ptx::pack_bf16(p0, p1));
        const uint32_t b1 = transpose8(KV8 ? pack_f16(p2, p3) : ptx::pack_bf16(p2, p3));
        // ---- O^T[d][head] += V^T[d][token] P^T[token][head]
        if constexpr (KV8) {
          // fragment j's rows gr and gr + 8 are d = 16 gr + 2 j and + 1: the bytes 2 j and 2 j + 1 of this
          // thread's value bytes, of the token pairs (2 tq, 2 tq + 1) and (2 tq + 8, 2 tq + 9)
          const uint32_t va[4] = {vr[0].x, vr[0].y, vr[0].z, vr[0].w}, vb[4] = {vr[1].x, vr[1].y, vr[1].z, vr[1].w};
          const uint32_t vc[4] = {vr[2].x, vr[2].y, vr[2].z, vr[2].w}, vd[4] = {vr[3].x, vr[3].y, vr[3].z, vr[3].w};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
            const uint32_t lo2 = prmt(va[j >> 1], vb[j >> 1], sel), hi2 = prmt(vc[j >> 1], vd[j >> 1], sel);
            const uint32_t f[4] = {e4m3x2_to_f16x2(lo2 & 0xffffu), e4m3x2_to_f16x2(lo2 >> 16),
                                   e4m3x2_to_f16x2(hi2 & 0xffffu), e4m3x2_to_f16x2(hi2 >> 16)};
            mma_f16(z.acc[j], f, b0, b1);
          }
        } else {
          // masked tokens' V elements become zero in the fragments (0 times an infinity is not 0)
          uint32_t k0 = ~0u, k1 = ~0u;
          if (bits != 0xffffu) {
            k0 = (((bits >> (2 * tq)) & 1) ? 0xffffu : 0u) | (((bits >> (2 * tq + 1)) & 1) ? 0xffff0000u : 0u);
            k1 = (((bits >> (2 * tq + 8)) & 1) ? 0xffffu : 0u) | (((bits >> (2 * tq + 9)) & 1) ? 0xffff0000u : 0u);
          }
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t f[4];
            ptx::ldsm_x4_trans(unit_addr(vt, row0 + (lane & 7) + 8 * (lane >> 4), 2 * j + ((lane >> 3) & 1)), f);
            f[0] &= k0; f[1] &= k0; f[2] &= k1; f[3] &= k1;
            ptx::mma_16816(z.acc[j], f, b0, b1);
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&empty_bar[sl]);
        }
      }
      // ---- the next segment's pair and query rows, while the warps are joined
      const bool begins = off == 0, ends = lim == n;
      if (!CL && begins) {  // whether the pair goes on, and to which CTA
        const int last = sh.of(place + kSegment + n - 1);
        // (debug builds) the pieces that the join will read are those of CTAs of this launch
        const bool joins = !ends && ptx::dbg_check(last >= c && last < (int)gridDim.x, a.status, &abort_flag, 0x404, last);
        const int4 r = make_int4(joins ? item : -1, c, last, 0);
        if (a.by_pair) {
          if (threadIdx.x == 0) a.rec[item] = r;
        } else if (!ends) {
          rec = r;
        }
      }
      more = !CL && step() && listed();
      if (more) load_q(item);
      // ---- join the warps
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        z.l0 += __shfl_xor_sync(0xffffffffu, z.l0, o);
        z.l1 += __shfl_xor_sync(0xffffffffu, z.l1, o);
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");  // the last join has been read
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int hd = 2 * tq + h;
        if (hd < grp) {
          float* r = red + (warp * grp + hd) * (D + 2);
          if (gr == 0) { r[0] = (h ? z.m1 : z.m0) - kLift<KV8>; r[1] = h ? z.l1 : z.l0; }
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const int d0 = KV8 ? 16 * gr + 2 * j : 16 * j + gr, d1 = KV8 ? d0 + 1 : d0 + 8;
            r[2 + d0] = z.acc[j][h];
            r[2 + d1] = z.acc[j][2 + h];
          }
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
      if (ok && !abort_flag) {
        float* part = CL ? reinterpret_cast<float*>(smem)  // (the ring is drained)
                         : a.part + ((size_t)2 * c + (begins ? 1 : 0)) * grp * (D + 2);
        for (int x = threadIdx.x; x < grp * D; x += kWarps * 32) {
          const int hd = x / D, d = x - hd * D;
          float m = -INFINITY;
#pragma unroll
          for (int v = 0; v < kWarps; ++v) m = fmaxf(m, red[(v * grp + hd) * (D + 2)]);
          float o = 0.f, l = 0.f;
#pragma unroll
          for (int v = 0; v < kWarps; ++v) {
            const float* r = red + (v * grp + hd) * (D + 2);
            const float f = r[0] == -INFINITY ? 0.f : ptx::ex2(r[0] - m);
            o += f * r[2 + d];
            l += f * r[1];
          }
          if (KV8) o *= a.v_scale;
          if (!CL && begins && ends) {  // the pair is finished here
            put_row<D>(a, (size_t)(h0 + hd), d, m, l, o);
          } else {
            part[hd * (D + 2) + 2 + d] = o;
            if (d == 0) { part[hd * (D + 2)] = m; part[hd * (D + 2) + 1] = l; }
          }
        }
      }
    }
  }
  // the joining kernel, or the next call's, may be set up now (it waits for these results; let in at the start
  // its blocks got in the way: one KV head of 128K 22.0 us against 20.2, one user with 8K 6.9 against 6.7)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (!CL) {
    if (!a.by_pair && threadIdx.x == 0) a.rec[c] = rec;
  } else {
    // ---- join the cluster's CTAs: each writes its part of the pair's outputs
    float* part = reinterpret_cast<float*>(smem);
    if (w0 >= w1 && (int)threadIdx.x < grp) {
      part[threadIdx.x * (D + 2)] = -INFINITY;
      part[threadIdx.x * (D + 2) + 1] = 0.f;
    }
    __syncwarp();
    cluster_sync();
    const int k = a.cluster, rank = c % k, each = (grp * D + k - 1) / k;
    for (int x = rank * each + threadIdx.x; x < imin(grp * D, (rank + 1) * each); x += kWarps * 32) {
      const int hd = x / D, d = x - hd * D;
      const float* p = part + hd * (D + 2);
      // (all loads of a kind are on their way before the first is used)
      float mr[kMaxCluster], lr[kMaxCluster], om[kMaxCluster], m = -INFINITY, o = 0.f, l = 0.f;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        mr[r] = -INFINITY;
        lr[r] = 0.f;
        if (r < k) mr[r] = cluster_ld(p, r);
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < k) {
          lr[r] = cluster_ld(p + 1, r);
          om[r] = cluster_ld(p + 2 + d, r);
        }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) m = fmaxf(m, mr[r]);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        const float f = mr[r] == -INFINITY ? 0.f : ptx::ex2(mr[r] - m);
        l += f * lr[r];  // (0 times NaN is NaN: a CTA that saw nothing else still counts)
        if (mr[r] != -INFINITY) o += f * om[r];  // (no such CTA, or its outputs were not written)
      }
      const size_t h = (size_t)first_item * grp + hd;
      put_row<D>(a, h, d, m, l, o);
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another still reads from it
  }
}

// Joins the pieces of a pair that several CTAs share; one block per (record, head of the group).  Warp w
// takes pieces w, w + warps, ..; the pieces' order is fixed.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const __grid_constant__ PagedDecodeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int hd = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int4 rec = a.rec[blockIdx.x];
  if (rec.x < 0) return;
  constexpr int E = D / 32;
  __shared__ float sm[kJoinWarps], sl[kJoinWarps], so[kJoinWarps][D];
  const int c = rec.y, n = rec.z - c + 1;
  const size_t slot = (size_t)a.grp * (D + 2);
  // piece 0 is CTA c's last segment, piece i CTA c + i's first
  auto piece = [&](int i) { return a.part + (i == 0 ? 2 * (size_t)c + 1 : 2 * ((size_t)c + i)) * slot + hd * (D + 2); };
  float m = -INFINITY;
  for (int i = threadIdx.x; i < n; i += blockDim.x) m = fmaxf(m, piece(i)[0]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) sm[warp] = m;
  __syncthreads();
  m = sm[0];
  for (int w = 1; w < warps; ++w) m = fmaxf(m, sm[w]);
  float acc[E] = {}, l = 0.f;
#pragma unroll 8
  for (int i = warp; i < n; i += warps) {
    const float* p = piece(i);
    const float f = p[0] == -INFINITY ? 0.f : ptx::ex2(p[0] - m);
    l += f * p[1];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += f * p[2 + lane + 32 * e];
  }
  if (lane == 0) sl[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = acc[e];
  __syncthreads();
  if (threadIdx.x >= D) return;
  const int d = threadIdx.x;
  l = sl[0];
  float o = so[0][d];
  for (int w = 1; w < warps; ++w) { l += sl[w]; o += so[w][d]; }
  const size_t h = (size_t)rec.x * a.grp + hd;
  put_row<D>(a, h, d, m, l, o);
}

template <int D, bool KV8, bool BIG>
cudaError_t launch_paged_t(const PagedDecodeArgs& a, cudaStream_t s) {
  const int bytes = Geo<D, KV8, BIG>::smem(a.grp);
  // the kernels are set up while the one before them runs, and wait for its results themselves
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e;
  // (what a kernel may ask for is set to the same value by every call: calls of other groups may be between
  // this and their launch in other threads)
  constexpr int most = Geo<D, KV8, BIG>::kMostSmem;
  if (a.cluster > 0) {
    auto kern = paged_split_kernel<D, KV8, true, BIG>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most)) != cudaSuccess) return e;
    if (a.cluster > 8 &&
        (e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
      return e;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = a.cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3((unsigned)(a.B * a.Hkv * a.cluster));
    return cudaLaunchKernelEx(&cfg, kern, a);
  }
  auto kern = paged_split_kernel<D, KV8, false, BIG>;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most)) != cudaSuccess) return e;
  cfg.gridDim = dim3(a.grid);
  if ((e = cudaLaunchKernelEx(&cfg, kern, a)) != cudaSuccess) return e;
  // a pair in many pieces is one of few: more warps for it
  cfg.gridDim = dim3(a.by_pair ? a.B * a.Hkv : a.grid, a.grp);
  cfg.blockDim = dim3(a.grid >= 8 * a.B * a.Hkv ? kJoinWarps * 32 : 128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, a);
}

}  // namespace

// How a paged decode is laid out.  grid: CTAs that share the list of all tiles, as many as the GPU holds at
// once, and no more than there can be tiles (0: more tiles than the kernels can count).  cluster > 0:
// instead, a cluster of so many CTAs per pair: 16 if all fit one CTA an SM (16 at two an SM are slower
// than 8: 18.8 against 14.0 us for 16 pairs of 6,200 keys), else 8 or 4 with which all fit the GPU at
// once, if then no CTA can have more than kClusterTiles tiles.  With fewer than 4 the list is as fast or
// faster (296 pairs of up to 680 keys in the cluster form: 21.6 us full, 18.8 ragged; 22.4 and 13.6 as a list).
PagedPlan paged_decode_plan(const Pat& p, int B, int Hq, int Hkv, int d, bool kv8, int max_pages, int page_size) {
  const int grp = Hq / Hkv;
  const int most = 148 * (kv8       ? (grp > 5 ? Geo<128, true, true>::ctas(grp) : Geo<128, true, false>::ctas(grp))
                          : d == 128 ? Geo<128, false, false>::ctas(grp)
                                     : Geo<64, false, false>::ctas(grp));
  const int64_t cap = (int64_t)max_pages * page_size, R = (int64_t)p.T - p.S, pairs = (int64_t)B * Hkv;
  const int64_t wide = R > 0 ? (R + p.H - 1) / p.H : 0;
  auto tiles = [&](int64_t n) { return n > 0 ? ((n < cap ? n : cap) + kTok - 1) / kTok + 1 : 0; };
  int64_t n = tiles(p.S) + tiles(wide) + tiles(p.L);
  const int64_t all = (cap + kTok - 1) / kTok + 2;  // (the ranges lie in the cache, and do not overlap)
  n = n < all ? n : all;
  PagedPlan plan{0, 0};
  const int kSegment = kv8 ? kSegmentOf<true> : kSegmentOf<false>;
  if (n + kSegment > 0x7fffffff / pairs) return plan;  // the kernels count tiles in 32 bits
  plan.grid = (int)((n + kSegment) * pairs < most ? (n + kSegment) * pairs : most);
  const int k = pairs * 16 <= 148 ? 16 : (pairs * 8 <= most ? 8 : 4);
  if (pairs * k <= most && (n + k - 1) / k <= kClusterTiles) plan.cluster = k;
  return plan;
}

size_t paged_decode_bytes(int grid, int grp, int d) {
  return align_up((size_t)grid * sizeof(int4), 256) + align_up((size_t)2 * grid * grp * (d + 2) * sizeof(float), 256);
}

cudaError_t launch_paged_decode(const PagedDecodeArgs& a, int d, bool kv8, cudaStream_t s) {
  if (kv8 && d == 128) return a.grp > 5 ? launch_paged_t<128, true, true>(a, s) : launch_paged_t<128, true, false>(a, s);
  if (!kv8 && d == 64) return launch_paged_t<64, false, false>(a, s);
  if (!kv8 && d == 128) return launch_paged_t<128, false, false>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace cowa
