// cowa_rope.cu -- rotary positions with one to four axes, and the write of a step's tokens into a
// paged cache (the queries and keys rotated on the way).
//
// A rotation turns pairs (a, b) of a head's elements by an angle that depends on the token:
//   angle(t, i) = pos[axis(i)][t] * inv_freq[i],   i = 0 .. r/2 - 1
//   (a, b) -> scale * (a cos - b sin, b cos + a sin)
// Pair i is (i, i + r/2) or, interleaved, (2i, 2i + 1); elements r .. d-1 pass through.  Its
// transpose, which the backward pass needs, is the rotation by the negated angle.
//
// Angles are formed in 64 bits (int32 position times fp32 frequency) and reduced to a fraction of a
// turn there: at position 100000 an fp32 product is off by 0.004 radians.  Sine and cosine of the
// reduced angle, and the rotation itself, are in 32 bits; the result is rounded once.  (Keys that
// become E4M3 codes are rotated in 64 bits, see below.)
//
// Bound: every element is read and written once, so HBM.  A block owns a few tokens and all their
// heads: the angles of a token are computed once, into shared memory, and used by all its heads; the
// rows are then moved with 16-byte loads and stores, each thread fetching its next row before it
// turns the one it has.
#include <cuda_bf16.h>

#include "cowa_internal.h"

namespace cowa {
namespace {

constexpr int kMaxTok = 8;  // tokens per block, at most

// How a row is cut into units of work:
//   kSplit  8 pairs (i, i + r/2): two 16-byte pieces r/2 elements apart   (r/2 a multiple of 8)
//   kInter  8 pairs (2i, 2i + 1): two 16-byte pieces side by side          (r a multiple of 8; also no
//           rotation at all); with r = 8 mod 16 the last unit's second piece passes through
//   kAny    one 16-byte piece, its partners wherever they are, through shared memory
enum { kSplit, kInter, kAny };
// What becomes of the rows: rotated copies; bf16 pages; pages of E4M3 codes
enum { kTurn, kPagesBf16, kPagesE4m3 };
// Threads of a block.  (E4M3 pages, where the angles in 64 bits take long: smaller blocks wait for them
// in smaller numbers, 41.4 us against 43.3 for 8K tokens; the others lose 2% that way.)
template <int MODE>
constexpr int kThreadsOf = MODE == kPagesE4m3 ? 128 : 256;

// bytes of a block's fp32 cos and sin tables (whole units of 8 pairs), and of all its shared memory
__host__ __device__ inline int whole_pairs(int half) { return (half + 7) / 8 * 8; }
__host__ __device__ inline size_t table_bytes(int tok, int half) { return (size_t)tok * whole_pairs(half) * 8; }
inline size_t smem_bytes(int mode, int tok, int half, int Hk) {
  return table_bytes(tok, half) + (mode == kPagesE4m3 ? (size_t)tok * whole_pairs(half) * 16 : 0) + (mode == kTurn ? 0 : (size_t)tok * Hk * 16);
}

struct Row {
  uint4 lo, hi;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void widen8(const uint4& v, float* x) {
  x[0] = bf_lo(v.x); x[1] = bf_hi(v.x); x[2] = bf_lo(v.y); x[3] = bf_hi(v.y);
  x[4] = bf_lo(v.z); x[5] = bf_hi(v.z); x[6] = bf_lo(v.w); x[7] = bf_hi(v.w);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 narrow8(const float* x) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
// E4M3 codes of x * inv: a float32 product, then round to nearest even, saturating (as the quantiser)
__device__ __forceinline__ uint2 codes8(const float* x, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(x[2 * i + 1] * inv), "f"(x[2 * i] * inv));
    w[i] = c;
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <int MODE, int CUT>
__global__ void __launch_bounds__(kThreadsOf<MODE>, 1024 / kThreadsOf<MODE>)
    turn_kernel(const __grid_constant__ RopeArgs a, int tok_per_block) {
  constexpr int kThreads = kThreadsOf<MODE>;
  // cos and sin of the block's tokens.  kSplit and kInter: [token][piece][unit] of float4, the pieces
  // being the unit's 8 cosines and then its 8 sines, so that neighbouring units are neighbours in
  // memory.  kAny: [token][pair] of (cos, sin).
  extern __shared__ __align__(16) unsigned char smem[];
  float* tab = reinterpret_cast<float*>(smem);
  // E4M3 keys: cos and sin in 64 bits, [token][pair of the unit][unit] (kAny: [token][pair])
  double2* tab64 = reinterpret_cast<double2*>(smem + table_bytes(tok_per_block, a.half));
  // element offset of each (token, KV head)'s key and value row in the pools, -1 for none
  longlong2* dst = reinterpret_cast<longlong2*>(tab64 + (MODE == kPagesE4m3 ? tok_per_block * whole_pairs(a.half) : 0));
  __shared__ int live[kMaxTok];
  __shared__ __align__(16) __nv_bfloat16 stage[CUT == kAny ? kThreads * 8 : 8];

  // set up while the kernel before it in the stream ran (it waits for that one's results here), as the
  // one after it may be
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const long long m0 = (long long)blockIdx.x * tok_per_block;
  const int nt = (int)(a.M - m0 < tok_per_block ? a.M - m0 : tok_per_block);
  const int b0 = MODE == kTurn ? (int)(m0 / a.N) : 0, t0 = (int)(m0 - (long long)b0 * a.N);  // of the first token
  const int half = a.half, rd = 2 * half;
  const int rot_units = CUT == kAny ? 0 : (half + 7) / 8;
  const int units = CUT == kSplit ? rot_units + (a.d - rd) / 8 : (CUT == kInter ? a.d / 16 : a.d / 8);
  const int lanes = kThreads / units;  // rows in flight
  const int heads = a.Hq + a.Hk + (MODE == kTurn ? 0 : a.Hk);
  const int u = tid % units;
  const bool active = tid < lanes * units;

  // The block's rows in order of (token, head); a thread's next one is `lanes` further on.  (b, t): the
  // token's place in its tensors; an append has one axis of tokens, and needs neither.
  struct At {
    int tok, head, b, t;
  };
  auto t_of = [&](const At& x) -> int64_t { return MODE == kTurn ? x.t : t0 + x.tok; };
  const int step_tok = lanes / heads, step_head = lanes % heads;
  At at{(tid / units) / heads, (tid / units) % heads, b0, t0};
  at.t += at.tok;
  auto wrap = [&](At& x) {
    if (MODE == kTurn)
      while (x.t >= a.N) { x.t -= a.N; ++x.b; }
  };
  wrap(at);
  auto next = [&](At& x) {
    int n = step_tok;
    x.head += step_head;
    if (x.head >= heads) { x.head -= heads; ++n; }
    x.tok += n;
    if (MODE == kTurn) {
      x.t += n;
      wrap(x);
    }
  };
  auto fetch = [&](const At& x) -> Row {
    const __nv_bfloat16* p;
    const int64_t t = t_of(x);
    if (x.head < a.Hq) p = a.q + (MODE == kTurn ? x.b * a.q_sb : 0) + t * a.q_st + x.head * a.q_sh;
    else if (MODE == kTurn) p = a.k + x.b * a.k_sb + t * a.k_st + (x.head - a.Hq) * a.k_sh;
    else if (x.head < a.Hq + a.Hk) p = a.k + t * a.k_st + (x.head - a.Hq) * a.k_sh;
    else p = a.v + t * a.v_st + (x.head - a.Hq - a.Hk) * a.v_sh;
    Row r;
    r.hi = make_uint4(0, 0, 0, 0);
    if (CUT == kSplit && u < rot_units) {
      r.lo = *reinterpret_cast<const uint4*>(p + 8 * u);
      r.hi = *reinterpret_cast<const uint4*>(p + half + 8 * u);
    } else if (CUT == kInter) {
      r.lo = *reinterpret_cast<const uint4*>(p + 16 * u);
      r.hi = *reinterpret_cast<const uint4*>(p + 16 * u + 8);
    } else {
      r.lo = *reinterpret_cast<const uint4*>(p + (CUT == kSplit ? rd + 8 * (u - rot_units) : 8 * u));
    }
    return r;
  };
  // the rows at hand, fetched before the angles are computed; kRows of them, so that enough bytes
  // are on their way
  constexpr int kRows = CUT == kAny ? 2 : 1;
  Row cur[kRows];
  At where[kRows];
  auto refill = [&]() {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      where[i] = at;
      if (active && at.tok < nt) cur[i] = fetch(at);
      next(at);
    }
  };
  refill();

  for (int x = tid; x < nt * half; x += kThreads) {
    const int tk = x / half, i = x - tk * half;
    const int axis = (i >= a.end0) + (i >= a.end1) + (i >= a.end2);
    int p;
    if (a.pos) {
      At x0{0, 0, b0, t0 + tk};
      wrap(x0);
      p = a.pos[axis * a.pos_sa + x0.b * a.pos_sb + x0.t];
    } else if (MODE == kTurn) {
      At x0{0, 0, b0, t0 + tk};
      wrap(x0);
      p = x0.t;
    } else {
      p = a.cache_pos[m0 + tk];
    }
    double turns = (double)p * (double)a.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    if (MODE == kPagesE4m3) {
      double s64, c64;
      sincospi(2.0 * turns, &s64, &c64);
      s64 *= (double)a.sin_scale;
      c64 *= (double)a.scale;
      tab64[CUT == kAny ? x : (tk * 8 + i % 8) * rot_units + i / 8] = make_double2(c64, s64);
      s = (float)s64;
      c = (float)c64;
    } else {
      sincospif((float)(2.0 * turns), &s, &c);
      c *= a.scale;
      s *= a.sin_scale;
    }
    if (CUT == kAny) {
      reinterpret_cast<float2*>(tab)[x] = make_float2(c, s);
    } else {
      const int un = i / 8, j = i % 8;
      float* base = tab + (size_t)tk * 16 * rot_units + 4 * un + (j & 3);
      base[(j >> 2) * 4 * rot_units] = c;
      base[(2 + (j >> 2)) * 4 * rot_units] = s;
    }
  }
  if (MODE != kTurn) {
    for (int x = tid; x < nt * a.Hk; x += kThreads) {
      const int tk = x / a.Hk, g = x - tk * a.Hk;
      const int p = a.cache_pos[m0 + tk];
      const long long sq = a.seq ? a.seq[m0 + tk] : m0 + tk;
      const bool on = p >= 0 && sq >= 0 && sq < a.tab.n_seq;
      long long ok = -1, ov = -1;
      if (on && p / a.tab.page_size < a.tab.max_pages) {
        const int page = a.tab.ptr[sq * a.tab.sb + g * a.tab.sh + p / a.tab.page_size];
        if (page >= 0 && page < a.tab.n_pages) {
          const int slot = p % a.tab.page_size, gh = a.tab.sh ? 0 : g;
          ok = page * a.kp_sp + slot * a.kp_st + gh * a.kp_sh;
          ov = page * a.vp_sp + slot * a.vp_st + gh * a.vp_sh;
        }
      }
      dst[x] = make_longlong2(ok, ov);
      if (g == 0) live[tk] = on;
    }
  }
  __syncthreads();

  // turns one row's unit and writes it where it belongs
  auto put = [&](const Row& r, const At& x, bool mine) {
    if (CUT == kAny) {
      // the row's pieces side by side in shared memory, for the partners of this one's elements
      __syncthreads();
      if (mine) *reinterpret_cast<uint4*>(stage + 8 * tid) = r.lo;
      __syncthreads();
    }
    if (!mine) return;
    const bool is_q = x.head < a.Hq, is_v = MODE != kTurn && x.head >= a.Hq + a.Hk;
    float lo[8], hi[8];
    widen8(r.lo, lo);
    if (CUT != kAny) widen8(r.hi, hi);
    const bool exact = MODE == kPagesE4m3 && !is_q;
    if (!is_v) {
      if (CUT == kAny) {
        const __nv_bfloat16* whole = stage + 8 * (tid - u);
        for (int e = 0; e < 8; ++e) {
          const int n = 8 * u + e;
          if (n >= rd) break;
          const int i = a.interleaved ? n >> 1 : (n < half ? n : n - half);
          const bool second = a.interleaved ? (n & 1) : n >= half;
          const int y = a.interleaved ? n ^ 1 : (second ? n - half : n + half);
          const float other = __bfloat162float(whole[y]);
          if (exact) {
            const double2 cs = tab64[x.tok * half + i];
            lo[e] = (float)(second ? fma((double)lo[e], cs.x, (double)other * cs.y)
                                   : fma((double)lo[e], cs.x, -((double)other * cs.y)));
          } else {
            const float2 cs = reinterpret_cast<const float2*>(tab)[x.tok * half + i];
            lo[e] = second ? fmaf(lo[e], cs.x, other * cs.y) : fmaf(lo[e], cs.x, -(other * cs.y));
          }
        }
      } else if (u < rot_units) {
        if (exact) {
          const double2* cs = tab64 + x.tok * 8 * rot_units + u;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (CUT == kInter && j >= 4 && 8 * u + j >= half) break;
            float& ea = CUT == kSplit ? lo[j] : (j < 4 ? lo[2 * j] : hi[2 * j - 8]);
            float& eb = CUT == kSplit ? hi[j] : (j < 4 ? lo[2 * j + 1] : hi[2 * j - 7]);
            const double2 t = cs[j * rot_units];
            const double xa = ea, xb = eb, c = t.x, s = t.y;
            ea = (float)fma(xa, c, -(xb * s));
            eb = (float)fma(xb, c, xa * s);
          }
        } else {
          const float4* cs = reinterpret_cast<const float4*>(tab + (size_t)x.tok * 16 * rot_units) + u;
          float c[8], s[8];
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const float4 cw = cs[w * rot_units], sw = cs[(2 + w) * rot_units];
            c[4 * w] = cw.x; c[4 * w + 1] = cw.y; c[4 * w + 2] = cw.z; c[4 * w + 3] = cw.w;
            s[4 * w] = sw.x; s[4 * w + 1] = sw.y; s[4 * w + 2] = sw.z; s[4 * w + 3] = sw.w;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (CUT == kInter && j >= 4 && 8 * u + j >= half) break;
            float& ea = CUT == kSplit ? lo[j] : (j < 4 ? lo[2 * j] : hi[2 * j - 8]);
            float& eb = CUT == kSplit ? hi[j] : (j < 4 ? lo[2 * j + 1] : hi[2 * j - 7]);
            const float xa = ea, xb = eb;
            ea = fmaf(xa, c[j], -(xb * s[j]));
            eb = fmaf(xb, c[j], xa * s[j]);
          }
        }
      }
    }
    // elements [e1, e1 + 8) and, where the unit has two pieces, [e2, e2 + 8)
    const bool two = CUT == kInter || (CUT == kSplit && u < rot_units);
    const int e1 = CUT == kSplit && !two ? rd + 8 * (u - rot_units) : (CUT == kInter ? 16 * u : 8 * u);
    const int e2 = CUT == kInter ? e1 + 8 : half + 8 * u;
    if (MODE == kTurn || is_q) {
      if (MODE != kTurn && !live[x.tok]) return;
      const int64_t t = t_of(x);
      __nv_bfloat16* o = is_q ? a.qo + (MODE == kTurn ? x.b * a.qo_sb : 0) + t * a.qo_st + x.head * a.qo_sh
                              : a.ko + x.b * a.ko_sb + t * a.ko_st + (x.head - a.Hq) * a.ko_sh;
      *reinterpret_cast<uint4*>(o + e1) = narrow8(lo);
      if (two) *reinterpret_cast<uint4*>(o + e2) = narrow8(hi);
    } else {
      const int g = x.head - a.Hq - (is_v ? a.Hk : 0);
      const longlong2 at_kv = dst[x.tok * a.Hk + g];
      const long long off = is_v ? at_kv.y : at_kv.x;
      if (off < 0) return;
      if (MODE == kPagesBf16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(is_v ? a.vp : a.kp) + off;
        *reinterpret_cast<uint4*>(o + e1) = narrow8(lo);
        if (two) *reinterpret_cast<uint4*>(o + e2) = narrow8(hi);
      } else {
        uint8_t* o = static_cast<uint8_t*>(is_v ? a.vp : a.kp) + off;
        const float inv = is_v ? a.inv_v : a.inv_k;
        *reinterpret_cast<uint2*>(o + e1) = codes8(lo, inv);
        if (two) *reinterpret_cast<uint2*>(o + e2) = codes8(hi, inv);
      }
    }
  };

  // a whole number of passes for every thread: kAny exchanges pieces within the block
  const int passes = (nt * heads + kRows * lanes - 1) / (kRows * lanes);
  for (int it = 0; it < passes; ++it) {
    Row row[kRows];
    At of[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) { row[i] = cur[i]; of[i] = where[i]; }
    if (it + 1 < passes) refill();
#pragma unroll
    for (int i = 0; i < kRows; ++i) put(row[i], of[i], active && of[i].tok < nt);
  }
}

template <int MODE>
cudaError_t launch_turn(const RopeArgs& a, cudaStream_t s) {
  const int rd = 2 * a.half;
  const int cut = a.half == 0 || (a.interleaved && rd % 8 == 0) ? kInter
                  : !a.interleaved && a.half % 8 == 0           ? kSplit
                                                                : kAny;
  const int units = cut == kSplit ? a.half / 8 + (a.d - rd) / 8 : (cut == kInter ? a.d / 16 : a.d / 8);
  const int heads = a.Hq + (MODE == kTurn ? 1 : 2) * a.Hk;
  const int lanes = kThreadsOf<MODE> / units;
  // Tokens per block: what takes the fewest passes over rows, in the turns that the blocks take on the SMs; a
  // block's start costs about half a pass, an angle a thread 0.2 (in 64 bits 0.6), one more block on an SM
  // 0.1.  (Against powers of two as large as leave eight blocks an SM: 4K tokens of 32/8 heads 18.3 -> 16.6 us
  // with 7, 2K of 40/8 13.0 -> 11.1 with 4, 8K appended as E4M3 codes 41.2 -> 39.9 with 7, 7.5K of 8/1
  // appended in bf16 15.7 -> 12.3; 32K the same.)
  int tok = 1;
  double least = 1e30;
  for (int n = 1; n <= kMaxTok && (n == 1 || smem_bytes(MODE, n, a.half, a.Hk) <= 32 * 1024); ++n) {
    const int at_once = 148 * imin(1024 / kThreadsOf<MODE>, (int)(228 * 1024 / (smem_bytes(MODE, n, a.half, a.Hk) + 1024)));
    const long long blocks = (a.M + n - 1) / n, turns = (blocks + at_once - 1) / at_once;
    const long long rows = (long long)lanes * (cut == kAny ? 2 : 1), passes = ((long long)n * heads + rows - 1) / rows;
    const int angles = (n * a.half + kThreadsOf<MODE> - 1) / kThreadsOf<MODE>;  // a thread's
    const double cost = (double)turns * (passes + 0.5 + (MODE == kPagesE4m3 ? 0.6 : 0.2) * angles) +
                        0.1 * ((blocks + 147) / 148);
    if (cost < least || (cost == least && turns > 1)) { least = cost; tok = n; }
  }
  const long long blocks = (a.M + tok - 1) / tok;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const size_t smem = smem_bytes(MODE, tok, a.half, a.Hk);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreadsOf<MODE>);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  auto kern = cut == kSplit ? turn_kernel<MODE, kSplit> : (cut == kInter ? turn_kernel<MODE, kInter> : turn_kernel<MODE, kAny>);
  return cudaLaunchKernelEx(&cfg, kern, a, tok);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) { return launch_turn<kTurn>(a, s); }

cudaError_t launch_paged_append(const RopeArgs& a, bool e4m3, cudaStream_t s) {
  return e4m3 ? launch_turn<kPagesE4m3>(a, s) : launch_turn<kPagesBf16>(a, s);
}

}  // namespace cowa
