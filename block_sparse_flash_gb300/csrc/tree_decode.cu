// tree_decode.cu -- attention of a tree of drafted tokens over a paged cache
// (splash_paged_tree_decode in splash.h).  Compiled once for each cache type
// (SPLASH_TREE_E4M3 = 0, 1), so that the instantiations build in parallel.
//
// For a row (query head h, token l): s_j = scale q.k_j over the keys it sees --
// the context and its ancestors --, out = sum exp(s_j - m) v_j / sum exp(s_j - m),
// lse = m + ln sum exp(s_j - m), in one pass over the keys.
//
// A KV head has Hq/Hkv * T rows, up to hundreds, that share its keys: `rows` FLOP per
// byte of a bf16 cache, 2 rows of an e4m3 one.  By these reading the cache bounds the call up
// to some 290 rows in bf16 (190 with the second term of P, see the softmax) and 145 in e4m3, the
// products beyond, so that the rows are the 128 lanes of tensor memory and the cache is
// read once for 256 of them.
//
//  * Work.  As in paged_decode: the steps of 64 keys of all (sequence, KV head, row
//    group) segments form one list and every CTA, one per SM, takes an equal contiguous
//    part; a segment's start counts as nine more steps.  Segments in whole are finished
//    there, parts go to the workspace and a second kernel joins them in the order of the
//    keys: the result does not depend on timing.  Where there are few segments and none can
//    be very long, each takes a cluster of CTAs, whose parts are joined through distributed
//    shared memory: no scan, no workspace, no second kernel.
//  * Warps.  One loads boxes of the pages (TMA), one issues the products
//    (tcgen05.mma, S = Q K^T from shared memory, O += P V with P from tensor memory), two
//    groups of four do the softmax, a thread per row; for e4m3 four widen the keys and
//    values to fp16 on the way.  More than 128 rows: a group per tile of 128, both on the
//    same keys.  Fewer: the groups take even and odd steps, so that two softmaxes are
//    under way in either case.
//  * Masks.  A row's keys are a range of the context and 64 bits for the tree, from its
//    ancestors.  Only the steps at a window's start and at the tree are masked.
//
// Measured (device time, 32 query and 8 KV heads of 128 unless said; us, and what bounds
// it): 32 requests of 32 .. 4096 tokens and 32 drafts, bf16, 84 (floor 44: a step of 64
// keys arrives every 1700 cycles, 1390 at the copy rate, and a segment's start and end cost
// 19000 of which the other SMs hide nothing); 16 requests of up to 32768 tokens and 64 drafts,
// e4m3, 250 (floor 149, the products: shared memory, which the products' operands, the
// widening and the loads fill to 80 %); 1 request of 300 tokens and 16 drafts 10.0 (the launch,
// eight dependent reads, the first fetch of the code).  Of these the join of the parts is 12, 19
// and 0.  19 requests of 8192 tokens, 32 drafts, a segment a CTA: 121 (floor 95).
//
// Up to 16 rows of a KV head go to paged_decode's kernel (kFewRows below).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <mutex>

#include "cluster.cuh"
#include "dependent_launch.cuh"
#include "internal.h"
#include "sm103_ptx.cuh"

namespace splash {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

constexpr int kMaxCtas = 160;              // of the grid; the workspace holds two parts for each
// A piece's start and end cost a CTA about as much as this many steps: a segment
// counts for so many more when the list is cut into equal parts.  (With 2, 6, 9, 12 and 16,
// us: 32 requests of up to 4096 tokens, 8 drafts 79.5, 72.1, 73.1, 74.1, 76.0, 32 drafts 100.2,
// 86.0, 83.9, 84.4, 85.6, 64 drafts 128.2, 113.5, 114.8, 117.1, 119.1; in e4m3, up to 8192 tokens, 32
// drafts 147.5, 122.9, 120.5, 121.4, 123.0, 16 requests of up to 32768 and 64 drafts 282.9, 259.3,
// 250.1, 247.7, 249.0; segments of one length 121.4 with any.)
constexpr int kPieceSteps = 9;
constexpr uint64_t kTimeoutNs = 1000000000ull;  // of a wait

// A running maximum is only moved when a score passes it by more than this (in
// powers of two): until then exp2(s - m) stays below 2^8, and the output in
// tensor memory need not be rescaled.
constexpr float kSlack = 8.f;
// For an e4m3 cache the reference is this much below the maximum, so that the
// probabilities use fp16 from the top: 2^7 for the largest key, below 2^15 with
// the slack.  What is dropped at the bottom, half of fp16's 2^-24, is 2^-32 of the
// largest key.
constexpr float kBelowTop = 7.f;
// The smallest factor of the scores: a masked one (-inf) stays -inf times it.  (fp32's
// smallest number: with its smallest normal one a scale below that would be rounded up to it,
// which is wrong by any power of two where the queries are as large as the scale is small.)
constexpr float kTiny = 0x1p-149f;

struct Params {
  const char *q;
  int64_t q_b, q_h, q_l;  // byte strides
  const char *v;
  int64_t v_page, v_head, v_token;  // byte strides
  // coordinates of a head and a page in the tensor maps: times 0 where the tensor repeats
  // them; the first page coordinate outside, which reads as zeros
  int32_t k_head_on, v_head_on, k_page_on, v_page_on, k_page_end, v_page_end;
  const float *k_scale, *v_scale;
  const int32_t *block_table;
  int64_t block_table_stride;
  const int32_t *seq_lens, *parents;
  int64_t parents_stride;
  __nv_bfloat16 *out;
  float *lse;
  float *part_o, *part_ml;  // [2 * CTAs][part_rows][DV], [2 * CTAs][part_rows][2] (maximum, sum)
  int32_t *lost;            // [CTAs] whether it put zeros in the place of values
  int32_t *before;          // [B + 1] list entries (of one head and row group) before each sequence's
  int64_t num_pages;
  int32_t B, Hkv, T, G, nrows, row_groups, part_rows;  // nrows = G * T rows per KV head
  int32_t max_pages, page_shift, window;               // window < 0: none
  uint32_t over_T;                                     // rounded up 2^32 / T: n / T for n T < 2^32
  int32_t ctas;                                        // of the grid
  float scale, cap;                                    // cap <= 0: none
  bool out_wide;                                       // out is 32-byte aligned
  uint32_t *err;
};

// Steps of KW keys for two groups of four softmax warps.  PAIR: 129 rows of a KV head
// and more, two tiles of 128 rows that share the keys.  Otherwise one tile of rows,
// and the groups take turns: even and odd steps, each with its own maximum, sum and
// output, joined at a piece's end.
template <int DQK_, int DV_, bool E4M3_, bool PAIR_>
struct Config {
  static constexpr int DQK = DQK_, DV = DV_, KW = 64;
  static constexpr bool E4M3 = E4M3_, PAIR = PAIR_;
  static constexpr int NT = PAIR ? 2 : 1, TILE = 128 * NT;                   // tiles of rows, rows
  static constexpr int RK = DQK * (E4M3 ? 1 : 2), RV = DV * (E4M3 ? 1 : 2);  // bytes of a cache row
  // Operand tiles in shared memory: 64-element (128-byte) columns of rows, 128-byte swizzle.
  static constexpr int COLUMN = KW * 128, K_BYTES = KW * DQK * 2, STAGE = K_BYTES + KW * DV * 2;
  static constexpr int Q_COLUMN = 128 * 128, Q_BYTES = 128 * DQK * 2;
  static constexpr int RAW = E4M3 ? KW * (RK + RV) : 0;  // an e4m3 step as it is in the cache
  static constexpr int ROOM = 222 * 1024 - NT * Q_BYTES;
  // (a step's scores are computed LOOK steps before its products with the values)
  static constexpr int LOOK = PAIR ? 1 : 2;
  static constexpr int STAGES = E4M3 ? (ROOM >= 4 * STAGE + 3 * RAW ? 4 : ROOM >= 3 * STAGE + 2 * RAW ? 3 : 2)
                                     : std::min(8, ROOM / STAGE);
  static constexpr int RAWS = E4M3 ? std::min(6, (ROOM - STAGES * STAGE) / std::max(RAW, 1)) : 0;
  static constexpr int TILES = NT * Q_BYTES + STAGES * STAGE + RAWS * RAW;
  static_assert(STAGES > LOOK && (!E4M3 || RAWS >= 2), "a step's stage is free before it is waited for");
  static_assert(TILE * (DV + 4) * 4 <= TILES, "a cluster's parts fit where the operands were");
  // Barriers: full[STAGES] empty[STAGES], per group s_full[2] p_full[2] q_full o_last, drain, raw_full[RAWS] raw_empty[RAWS]
  static constexpr int BARS = 2 * STAGES + 13 + 2 * RAWS;
  static constexpr int SMEM = 1024 + TILES + BARS * 8;
  // Warps: softmax (8), for e4m3 four that widen, then loads and products.
  static constexpr int LOAD = E4M3 ? 12 : 8, MMA = LOAD + 1, WARPS = MMA + 1, THREADS = 32 * WARPS;
  // Tensor memory: per group two buffers of scores (64 columns each, P in their place) and O.
  static constexpr int GROUP_COLS = 2 * KW + DV, COLS = 512;
  static constexpr uint32_t FORMAT = E4M3 ? 0u : (1u << 7) | (1u << 10);  // fp16 or bf16 operands
  static constexpr uint32_t IDESC_QK = (idesc_bf16_f32(128, KW, false) & ~((1u << 7) | (1u << 10))) | FORMAT;
  static constexpr uint32_t IDESC_PV = (idesc_bf16_f32(128, DV, true) & ~((1u << 7) | (1u << 10))) | FORMAT;
};

// The keys of sequence b that some token sees, in steps of KW.
struct Span {
  int32_t n, ctx, lo;  // keys [lo, n), the tree's from ctx on (negative: some of it has no slot)
  int32_t step0, nst;  // steps step0 .. step0 + nst - 1; at least one, so that empty rows are written too
};

template <int KW>
__device__ __forceinline__ Span span_of(const Params &p, int32_t n) {  // n: the sequence's length as given
  Span s;
  const int64_t most = (int64_t)p.max_pages << p.page_shift;
  s.n = n < 0 ? 0 : n > most ? (int32_t)most : n;
  s.ctx = s.n - p.T;
  s.lo = p.window < 0 ? 0 : max(0, s.ctx - p.window);
  s.step0 = s.lo / KW;
  s.nst = max(1, (s.n + KW - 1) / KW - s.step0);
  return s;
}

// Whether every token sees all of a step's keys.
template <int KW>
__device__ __forceinline__ bool whole(const Params &p, const Span &s, int32_t key0) {
  return key0 + KW <= s.ctx && (p.window < 0 || key0 >= s.ctx + p.T - 1 - p.window);
}

// Equal contiguous parts of T entries: CTA w takes [begin(w), begin(w + 1)).  A segment has kPieceSteps entries for its start, then one
// for each step.
struct Parts {
  int32_t total, count, each, more;  // the first `more` take one entry more
  __device__ __forceinline__ Parts(const Params &p, int32_t T)
      : total(T), count(max(1, min(p.ctas, T))), each((uint32_t)T / (uint32_t)count), more(T - each * count) {}
  __device__ __forceinline__ int32_t begin(int32_t w) const { return w >= count ? total : each * w + min(w, more); }
  __device__ __forceinline__ int32_t owner(int32_t u) const {
    const int32_t cut = (each + 1) * more;
    return u < cut ? (uint32_t)u / (uint32_t)(each + 1) : more + (uint32_t)(u - cut) / (uint32_t)each;
  }
};

// A CTA's way through its part of the list: pieces, each some steps of one segment
// (sequence b, head and row group seg).
struct Piece {
  int32_t b, seg, step, steps;
  Span s;
  // Where a part of the segment goes in the workspace, -1 for a segment in whole.  A CTA has
  // at most one that begins a segment and one that goes on with another.
  __device__ __forceinline__ int slot(int cta) const { return steps == s.nst ? -1 : 2 * cta + (step == 0 ? 1 : 0); }
};
template <int KW>
struct Walk {
  const Params &p;
  int32_t u, end, per_seq;
  int32_t b, seg, entry;  // the entry of segment seg that u is
  int32_t length;         // of sequence b, as given (read when b is entered, needed at its first piece)
  __device__ __forceinline__ bool next(Piece &x) {
    while (u < end) {
      const Span s = span_of<KW>(p, length);
      const int32_t to = min(s.nst + kPieceSteps, entry + (end - u));
      x.b = b;
      x.seg = seg;
      x.step = max(entry - kPieceSteps, 0);
      x.steps = max(to - kPieceSteps, 0) - x.step;
      x.s = s;
      u += to - entry;
      entry = 0;
      if (++seg == per_seq) {
        seg = 0;
        ++b;
        if (u < end) length = p.seq_lens[b];
      }
      if (x.steps > 0) return true;
    }
    return false;
  }
};

// A token's place in its tree: which tokens it sees (itself among them; none for
// padding), and how many ancestors it has.
struct Branch {
  uint64_t seen;
  int32_t depth;
};

__device__ __forceinline__ Branch branch_of(const int32_t *parents, int l, int first, int window, bool *bad) {
  Branch x = {0, 0};
  int at = l;
  for (;;) {
    if (window < 0 || x.depth <= window) x.seen |= 1ull << at;
    const int32_t up = at < first ? -2 : parents[at];
    if (up == -1) return x;
    if (up < 0 || up >= at) {
      *bad |= up >= at;
      return {0, 0};
    }
    at = up;
    ++x.depth;
  }
}

// The keys of [key0, key0 + 64) that a row sees, as bits: context keys from lo
// on, and its branch.
__device__ __forceinline__ uint64_t visible(int32_t key0, int32_t ctx, int32_t lo, uint64_t seen) {
  const int32_t a = max(0, lo - key0), b = min(64, ctx - key0), d = ctx - key0;
  uint64_t m = b > a ? (b - a >= 64 ? ~0ull : (1ull << (b - a)) - 1) << a : 0;
  m |= d >= 64 || d <= -64 ? 0 : d >= 0 ? seen << d : seen >> -d;
  return seen != 0 ? m : 0;
}

__device__ __forceinline__ uint4 load_shared4(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
  return x;
}
// 4-D tiled load of the box at (x, y, z, w), completing its bytes on the mbarrier; issued by the
// lane of a converged warp whose `leader` is not 0.
__device__ __forceinline__ void load_box(uint32_t leader, uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z, int32_t w,
                                         uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %7, 0;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// Four e4m3 values to two pairs of fp16 (exact).
[[maybe_unused]] __device__ __forceinline__ void widen(uint32_t x, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^x as the factor of a sum of parts: never 0, so that an infinite part stays one (0 x
// infinity would be NaN); 2^-149 of a finite one is nothing.
__device__ __forceinline__ float factor_of(float x) { return fmaxf(ex2_approx(x), 0x1p-149f); }
// A number cut off to bf16.
__device__ __forceinline__ float cut(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// The larger exponent field of a word's two bf16 values, and the word as fp16
// values times `down`.
__device__ __forceinline__ uint32_t exponent(uint32_t x) { return max((x >> 7) & 255u, (x >> 23) & 255u); }
__device__ __forceinline__ uint32_t to_half(uint32_t x, float down) {
  return pack_half2(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xffff0000u) * down);
}

// A word's 16-bit values that are not finite (exponent bits `top` all set) become 0.
__device__ __forceinline__ uint32_t finite(uint32_t x, uint32_t top) {
  if ((x & top) == top) x &= 0xffff0000u;
  if ((x >> 16 & top) == top) x &= 0xffffu;
  return x;
}

// tanh for the soft cap.  Up to 0.25 the forward's polynomial (attention_fwd.cu):
// t (1 + u (c1 + c2 u)), u = t^2, a minimax fit of tanh(t)/t with a relative error
// of 4.8e-7, so that cap * tanh(s / cap) keeps the score's low bits however large
// the cap; above it tanh|x| = (1 - e) / (1 + e), e = exp(-2|x|), whose error is
// absolute.
constexpr float kTanhC1 = -0.33324610f, kTanhC2 = 0.12877172f, kTanhSeriesLimit = 0.25f;
__device__ __forceinline__ float tanh_of(float x) {
  const float u = x * x, e = ex2_approx(-2.f * kLog2e * fabsf(x));
  return fabsf(x) <= kTanhSeriesLimit ? fmaf(x * u, fmaf(u, kTanhC2, kTanhC1), x) : copysignf(__fdividef(1.f - e, 1.f + e), x);
}

// A chunk of 16 e4m3 values into a row of an operand tile.
template <class C>
__device__ __forceinline__ void widen_chunk(const uint4 &y, uint32_t dst, int row, int c) {
  uint32_t w[8];
  widen(y.x, w[0], w[1]);
  widen(y.y, w[2], w[3]);
  widen(y.z, w[4], w[5]);
  widen(y.w, w[6], w[7]);
  dst += (c >> 2) * C::COLUMN + row * 128;
  const int cc = 2 * (c & 3);
  st_shared_v4(dst + ((cc ^ (row & 7)) << 4), w[0], w[1], w[2], w[3]);
  st_shared_v4(dst + (((cc + 1) ^ (row & 7)) << 4), w[4], w[5], w[6], w[7]);
}

template <class C>
struct Bars {
  uint32_t base;
  __device__ __forceinline__ uint32_t full(int s) const { return base + 8u * s; }
  __device__ __forceinline__ uint32_t empty(int s) const { return base + 8u * (C::STAGES + s); }
  __device__ __forceinline__ uint32_t s_full(int t, int x) const { return base + 8u * (2 * C::STAGES + 6 * t + x); }
  __device__ __forceinline__ uint32_t p_full(int t, int x) const { return base + 8u * (2 * C::STAGES + 6 * t + 2 + x); }
  __device__ __forceinline__ uint32_t q_full(int t) const { return base + 8u * (2 * C::STAGES + 6 * t + 4); }
  __device__ __forceinline__ uint32_t o_last(int t) const { return base + 8u * (2 * C::STAGES + 6 * t + 5); }
  __device__ __forceinline__ uint32_t drain() const { return base + 8u * (2 * C::STAGES + 12); }
  __device__ __forceinline__ uint32_t raw_full(int s) const { return base + 8u * (2 * C::STAGES + 13 + s); }
  __device__ __forceinline__ uint32_t raw_empty(int s) const { return base + 8u * (2 * C::STAGES + 13 + C::RAWS + s); }
};

__device__ __forceinline__ void give_up(const Params &p, volatile int *abort, uint32_t bit) {
  atomicOr(p.err, bit);
  *abort = 1;
}

// ------------------------------------------------------------------ loads
// One warp brings the steps of the CTA's part in order, across the borders of
// pieces: boxes of up to 64 rows (16-row pages: four) of the pages, bf16 straight into
// the swizzled operand tiles (a box per 64 columns), e4m3 as it is into a ring of raw
// steps.  The lanes look up 32 blocks at a time and as many ahead (a step at a time, the
// look up cost each step 700 cycles); the warp issues the boxes together.  A box with no visible key, or
// of a page that does not exist, lies outside the tensor and arrives as zeros; a box's
// other rows that no token sees are masked by the softmax.
template <class C>
__device__ __forceinline__ void run_loads(const Params &p, Walk<C::KW> walk, const Bars<C> bar, const CUtensorMap *map_k,
                                          const CUtensorMap *map_v, uint32_t stages, uint32_t raws, volatile int *abort) {
  constexpr int KW = C::KW, CK = C::E4M3 ? 1 : C::DQK / 64, CV = C::E4M3 ? 1 : C::DV / 64;  // boxes of a block's rows
  constexpr int RING = C::E4M3 ? C::RAWS : C::STAGES;
  const int lane = threadIdx.x & 31;
  const uint32_t leader = elect_one_sync();
  const int shift = min(6, p.page_shift), rows = 1 << shift, blocks = KW >> shift, in_page = (1 << p.page_shift) - 1;
  uint32_t n = 0, st = 0, turn = 1;  // steps asked for; the next one's slot, and the parity of its last use
  bool ok = true;
  Piece x;
  while (ok && walk.next(x)) {
    const int head = x.seg / p.row_groups, head_k = head * p.k_head_on, head_v = head * p.v_head_on;
    const int32_t *pages = p.block_table + x.b * p.block_table_stride;
    int32_t key0 = (x.s.step0 + x.step) * KW;
    // the pages of the next 32 blocks, one a lane: -1 where no key is seen, -2 where it does not exist
    auto look = [&](int32_t at) {
      at += lane * rows;
      if (at >= x.s.n || at + rows <= x.s.lo) return -1;
      const int32_t page = pages[at >> p.page_shift];
      return page >= 0 && page < p.num_pages ? page : -2;
    };
    int32_t entries = look(key0), ahead = look(key0 + 32 * rows);
    for (int i = 0, block = 0; i < x.steps; ++i, ++n, key0 += KW, block += blocks) {
      if (block == 32) {
        block = 0;
        entries = ahead;
        ahead = look(key0 + 32 * rows);
      }
      const uint32_t full = C::E4M3 ? bar.raw_full(st) : bar.full(st), empty = C::E4M3 ? bar.raw_empty(st) : bar.empty(st);
      if (n >= RING && !(ok = __all_sync(~0u, mbar_wait(empty, turn, abort, kTimeoutNs)))) break;
      if (leader) mbar_arrive_expect_tx(full, C::E4M3 ? C::RAW : C::STAGE);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= blocks) break;
        const int32_t page = __shfl_sync(~0u, entries, block + j), slot = (key0 + j * rows) & in_page;
        if (page == -2 && leader) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
        const int32_t page_k = page < 0 ? p.k_page_end : page * p.k_page_on, page_v = page < 0 ? p.v_page_end : page * p.v_page_on;
        if constexpr (C::E4M3) {
          const uint32_t to = raws + st * C::RAW;
          load_box(leader, to + j * rows * C::RK, map_k, 0, slot, head_k, page_k, full);
          load_box(leader, to + KW * C::RK + j * rows * C::RV, map_v, 0, slot, head_v, page_v, full);
        } else {
          const uint32_t to = stages + st * C::STAGE + j * rows * 128;
#pragma unroll
          for (int c = 0; c < CK; ++c) load_box(leader, to + c * C::COLUMN, map_k, 64 * c, slot, head_k, page_k, full);
#pragma unroll
          for (int c = 0; c < CV; ++c) load_box(leader, to + C::K_BYTES + c * C::COLUMN, map_v, 64 * c, slot, head_v, page_v, full);
        }
      }
      if (++st == RING) st = 0, turn ^= 1u;
    }
  }
  if (!ok && lane == 0) give_up(p, abort, SPLASH_DEV_TIMEOUT_PRODUCER);
  // the last load into every slot has landed before the memory is given back
  bool landed = true;
  for (uint32_t k = n > RING ? n - RING : 0; k < n; ++k)
    landed &= mbar_wait_drain(C::E4M3 ? bar.raw_full(k % RING) : bar.full(k % RING), (k / RING) & 1u, kTimeoutNs);
  if (!landed && lane == 0) atomicOr(p.err, SPLASH_DEV_TIMEOUT_DRAIN);
}

// e4m3: four warps widen the raw steps to fp16 operand tiles.
template <class C>
__device__ __forceinline__ void run_widen(const Params &p, Walk<C::KW> walk, const Bars<C> bar, uint32_t stages, uint32_t raws, int tid,
                                          volatile int *abort) {
  constexpr int KW = C::KW, CK = C::RK / 16, CV = C::RV / 16, RING = C::E4M3 ? C::RAWS : 1;  // 16-byte chunks of a row
  Piece x;
  uint32_t steps = 0;
  while (walk.next(x)) steps += x.steps;
  for (uint32_t n = 0; n < steps; ++n) {
    const uint32_t st = n % C::STAGES, slot = n % RING;
    bool ok = mbar_wait(bar.raw_full(slot), (n / RING) & 1u, abort, kTimeoutNs);
    ok = ok && (n < C::STAGES || mbar_wait(bar.empty(st), (n / C::STAGES - 1) & 1u, abort, kTimeoutNs));
    if (!ok) {
      give_up(p, abort, SPLASH_DEV_TIMEOUT_PRODUCER);
      return;
    }
    const uint32_t stage = stages + st * C::STAGE, raw = raws + slot * C::RAW;
    // (all reads before the first write: a thread's chunks of a step wait for shared memory once)
    constexpr int EK = KW * CK / 128, EV = KW * CV / 128;
    uint4 y[EK + EV];
#pragma unroll
    for (int i = 0; i < EK + EV; ++i) y[i] = load_shared4(raw + (tid + 128 * i) * 16);
    mbar_arrive(bar.raw_empty(slot));
#pragma unroll
    for (int i = 0; i < EK; ++i) widen_chunk<C>(y[i], stage, (tid + 128 * i) / CK, (tid + 128 * i) % CK);
#pragma unroll
    for (int i = 0; i < EV; ++i) widen_chunk<C>(y[EK + i], stage + C::K_BYTES, (tid + 128 * i) / CV, (tid + 128 * i) % CV);
    fence_proxy_async_shared();
    mbar_arrive(bar.full(st));
  }
}

// ------------------------------------------------------------------ products
// One warp: S = Q K^T of a step, LOOK steps ahead of its O += P V.  For a bf16 cache
// P is two terms (see the softmax), each a product.
template <class C>
__device__ __forceinline__ void run_mma(const Params &p, Walk<C::KW> walk, const Bars<C> bar, uint32_t tmem, uint32_t q_addr,
                                        uint32_t stages, volatile int *abort) {
  constexpr uint32_t HI = sdesc_hi_sw128(1024);
  constexpr int KW = C::KW;
  const uint32_t leader = elect_one_sync();
  uint32_t cnt[2] = {0, 0}, pieces[2] = {0, 0}, step = 0;  // of each group, of the CTA
  bool ok = true;
  Piece x;
  // S of step i of the piece for group t, its j-th
  auto scores = [&](int t, uint32_t j, uint32_t kd) {
    const uint32_t buf = j & 1u, qd = sdesc_lo(q_addr + (C::PAIR ? t * C::Q_BYTES : 0), 16), d = tmem + t * C::GROUP_COLS + buf * KW;
#pragma unroll
    for (int kk = 0; kk < C::DQK / 16; ++kk)
      mma_ss_lhp(leader, d, qd + (uint32_t)(((kk / 4) * C::Q_COLUMN + (kk % 4) * 32) >> 4), HI,
                 kd + (uint32_t)(((kk / 4) * C::COLUMN + (kk % 4) * 32) >> 4), HI, C::IDESC_QK, kk != 0);
    tc_commit_p(leader, bar.s_full(t, buf));
  };
  auto values = [&](int t, uint32_t j, bool first, bool last, uint32_t vd) {
    const uint32_t buf = j & 1u;
    if (!mbar_wait(bar.p_full(t, buf), (j >> 1) & 1u, abort, kTimeoutNs)) return false;
    tc_fence_after();
    const uint32_t pa = tmem + t * C::GROUP_COLS + buf * KW, o = tmem + t * C::GROUP_COLS + 2 * KW;
#pragma unroll
    for (int kk = 0; kk < KW / 16; ++kk)
      mma_ts_lhp(leader, o, pa + 8u * kk, vd + (uint32_t)((kk * 2048) >> 4), HI, C::IDESC_PV, !first || kk > 0);
    if constexpr (!C::E4M3) {
#pragma unroll
      for (int kk = 0; kk < KW / 16; ++kk)
        mma_ts_lhp(leader, o, pa + KW / 2 + 8u * kk, vd + (uint32_t)((kk * 2048) >> 4), HI, C::IDESC_PV, 1);
    }
    if (last) tc_commit_p(leader, bar.o_last(C::PAIR ? t : 0));
    return true;
  };
  while (ok && walk.next(x)) {
    const int groups = C::PAIR && p.nrows - (x.seg % p.row_groups) * C::TILE <= 128 ? 1 : 2;  // (a last tile may be missing)
#pragma unroll
    for (int t = 0; t < C::NT; ++t)
      if (t < groups) ok = ok && mbar_wait(bar.q_full(t), pieces[t]++ & 1u, abort, kTimeoutNs);
    if (!ok) break;
    tc_fence_after();
    for (int i = 0; i < x.steps + C::LOOK && ok; ++i) {
      if (i < x.steps) {
        const uint32_t u = step + i, st = u % C::STAGES;
        if (!(ok = mbar_wait(bar.full(st), (u / C::STAGES) & 1u, abort, kTimeoutNs))) break;
        tc_fence_after();
        const uint32_t kd = sdesc_lo(stages + st * C::STAGE, 16);
        if constexpr (C::PAIR) {
          scores(0, cnt[0] + i, kd);
          if (groups > 1) scores(1, cnt[1] + i, kd);
        } else {
          scores(i & 1, (i & 1 ? cnt[1] : cnt[0]) + (i >> 1), kd);
        }
      }
      const int k = i - C::LOOK;
      if (k >= 0) {
        const uint32_t st = (step + k) % C::STAGES, vd = sdesc_lo(stages + st * C::STAGE + C::K_BYTES, C::COLUMN);
        if constexpr (C::PAIR) {
          ok = values(0, cnt[0] + k, k == 0, k + 1 == x.steps, vd) && (groups < 2 || values(1, cnt[1] + k, k == 0, k + 1 == x.steps, vd));
        } else {
          ok = values(k & 1, (k & 1 ? cnt[1] : cnt[0]) + (k >> 1), k < 2, k + 1 == x.steps, vd);
        }
        if (ok) tc_commit_p(leader, bar.empty(st));
      }
    }
    step += x.steps;
    cnt[0] += C::PAIR ? x.steps : (x.steps + 1) / 2;
    if (groups > 1) cnt[1] += C::PAIR ? x.steps : x.steps / 2;
  }
  if (!ok && leader) give_up(p, abort, SPLASH_DEV_TIMEOUT_MMA);
  tc_commit_p(leader, bar.drain());
  if (!mbar_wait_drain(bar.drain(), 0, kTimeoutNs) && leader) atomicOr(p.err, SPLASH_DEV_TIMEOUT_DRAIN);
}

// ------------------------------------------------------------------ softmax
// The queries of a tile on their way from memory: eight lanes per row, 16 bytes of each
// of its 128-byte columns, and one thread's parents.
template <class C>
struct Queries {
  static constexpr int WARPS = C::PAIR ? 4 : 8, ROWS = 128 / (4 * WARPS), COLS = C::DQK / 64;  // rows of a lane
  uint4 q[ROWS][COLS];
  int32_t parent;
  float k_scale;

  __device__ __forceinline__ static int row(int k) {
    return 4 * ((int)(threadIdx.x >> 5) % WARPS) + ((threadIdx.x & 31) >> 3) + 4 * WARPS * k;
  }

  __device__ __forceinline__ void ask(const Params &p, const Piece &x, int row0, int rows) {
    const int head = x.seg / p.row_groups, thread = threadIdx.x % (32 * WARPS);
    const char *base = p.q + x.b * p.q_b + (int64_t)head * p.G * p.q_h + (threadIdx.x & 7) * 16;
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int i = row(k), g = p.T == 1 ? row0 + i : (int)__umulhi(row0 + i, p.over_T), l = row0 + i - g * p.T;
      const char *src = base + g * p.q_h + l * p.q_l;
#pragma unroll
      for (int c = 0; c < COLS; ++c) q[k][c] = i < rows ? *reinterpret_cast<const uint4 *>(src + c * 128) : make_uint4(0, 0, 0, 0);
    }
    parent = rows > 0 && thread < p.T ? p.parents[x.b * p.parents_stride + thread] : -2;
    k_scale = C::E4M3 && rows > 0 ? p.k_scale[head] : 1.f;
  }

  // Into the operand tile.  For an e4m3 cache the queries become fp16, a row scaled by the
  // power of two that brings its largest element into [1, 2): exact but for elements 2^14
  // times smaller, whose error, 2^-25 of the largest, is below that of an fp32 sum.  The
  // factors go to s_factor.
  __device__ __forceinline__ void put(const Params &p, uint32_t tile, int32_t *s_parents, float *s_factor) const {
    const int thread = threadIdx.x % (32 * WARPS), lane8 = threadIdx.x & 7;
    if (thread < p.T) s_parents[thread] = parent;
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int i = row(k);
      float down = k_scale < 0.f ? -1.f : 1.f;
      if (C::E4M3) {
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
          const uint4 y = q[k][c];
          top = max(top, max(max(exponent(y.x), exponent(y.y)), max(exponent(y.z), exponent(y.w))));
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
        top = min(max(top, 1u), 253u);
        down *= __uint_as_float((254u - top) << 23);
        if (lane8 == 0) s_factor[i] = __uint_as_float(top << 23);
      }
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        uint4 y = q[k][c];
        if (C::E4M3) y = make_uint4(to_half(y.x, down), to_half(y.y, down), to_half(y.z, down), to_half(y.w, down));
        st_shared_v4(tile + c * C::Q_COLUMN + i * 128 + ((lane8 ^ (i & 7)) << 4), y.x, y.y, y.z, y.w);
      }
    }
  }
};

// The values of a step that are not finite become zeros: the product adds 0 x value
// for the rows that do not see a key.  128 threads; returns whether there were any
// (then the join adds them where they are seen).
template <class C>
__device__ __forceinline__ bool clean_values(uint32_t tile, int tid) {
  constexpr uint32_t TOP = C::E4M3 ? 0x7c007c00u : 0x7f807f80u, STEP = C::E4M3 ? 0x04000400u : 0x00800080u;
  constexpr int EACH = C::KW * C::DV / 8 / 128;
  uint32_t high = 0;  // the top bit of a half: some exponent had all its bits set
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const uint4 y = load_shared4(tile + (tid + 128 * i) * 16);
    high |= ((y.x & TOP) + STEP) | ((y.y & TOP) + STEP) | ((y.z & TOP) + STEP) | ((y.w & TOP) + STEP);
  }
  if ((high & 0x80008000u) == 0) return false;
#pragma unroll 1
  for (int i = 0; i < EACH; ++i) {
    const uint32_t at = tile + (tid + 128 * i) * 16;
    const uint4 y = load_shared4(at);
    st_shared_v4(at, finite(y.x, TOP & 0xffffu), finite(y.y, TOP & 0xffffu), finite(y.z, TOP & 0xffffu), finite(y.w, TOP & 0xffffu));
  }
  fence_proxy_async_shared();
  return true;
}

// What a row has when its piece's steps are done.
struct Done {
  int64_t row;     // of the result, or of the parts
  float scale;     // of the values
  float m, sum;    // of both groups
  float f0, f1;    // the outputs' factors: f0 O_0 + f1 O_1
  bool complete;   // the result's
  bool empty;      // padding
  bool two;        // O_1 is there
};

// Writes a finished piece: rows of the result, or this CTA's part of them.  A lane has a
// row, so that a store touches 32 lines however little it writes to each: 32 bytes a lane.
// In a cluster parts go to shared memory, at `rows`, each followed by 16 bytes that keep
// neighbours on different banks.
template <class C, bool TOGETHER>
__device__ __forceinline__ void write_rows(const Params &p, const Done &d, uint32_t o_0, int t, bool real, uint32_t rows, float2 *s_part) {
  constexpr bool PAIR = C::PAIR;
  const bool empty = d.sum == 0.f || d.empty;
  const float inv = __fdividef(d.scale, d.sum);
  // (groups that share a tile take a half of the columns each)
  constexpr int COLS = PAIR ? C::DV : C::DV / 2;
#pragma unroll 1
  for (int c = PAIR ? 0 : t * COLS; c < (PAIR ? COLS : (t + 1) * COLS); c += 32) {
    uint32_t y[32];
    float o[32];
    tmem_ld32(o_0 + c, y);
    tmem_wait_ld();
    reg_fence32(y);
#pragma unroll
    for (int j = 0; j < 32; ++j) o[j] = d.two ? d.f0 * __uint_as_float(y[j]) : __uint_as_float(y[j]);
    if (d.two) {
      tmem_ld32(o_0 + C::GROUP_COLS + c, y);
      tmem_wait_ld();
      reg_fence32(y);
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] += d.f1 * __uint_as_float(y[j]);
    }
    if (TOGETHER) {
      const uint32_t dst = rows + ((uint32_t)d.row * (C::DV + 4) + c) * 4;
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        if (real)
          st_shared_v4(dst + 4 * j, empty ? 0u : __float_as_uint(o[j]), empty ? 0u : __float_as_uint(o[j + 1]),
                       empty ? 0u : __float_as_uint(o[j + 2]), empty ? 0u : __float_as_uint(o[j + 3]));
    } else if (real && d.complete) {
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = empty ? 0u : pack_bf16x2(o[2 * j] * inv, o[2 * j + 1] * inv);
      __nv_bfloat16 *dst = p.out + d.row * C::DV + c;
      if (p.out_wide) {
        st_global_v8(dst, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
        st_global_v8(dst + 16, w[8], w[9], w[10], w[11], w[12], w[13], w[14], w[15]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) reinterpret_cast<uint4 *>(dst)[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
      }
    } else if (real) {
      float *dst = p.part_o + d.row * C::DV + c;
      uint32_t w[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) w[j] = empty ? 0u : __float_as_uint(o[j]);
#pragma unroll
      for (int j = 0; j < 32; j += 8) st_global_v8(dst + j, w[j], w[j + 1], w[j + 2], w[j + 3], w[j + 4], w[j + 5], w[j + 6], w[j + 7]);
    }
    __syncwarp();
  }
  if (real && (PAIR || t == 0)) {
    if (TOGETHER)
      s_part[d.row] = empty ? make_float2(-INFINITY, 0.f) : make_float2(d.m, d.sum);
    else if (d.complete)
      p.lse[d.row] = empty ? -INFINITY : (d.m + log2f(d.sum)) * kLn2;
    else
      *reinterpret_cast<float2 *>(p.part_ml + 2 * d.row) = empty ? make_float2(-INFINITY, 0.f) : make_float2(d.m, d.sum);
  }
}

// Two groups of four warps, a thread per row of a tile: group t has tile t (PAIR) or
// every other step.  From piece to piece: the next queries are read while the last
// products run, go to shared memory as soon as those are done, and the finished rows
// are written while the next piece's first scores are computed.
template <class C, bool TOGETHER>
__device__ __forceinline__ void run_softmax(const Params &p, Walk<C::KW> walk, const Bars<C> bar, uint32_t tmem, uint32_t q_addr,
                                            uint32_t stages, int32_t *s_parents, float *s_factor, float2 (*s_ml)[128], float2 *s_part, int t,
                                            volatile int *abort, volatile int *lost) {
  constexpr int KW = C::KW;
  constexpr bool E4M3 = C::E4M3, PAIR = C::PAIR;
  const int tid = threadIdx.x & 127, warp = tid >> 5;
  const uint32_t lanes = (uint32_t)(32 * warp) << 16, base = tmem + t * C::GROUP_COLS + lanes, o_col = base + 2 * KW;
  const uint32_t o_0 = tmem + (PAIR ? t * C::GROUP_COLS : 0) + lanes + 2 * KW, q_tile = q_addr + (PAIR ? t * C::Q_BYTES : 0);
  const int bar_id = PAIR ? 1 + t : 1, bar_threads = PAIR ? 128 : 256;
  uint32_t cnt = 0, pieces = 0, step = 0, skipped = 0;  // of this group; steps of the CTA before x
  int row0 = 0, rows = 0, done_rows = 0, tree = -1;
  bool ok = true, some = false;  // some: a piece is finished and not written
  Piece x = {};
  Done d;
  Queries<C> queries;
  Branch me = {0, 0};
  // the next piece that has rows for this group (the second tile of a last row group may be missing)
  auto advance = [&]() {
    while (walk.next(x)) {
      row0 = (x.seg % p.row_groups) * C::TILE + (PAIR ? t * 128 : 0);
      rows = min(128, p.nrows - row0);
      if (rows > 0) return true;
      skipped += x.steps;
    }
    return false;
  };
  bool more = advance();
  queries.ask(p, x, row0, more ? rows : 0);
  while (more || some) {
    if (more) {
      queries.put(p, q_tile, s_parents, s_factor);
      fence_proxy_async_shared();
      mbar_arrive(bar.q_full(PAIR ? t : 0));
    }
    if (some) {
      tc_fence_after();
      if (32 * warp < done_rows) write_rows<C, TOGETHER>(p, d, o_0, t, tid < done_rows, q_addr, s_part);
      tc_fence_before();
      some = false;
    }
    if (!more) break;
    bar_sync(bar_id, bar_threads);  // (tree and factors are there; nobody still reads an output that the next products replace)
    const bool real = tid < rows, busy = 32 * warp < rows;
    step += skipped;
    skipped = 0;
    if (tree != x.b || p.row_groups > 1) {
      const int r = row0 + tid;
      bool bad = false;
      me = {0, 0};
      const int l = p.T == 1 ? 0 : r - (int)__umulhi(r, p.over_T) * p.T;
      if (real) me = branch_of(s_parents, l, max(0, -x.s.ctx), p.window, &bad);
      if (bad) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
      tree = x.b;
    }
    const int32_t lo = p.window < 0 ? 0 : max(0, x.s.ctx + me.depth - p.window);
    float factor = (p.cap > 0.f ? p.scale / p.cap : p.scale * kLog2e) * fabsf(queries.k_scale);
    if (E4M3) factor *= s_factor[tid];
    if (factor < kTiny) factor = kTiny;  // (NaN stays)
    if (factor > FLT_MAX) factor = FLT_MAX;  // (0 times it stays 0)
    const float times = p.cap > 0.f ? 1.f : factor;
    float m = -INFINITY, sum = 0.f;

    for (int i = PAIR ? 0 : t; i < x.steps; i += PAIR ? 1 : 2, ++cnt) {
      const uint32_t buf = cnt & 1u;
      if (!(ok = __all_sync(~0u, mbar_wait(bar.s_full(t, buf), (cnt >> 1) & 1u, abort, kTimeoutNs)))) break;
      const int32_t key0 = (x.s.step0 + x.step + i) * KW;
      const bool all = whole<KW>(p, x.s, key0);
      if (!all && (!PAIR || t == 0)) {
        // (the step's products wait for these threads, for the first tile's before the second's)
        const uint32_t st = (step + i) % C::STAGES;
        if (!(ok = __all_sync(~0u, mbar_wait(bar.full(st), ((step + i) / C::STAGES) & 1u, abort, kTimeoutNs)))) break;
        if (clean_values<C>(stages + st * C::STAGE + C::K_BYTES, tid)) *lost = 1;
      }
      if (busy) {
        tc_fence_after();
        uint32_t a[32], b[32];
        tmem_ld32(base + buf * KW, a);
        tmem_ld32(base + buf * KW + 32, b);
        tmem_wait_ld();
        reg_fence32(a);
        reg_fence32(b);
        float s[KW];
#pragma unroll
        for (int j = 0; j < 32; ++j) s[j] = __uint_as_float(a[j]), s[32 + j] = __uint_as_float(b[j]);
        if (p.cap > 0.f) {
          // tanh by the series alone where it holds for the whole warp's step
          const float cap = p.cap * kLog2e;
          float most = 0.f;
#pragma unroll
          for (int j = 0; j < KW; ++j) most = fmaxf(most, fabsf(s[j]));
          if (__any_sync(~0u, most * factor > kTanhSeriesLimit)) {  // (NaN stays NaN either way)
#pragma unroll
            for (int j = 0; j < KW; ++j) s[j] = cap * tanh_of(s[j] * factor);
          } else {
#pragma unroll
            for (int j = 0; j < KW; j += 2) {
              const f32x2 x = fmul2({s[j], s[j + 1]}, {factor, factor}), u = fmul2(x, x);
              const f32x2 y = fmul2(ffma2(fmul2(x, u), ffma2(u, {kTanhC2, kTanhC2}, {kTanhC1, kTanhC1}), x), {cap, cap});
              s[j] = y.x;
              s[j + 1] = y.y;
            }
          }
        }
        if (!all) {
          const uint64_t see = visible(key0, x.s.ctx, lo, me.seen);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (!((uint32_t)see >> j & 1u)) s[j] = -INFINITY;
            if (!((uint32_t)(see >> 32) >> j & 1u)) s[32 + j] = -INFINITY;
          }
        }
        float top;
        {
          float y[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int j = 4; j + 7 < KW; j += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = fmax3(y[k], s[j + k], s[j + 4 + k]);
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = fmaxf(y[k], s[KW - 4 + k]);
          top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) * times;
        }
        if (E4M3) top -= kBelowTop;
        if (__any_sync(~0u, top > m + kSlack)) {
          const float high = fmaxf(top, m), alpha = m == -INFINITY ? 0.f : ex2_approx(m - high);
          m = high;
          sum *= alpha;
          if (i >= (PAIR ? 1 : 2)) {
            // (these scores came after the products of all the group's steps but the one before: its stage is free when
            // that one is done)
            const uint32_t u = step + i - (PAIR ? 1 : 2);
            if (!(ok = __all_sync(~0u, mbar_wait(bar.empty(u % C::STAGES), (u / C::STAGES) & 1u, abort, kTimeoutNs)))) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < C::DV / 32; ++c) {
              uint32_t y[32];
              tmem_ld32(o_col + 32 * c, y);
              tmem_wait_ld();
              reg_fence32(y);
#pragma unroll
              for (int j = 0; j < 32; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * alpha);
              tmem_st32(o_col + 32 * c, y);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        // P in 16 bits, half of the keys at a time (the registers of their scores are free then).
        // fp16 for an e4m3 cache; for bf16 two terms, cut off and rest: 2^-16 of each p, where
        // bf16 alone loses 2^-8, as much as the rounding of the result.  The rest is taken of
        // (1 + 2^-23) p, which keeps it above 0 where p is: an infinite value times either term
        // then has its sign, and the sum is that infinity (0 x infinity is NaN, as it is where p
        // itself is below 2^-126).
        constexpr float above = 1.f + 0x1p-23f;
        f32x2 acc[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t u[16], v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int k = 32 * h + 2 * j;
            const f32x2 y = ffma2({s[k], s[k + 1]}, {times, times}, {-ref, -ref});
            const f32x2 e = {ex2_approx(y.x), ex2_approx(y.y)};
            acc[j & 3] = fadd2(acc[j & 3], e);
            if (E4M3) {
              u[j] = pack_half2(e.x, e.y);
            } else {
              u[j] = __byte_perm(__float_as_uint(e.x), __float_as_uint(e.y), 0x7632);
              const f32x2 rest = ffma2(e, {above, above}, {-cut(e.x), -cut(e.y)});
              v[j] = pack_bf16x2(rest.x, rest.y);
            }
          }
          tmem_st16(base + buf * KW + 16 * h, u);
          if (!E4M3) tmem_st16(base + buf * KW + 32 + 16 * h, v);
        }
        acc[0] = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
        sum += acc[0].x + acc[0].y;
        tmem_wait_st();
        tc_fence_before();
      }
      mbar_arrive(bar.p_full(t, buf));
    }
    if (!ok) break;

    const int head = x.seg / p.row_groups, slot = TOGETHER ? 0 : x.slot(blockIdx.x);
    d.complete = slot < 0;
    d.row = slot < 0 ? ((int64_t)x.b * p.Hkv + head) * p.nrows + row0 + tid : (int64_t)slot * p.part_rows + (PAIR ? t * 128 : 0) + tid;
    d.scale = E4M3 ? p.v_scale[head] : 1.f;
    d.empty = me.seen == 0;
    d.m = m;
    d.sum = sum;
    d.f0 = 1.f;
    d.f1 = 0.f;
    d.two = !PAIR && x.steps > 1;  // the other group has steps too
    done_rows = rows;
    some = true;
    step += x.steps;
    more = advance();
    queries.ask(p, x, row0, more ? rows : 0);  // (always: nothing of the last ones stays in registers)
    // (a barrier of its own: one with a phase per step may be two behind here, which its parity would not tell)
    if (!(ok = __all_sync(~0u, mbar_wait(bar.o_last(PAIR ? t : 0), pieces++ & 1u, abort, kTimeoutNs)))) break;
    if (TOGETHER && PAIR && p.nrows - (row0 - t * 128) > 128) {  // (the rows go where the other tile's operands are)
      if (!(ok = __all_sync(~0u, mbar_wait(bar.o_last(t ^ 1), 0u, abort, kTimeoutNs)))) break;
    }
    if (!PAIR) {
      s_ml[t][tid] = make_float2(m, sum);
      bar_sync(bar_id, bar_threads);
      const float2 z = s_ml[t ^ 1][tid];
      if (d.two) {
        const float high = fmaxf(m, z.x), ref = high == -INFINITY ? 0.f : high;
        const float mine = factor_of(m - ref), theirs = factor_of(z.x - ref);
        d.sum = sum * mine + z.y * theirs;
        d.m = high;
        d.f0 = t == 0 ? mine : theirs;
        d.f1 = t == 0 ? theirs : mine;
      } else if (t == 1) {
        d.m = z.x;
        d.sum = z.y;
      }
    }
  }
  if (!ok && (threadIdx.x & 31) == 0) give_up(p, abort, SPLASH_DEV_TIMEOUT_SOFTMAX);
}

// Adds to a row's columns the values that are not finite of the keys that it sees in the
// segment's steps that are not whole (the products had zeros in their place): a value
// that is infinite or NaN is the result's, whatever else is in it.  A warp; returns
// whether there were any.
template <int DV, bool E4M3>
__device__ __noinline__ bool add_lost(const Params &p, const Span &s, int b, int head, int row, float (&acc)[DV / 32]) {
  constexpr int KW = 64, PER = DV / 32;
  bool bad = false, found = false;
  const Branch me = branch_of(p.parents + b * p.parents_stride, row % p.T, max(0, -s.ctx), p.window, &bad);
  const int32_t lo = p.window < 0 ? 0 : max(0, s.ctx + me.depth - p.window);
  for (int i = 0; i < s.nst; ++i) {
    const int32_t key0 = (s.step0 + i) * KW;
    if (whole<KW>(p, s, key0)) continue;
    for (uint64_t m = visible(key0, s.ctx, lo, me.seen); m != 0; m &= m - 1) {
      const int32_t key = key0 + __ffsll((long long)m) - 1;
      const int32_t page = p.block_table[b * p.block_table_stride + (key >> p.page_shift)];
      if (page < 0 || page >= p.num_pages) continue;
      const char *v = p.v + page * p.v_page + head * p.v_head + (key & ((1 << p.page_shift) - 1)) * p.v_token;
#pragma unroll
      for (int c = 0; c < PER; ++c) {
        const int col = (threadIdx.x & 31) * PER + c;
        const float y = E4M3 ? (float)reinterpret_cast<const __nv_fp8_e4m3 *>(v)[col]
                             : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(v)[col]);
        if (!(fabsf(y) < INFINITY)) acc[c] += y, found = true;
      }
    }
  }
  return __any_sync(~0u, found);
}

// Where CTA `rank` of a cluster (of a power of two) begins in n steps.
__device__ __forceinline__ int32_t share(int32_t n, uint32_t rank, uint32_t ctas) {
  return (int32_t)((int64_t)n * rank >> (31 - __clz((int)ctas)));
}

// TOGETHER: a cluster of CTAs per segment, which share its steps; otherwise equal parts of the list.
// The registers do not hold all (52 .. 140 bytes are spilled, 180 .. 308 for e4m3), but the
// steps hardly notice: a softmax warp reads one to three of them a step, all warps together 8 and 12
// of a step's 3800 and 1900 instructions (PAIR and not; e4m3 16 of 3100 and 20 of 1900), and writes none.
template <class C, bool TOGETHER>
__global__ void __launch_bounds__(C::THREADS, 1) tree_decode_kernel(const __grid_constant__ CUtensorMap map_k,
                                                                  const __grid_constant__ CUtensorMap map_v, const Params p) {
  constexpr int KW = C::KW;
  extern __shared__ char smem_raw[];
  __shared__ int32_t s_scan[C::WARPS], s_seq, s_before, s_parents[C::NT][SPLASH_MAX_TREE_TOKENS];
  __shared__ float2 s_ml[2][128];  // (maximum, sum) of the groups' rows
  __shared__ float2 s_part[TOGETHER ? C::TILE : 1];  // of this CTA's part of them
  __shared__ float s_factor[C::NT][128];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_lost;
  const uint32_t tiles = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const Bars<C> bar{tiles + C::TILES};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == C::MMA) {
    tmem_alloc(smem_u32(&s_tmem), C::COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar.full(s), C::E4M3 ? 128 : 1);
      mbar_init(bar.empty(s), 1);
    }
    for (int s = 0; s < C::RAWS; ++s) {
      mbar_init(bar.raw_full(s), 1);
      mbar_init(bar.raw_empty(s), 128);
    }
    for (int t = 0; t < 2; ++t) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(bar.s_full(t, x), 1);
        mbar_init(bar.p_full(t, x), 128);
      }
      mbar_init(bar.o_last(t), 1);
      mbar_init(bar.q_full(t), C::PAIR ? 128 : 256);
    }
    mbar_init(bar.drain(), 1);
    mbar_fence_init();
    s_abort = s_lost = 0;
  }
  if (tid == 32 * C::LOAD) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  // (the allocation comes before the next kernel may start: one that waits for this one cannot
  // hold what this one still needs)
  grid_dependency();

  const int per_seq = p.Hkv * p.row_groups;
  Walk<KW> walk{p, 0, 0, per_seq, 0, 0, 0, 0};
  if constexpr (TOGETHER) {
    const uint32_t ctas = cluster_size(), rank = cluster_rank(), segment = blockIdx.x / ctas;
    walk.b = segment / per_seq;
    walk.seg = segment % per_seq;
    walk.length = p.seq_lens[walk.b];
    const Span s = span_of<KW>(p, walk.length);
    walk.u = walk.entry = kPieceSteps + share(s.nst, rank, ctas);
    walk.end = kPieceSteps + share(s.nst, rank + 1, ctas);
    if (walk.seg == 0 && rank == 0 && tid == 0 && s.n != walk.length) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  } else {
    // ---- this CTA's part of the list: a scan over the sequences
    const int per = (p.B + C::THREADS - 1) / C::THREADS;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int32_t own = 0;
    for (int b = b0; b < b1; ++b) own += span_of<KW>(p, p.seq_lens[b]).nst + kPieceSteps;
    int32_t before = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(~0u, before, o);
      if (lane >= o) before += y;
    }
    if (lane == 31) s_scan[warp] = before;
    before -= own;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int32_t total = 0;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    const Parts parts(p, total * per_seq);
    const int32_t begin = parts.begin(blockIdx.x);
    walk.end = parts.begin(blockIdx.x + 1);
    if (blockIdx.x == 0 || (begin >= before * per_seq && begin < (before + own) * per_seq)) {
      int32_t at = before;
      for (int b = b0; b < b1; ++b) {
        const Span s = span_of<KW>(p, p.seq_lens[b]);
        const int32_t entries = s.nst + kPieceSteps;
        if (begin >= at * per_seq && begin < (at + entries) * per_seq) s_seq = b, s_before = at;
        if (blockIdx.x == 0) {
          p.before[b] = at;
          if (b == p.B - 1) p.before[p.B] = at + entries;
          if (s.n != p.seq_lens[b]) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
        }
        at += entries;
      }
    }
    __syncthreads();
    walk.u = begin;
    if (begin < walk.end) {
      walk.b = s_seq;
      walk.length = p.seq_lens[walk.b];
      const int32_t entries = span_of<KW>(p, walk.length).nst + kPieceSteps, in_seq = begin - s_before * per_seq;
      walk.seg = (uint32_t)in_seq / (uint32_t)entries;
      walk.entry = in_seq - walk.seg * entries;
    }
  }
  const int32_t mine_b = walk.b, mine_seg = walk.seg;
  if (walk.u < walk.end) {
    const uint32_t q_addr = tiles, stages = tiles + C::NT * C::Q_BYTES, raws = stages + C::STAGES * C::STAGE;
    // (registers for e4m3: 14 warps are launched with 128 a thread; 8 take 152 and 4 leave 48 each)
    if (warp < 8) {
      if constexpr (C::E4M3) regs_increase<152>();
      const int t = warp >> 2, tile = C::PAIR ? t : 0;
      run_softmax<C, TOGETHER>(p, walk, bar, s_tmem, q_addr, stages, s_parents[tile], s_factor[tile], s_ml, s_part, t, &s_abort, &s_lost);
    } else if (warp == C::MMA) {
      run_mma<C>(p, walk, bar, s_tmem, q_addr, stages, &s_abort);
    } else if (warp == C::LOAD) {
      run_loads<C>(p, walk, bar, &map_k, &map_v, stages, raws, &s_abort);
    } else if constexpr (C::E4M3) {
      regs_decrease<80>();
      run_widen<C>(p, walk, bar, stages, raws, tid - 256, &s_abort);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (!TOGETHER && tid == 0) p.lost[blockIdx.x] = s_lost;
  if (warp == C::MMA) {
    tc_fence_after();
    tmem_dealloc(s_tmem, C::COLS);
  }
  if constexpr (TOGETHER) {
    // ---- the segment's rows: every CTA finishes some of them, a warp a row
    constexpr int PER = C::DV / 32;
    const uint32_t ctas = cluster_size(), rank = cluster_rank();
    cluster_sync();
    const Span s = span_of<KW>(p, p.seq_lens[mine_b]);
    const int head = mine_seg / p.row_groups, tile0 = (mine_seg % p.row_groups) * C::TILE, rows = min(C::TILE, p.nrows - tile0);
    const float v_scale = C::E4M3 ? p.v_scale[head] : 1.f;
    auto has = [&](uint32_t k) { return share(s.nst, k, ctas) < share(s.nst, k + 1, ctas); };
    const bool lost = __any_sync(~0u, lane < ctas && load_cluster(in_cta(smem_u32(&s_lost), lane)) != 0);
    const int r1 = (int)(rows * (rank + 1) / ctas);
    for (int r = (int)(rows * rank / ctas) + warp; r < r1; r += C::WARPS) {
      const uint32_t ml = smem_u32(&s_part[r]), from = tiles + (r * (C::DV + 4) + lane * PER) * 4;
      const float2 mine = lane < ctas && has(lane) ? load_cluster2(in_cta(ml, lane)) : make_float2(-INFINITY, 0.f);
      float top = mine.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      const float f = factor_of(mine.x - (top == -INFINITY ? 0.f : top));
      float sum = f * mine.y, acc[PER];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll 4
      for (uint32_t k = 0; k < ctas; ++k) {
        const float g = __shfl_sync(~0u, f, k);
        if (!has(k)) continue;
        if constexpr (PER == 4) {
          const float4 x = load_cluster4(in_cta(from, k));
          acc[0] += g * x.x, acc[1] += g * x.y, acc[2] += g * x.z, acc[3] += g * x.w;
        } else {
          const float2 x = load_cluster2(in_cta(from, k));
          acc[0] += g * x.x, acc[1] += g * x.y;
        }
      }
      const float inv = sum == 0.f ? 0.f : v_scale / sum;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] *= inv;
      if (lost) add_lost<C::DV, C::E4M3>(p, s, mine_b, head, tile0 + r, acc);
      const int64_t row = ((int64_t)mine_b * p.Hkv + head) * p.nrows + tile0 + r;
      uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + row * C::DV) + lane * (PER / 2);
      if constexpr (PER == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
      else
        *dst = pack_bf16x2(acc[0], acc[1]);
      if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
    cluster_sync();  // (no CTA ends while another reads its shared memory)
  }
}

// Joins the parts of a segment that several CTAs computed: with (m_c, l_c, o_c) of part c
// of a row and m = max m_c: out = sum exp(m_c - m) o_c / sum exp(m_c - m) l_c, in the
// order of the keys.  A CTA takes `each` rows of a segment, a warp one at a time.  (CTAs for each
// place where a segment goes on in another CTA, instead of for each segment: 32 requests of 32
// drafts 83.2 -> 82.3 us, but 1 request of 16384 tokens, in parts of all CTAs, 33.7 -> 45.)
constexpr int kJoinWarps = 8;
template <int DV, int TILE, bool E4M3>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const Params p, int slices, int each) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int PER = DV / 32, AHEAD = 8;  // columns of a lane; parts read at once
  const int per_seq = p.Hkv * p.row_groups;
  const int64_t segment = blockIdx.x / slices;
  const int b = (int)(segment / per_seq), seg = (int)(segment % per_seq), head = seg / p.row_groups;
  grid_dependency();
  const Parts parts(p, p.before[p.B] * per_seq);
  const int32_t entries = p.before[b + 1] - p.before[b];
  const int32_t u0 = p.before[b] * per_seq + entries * seg + kPieceSteps, u1 = u0 + entries - kPieceSteps - 1;
  const int c0 = parts.owner(u0), c1 = parts.owner(u1);
  bool lost = false;
  for (int c = c0 + lane; c <= c1; c += 32) lost |= p.lost[c] != 0;
  lost = __any_sync(~0u, lost);
  if (c0 == c1 && !lost) return;  // written by that CTA
  const int tile0 = (seg % p.row_groups) * TILE, rows = min(TILE, p.nrows - tile0);
  const float v_scale = E4M3 ? p.v_scale[head] : 1.f;
  const int r0 = blockIdx.x % slices * each, r1 = min(rows, r0 + each);
  for (int r = r0 + warp; r < r1; r += kJoinWarps) {
    const int64_t row = ((int64_t)b * p.Hkv + head) * p.nrows + tile0 + r;
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + row * DV) + lane * (PER / 2);
    float top = -INFINITY, sum = 0.f, acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
    for (int c = c0; c <= c1 && c0 < c1; c += AHEAD) {
      float2 ml[AHEAD];
      float x[AHEAD][PER];
      float above = top;
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        ml[a] = make_float2(-INFINITY, 0.f);
        if (c + a <= c1) {
          const int64_t at = (int64_t)(2 * (c + a) + (c + a == c0 ? 1 : 0)) * p.part_rows + r;
          ml[a] = *reinterpret_cast<const float2 *>(p.part_ml + at * 2);
          if constexpr (PER == 4)
            *reinterpret_cast<float4 *>(x[a]) = reinterpret_cast<const float4 *>(p.part_o + at * DV)[lane];
          else
            *reinterpret_cast<float2 *>(x[a]) = reinterpret_cast<const float2 *>(p.part_o + at * DV)[lane];
        }
      }
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) above = fmaxf(above, ml[a].x);
      const float ref = above == -INFINITY ? 0.f : above, f0 = factor_of(top - ref);
      sum *= f0;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] *= f0;
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        if (c + a > c1) break;
        const float f = factor_of(ml[a].x - ref);
        sum += f * ml[a].y;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] += f * x[a][i];
      }
      top = above;
    }
    const float inv = sum == 0.f ? 0.f : v_scale / sum;
    if (c0 < c1 && lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = c0 < c1 ? acc[i] * inv : __bfloat162float(p.out[row * DV + lane * PER + i]);
    bool changed = false;
    if (lost) {
      float w[PER];  // (in memory: the call takes its address)
#pragma unroll
      for (int i = 0; i < PER; ++i) w[i] = acc[i];
      changed = add_lost<DV, E4M3>(p, span_of<64>(p, p.seq_lens[b]), b, head, tile0 + r, w);
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = w[i];
    }
    if (c0 == c1 && !changed) continue;
    if constexpr (PER == 4)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
    else
      *dst = pack_bf16x2(acc[0], acc[1]);
  }
}

int64_t align16(int64_t x) { return (x + 15) & ~(int64_t)15; }

// Steps that a sequence can have, from its row of pages and the window.  (A window of all
// its keys is none: with T added the largest ones would overflow.)
int64_t most_steps(int32_t T, int32_t max_pages, int32_t page_size, int64_t window) {
  const int64_t keys = (int64_t)max_pages * page_size, most = (keys + 63) / 64;
  return window < 0 || window >= keys ? most : std::min(most, (window + T) / 64 + 3);
}

// A cache as a 4-D tensor [pages][heads][tokens][d]; boxes of `rows` rows by 64 bf16 columns
// (swizzled) or by a whole e4m3 row.  Dimensions of one entry, and those that repeat it
// (stride 0), have one entry in the map.
splash_status make_map(CUtensorMap *map, const splash_cache_view &v, int64_t pages, int32_t heads, int32_t page_size, int32_t d,
                       bool e4m3, int32_t *head_on, int32_t *page_on, int32_t *page_end) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  if (encode == nullptr) return SPLASH_ERR_CUDA;
  const int64_t size = e4m3 ? 1 : 2;
  *head_on = heads > 1 && v.stride_head > 0;
  *page_on = pages > 1 && v.stride_page > 0;
  *page_end = *page_on ? (int32_t)pages : 1;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)page_size, (cuuint64_t)(*head_on ? heads : 1), (cuuint64_t)*page_end};
  const cuuint64_t strides[3] = {(cuuint64_t)(size * v.stride_token), (cuuint64_t)(size * (*head_on ? v.stride_head : d)),
                                 (cuuint64_t)(size * (*page_on ? v.stride_page : d))};
  const cuuint32_t box[4] = {(cuuint32_t)(e4m3 ? d : 64), (cuuint32_t)std::min(page_size, 64), 1, 1}, ones[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.ptr, dims, strides, box,
                            ones, CU_TENSOR_MAP_INTERLEAVE_NONE, e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SPLASH_OK : SPLASH_ERR_CUDA;
}

// Sets the kernels up on first use and picks the CTAs per segment (0: the list): the
// largest cluster of which one for every segment runs at the same time, where its share of
// the longest possible sequence is at most what the list would take for sequences four fifths
// as long, and three steps for the second kernel.  (32 / 8 heads of 128, list -> clusters:
// 1 request of 300 keys and 16 drafts 12.4 -> 10.0 us, 64 drafts 16.2 -> 15.3; 8 requests of
// up to 2048 keys 23.5 -> 22.7; but 1 request of 16384 keys 28.1 -> 33.3, as clusters of 16
// have room for 7 segments and those of 8 leave half of the SMs idle.)
template <class C>
splash_status cluster_for(int dev, int sms, int64_t segments, int64_t most, int *cluster) {
  static std::atomic<uint64_t> room[64];  // per device: 12 bits each for clusters of 1, 2, 4, 8, 16 CTAs; 0: not asked yet
  uint64_t fits = room[dev & 63].load(std::memory_order_acquire);
  if (fits == 0) {
    SPLASH_CUDA_TRY(cudaFuncSetAttribute(tree_decode_kernel<C, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
    SPLASH_CUDA_TRY(cudaFuncSetAttribute(tree_decode_kernel<C, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
    SPLASH_CUDA_TRY(cudaFuncSetAttribute(tree_decode_kernel<C, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    fits = (uint64_t)1 << 60;
    for (int i = 0; i < 5; ++i) {
      cudaLaunchConfig_t config = {};
      config.gridDim = dim3(1u << i);
      config.blockDim = dim3(C::THREADS);
      config.dynamicSmemBytes = C::SMEM;
      cudaLaunchAttribute attr = {};
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 1u << i;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      config.attrs = &attr;
      config.numAttrs = 1;
      int clusters = 0;
      if (cudaOccupancyMaxActiveClusters(&clusters, tree_decode_kernel<C, true>, &config) != cudaSuccess) {
        (void)cudaGetLastError();  // (a size that the device does not place)
        clusters = 0;
      }
      fits |= (uint64_t)std::min(clusters, 4095) << (12 * i);
    }
    room[dev & 63].store(fits, std::memory_order_release);
  }
  *cluster = 0;
  for (int i = 4; i >= 0; --i) {
    if ((int64_t)(fits >> (12 * i) & 4095u) < segments || ((int64_t)1 << i) >= 2 * most) continue;
    if ((((most + ((int64_t)1 << i) - 1) >> i) - 3) * 5 * sms <= (most + kPieceSteps) * segments * 4) *cluster = 1 << i;
    break;
  }
  return SPLASH_OK;
}

template <class C>
splash_status launch(const splash_paged_decode_args &a, Params p, cudaStream_t stream) {
  CUtensorMap map_k, map_v;
  splash_status st = make_map(&map_k, a.k_cache, a.num_pages, a.Hkv, a.page_size, a.dqk, C::E4M3, &p.k_head_on, &p.k_page_on, &p.k_page_end);
  if (st != SPLASH_OK) return st;
  st = make_map(&map_v, a.v_cache, a.num_pages, a.Hkv, a.page_size, a.dv, C::E4M3, &p.v_head_on, &p.v_page_on, &p.v_page_end);
  if (st != SPLASH_OK) return st;
  p.row_groups = (p.nrows + C::TILE - 1) / C::TILE;
  p.part_rows = std::min(p.nrows, C::TILE);
  char *ws = static_cast<char *>(a.workspace);
  p.before = reinterpret_cast<int32_t *>(ws);
  ws += align16(4 * ((int64_t)p.B + 1));
  p.lost = reinterpret_cast<int32_t *>(ws);
  ws += 4 * kMaxCtas;
  p.part_ml = reinterpret_cast<float *>(ws);
  ws += (int64_t)2 * kMaxCtas * p.part_rows * 2 * 4;
  p.part_o = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(ws) + 31) & ~(uintptr_t)31);
  const int64_t most = most_steps(a.Lq, a.max_pages, a.page_size, a.window_left), segments = (int64_t)p.B * p.Hkv * p.row_groups;
  int dev = 0, sms = 0, cluster = 0;
  SPLASH_CUDA_TRY(cudaGetDevice(&dev));
  SPLASH_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  if ((st = cluster_for<C>(dev, sms, segments, most, &cluster)) != SPLASH_OK) return st;
  if (cluster > 0) {
    SPLASH_CUDA_TRY(launch_dependent(tree_decode_kernel<C, true>, dim3((unsigned)(segments * cluster)), dim3(C::THREADS), C::SMEM, cluster,
                                     stream, map_k, map_v, p));
    splash_count_launches(1);
    return SPLASH_OK;
  }
  p.ctas = (int)std::min<int64_t>({most * segments, (int64_t)sms, (int64_t)kMaxCtas});
  SPLASH_CUDA_TRY(launch_dependent(tree_decode_kernel<C, false>, dim3(p.ctas), dim3(C::THREADS), C::SMEM, 1, stream, map_k, map_v, p));
  splash_count_launches(1);
  // a row per warp, or four where that still fills the GPU
  const int each = segments * p.part_rows >= 32 * 1024 ? 4 * kJoinWarps : kJoinWarps, slices = (p.part_rows + each - 1) / each;
  SPLASH_CUDA_TRY(launch_dependent(tree_join_kernel<C::DV, C::TILE, C::E4M3>, dim3((unsigned)(segments * slices)), dim3(32 * kJoinWarps), 0, 1,
                                   stream, p, slices, each));
  splash_count_launches(1);
  return SPLASH_OK;
}

template <int DQK, int DV>
splash_status pick(const splash_paged_decode_args &a, const Params &p, cudaStream_t stream) {
  constexpr bool E4M3 = SPLASH_TREE_E4M3 != 0;
  return p.nrows <= 128 ? launch<Config<DQK, DV, E4M3, false>>(a, p, stream) : launch<Config<DQK, DV, E4M3, true>>(a, p, stream);
}

}  // namespace
}  // namespace splash

#if !SPLASH_TREE_E4M3
int64_t splash_paged_tree_decode_entries(int32_t B, int32_t Hq, int32_t Hkv, int32_t T, int32_t max_pages, int32_t page_size,
                                         int64_t window) {
  const int64_t rows = (int64_t)(Hq / Hkv) * T, tile = rows <= 128 ? 128 : 256;
  return (splash::most_steps(T, max_pages, page_size, window) + splash::kPieceSteps) * B * Hkv * ((rows + tile - 1) / tile);
}

// Up to this many rows of a KV head paged_decode's kernel takes the tree: its tiles of 8
// and 16 rows keep four times the SMs' warps busy with loads, where here one warp in four
// has rows, and a step of 64 keys takes as long as with 128 rows.  (Device time, here -> there: 64
// requests of up to 4096 tokens, 32 / 8 heads of 128, 1 draft 117 -> 92 us, 4 drafts 123 ->
// 110; in e4m3, up to 8192 tokens, 186 -> 104 and 160 -> 122; 7 drafts, 128 / 128 heads of 192, window
// of 1023, cap 129 -> 94, 16 drafts without them 137 -> 112, in e4m3 254 -> 116; 1 request of
// 300 tokens, 4 drafts 9.4 -> 6.1.  With 32 rows: 8 drafts of 32 requests 72 here, and half
// of the 223 us that 4 tokens of 64 requests with 64 / 8 heads take there.)
constexpr int kFewRows = 16;

bool splash_paged_tree_decode_few_rows(int32_t Hq, int32_t Hkv, int32_t T) { return (int64_t)(Hq / Hkv) * T <= kFewRows; }

size_t splash_paged_tree_decode_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t T, int32_t dqk, int32_t dv,
                                                int32_t max_pages, int32_t page_size, int32_t type, int64_t window) {
  if (splash_paged_tree_decode_few_rows(Hq, Hkv, T))
    return splash_paged_decode_workspace_bytes(B, Hq, Hkv, T, dqk, dv, max_pages, page_size, type, window);
  const int64_t rows = std::min<int64_t>((int64_t)(Hq / Hkv) * T, 256);
  return (size_t)(16 + splash::align16(4 * ((int64_t)B + 1)) + 4 * splash::kMaxCtas + (int64_t)2 * splash::kMaxCtas * rows * 4 * (dv + 2));
}

splash_status splash_paged_tree_decode_launch(const splash_paged_tree_decode_args &args, cudaStream_t stream, uint32_t *err_word) {
  const bool e4m3 = args.decode.cache_type == SPLASH_CACHE_E4M3;
  if (splash_paged_tree_decode_few_rows(args.decode.Hq, args.decode.Hkv, args.decode.Lq))
    return e4m3 ? splash_paged_tree_rows_launch_e4m3(args, stream, err_word) : splash_paged_tree_rows_launch_bf16(args, stream, err_word);
  return e4m3 ? splash_paged_tree_decode_launch_e4m3(args, stream, err_word)
              : splash_paged_tree_decode_launch_bf16(args, stream, err_word);
}
#endif

#if SPLASH_TREE_E4M3
splash_status splash_paged_tree_decode_launch_e4m3(const splash_paged_tree_decode_args &args, cudaStream_t stream, uint32_t *err_word) {
#else
splash_status splash_paged_tree_decode_launch_bf16(const splash_paged_tree_decode_args &args, cudaStream_t stream, uint32_t *err_word) {
#endif
  using namespace splash;
  const splash_paged_decode_args &a = args.decode;
  const int64_t size = a.cache_type == SPLASH_CACHE_E4M3 ? 1 : 2;
  Params p = {};
  p.q = static_cast<const char *>(a.q.ptr);
  p.q_b = 2 * a.q.stride_b;
  p.q_h = 2 * a.q.stride_h;
  p.q_l = 2 * a.q.stride_l;
  p.v = static_cast<const char *>(a.v_cache.ptr);
  p.v_page = size * a.v_cache.stride_page;
  p.v_head = size * a.v_cache.stride_head;
  p.v_token = size * a.v_cache.stride_token;
  p.k_scale = size == 1 ? a.k_scale : nullptr;
  p.v_scale = size == 1 ? a.v_scale : nullptr;
  p.block_table = a.block_table;
  p.block_table_stride = a.block_table_stride;
  p.seq_lens = a.seq_lens;
  p.parents = args.parents;
  p.parents_stride = args.parents_stride_b;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  p.out_wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  p.num_pages = a.num_pages;
  p.B = a.B;
  p.Hkv = a.Hkv;
  p.T = a.Lq;
  p.G = a.Hq / a.Hkv;
  p.nrows = p.G * a.Lq;
  p.over_T = (uint32_t)((((uint64_t)1 << 32) + a.Lq - 1) / a.Lq);
  p.max_pages = a.max_pages;
  p.page_shift = __builtin_ctz((unsigned)a.page_size);
  // (differences of positions stay below 2^31 - 64)
  p.window = a.window_left < 0 ? -1 : (int32_t)std::min<int64_t>(a.window_left, INT32_MAX - 64);
  p.scale = a.scale;
  // (cap log2 e would overflow next to fp32's end; from 2^100 on tanh leaves every
  // score below 2^88 as it is)
  p.cap = a.softcap < 0x1p100f ? a.softcap : 0.f;
  p.err = err_word;
  if (a.dqk == 64) return pick<64, 64>(a, p, stream);
  if (a.dqk == 128) return pick<128, 128>(a, p, stream);
  return pick<192, 128>(a, p, stream);
}
