// tree_decode.cu -- attention of a tree of drafted tokens over a paged cache
// (splash_paged_tree_decode in splash.h).
//
// For a row (query head h, token l): s_j = scale q.k_j over the keys it sees --
// the context and its ancestors --, out = sum exp(s_j - m) v_j / sum exp(s_j - m),
// lse = m + ln sum exp(s_j - m), in one pass over the keys.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "dependent_launch.cuh"
#include "internal.h"
#include "sm103_ptx.cuh"

namespace splash {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

constexpr int kMaxCtas = 160;              // of the grid; the workspace holds two parts for each
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
// The smallest factor of the scores: a masked one (-inf) stays -inf times it.
constexpr float kTiny = 0x1p-126f;

struct Params {
  const char *q;
  int64_t q_b, q_h, q_l;  // byte strides
  const char *k, *v;
  int64_t k_page, k_head, k_token, v_page, v_head, v_token;  // byte strides
  const float *k_scale, *v_scale;
  const int32_t *block_table;
  int64_t block_table_stride;
  const int32_t *seq_lens, *parents;
  int64_t parents_stride;
  __nv_bfloat16 *out;
  float *lse;
  float *part_o, *part_ml;  // [2 * CTAs][part_rows][DV], [2 * CTAs][part_rows][2] (maximum, sum)
  int32_t *before;          // [B + 1] list entries (of one head and row group) before each sequence
  int64_t num_pages;
  int32_t B, Hkv, T, G, nrows, row_groups, part_rows;  // nrows = G * T rows per KV head
  int32_t max_pages, page_shift, window;               // window < 0: none
  int32_t ctas, min_steps;                             // of the grid; least steps of a CTA's part
  float scale, cap;                                    // cap <= 0: none
  uint32_t *err;
};

// A tile of NT x 128 rows of a KV head and steps of KW keys.
template <int DQK_, int DV_, bool E4M3_, int NT_>
struct Config {
  static constexpr int DQK = DQK_, DV = DV_, NT = NT_, KW = 64;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int RK = DQK * (E4M3 ? 1 : 2), RV = DV * (E4M3 ? 1 : 2);  // bytes of a cache row
  // Operand tiles in shared memory: 64-element (128-byte) columns of rows, 128-byte swizzle.
  static constexpr int COLUMN = KW * 128, K_BYTES = KW * DQK * 2, STAGE = K_BYTES + KW * DV * 2;
  static constexpr int Q_COLUMN = 128 * 128, Q_BYTES = 128 * DQK * 2;
  static constexpr int RAW = E4M3 ? KW * (RK + RV) : 0;  // an e4m3 step as it is in the cache
  static constexpr int BUDGET = 222 * 1024 - NT * Q_BYTES;
  static constexpr int STAGES = E4M3 ? (BUDGET >= 3 * STAGE + 2 * RAW ? 3 : 2) : std::min(8, BUDGET / STAGE);
  static constexpr int RAWS = E4M3 ? std::min(6, (BUDGET - STAGES * STAGE) / std::max(RAW, 1)) : 0;
  static constexpr int RING = E4M3 ? RAWS : 1;
  static constexpr int TILES = NT * Q_BYTES + STAGES * STAGE + RAWS * RAW;
  static_assert(E4M3 ? STAGES >= 2 && RAWS >= 2 : STAGES >= 3, "the loader's lookahead");
  // Barriers: full[STAGES] empty[STAGES], per tile s_full[2] p_full[2] o_done q_full, then drain
  static constexpr int BARS = 2 * STAGES + 6 * NT + 1;
  static constexpr int SMEM = 1024 + TILES + BARS * 8;
  static constexpr int WARPS = 4 * NT + 5, THREADS = 32 * WARPS;  // softmax, loaders, MMA
  // Tensor memory: per tile two buffers of scores (64 columns each, P in their place) and O.
  static constexpr int TILE_COLS = 2 * KW + DV, COLS = NT * TILE_COLS <= 256 ? 256 : 512;
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
__device__ __forceinline__ Span span_of(const Params &p, int b) {
  Span s;
  const int64_t most = (int64_t)p.max_pages << p.page_shift;
  const int32_t n = p.seq_lens[b];
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

// Equal contiguous parts of T entries, of at least p.min_steps each: CTA w takes
// [begin(w), begin(w + 1)).
struct Parts {
  int32_t total, count, each, more;  // the first `more` take one entry more
  __device__ __forceinline__ Parts(const Params &p, int32_t T)
      : total(T), count(max(1, min(p.ctas, T / p.min_steps))), each((uint32_t)T / (uint32_t)count), more(T - each * count) {}
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
  bool complete;  // all of the segment's steps
};
template <int KW>
struct Walk {
  const Params &p;
  int32_t u, end, per_seq;
  int32_t b, seg, step;
  Span s;
  __device__ __forceinline__ bool next(Piece &x) {
    if (u >= end) return false;
    x.b = b;
    x.seg = seg;
    x.step = step;
    x.steps = min(s.nst - step, end - u);
    x.s = s;
    x.complete = x.steps == s.nst;
    u += x.steps;
    step = 0;
    if (++seg == per_seq) {
      seg = 0;
      ++b;
      if (u < end) s = span_of<KW>(p, b);
    }
    return true;
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

__device__ __forceinline__ void copy16(uint32_t dst, const char *src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 load_shared4(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// Four e4m3 values to two pairs of fp16 (exact).
__device__ __forceinline__ void widen(uint32_t x, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// A number cut off to bf16.
__device__ __forceinline__ float cut(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The larger exponent field of a word's two bf16 values, and the word as fp16
// values times `down`.
__device__ __forceinline__ uint32_t exponent(uint32_t x) { return max((x >> 7) & 255u, (x >> 23) & 255u); }
__device__ __forceinline__ uint32_t to_half(uint32_t x, float down) {
  return pack_half2(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xffff0000u) * down);
}

// A word's 16-bit values that are not finite (exponent bits `top` all set) become 0.
__device__ __forceinline__ uint32_t finite(uint32_t x, uint32_t top, bool &lost) {
  if ((x & top) == top) x &= 0xffff0000u, lost = true;
  if ((x >> 16 & top) == top) x &= 0xffffu, lost = true;
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

template <class C>
struct Bars {
  uint32_t base;
  __device__ __forceinline__ uint32_t full(int s) const { return base + 8u * s; }
  __device__ __forceinline__ uint32_t empty(int s) const { return base + 8u * (C::STAGES + s); }
  __device__ __forceinline__ uint32_t s_full(int t, int x) const { return base + 8u * (2 * C::STAGES + 6 * t + x); }
  __device__ __forceinline__ uint32_t p_full(int t, int x) const { return base + 8u * (2 * C::STAGES + 6 * t + 2 + x); }
  __device__ __forceinline__ uint32_t o_done(int t) const { return base + 8u * (2 * C::STAGES + 6 * t + 4); }
  __device__ __forceinline__ uint32_t q_full(int t) const { return base + 8u * (2 * C::STAGES + 6 * t + 5); }
  __device__ __forceinline__ uint32_t drain() const { return base + 8u * (2 * C::STAGES + 6 * C::NT); }
};

__device__ __forceinline__ void give_up(const Params &p, volatile int *abort, uint32_t bit) {
  atomicOr(p.err, bit);
  *abort = 1;
}

// ------------------------------------------------------------------ loaders
// Four warps bring the steps of the CTA's part in order, running ahead of the
// products and across the borders of pieces: bf16 rows by 16-byte asynchronous
// copies straight into the swizzled operand tiles, e4m3 rows by way of a ring of
// raw steps, from which the thread that asked for a chunk widens it to fp16.
// Rows that no token sees become zeros and are not read.  In a step that only some
// tokens see in whole, values that are not finite become zeros too, since the
// product adds 0 x value for the others; `lost` then tells the epilogue to add
// them where they are seen.
// A thread's copies of a step's rows of CH 16-byte chunks.
template <class C, int CH>
__device__ __forceinline__ void ask(uint32_t stage, uint32_t raw, const char *const (&from)[C::KW / 16],
                                    const bool (&there)[C::KW / 16], int64_t token, const char *base, int32_t key0, const Span &s,
                                    int tid) {
  if constexpr (C::E4M3) {
#pragma unroll
    for (int e = 0; e < C::KW * CH / 128; ++e) {
      const int at = tid + 128 * e, row = at / CH, c = at % CH, block = row >> 4;
      const char *src = block == 0 ? from[0] : block == 1 ? from[1] : block == 2 ? from[2] : from[3];
      const bool in = block == 0 ? there[0] : block == 1 ? there[1] : block == 2 ? there[2] : there[3];
      const int32_t key = key0 + row;
      const bool read = in && key >= s.lo && key < s.n;
      copy16(raw + at * 16, read ? src + (row & 15) * token + c * 16 : base, read);
    }
  } else {
#pragma unroll
    for (int j = 0; j < C::KW / 16; ++j) {
      const int row = 16 * j + (tid >> 3), c = tid & 7;
      const int32_t key = key0 + row;
      const bool read = there[j] && key >= s.lo && key < s.n;
      const char *src = read ? from[j] + (tid >> 3) * token + c * 16 : base;
#pragma unroll
      for (int x = 0; x < CH / 8; ++x)
        copy16(stage + x * C::COLUMN + row * 128 + ((c ^ (row & 7)) << 4), read ? src + x * 128 : base, read);
    }
  }
}

// A chunk of 16 e4m3 values into a row of an operand tile.
template <class C>
__device__ __forceinline__ void widen_chunk(uint32_t src, uint32_t dst, int row, int c, bool check, bool &found) {
  const uint4 y = load_shared4(src);
  uint32_t w[8];
  widen(y.x, w[0], w[1]);
  widen(y.y, w[2], w[3]);
  widen(y.z, w[4], w[5]);
  widen(y.w, w[6], w[7]);
  if (check) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = finite(w[i], 0x7c00u, found);
  }
  dst += (c >> 2) * C::COLUMN + row * 128;
  const int cc = 2 * (c & 3);
  st_shared_v4(dst + ((cc ^ (row & 7)) << 4), w[0], w[1], w[2], w[3]);
  st_shared_v4(dst + (((cc + 1) ^ (row & 7)) << 4), w[4], w[5], w[6], w[7]);
}

template <class C>
__device__ __forceinline__ void run_loader(const Params &p, Walk<C::KW> walk, const Bars<C> bar, uint32_t stages, uint32_t raws,
                                           int tid, volatile int *abort, volatile int *lost) {
  constexpr int KW = C::KW, BLOCKS = KW / 16;
  constexpr int AHEAD = C::E4M3 ? C::RAWS - 1 : C::STAGES - 2;  // steps asked for before one is handed over
  constexpr int CK = C::RK / 16, CV = C::RV / 16, EK = KW * CK / 128, EV = KW * CV / 128;  // chunks of a row, of a thread
  uint32_t asked = 0, given = 0, partial = 0;  // partial: a bit for each step asked for, the newest lowest
  Piece x;
  int32_t entry[BLOCKS];
  bool ok = true;

  auto hand_over = [&]() {
    const int st = given % C::STAGES;
    const bool clean = (partial >> (asked - given - 1) & 1u) != 0;
    const uint32_t stage = stages + st * C::STAGE;
    bool found = false;
    if constexpr (C::E4M3) {
      if (given >= C::STAGES && !mbar_wait(bar.empty(st), (given / C::STAGES - 1) & 1u, abort, kTimeoutNs)) return false;
      const uint32_t raw = raws + (given % C::RING) * C::RAW;
#pragma unroll
      for (int i = 0; i < EK; ++i) {
        const int at = tid + 128 * i;
        widen_chunk<C>(raw + at * 16, stage, at / CK, at % CK, false, found);
      }
#pragma unroll
      for (int i = 0; i < EV; ++i) {
        const int at = tid + 128 * i;
        widen_chunk<C>(raw + KW * C::RK + at * 16, stage + C::K_BYTES, at / CV, at % CV, clean, found);
      }
    } else if (clean) {
#pragma unroll 1
      for (int i = 0; i < BLOCKS * (CV / 8); ++i) {
        const int row = 16 * (i / (CV / 8)) + (tid >> 3);
        const uint32_t at = stage + C::K_BYTES + (i % (CV / 8)) * C::COLUMN + row * 128 + (((tid & 7) ^ (row & 7)) << 4);
        const uint4 y = load_shared4(at);
        bool here = false;
        const uint32_t w[4] = {finite(y.x, 0x7f80u, here), finite(y.y, 0x7f80u, here), finite(y.z, 0x7f80u, here),
                               finite(y.w, 0x7f80u, here)};
        if (here) st_shared_v4(at, w[0], w[1], w[2], w[3]);
        found |= here;
      }
    }
    if (found) *lost = 1;
    __threadfence_block();
    fence_proxy_async_shared();
    mbar_arrive(bar.full(st));
    ++given;
    return true;
  };

  while (ok && walk.next(x)) {
    const int head = x.seg / p.row_groups;
    const char *k = p.k + head * p.k_head, *v = p.v + head * p.v_head;
    const int32_t *pages = p.block_table + x.b * p.block_table_stride;
    auto look = [&](int32_t key0) {
#pragma unroll
      for (int i = 0; i < BLOCKS; ++i) {
        const int32_t key = key0 + 16 * i;
        entry[i] = key < x.s.n && key + 16 > x.s.lo ? pages[key >> p.page_shift] : 0;
      }
    };
    int32_t key0 = (x.s.step0 + x.step) * KW;
    look(key0);
    for (int i = 0; i < x.steps && ok; ++i, key0 += KW) {
      const int st = asked % C::STAGES;
      if (!C::E4M3 && asked >= C::STAGES && !mbar_wait(bar.empty(st), (asked / C::STAGES - 1) & 1u, abort, kTimeoutNs)) {
        ok = false;
        break;
      }
      const char *from_k[BLOCKS], *from_v[BLOCKS];
      bool there[BLOCKS];
#pragma unroll
      for (int j = 0; j < BLOCKS; ++j) {
        const int32_t key = key0 + 16 * j;
        there[j] = entry[j] >= 0 && entry[j] < p.num_pages;
        if (!there[j] && tid == 0) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
        const int64_t page = there[j] ? entry[j] : 0, slot = key & ((1 << p.page_shift) - 1);
        from_k[j] = k + page * p.k_page + slot * p.k_token;
        from_v[j] = v + page * p.v_page + slot * p.v_token;
      }
      if (i + 1 < x.steps) look(key0 + KW);
      const uint32_t stage = stages + st * C::STAGE, raw = raws + (C::E4M3 ? asked % C::RING : 0u) * C::RAW;
      ask<C, CK>(stage, raw, from_k, there, p.k_token, k, key0, x.s, tid);
      ask<C, CV>(stage + C::K_BYTES, raw + KW * C::RK, from_v, there, p.v_token, v, key0, x.s, tid);
      copy_commit();
      partial = partial << 1 | (whole<KW>(p, x.s, key0) ? 0u : 1u);
      ++asked;
      if (asked - given > AHEAD) {
        copy_wait<AHEAD>();
        ok = hand_over();
      }
    }
  }
  copy_wait<0>();
  while (ok && given < asked) ok = hand_over();
  if (!ok) give_up(p, abort, SPLASH_DEV_TIMEOUT_PRODUCER);
}

// ------------------------------------------------------------------ products
// One warp: S = Q K^T of a step for each tile, one step ahead of the softmax, and
// O += P V.  For a bf16 cache P is two terms (see the softmax), each a product.
template <class C>
__device__ __forceinline__ void run_mma(const Params &p, Walk<C::KW> walk, const Bars<C> bar, uint32_t tmem, uint32_t q_addr,
                                        uint32_t stages, volatile int *abort) {
  constexpr uint32_t HI = sdesc_hi_sw128(1024);
  constexpr int KW = C::KW;
  const uint32_t leader = elect_one_sync();
  uint32_t cnt[2] = {0, 0}, pieces[2] = {0, 0}, step = 0;  // of each tile, of the CTA
  bool ok = true;
  Piece x;
  while (ok && walk.next(x)) {
    const int rows = min(C::NT * 128, p.nrows - (x.seg % p.row_groups) * C::NT * 128), tiles = (rows + 127) / 128;
#pragma unroll
    for (int t = 0; t < C::NT; ++t)
      if (t < tiles) ok = ok && mbar_wait(bar.q_full(t), pieces[t]++ & 1u, abort, kTimeoutNs);
    if (!ok) break;
    tc_fence_after();
    for (int i = 0; i <= x.steps && ok; ++i) {
      if (i < x.steps) {
        const uint32_t u = step + i, st = u % C::STAGES;
        if (!(ok = mbar_wait(bar.full(st), (u / C::STAGES) & 1u, abort, kTimeoutNs))) break;
        tc_fence_after();
        const uint32_t kd = sdesc_lo(stages + st * C::STAGE, 16);
#pragma unroll
        for (int t = 0; t < C::NT; ++t) {
          if (t >= tiles) break;
          const uint32_t buf = (cnt[t] + i) & 1u, qd = sdesc_lo(q_addr + t * C::Q_BYTES, 16);
          const uint32_t d = tmem + t * C::TILE_COLS + buf * KW;
#pragma unroll
          for (int kk = 0; kk < C::DQK / 16; ++kk)
            mma_ss_lhp(leader, d, qd + (uint32_t)(((kk / 4) * C::Q_COLUMN + (kk % 4) * 32) >> 4), HI,
                       kd + (uint32_t)(((kk / 4) * C::COLUMN + (kk % 4) * 32) >> 4), HI, C::IDESC_QK, kk != 0);
          tc_commit_p(leader, bar.s_full(t, buf));
        }
      }
      if (i > 0) {
        const uint32_t u = step + i - 1, st = u % C::STAGES;
        const uint32_t vd = sdesc_lo(stages + st * C::STAGE + C::K_BYTES, C::COLUMN);
#pragma unroll
        for (int t = 0; t < C::NT; ++t) {
          if (t >= tiles) break;
          const uint32_t c = cnt[t] + i - 1, buf = c & 1u;
          if (!(ok = mbar_wait(bar.p_full(t, buf), (c >> 1) & 1u, abort, kTimeoutNs))) break;
          tc_fence_after();
          const uint32_t pa = tmem + t * C::TILE_COLS + buf * KW, o = tmem + t * C::TILE_COLS + 2 * KW;
#pragma unroll
          for (int kk = 0; kk < KW / 16; ++kk)
            mma_ts_lhp(leader, o, pa + 8u * kk, vd + (uint32_t)((kk * 2048) >> 4), HI, C::IDESC_PV, i > 1 || kk > 0);
          if constexpr (!C::E4M3) {
#pragma unroll
            for (int kk = 0; kk < KW / 16; ++kk)
              mma_ts_lhp(leader, o, pa + KW / 2 + 8u * kk, vd + (uint32_t)((kk * 2048) >> 4), HI, C::IDESC_PV, 1);
          }
          tc_commit_p(leader, bar.o_done(t));
        }
        if (ok) tc_commit_p(leader, bar.empty(st));
      }
    }
    step += x.steps;
#pragma unroll
    for (int t = 0; t < C::NT; ++t)
      if (t < tiles) cnt[t] += x.steps;
  }
  if (!ok && leader) give_up(p, abort, SPLASH_DEV_TIMEOUT_MMA);
  tc_commit_p(leader, bar.drain());
  if (!mbar_wait_drain(bar.drain(), 0, kTimeoutNs) && leader) atomicOr(p.err, SPLASH_DEV_TIMEOUT_DRAIN);
}

// ------------------------------------------------------------------ softmax
// A row's queries, the row of its tile; zeros for rows that do not exist.  For an
// e4m3 cache they become fp16, scaled by the power of two that brings the row's
// largest element into [1, 2): exact but for elements 2^14 times smaller, whose
// error, 2^-25 of the largest, is below that of an fp32 sum.  Returns the factor.
template <class C>
__device__ __forceinline__ float load_query(const char *q, bool real, uint32_t dst, int row, bool negate) {
  float down = negate ? -1.f : 1.f, factor = 1.f;
  if (C::E4M3 && real) {
    uint32_t top = 0;
#pragma unroll 4
    for (int c = 0; c < C::DQK / 8; ++c) {
      const uint4 y = reinterpret_cast<const uint4 *>(q)[c];
      top = max(max(top, max(exponent(y.x), exponent(y.y))), max(exponent(y.z), exponent(y.w)));
    }
    top = min(max(top, 1u), 253u);
    down *= __uint_as_float((254u - top) << 23);
    factor = __uint_as_float(top << 23);
  }
#pragma unroll 4
  for (int c = 0; c < C::DQK / 8; ++c) {
    uint4 y = make_uint4(0, 0, 0, 0);
    if (real) y = reinterpret_cast<const uint4 *>(q)[c];
    if (C::E4M3) y = make_uint4(to_half(y.x, down), to_half(y.y, down), to_half(y.z, down), to_half(y.w, down));
    st_shared_v4(dst + (c >> 3) * C::Q_COLUMN + row * 128 + (((c & 7) ^ (row & 7)) << 4), y.x, y.y, y.z, y.w);
  }
  return factor;
}

// Adds to 32 columns of a row the values that are not finite of the keys it sees in
// a piece's steps that are not whole (the product had zeros in their place).
template <class C>
__device__ __noinline__ void add_lost(const Params &p, const Piece &x, int head, int32_t lo, uint64_t seen, int col, float (&o)[32]) {
  for (int i = 0; i < x.steps; ++i) {
    const int32_t key0 = (x.s.step0 + x.step + i) * C::KW;
    if (whole<C::KW>(p, x.s, key0)) continue;
    for (uint64_t m = visible(key0, x.s.ctx, lo, seen); m != 0; m &= m - 1) {
      const int32_t key = key0 + __ffsll(m) - 1;
      const int32_t page = p.block_table[x.b * p.block_table_stride + (key >> p.page_shift)];
      if (page < 0 || page >= p.num_pages) continue;
      const char *v = p.v + page * p.v_page + head * p.v_head + (key & ((1 << p.page_shift) - 1)) * p.v_token;
#pragma unroll 1
      for (int c = 0; c < 32; ++c) {
        const float y = C::E4M3 ? (float)reinterpret_cast<const __nv_fp8_e4m3 *>(v)[col + c]
                                : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(v)[col + c]);
        if (!(fabsf(y) < INFINITY)) o[c] += y;
      }
    }
  }
}

// Four warps per tile, a thread per row.
template <class C>
__device__ __forceinline__ void run_softmax(const Params &p, Walk<C::KW> walk, const Bars<C> bar, uint32_t tmem, uint32_t q_addr,
                                            int32_t *s_parents, int t, int part, volatile int *abort, volatile int *lost) {
  constexpr int KW = C::KW;
  constexpr bool E4M3 = C::E4M3;
  const int tid = threadIdx.x & 127, warp = tid >> 5;
  const uint32_t base = tmem + t * C::TILE_COLS + ((uint32_t)(32 * warp) << 16), o_col = base + 2 * KW;
  uint32_t cnt = 0;
  bool ok = true;
  Piece x;
  while (ok && walk.next(x)) {
    const int head = x.seg / p.row_groups, row0 = (x.seg % p.row_groups) * C::NT * 128;
    const int rows = min(128, p.nrows - row0 - t * 128);  // of this tile (none: <= 0)
    const int slot = part;
    part |= 1;  // what follows the first piece and is not complete is the last one
    if (rows <= 0) continue;
    const bool real = tid < rows, busy = 32 * warp < rows;
    const int r = row0 + t * 128 + tid, g = real ? r / p.T : 0, l = real ? r - g * p.T : 0;
    bar_sync(1 + t, 128);  // (the tree before is no longer read)
    if (tid < p.T) s_parents[tid] = p.parents[x.b * p.parents_stride + tid];
    const float ks = E4M3 ? p.k_scale[head] : 1.f;
    const char *q = p.q + x.b * p.q_b + ((int64_t)head * p.G + g) * p.q_h + l * p.q_l;
    float factor = (p.cap > 0.f ? p.scale / p.cap : p.scale * kLog2e) * fabsf(ks);
    factor *= load_query<C>(q, real, q_addr + t * C::Q_BYTES, tid, ks < 0.f);
    if (factor < kTiny) factor = kTiny;  // (NaN stays)
    fence_proxy_async_shared();
    mbar_arrive(bar.q_full(t));
    bar_sync(1 + t, 128);
    Branch me = {0, 0};
    if (real) {
      bool bad = false;
      me = branch_of(s_parents, l, max(0, -x.s.ctx), p.window, &bad);
      if (bad) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
    }
    const int32_t lo = p.window < 0 ? 0 : max(0, x.s.ctx + me.depth - p.window);
    float m = -INFINITY, sum = 0.f;

    for (int i = 0; i < x.steps; ++i, ++cnt) {
      const uint32_t buf = cnt & 1u;
      if (!(ok = __all_sync(~0u, mbar_wait(bar.s_full(t, buf), (cnt >> 1) & 1u, abort, kTimeoutNs)))) break;
      if (busy) {
        tc_fence_after();
        const int32_t key0 = (x.s.step0 + x.step + i) * KW;
        const bool all = whole<KW>(p, x.s, key0);
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
          const float cap = p.cap * kLog2e;
#pragma unroll
          for (int j = 0; j < KW; ++j) s[j] = cap * tanh_of(s[j] * factor);
        }
        if (!all) {
          const uint64_t see = visible(key0, x.s.ctx, lo, me.seen);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (!((uint32_t)see >> j & 1u)) s[j] = -INFINITY;
            if (!((uint32_t)(see >> 32) >> j & 1u)) s[32 + j] = -INFINITY;
          }
        }
        const float times = p.cap > 0.f ? 1.f : factor;
        float top = s[0];
#pragma unroll
        for (int j = 1; j + 1 < KW; j += 2) top = fmax3(top, s[j], s[j + 1]);
        top = fmaxf(top, s[KW - 1]) * times;
        if (E4M3) top -= kBelowTop;
        if (__any_sync(~0u, top > m + kSlack)) {
          const float high = fmaxf(top, m), alpha = m == -INFINITY ? 0.f : ex2_approx(m - high);
          m = high;
          sum *= alpha;
          if (i > 0) {
            // (only the product of the step before can still be running: this one's waits for us)
            if (!(ok = __all_sync(~0u, mbar_wait(bar.o_done(t), (cnt - 1) & 1u, abort, kTimeoutNs)))) break;
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
        f32x2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
        for (int j = 0; j < KW; j += 2) {
          const f32x2 y = ffma2({s[j], s[j + 1]}, {times, times}, {-ref, -ref});
          s[j] = ex2_approx(y.x);
          s[j + 1] = ex2_approx(y.y);
          acc[j / 2 & 1] = fadd2(acc[j / 2 & 1], {s[j], s[j + 1]});
        }
        acc[0] = fadd2(acc[0], acc[1]);
        sum += acc[0].x + acc[0].y;
        if constexpr (E4M3) {
#pragma unroll
          for (int j = 0; j < 32; ++j) a[j] = pack_half2(s[2 * j], s[2 * j + 1]);
          tmem_st32(base + buf * KW, a);
        } else {
          // P in two bf16 terms, cut off and rest: 2^-16 of each p, where bf16 alone
          // loses 2^-8, as much as the rounding of the result.  The rest is kept above 0 in
          // whole steps: an infinite value times either term then has its sign, and the
          // sum is that infinity (0 x infinity is NaN); the floor, the smallest normal
          // number, adds 2^-126 of a value.  In the other steps values are finite.
          const uint32_t floor = all ? 0x00800080u : 0u;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            a[j] = __byte_perm(__float_as_uint(s[2 * j]), __float_as_uint(s[2 * j + 1]), 0x7632);
            const f32x2 rest = fadd2({s[2 * j], s[2 * j + 1]}, {-cut(s[2 * j]), -cut(s[2 * j + 1])});
            b[j] = max_bf16x2(pack_bf16x2(rest.x, rest.y), floor);
          }
          tmem_st32(base + buf * KW, a);
          tmem_st32(base + buf * KW + 32, b);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      mbar_arrive(bar.p_full(t, buf));
    }
    if (!ok) break;

    // ---- finished rows, or this CTA's part of them
    if (!(ok = __all_sync(~0u, mbar_wait(bar.o_done(t), (cnt - 1) & 1u, abort, kTimeoutNs)))) break;
    tc_fence_after();
    if (busy) {
      const bool empty = sum == 0.f || me.seen == 0;
      const float inv = (E4M3 ? p.v_scale[head] : 1.f) / sum;
      const int64_t row = x.complete ? ((int64_t)x.b * p.Hkv + head) * p.nrows + r : (int64_t)slot * p.part_rows + t * 128 + tid;
#pragma unroll 1
      for (int c = 0; c < C::DV / 32; ++c) {
        uint32_t y[32];
        float o[32];
        tmem_ld32(o_col + 32 * c, y);
        tmem_wait_ld();
        reg_fence32(y);
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = __uint_as_float(y[j]);
        if (*lost && real) {
          float z[32];  // (in memory: the call takes its address)
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] = o[j];
          add_lost<C>(p, x, head, lo, me.seen, 32 * c, z);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = z[j];
        }
        if (real && x.complete) {
          uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * C::DV + 32 * c);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = empty ? 0.f : o[j] * inv;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            dst[j] = make_uint4(pack_bf16x2(o[8 * j], o[8 * j + 1]), pack_bf16x2(o[8 * j + 2], o[8 * j + 3]),
                                pack_bf16x2(o[8 * j + 4], o[8 * j + 5]), pack_bf16x2(o[8 * j + 6], o[8 * j + 7]));
        } else if (real) {
          float4 *dst = reinterpret_cast<float4 *>(p.part_o + row * C::DV + 32 * c);
#pragma unroll
          for (int j = 0; j < 8; ++j) dst[j] = empty ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
        __syncwarp();
      }
      if (real) {
        if (x.complete)
          p.lse[row] = empty ? -INFINITY : (m + log2f(sum)) * kLn2;
        else
          *reinterpret_cast<float2 *>(p.part_ml + 2 * row) = empty ? make_float2(-INFINITY, 0.f) : make_float2(m, sum);
      }
      tc_fence_before();
    }
  }
  if (!ok && (threadIdx.x & 31) == 0) give_up(p, abort, SPLASH_DEV_TIMEOUT_SOFTMAX);
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) tree_decode_kernel(const Params p) {
  constexpr int KW = C::KW;
  extern __shared__ char smem_raw[];
  __shared__ int32_t s_scan[C::WARPS], s_seq, s_before, s_parents[C::NT][SPLASH_MAX_TREE_TOKENS];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_lost;
  const uint32_t tiles = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const Bars<C> bar{tiles + C::TILES};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == C::WARPS - 1) {
    tmem_alloc(smem_u32(&s_tmem), C::COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar.full(s), 128);
      mbar_init(bar.empty(s), 1);
    }
    for (int t = 0; t < C::NT; ++t) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(bar.s_full(t, x), 1);
        mbar_init(bar.p_full(t, x), 128);
      }
      mbar_init(bar.o_done(t), 1);
      mbar_init(bar.q_full(t), 128);
    }
    mbar_init(bar.drain(), 1);
    mbar_fence_init();
    s_abort = s_lost = 0;
  }
  // (the allocation comes before the next kernel may start: one that waits for this one cannot
  // hold what this one still needs)
  grid_dependency();

  // ---- this CTA's part of the list: a scan over the sequences
  const int per_seq = p.Hkv * p.row_groups;
  const int per = (p.B + C::THREADS - 1) / C::THREADS;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int32_t own = 0;
  for (int b = b0; b < b1; ++b) own += span_of<KW>(p, b).nst;
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
  const int32_t begin = parts.begin(blockIdx.x), end = parts.begin(blockIdx.x + 1);
  if (blockIdx.x == 0 || (begin >= before * per_seq && begin < (before + own) * per_seq)) {
    int32_t at = before;
    for (int b = b0; b < b1; ++b) {
      const Span s = span_of<KW>(p, b);
      if (begin >= at * per_seq && begin < (at + s.nst) * per_seq) s_seq = b, s_before = at;
      if (blockIdx.x == 0) {
        p.before[b] = at;
        if (b == p.B - 1) p.before[p.B] = at + s.nst;
        if (s.n != p.seq_lens[b]) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
      }
      at += s.nst;
    }
  }
  __syncthreads();
  if (begin < end) {
    Walk<KW> walk{p, begin, end, per_seq, s_seq, 0, 0, {}};
    walk.s = span_of<KW>(p, walk.b);
    const int32_t in_seq = begin - s_before * per_seq;
    walk.seg = (uint32_t)in_seq / (uint32_t)walk.s.nst;
    walk.step = in_seq - walk.seg * walk.s.nst;
    const uint32_t q_addr = tiles, stages = tiles + C::NT * C::Q_BYTES, raws = stages + C::STAGES * C::STAGE;
    // (registers: 13 warps are launched with 128 a thread; 2 x 128 x 152 + 128 x 80 + 32 x 128 of them)
    if (warp < 4 * C::NT) {
      if constexpr (C::NT == 2) regs_increase<152>();
      run_softmax<C>(p, walk, bar, s_tmem, q_addr, s_parents[warp >> 2], warp >> 2, 2 * blockIdx.x, &s_abort, &s_lost);
    } else if (warp < C::WARPS - 1) {
      if constexpr (C::NT == 2) regs_decrease<80>();
      run_loader<C>(p, walk, bar, stages, raws, tid - 128 * C::NT, &s_abort, &s_lost);
    } else {
      run_mma<C>(p, walk, bar, s_tmem, q_addr, stages, &s_abort);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::WARPS - 1) {
    tc_fence_after();
    tmem_dealloc(s_tmem, C::COLS);
  }
}

// Joins the parts of a row that several CTAs computed: with (m_c, l_c, o_c) of
// part c and m = max m_c: out = sum exp(m_c - m) o_c / sum exp(m_c - m) l_c, in the
// order of the keys.  One CTA per row, its warps taking every fourth part.
constexpr int kJoinWarps = 4;
template <int DV, int TILE>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const Params p) {
  __shared__ float s_o[kJoinWarps][DV], s_sum[kJoinWarps], s_top[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int PER = DV / 32;
  const int64_t row = blockIdx.x;  // (b, KV head, row)
  const int head_row = (int)(row % p.nrows), head = (int)(row / p.nrows % p.Hkv), b = (int)(row / p.nrows / p.Hkv);
  const int per_seq = p.Hkv * p.row_groups;
  grid_dependency();
  const Parts parts(p, p.before[p.B] * per_seq);
  const int32_t entries = p.before[b + 1] - p.before[b];
  const int32_t u0 = p.before[b] * per_seq + entries * (head * p.row_groups + head_row / TILE);
  const int c0 = parts.owner(u0), c1 = parts.owner(u0 + entries - 1);
  if (c0 == c1) return;  // written by that CTA
  const int r = head_row % TILE;
  // It is the first piece of CTA c0 if nothing of the one before is that CTA's.
  const int64_t first = (int64_t)2 * c0 + (parts.begin(c0) >= u0 ? 0 : 1);
  constexpr int AHEAD = 4;  // parts read at once
  float top = -INFINITY, sum = 0.f, acc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  // (an infinite value stays one however small its part's factor: 0 x infinity would be NaN)
  auto scaled = [](float f, float x) { return fabsf(x) == INFINITY ? x : f * x; };
  for (int c = c0 + warp; c <= c1; c += kJoinWarps * AHEAD) {
    float2 ml[AHEAD];
    float x[AHEAD][PER];
    float above = top;
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int ca = c + a * kJoinWarps;
      ml[a] = make_float2(-INFINITY, 0.f);
      if (ca <= c1) {
        const int64_t at = (ca == c0 ? first : (int64_t)2 * ca) * p.part_rows + r;
        ml[a] = *reinterpret_cast<const float2 *>(p.part_ml + at * 2);
#pragma unroll
        for (int i = 0; i < PER; ++i) x[a][i] = p.part_o[at * DV + i * 32 + lane];
      }
    }
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) above = fmaxf(above, ml[a].x);
    const float ref = above == -INFINITY ? 0.f : above, f0 = ex2_approx(top - ref);
    sum *= f0;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = scaled(f0, acc[i]);
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      if (c + a * kJoinWarps > c1) break;
      const float f = ex2_approx(ml[a].x - ref);
      sum += f * ml[a].y;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] += scaled(f, x[a][i]);
    }
    top = above;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) s_o[warp][i * 32 + lane] = acc[i];
  if (lane == 0) s_sum[warp] = sum, s_top[warp] = top;
  __syncthreads();
  float f[kJoinWarps];
  top = -INFINITY;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_top[w]);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    f[w] = ex2_approx(s_top[w] - (top == -INFINITY ? 0.f : top));
    sum += f[w] * s_sum[w];
  }
  const float inv = sum == 0.f ? 0.f : (p.v_scale != nullptr ? p.v_scale[head] : 1.f) / sum;
  if ((int)threadIdx.x < DV / 2) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      x += scaled(f[w], s_o[w][2 * threadIdx.x]);
      y += scaled(f[w], s_o[w][2 * threadIdx.x + 1]);
    }
    reinterpret_cast<uint32_t *>(p.out + row * DV)[threadIdx.x] = pack_bf16x2(x * inv, y * inv);
  }
  if (threadIdx.x == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

int64_t align16(int64_t x) { return (x + 15) & ~(int64_t)15; }

// Steps that a sequence can have, from its row of pages and the window.
int64_t most_steps(int32_t T, int32_t max_pages, int32_t page_size, int64_t window) {
  const int64_t most = ((int64_t)max_pages * page_size + 63) / 64;
  return window < 0 ? most : std::min(most, (window + T) / 64 + 3);
}

template <class C>
splash_status launch(const splash_paged_decode_args &a, Params p, cudaStream_t stream) {
  p.row_groups = (p.nrows + C::NT * 128 - 1) / (C::NT * 128);
  p.part_rows = std::min(p.nrows, C::NT * 128);
  char *ws = static_cast<char *>(a.workspace);
  p.before = reinterpret_cast<int32_t *>(ws);
  ws += align16(4 * ((int64_t)p.B + 1));
  p.part_ml = reinterpret_cast<float *>(ws);
  ws += (int64_t)2 * kMaxCtas * p.part_rows * 2 * 4;
  p.part_o = reinterpret_cast<float *>(ws);
  int dev = 0, sms = 0;
  SPLASH_CUDA_TRY(cudaGetDevice(&dev));
  SPLASH_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  static std::atomic<bool> ready[64];  // per device: the kernel may use its shared memory
  if (!ready[dev & 63].load(std::memory_order_acquire)) {
    SPLASH_CUDA_TRY(cudaFuncSetAttribute(tree_decode_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
    ready[dev & 63].store(true, std::memory_order_release);
  }
  const int64_t most = most_steps(a.Lq, a.max_pages, a.page_size, a.window_left), segments = (int64_t)p.B * p.Hkv * p.row_groups;
  p.min_steps = 1;
  p.ctas = (int)std::min<int64_t>({most * segments, (int64_t)sms, (int64_t)kMaxCtas});
  SPLASH_CUDA_TRY(launch_dependent(tree_decode_kernel<C>, dim3(p.ctas), dim3(C::THREADS), C::SMEM, 1, stream, p));
  splash_count_launches(1);
  if (most <= 1) return SPLASH_OK;  // (no segment has more than one step: nothing to join)
  const dim3 rows((unsigned)((int64_t)p.B * p.Hkv * p.nrows));
  SPLASH_CUDA_TRY(launch_dependent(tree_join_kernel<C::DV, C::NT * 128>, rows, dim3(32 * kJoinWarps), 0, 1, stream, p));
  splash_count_launches(1);
  return SPLASH_OK;
}

template <int DQK, int DV, bool E4M3>
splash_status pick(const splash_paged_decode_args &a, const Params &p, cudaStream_t stream) {
  return p.nrows <= 128 ? launch<Config<DQK, DV, E4M3, 1>>(a, p, stream) : launch<Config<DQK, DV, E4M3, 2>>(a, p, stream);
}

}  // namespace
}  // namespace splash

size_t splash_paged_tree_decode_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t T, int32_t, int32_t dv, int32_t, int32_t,
                                                int32_t, int64_t) {
  const int64_t rows = std::min<int64_t>((int64_t)(Hq / Hkv) * T, 256);
  return (size_t)(splash::align16(4 * ((int64_t)B + 1)) + (int64_t)2 * splash::kMaxCtas * rows * 4 * (dv + 2));
}

splash_status splash_paged_tree_decode_launch(const splash_paged_tree_decode_args &args, cudaStream_t stream, uint32_t *err_word) {
  using namespace splash;
  const splash_paged_decode_args &a = args.decode;
  const int64_t size = a.cache_type == SPLASH_CACHE_E4M3 ? 1 : 2;
  Params p = {};
  p.q = static_cast<const char *>(a.q.ptr);
  p.q_b = 2 * a.q.stride_b;
  p.q_h = 2 * a.q.stride_h;
  p.q_l = 2 * a.q.stride_l;
  p.k = static_cast<const char *>(a.k_cache.ptr);
  p.k_page = size * a.k_cache.stride_page;
  p.k_head = size * a.k_cache.stride_head;
  p.k_token = size * a.k_cache.stride_token;
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
  p.num_pages = a.num_pages;
  p.B = a.B;
  p.Hkv = a.Hkv;
  p.T = a.Lq;
  p.G = a.Hq / a.Hkv;
  p.nrows = p.G * a.Lq;
  p.max_pages = a.max_pages;
  p.page_shift = __builtin_ctz((unsigned)a.page_size);
  // (differences of positions stay below 2^31 - 64)
  p.window = a.window_left < 0 ? -1 : (int32_t)std::min<int64_t>(a.window_left, INT32_MAX - 64);
  p.scale = a.scale;
  // (cap log2 e would overflow next to fp32's end; from 2^100 on tanh leaves every
  // score below 2^88 as it is)
  p.cap = a.softcap < 0x1p100f ? a.softcap : 0.f;
  p.err = err_word;
  const auto f = size == 1 ? (a.dqk == 64 ? pick<64, 64, true> : a.dqk == 128 ? pick<128, 128, true> : pick<192, 128, true>)
                           : (a.dqk == 64 ? pick<64, 64, false> : a.dqk == 128 ? pick<128, 128, false> : pick<192, 128, false>);
  return f(a, p, stream);
}
