// paged_decode.cu -- attention of new tokens over a paged key/value cache
// (splash_paged_decode in splash.h).  Compiled once for each cache type
// (SPLASH_DECODE_E4M3 = 0, 1), so that the instantiations build in parallel.
//
// For a query row: s_j = scale q.k_j, m = max s_j, l = sum exp(s_j - m),
// out = sum exp(s_j - m) v_j / l, lse = m + ln l, in one pass over the keys.
// Every key and value is used by the Hq/Hkv * Lq rows of its head only, a few
// FLOP per byte: reading the cache bounds the call, so the kernel is built to
// keep the memory system full.  64 requests of 64 .. 4096 tokens (32 query, 8 KV
// heads of 128, bf16) take 89 .. 91 us (box to box), 6.1 TB/s with the launches;
// 64 requests of up to 32768 tokens with an e4m3 cache 316 .. 323 us, 6.8 .. 6.9
// TB/s; DRAM reads are the cache's bytes (546 MB of 546 for the first).  One
// request of 300 tokens takes 4.7 us: the launch, three dependent reads (length,
// page, keys) and the join.  Up to 32 rows share a reading; 64 rows read the cache
// twice and take twice the time (64 requests of up to 4096 tokens, 64 / 8 heads: 4
// tokens each 223 us, 8 tokens 465), as their products, not DRAM, bound them.
//
//  * Work.  The keys of each (sequence, KV head, group of rows) are cut into
//    steps of KW keys; all steps form one list, and every warp of a grid that
//    fills the GPU once takes an equal, contiguous part of it.  Long and short
//    sequences thus load every SM alike.  A (sequence, head) that one warp
//    covers is finished there; parts of one that several warps share go to the
//    workspace as (maximum, sum, unnormalised output) and a second kernel joins
//    them, in the order of the keys, so that the result does not depend on
//    timing.  Where there are too few segments to fill the GPU and none can be
//    very long, each takes a cluster of CTAs instead: their warps share the keys
//    equally and join through distributed shared memory, which saves the scan,
//    the workspace and the second kernel.
//  * Loads.  Each warp keeps a ring of stages in shared memory, filled by
//    16-byte asynchronous copies that run ahead of the products and across the
//    borders of sequences; there is no barrier between warps.  Two CTAs of four
//    warps per SM with 2 to 6 stages of 4 to 10 KB saturate DRAM (the 32-row tile of
//    192-wide heads has room for one CTA); more in flight (prefetching into L2)
//    measured slower.  Rows outside the keys that some query sees are filled with
//    zeros instead of being read, so that whatever they hold cannot reach a
//    product.
//  * Products.  16 rows x 16 keys per tensor instruction (mma.sync: with 4 to 32
//    rows a tile is memory-bound many times over, and the accumulators stay in
//    registers next to the softmax).  P goes to the second product from the
//    registers that the first one left it in.  With two CTAs of 128 threads per
//    SM a thread has 255 registers: the tiles of 32 rows, and those of several
//    queries with up to 8 rows, need up to 88 bytes more, which spill.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "dependent_launch.cuh"
#include "internal.h"
#include "sm103_ptx.cuh"

namespace splash {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kMaxWarps = 1216;  // of the grid; the workspace holds two parts for each

// A running maximum is only moved when a score passes it by more than this
// (in powers of two): until then exp2(s - m) stays below 2^8, which neither
// the sums (fp32) nor P's 16-bit types mind, and no shuffles or rescaling of
// the output are needed (4 tokens of 8 requests 32.6 us, against 33.4 without).
constexpr float kSlack = 8.f;

// For an e4m3 cache the reference is this much below the maximum, so that
// probabilities use fp16 from the top: 2^7 for the largest key, below 2^15 with
// the slack (fp16 ends at 65504).  At the bottom fp16 steps by 2^-24, which is
// 2^-31 of the largest key: what is dropped below half of that stays under the
// output's own rounding (2^-8) up to 2^23 keys in one warp, where a reference
// at the maximum itself stopped at 2^16.  bf16 has fp32's range.
constexpr float kBelowTop = 7.f;

struct Params {
  const char *q;
  int64_t q_b, q_h, q_l;  // byte strides
  const char *k, *v;
  int64_t k_page, k_head, k_token, v_page, v_head, v_token;  // byte strides
  const float *k_scale, *v_scale;
  const int32_t *block_table;
  int64_t block_table_stride;
  const int32_t *seq_lens;
  __nv_bfloat16 *out;
  float *lse;
  float *part_o, *part_ml;  // [2 * warps][part_rows][DV], [2 * warps][part_rows][2] (maximum, sum)
  int32_t *before;          // [B + 1] list entries (of one head and row group) before each sequence
  int64_t num_pages;
  int32_t B, Hkv, Lq, G, nrows, row_groups, part_rows;  // nrows = G * Lq rows per KV head
  int32_t max_pages, page_shift, window;         // window < 0: none
  float scale, cap;                              // cap <= 0: none
  uint32_t *err;
};

// Keys of a step, from the bytes of a key and its value: 8 KB or so per step.
constexpr int keys_per_step(int bytes) { return bytes >= 512 ? 16 : 32; }

// ROWS: query rows of a tile, 8, 16 or 32.  Eight rows (up to 8 query heads per
// KV head, one new token) leave half of each 16-row product free: it takes what
// rounding P to 16 bits loses.  With more rows that has a product of its own for a
// bf16 cache (REST), see below.
template <int DQK_, int DV_, bool E4M3_, int ROWS_, bool MULTI_>
struct Config {
  static constexpr int DQK = DQK_, DV = DV_, ROWS = ROWS_;
  static constexpr bool MULTI = MULTI_;          // more than one query per sequence and head
  static constexpr int MT = ROWS <= 16 ? 1 : 2;  // products of 16 rows
  static constexpr int E = ROWS == 8 ? 1 : 2;    // halves of them that hold rows
  static constexpr bool E4M3 = E4M3_;
  static constexpr bool REST = !E4M3 && E == 2;  // what rounding P loses has a product of its own
  static constexpr int RK = DQK * (E4M3 ? 1 : 2), RV = DV * (E4M3 ? 1 : 2);  // bytes of a row
  static constexpr int KW = keys_per_step(RK + RV), NB = KW / 16;            // keys and 16-key blocks of a step
  static constexpr int STAGE = KW * (RK + RV);
  static constexpr int QBYTES = MT == 1 ? 0 : ROWS * DQK * 2;  // queries of 16 rows stay in registers
  // two CTAs per SM, if at least two stages fit
  static constexpr int STAGES = std::max(2, (108 * 1024 / kWarps - QBYTES) / STAGE);
  static constexpr int WARP_BYTES = STAGES * STAGE + QBYTES;
  static constexpr int SMEM = kWarps * WARP_BYTES;
  static constexpr int CTAS = SMEM <= 110 * 1024 ? 2 : 1;  // per SM
  static constexpr int ODIM = DV + 4;                      // floats of a row in a CTA's join
  static_assert(WARP_BYTES >= ROWS * ODIM * 4, "the join of a CTA's warps uses their stages");
};

// The keys of sequence b that its queries see, in steps of KW.
struct Span {
  int32_t n, lo;       // keys [lo, n) are visible to some query
  int32_t step0, nst;  // steps step0 .. step0 + nst - 1; at least one, so that empty rows are written too
};

__device__ __forceinline__ void check_length(const Params &p, int b) {
  const int32_t n = p.seq_lens[b];
  if (n < 0 || n > (int64_t)p.max_pages << p.page_shift) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
}

template <int KW>
__device__ __forceinline__ Span span_of(const Params &p, int b) {
  Span s;
  const int64_t most = (int64_t)p.max_pages << p.page_shift;
  const int32_t n = p.seq_lens[b];
  s.n = n < 0 ? 0 : n > most ? (int32_t)most : n;
  s.lo = p.window < 0 ? 0 : max(0, s.n - p.Lq - p.window);
  s.step0 = s.lo / KW;
  s.nst = max(1, (s.n + KW - 1) / KW - s.step0);
  return s;
}

// Equal contiguous parts of T entries: warp w takes [begin(w), begin(w + 1)).
// (The host keeps T below 2^31: with 64-bit divisions the start of a call took
// 0.65 us longer.)
struct Parts {
  int32_t each, more;  // the first `more` warps take one entry more
  __device__ __forceinline__ Parts(int32_t T, int32_t warps)
      : each((uint32_t)T / (uint32_t)warps), more(T - each * warps) {}
  __device__ __forceinline__ int32_t begin(int32_t w) const { return each * w + min(w, more); }
  __device__ __forceinline__ int32_t owner(int32_t u) const {
    const int32_t cut = (each + 1) * more;
    return u < cut ? (uint32_t)u / (uint32_t)(each + 1) : more + (uint32_t)(u - cut) / (uint32_t)each;
  }
};

// A warp's place in its part of the list.
template <int KW>
struct Cursor {
  int32_t u;  // list entry of the current step
  int32_t b, seg, step;  // segment seg (head, row group) of sequence b, its step
  Span s;
  // returns true when the segment changed; s is that of b as long as u < end
  __device__ __forceinline__ bool advance(const Params &p, int per_seq, int32_t end) {
    ++u;
    if (++step < s.nst) return false;
    step = 0;
    if (++seg == per_seq) {
      seg = 0;
      ++b;
      if (u < end) s = span_of<KW>(p, b);
    }
    return true;
  }
};

// 16-byte chunk c of row r in a tile of rows of ROWB bytes: permuted so that
// the 8 rows of an ldmatrix fall on different banks.
template <int ROWB>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return r * ROWB + ((c ^ (ROWB % 128 == 0 ? (r & 7) : ((r >> 1) & 3))) << 4);
}

__device__ __forceinline__ void copy16(uint32_t dst, const char *src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const char *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// d += a (16 x 16) b (16 x 8); fp16 operands for an e4m3 cache (every e4m3
// value is an fp16 value), bf16 otherwise.
template <bool HALF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (HALF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four e4m3 values to two pairs of fp16 (exact).
__device__ __forceinline__ void widen(uint32_t x, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

template <bool HALF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (!HALF) return pack_bf16x2(lo, hi);
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two positive numbers cut off to bf16, and what that leaves of them.
__device__ __forceinline__ uint32_t cut_bf16x2(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
__device__ __forceinline__ float rest_of(float x) {
  return fmaxf(x - __uint_as_float(__float_as_uint(x) & 0xffff0000u), __uint_as_float(0x00800000u));
}
__device__ __forceinline__ uint32_t rest_bf16x2(float lo, float hi) { return pack_bf16x2(rest_of(lo), rest_of(hi)); }

// The larger exponent field of a word's two bf16 values, and the word as fp16
// values over 2^(top - 127).
__device__ __forceinline__ uint32_t exponent(uint32_t x) { return max((x >> 7) & 255u, (x >> 23) & 255u); }
__device__ __forceinline__ uint32_t to_half(uint32_t x, uint32_t top) {
  const float down = __uint_as_float((254u - top) << 23);
  return pack2<true>(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xffff0000u) * down);
}

// tanh for the soft cap.  Up to 0.25 the forward's polynomial (attention_fwd.cu):
// t (1 + u (c1 + c2 u)), u = t^2, a minimax fit of tanh(t)/t with a relative error
// of 4.8e-7, so that cap * tanh(s / cap) keeps the score's low bits however large
// the cap; above it tanh|x| = (1 - e) / (1 + e), e = exp(-2|x|), whose error is
// absolute.
constexpr float kTanhC1 = -0.33324610f, kTanhC2 = 0.12877172f, kTanhSeriesLimit = 0.25f;

__device__ __forceinline__ float tanh_series(float x) {
  const float u = x * x;
  return fmaf(x * u, fmaf(u, kTanhC2, kTanhC1), x);
}
__device__ __forceinline__ float tanh_of(float x) {
  const float e = ex2_approx(-2.f * kLog2e * fabsf(x));
  return fabsf(x) <= kTanhSeriesLimit ? tanh_series(x) : copysignf(__fdividef(1.f - e, 1.f + e), x);
}

// A warp's copies: the steps of its part of the list, in order.
template <class C>
struct Loader {
  const Params &p;
  const int lane, per_seq;
  const int32_t end;
  Cursor<C::KW> at;
  const char *k, *v;  // the head's rows of page 0
  const int32_t *pages;
  int32_t entry[C::NB];  // the step's page entries, read one step ahead

  __device__ __forceinline__ void enter() {
    const int head = at.seg / p.row_groups;
    k = p.k + head * p.k_head;
    v = p.v + head * p.v_head;
    pages = p.block_table + at.b * p.block_table_stride;
  }

  __device__ __forceinline__ void look() {
#pragma unroll
    for (int i = 0; i < C::NB; ++i) {
      const int32_t key = (at.s.step0 + at.step) * C::KW + 16 * i;
      entry[i] = key < at.s.n && key + 16 > at.s.lo ? pages[key >> p.page_shift] : 0;
    }
  }

  template <int ROWB>
  __device__ __forceinline__ void block(uint32_t dst, const char *base, int64_t token, int32_t key, bool ok, bool whole) const {
    constexpr int SEG = ROWB % 128 == 0 ? 128 : 64;  // a row's contiguous bytes per instruction
    constexpr int LPS = SEG / 16, RPI = 32 / LPS;
    const int r0 = lane / LPS, c0 = lane % LPS;
    const char *src = base + r0 * token + c0 * 16;
    if (whole) {
#pragma unroll
      for (int rg = 0; rg < 16 / RPI; ++rg)
#pragma unroll
        for (int part = 0; part < ROWB / SEG; ++part)
          copy16(dst + chunk_at<ROWB>(rg * RPI + r0, part * LPS + c0), src + rg * RPI * token + part * SEG);
    } else {
#pragma unroll 1
      for (int rg = 0; rg < 16 / RPI; ++rg) {
        const int r = rg * RPI + r0;
        const bool read = ok && key + r >= at.s.lo && key + r < at.s.n;
#pragma unroll
        for (int part = 0; part < ROWB / SEG; ++part)
          copy16(dst + chunk_at<ROWB>(r, part * LPS + c0), read ? src + rg * RPI * token + part * SEG : base, read);
      }
    }
  }

  // the current step into a stage (nothing once the part is done), as one
  // group of copies; then on to the next
  __device__ __forceinline__ void step(uint32_t stage) {
    if (at.u < end) {
#pragma unroll
      for (int i = 0; i < C::NB; ++i) {
        const int32_t key = (at.s.step0 + at.step) * C::KW + 16 * i, page = entry[i];
        const bool ok = page >= 0 && page < p.num_pages;
        if (!ok && lane == 0) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
        const int32_t slot = key & ((1 << p.page_shift) - 1);
        const int64_t pg = ok ? page : 0;
        const bool whole = ok && key >= at.s.lo && key + 16 <= at.s.n;
        block<C::RK>(stage + i * 16 * C::RK, k + pg * p.k_page + slot * p.k_token, p.k_token, key, ok, whole);
        block<C::RV>(stage + C::KW * C::RK + i * 16 * C::RV, v + pg * p.v_page + slot * p.v_token, p.v_token, key, ok, whole);
      }
      if (at.advance(p, per_seq, end) && at.u < end) enter();
      if (at.u < end) look();
    }
    copy_commit();
  }
};

// A thread's columns of a row of the accumulators (e: the lower or upper 8 rows).
template <class C>
__device__ __forceinline__ void store_row(float *dst, const float (&o)[C::DV / 8][4], int e, int tq) {
  if (C::E4M3) {
#pragma unroll
    for (int j = 0; j < C::DV / 16; ++j)
      *reinterpret_cast<float4 *>(dst + 16 * j + 4 * tq) =
          make_float4(o[2 * j][2 * e], o[2 * j + 1][2 * e], o[2 * j][2 * e + 1], o[2 * j + 1][2 * e + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < C::DV / 8; ++j)
      *reinterpret_cast<float2 *>(dst + 8 * j + 2 * tq) = make_float2(o[j][2 * e], o[j][2 * e + 1]);
  }
}

// acc and sum += a part (maximum, sum, x), both taken relative to `high`.
__device__ __forceinline__ void add_part(float4 &acc, float &sum, float high, float2 ml, float4 x) {
  const float f = ex2_approx(ml.x - (high == -INFINITY ? 0.f : high));
  sum += f * ml.y;
  acc.x += f * x.x;
  acc.y += f * x.y;
  acc.z += f * x.z;
  acc.w += f * x.w;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
// Every thread of every CTA of the cluster arrives and waits.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// The same shared memory address in another CTA of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 load_cluster4(uint32_t addr) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(addr)
               : "memory");
  return x;
}
__device__ __forceinline__ float2 load_cluster2(uint32_t addr) {
  float2 x;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(addr) : "memory");
  return x;
}

// The pairs of keys of a step that a query sees (2 tq, 2 tq + 1 and the same + 8
// of each 16), as masks of the value's pairs, and which of a thread's rows are
// that query's.
template <class C>
struct Seen {
  uint32_t keys[C::NB][2];
  bool row[C::MT][C::E];
};

// P in 16 bits as the product takes it, with its rest where that has a product
// of its own.
template <class C>
struct Weights {
  uint32_t p[C::MT][C::NB][4], rest[C::REST ? C::MT : 1][C::REST ? C::NB : 1][4];
};

template <class C, bool MASKED>
__device__ __forceinline__ void add_product(float (&o)[4], const Weights<C> &w, int mt, int nb, uint32_t b0, uint32_t b1,
                                            const bool (&row)[C::E]) {
  if constexpr (!MASKED) {
    mma<C::E4M3>(o, w.p[mt][nb], b0, b1);
  } else {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    mma<C::E4M3>(x, w.p[mt][nb], b0, b1);
    if constexpr (C::REST) mma<C::E4M3>(x, w.rest[mt][nb], b0, b1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row[C::E == 1 ? 0 : i >> 1]) o[i] += x[i];
  }
}

// O += P V for the step whose values are at vs; with MASKED only the rows and
// keys of `seen`.
template <class C, bool MASKED>
__device__ __forceinline__ void add_values(float (&o)[C::MT][C::DV / 8][4], const Weights<C> &w, uint32_t vs, int lane,
                                           const Seen<C> &seen) {
  const int v_row = (lane & 7) + ((lane >> 3) & 1) * 8, v_chunk = lane >> 4;
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb) {
    const uint32_t m0 = MASKED ? seen.keys[nb][0] : ~0u, m1 = MASKED ? seen.keys[nb][1] : ~0u;
#pragma unroll
    for (int j = 0; j < C::DV / 16; j += C::E4M3 ? 2 : 1) {
      uint32_t vb[4];
      ldsm4_trans(vb, vs + nb * 16 * C::RV + chunk_at<C::RV>(v_row, (C::E4M3 ? j : 2 * j) + v_chunk));
      if (C::E4M3) {
        // Each word holds two neighbouring columns of two keys: the even
        // columns of 16 go to one product, the odd ones to the next.
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t b0, b1, c0, c1;
          widen(__byte_perm(vb[2 * x], 0, 0x3120), b0, c0);
          widen(__byte_perm(vb[2 * x + 1], 0, 0x3120), b1, c1);
#pragma unroll
          for (int mt = 0; mt < C::MT; ++mt) {
            add_product<C, MASKED>(o[mt][2 * (j + (C::E4M3 ? x : 0))], w, mt, nb, b0 & m0, b1 & m1, seen.row[mt]);
            add_product<C, MASKED>(o[mt][2 * (j + (C::E4M3 ? x : 0)) + 1], w, mt, nb, c0 & m0, c1 & m1, seen.row[mt]);
          }
        }
      } else {
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
          add_product<C, MASKED>(o[mt][2 * j], w, mt, nb, vb[0] & m0, vb[1] & m1, seen.row[mt]);
          add_product<C, MASKED>(o[mt][2 * j + 1], w, mt, nb, vb[2] & m0, vb[3] & m1, seen.row[mt]);
        }
        if constexpr (C::REST && !MASKED) {  // (after the tiles' other products, which it would wait for)
#pragma unroll
          for (int mt = 0; mt < C::MT; ++mt) {
            mma<false>(o[mt][2 * j], w.rest[mt][nb], vb[0], vb[1]);
            mma<false>(o[mt][2 * j + 1], w.rest[mt][nb], vb[2], vb[3]);
          }
        }
      }
    }
  }
}

// TOGETHER: a cluster of CTAs per segment; otherwise equal parts of the list per warp.
template <class C, bool TOGETHER>
__global__ void __launch_bounds__(kThreads, 2) paged_decode_kernel(const Params p) {
  constexpr int DQK = C::DQK, DV = C::DV, MT = C::MT, NB = C::NB, E = C::E;
  constexpr bool E4M3 = C::E4M3;
  const int Lq = C::MULTI ? p.Lq : 1;
  extern __shared__ __align__(1024) char smem[];
  __shared__ int32_t s_scan[kWarps], s_before[kWarps], s_seq[kWarps];
  __shared__ float2 s_ml[kWarps][C::ROWS], s_cta[C::ROWS];  // (maximum, sum) of the rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quad = lane >> 2, tq = lane & 3;
  const uint32_t ring = smem_u32(smem + warp * C::WARP_BYTES);
  const uint32_t q_u = ring + C::STAGES * C::STAGE;
  char *q_smem = smem + warp * C::WARP_BYTES + C::STAGES * C::STAGE;

  grid_dependency();

  const int per_seq = p.Hkv * p.row_groups;
  const int wid = kWarps * blockIdx.x + warp;
  Cursor<C::KW> at;
  int32_t end;
  if constexpr (TOGETHER) {
    const uint32_t ctas = cluster_size(), rank = cluster_rank(), segment = blockIdx.x / ctas;
    at.b = segment / per_seq;
    at.seg = segment % per_seq;
    at.s = span_of<C::KW>(p, at.b);
    const Parts parts(at.s.nst, kWarps * ctas);
    at.u = at.step = parts.begin(rank * kWarps + warp);
    end = parts.begin(rank * kWarps + warp + 1);
    if (at.seg == 0 && rank == 0 && threadIdx.x == 0) check_length(p, at.b);
  } else {
    // the warps' parts of the list: a scan over the sequences
    int32_t T;
    {
      const int per = (p.B + kThreads - 1) / kThreads;
      const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
      int32_t own = 0;
      for (int b = b0; b < b1; ++b) own += span_of<C::KW>(p, b).nst;
      int32_t before = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(~0u, before, o);
        if (lane >= o) before += y;
      }
      if (lane == 31) s_scan[warp] = before;
      before -= own;
      __syncthreads();
      int32_t total = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
      }
      T = total * per_seq;
      const Parts parts(T, kWarps * gridDim.x);
      int32_t first[kWarps];
      bool mine = blockIdx.x == 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        first[w] = parts.begin(kWarps * blockIdx.x + w);
        mine |= first[w] >= before * per_seq && first[w] < (before + own) * per_seq;
      }
      if (mine) {
        int32_t at = before;
        for (int b = b0; b < b1; ++b) {
          const int32_t next = at + span_of<C::KW>(p, b).nst;
#pragma unroll
          for (int w = 0; w < kWarps; ++w)
            if (first[w] >= at * per_seq && first[w] < next * per_seq) s_seq[w] = b, s_before[w] = at;
          if (blockIdx.x == 0) {
            p.before[b] = at;
            if (b == p.B - 1) p.before[p.B] = next;
            check_length(p, b);
          }
          at = next;
        }
      }
      __syncthreads();
    }
    const Parts parts(T, kWarps * gridDim.x);
    at.u = parts.begin(wid);
    end = parts.begin(wid + 1);
    if (at.u >= end) return;
    at.b = s_seq[warp];
    at.s = span_of<C::KW>(p, at.b);
    const int32_t in_seq = at.u - s_before[warp] * per_seq;
    at.seg = (uint32_t)in_seq / (uint32_t)at.s.nst;
    at.step = in_seq - at.seg * at.s.nst;
  }
  Loader<C> load{p, lane, per_seq, end, at, nullptr, nullptr, nullptr, {}};
  if (at.u < end) {
    load.enter();
    load.look();
  }
#pragma unroll 1  // (one copy of the code: its first fetch is part of a short call's time)
  for (int s = 0; s < C::STAGES - 1; ++s) load.step(ring + s * C::STAGE);

  int slot = 0, part = 2 * wid;
  do {
    // ---- a segment: the rows' queries, 16 bits each.  For e4m3 they become
    // fp16, scaled by the power of two that brings the row's largest element
    // into [1, 2).  That is exact except for elements 2^14 times smaller (their
    // error, 2^-25 of the largest, is below that of an fp32 sum); the factor
    // goes to the row's scale.
    const int head = at.seg / p.row_groups, row0 = (at.seg % p.row_groups) * C::ROWS;
    const int rows = min(C::ROWS, p.nrows - row0);
    const bool from_start = at.step == 0;
    const Span sp = at.s;
    const int b = at.b;
    const char *q_head = p.q + b * p.q_b + (int64_t)head * p.G * p.q_h;
    const float base_factor = (p.cap > 0.f ? p.scale / p.cap : p.scale * kLog2e) * (E4M3 ? p.k_scale[head] : 1.f);
    uint32_t qa[MT == 1 ? DQK / 16 : 1][4];
    float factor[MT][E], m[MT][E], l[MT][E], o[MT][DV / 8][4];
    int32_t pos[MT][E];  // the row's position (rows past the last one see what the last query sees)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int r = mt * 16 + quad + 8 * e;
        const int g = (row0 + r) / Lq, lq = (row0 + r) - g * Lq;
        factor[mt][e] = base_factor;
        pos[mt][e] = sp.n - Lq + (r < rows ? lq : Lq - 1);
        m[mt][e] = -INFINITY;
        l[mt][e] = 0.f;
        if (MT == 1) {
          // An ldmatrix of e4m3 keys leaves elements 4t .. 4t+3 in the thread
          // that the product expects to hold 2t, 2t+1, 2t+8, 2t+9 of each 16:
          // the queries are taken in that order too.
          const char *src = q_head + (int64_t)g * p.q_h + lq * p.q_l;
#pragma unroll
          for (int kk = 0; kk < DQK / 16; ++kk) {
            uint2 x = make_uint2(0, 0);
            if (r < rows) {
              if (E4M3) {
                x = reinterpret_cast<const uint2 *>(src)[4 * kk + tq];
              } else {
                x.x = reinterpret_cast<const uint32_t *>(src)[8 * kk + tq];
                x.y = reinterpret_cast<const uint32_t *>(src)[8 * kk + tq + 4];
              }
            }
            qa[kk][e] = x.x;
            qa[kk][2 + e] = x.y;
            if (E == 1) qa[kk][1] = qa[kk][3] = 0;
          }
          if (E4M3) {
            uint32_t top = 0;  // exponent field of the largest element
#pragma unroll
            for (int kk = 0; kk < DQK / 16; ++kk) top = max(top, max(exponent(qa[kk][e]), exponent(qa[kk][2 + e])));
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            top = min(max(top, 1u), 253u);
#pragma unroll
            for (int kk = 0; kk < DQK / 16; ++kk) {
              qa[kk][e] = to_half(qa[kk][e], top);
              qa[kk][2 + e] = to_half(qa[kk][2 + e], top);
            }
            factor[mt][e] *= __uint_as_float(top << 23);
          }
        }
      }
    if (MT > 1) {  // more rows than the registers hold: in shared memory
      __syncwarp();
#pragma unroll 4
      for (int r = 0; r < C::ROWS; ++r) {
        constexpr int W = DQK / 64;  // words (two elements) per lane
        const int g = (row0 + r) / Lq, lq = (row0 + r) - g * Lq;
        uint32_t x[W];
#pragma unroll
        for (int i = 0; i < W; ++i)
          x[i] = r < rows ? reinterpret_cast<const uint32_t *>(q_head + (int64_t)g * p.q_h + lq * p.q_l)[i * 32 + lane] : 0;
        if (E4M3) {
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < W; ++i) top = max(top, exponent(x[i]));
          top = min(max(__reduce_max_sync(~0u, top), 1u), 253u);
#pragma unroll
          for (int i = 0; i < W; ++i) x[i] = to_half(x[i], top);
          if (quad == (r & 7)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < E; ++e)
                if (r >> 3 == 2 * mt + e) factor[mt][e] *= __uint_as_float(top << 23);
          }
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const int d = 2 * (i * 32 + lane);
          const int to = E4M3 ? (d & ~15) + 2 * ((d & 15) >> 2) + ((d & 2) ? 8 : 0) : d;  // (the order above)
          *reinterpret_cast<uint32_t *>(q_smem + chunk_at<DQK * 2>(r, to >> 3) + (to & 7) * 2) = x[i];
        }
      }
      __syncwarp();
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < DV / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][j][i] = 0.f;
    const uint32_t q_row = (lane & 7) + ((lane >> 3) & 1) * 8;

    // ---- its steps
    bool change = false;
    while (!change && at.u < end) {
      copy_wait<C::STAGES - 2>();
      __syncwarp();
      const int32_t key0 = (sp.step0 + at.step) * C::KW;
      const uint32_t ks = ring + slot * C::STAGE, vs = ks + C::KW * C::RK;
      load.step(ring + (slot == 0 ? C::STAGES - 1 : slot - 1) * C::STAGE);
      slot = slot == C::STAGES - 1 ? 0 : slot + 1;
      change = at.advance(p, per_seq, end);
      if (key0 >= sp.n) continue;  // no keys at all

      // S = Q K^T
      float s[MT][2 * NB][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[mt][j][i] = 0.f;
      const int k_row = (lane & 7) + (lane >> 4) * 8, k_chunk = (lane >> 3) & 1;
#pragma unroll
      for (int kk = 0; kk < DQK / 16; kk += E4M3 ? 2 : 1) {
        uint32_t a[E4M3 ? 2 : 1][MT][4];
#pragma unroll
        for (int x = 0; x < (E4M3 ? 2 : 1); ++x)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if (MT == 1) {
#pragma unroll
              for (int i = 0; i < 4; ++i) a[x][mt][i] = qa[kk + x][i];
            } else {
              ldsm4(a[x][mt], q_u + chunk_at<DQK * 2>(mt * 16 + q_row, 2 * (kk + x) + (lane >> 4)));
            }
          }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          uint32_t kb[4];
          ldsm4(kb, ks + nb * 16 * C::RK + chunk_at<C::RK>(k_row, (E4M3 ? kk : 2 * kk) + k_chunk));
          if (E4M3) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t b0, b1, c0, c1;
              widen(kb[x], b0, b1);
              widen(kb[2 + x], c0, c1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma<true>(s[mt][2 * nb], a[E4M3 ? x : 0][mt], b0, b1);
                mma<true>(s[mt][2 * nb + 1], a[E4M3 ? x : 0][mt], c0, c1);
              }
            }
          } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma<false>(s[mt][2 * nb], a[0][mt], kb[0], kb[1]);
              mma<false>(s[mt][2 * nb + 1], a[0][mt], kb[2], kb[3]);
            }
          }
        }
      }

      // scores in powers of two; masked where some row does not see some key
      const bool whole = key0 + C::KW <= sp.n - Lq + 1 && (p.window < 0 || key0 >= sp.n - 1 - p.window);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
          for (int i = 0; i < 2 * E; ++i) s[mt][j][i] *= factor[mt][i >> 1];
      if (p.cap > 0.f) {
        // tanh by the series alone where it holds for the whole step: 8
        // requests x 4 tokens with a cap of 30 take 35.2 us, against 36.0 with a
        // choice per score.
        const float cap = p.cap * kLog2e;
        float most = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
            for (int i = 0; i < 2 * E; ++i) most = fmaxf(most, fabsf(s[mt][j][i]));
        if (__any_sync(~0u, most > kTanhSeriesLimit)) {  // (NaN stays NaN either way)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
              for (int i = 0; i < 2 * E; ++i) s[mt][j][i] = cap * tanh_of(s[mt][j][i]);
        } else {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
              for (int i = 0; i < 2 * E; ++i) s[mt][j][i] = cap * tanh_series(s[mt][j][i]);
        }
      }
      if (!whole) {
        const uint32_t reach = p.window < 0 ? 0x7fffffffu : (uint32_t)p.window;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
            for (int i = 0; i < 2 * E; ++i) {
              // (as unsigned, a key ahead of the query is out of reach too)
              const uint32_t behind = (uint32_t)(pos[mt][i >> 1] - (key0 + 8 * j + 2 * tq + (i & 1)));
              if (behind > reach) s[mt][j][i] = -INFINITY;
            }
      }
      float top[MT][E];
      bool move = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          top[mt][e] = fmaxf(s[mt][0][2 * e], s[mt][0][2 * e + 1]);
#pragma unroll
          for (int j = 1; j < 2 * NB; ++j) top[mt][e] = fmax3(top[mt][e], s[mt][j][2 * e], s[mt][j][2 * e + 1]);
          if (E4M3) top[mt][e] -= kBelowTop;
          move |= top[mt][e] > m[mt][e] + kSlack;
        }
      if (__any_sync(~0u, move)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            float high = fmaxf(top[mt][e], m[mt][e]);
            high = fmaxf(high, __shfl_xor_sync(~0u, high, 1));
            high = fmaxf(high, __shfl_xor_sync(~0u, high, 2));
            const float alpha = high == -INFINITY ? 1.f : ex2_approx(m[mt][e] - high);
            m[mt][e] = high;
            l[mt][e] *= alpha;
#pragma unroll
            for (int j = 0; j < DV / 8; ++j) {
              o[mt][j][2 * e] *= alpha;
              o[mt][j][2 * e + 1] *= alpha;
              if (E == 1) o[mt][j][2] *= alpha, o[mt][j][3] *= alpha;
            }
          }
      }

      // P, O += P V.  The product takes P in 16 bits (its sum is taken before):
      // fp16 for an e4m3 cache, 2^-11 of each p, or bf16, 2^-8, which is as much as
      // the rounding of the result.
      //  * Eight rows: the free half of the product takes the rest, P - bf16(P) or
      //    P - fp16(P); the halves are added at the end, and the result carries
      //    one bf16 rounding, its own.  (e4m3: 8 requests of 1023 .. 8191 tokens
      //    27.0 us, 26.5 without, longer ones as before; bf16: no difference.)
      //  * More: bf16's rest has a product of its own into the same sums (4 tokens of
      //    64 requests take 107.1 us, 104.3 without, of 8 requests 36.1 and 33.8, 32
      //    rows of 192-wide heads 79.2 and 71.8; errors 1.7e-3 and 2.3e-3).  There P
      //    is cut off to bf16 and the rest kept above 0: an infinite value times
      //    either has its sign, and the sum is that infinity (0 x infinity and
      //    infinity - infinity are NaN).  The rest's floor, the smallest normal
      //    number, adds 2^-126 of a value.
      Weights<C> w;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float ref = m[mt][e] == -INFINITY ? 0.f : m[mt][e];
#pragma unroll
          for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float x = ex2_approx(s[mt][j][2 * e + i] - ref);
              s[mt][j][2 * e + i] = x;
              l[mt][e] += x;
            }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float *y = &s[mt][2 * nb + (i >> 1)][E == 1 ? 0 : 2 * (i & 1)];
            if constexpr (C::REST) {
              w.p[mt][nb][i] = cut_bf16x2(y[0], y[1]);
              w.rest[mt][nb][i] = rest_bf16x2(y[0], y[1]);
            } else if (E == 2 || (i & 1) == 0) {
              w.p[mt][nb][i] = pack2<E4M3>(y[0], y[1]);
            } else if (E4M3) {
              const uint32_t h = w.p[mt][nb][i - 1];
              const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
              w.p[mt][nb][i] = pack2<true>(y[0] - f.x, y[1] - f.y);
            } else {
              w.p[mt][nb][i] = pack_bf16x2(y[0] - __uint_as_float(w.p[mt][nb][i - 1] << 16),
                                           y[1] - __uint_as_float(w.p[mt][nb][i - 1] & 0xffff0000u));
            }
          }
      }
      if (!C::MULTI || whole) {
        add_values<C, false>(o, w, vs, lane, Seen<C>());
      } else if constexpr (C::MULTI) {
        // Some of the step's values are one query's and not another's: a
        // product for each query, with zeros in the place of the values that
        // it does not see, whatever they are (0 x infinity is not 0).
#pragma unroll 1
        for (int lq = 0; lq < Lq; ++lq) {
          const int32_t last = sp.n - Lq + lq;
          const uint32_t reach = p.window < 0 ? 0x7fffffffu : (uint32_t)p.window;
          Seen<C> seen;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t behind = (uint32_t)(last - (key0 + 16 * nb + 8 * i + 2 * tq));
              seen.keys[nb][i] = (behind <= reach ? 0xffffu : 0u) | (behind - 1u <= reach ? 0xffff0000u : 0u);
            }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < E; ++e) seen.row[mt][e] = pos[mt][e] == last;
          add_values<C, true>(o, w, vs, lane, seen);
        }
      }
    }

    if (E == 1) {
      // The halves' sum.  The rest of a P is 0 or negative too: an infinite value
      // times it is NaN or the other infinity, so that a sum which is not finite
      // stays as bf16(P) made it.
#pragma unroll
      for (int j = 0; j < DV / 8; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (fabsf(o[0][j][i]) < INFINITY) o[0][j][i] += o[0][j][i + 2];
    }
    if constexpr (TOGETHER) {
      copy_wait<0>();
      __syncwarp();
      float *own = reinterpret_cast<float *>(smem + warp * C::WARP_BYTES);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int r = mt * 16 + quad + 8 * e;
          float sum = l[mt][e];
          sum += __shfl_xor_sync(~0u, sum, 1);
          sum += __shfl_xor_sync(~0u, sum, 2);
          if (r >= rows) continue;
          if (tq == 0) s_ml[warp][r] = make_float2(m[mt][e], sum);
          store_row<C>(own + r * C::ODIM, o[mt], e, tq);
        }
      __syncthreads();
      // the CTA's rows, where the first warp's were
      constexpr int LANES = DV / 4;
      const int col = 4 * (threadIdx.x % LANES);
      for (int r = threadIdx.x / LANES; r < rows; r += kThreads / LANES) {
        float high = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) high = fmaxf(high, s_ml[w][r].x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          add_part(acc, sum, high, s_ml[w][r], *reinterpret_cast<const float4 *>(smem + w * C::WARP_BYTES + 4 * (r * C::ODIM + col)));
        *reinterpret_cast<float4 *>(smem + 4 * (r * C::ODIM + col)) = acc;
        if (col == 0) s_cta[r] = make_float2(high, sum);
      }
      // the cluster's: every CTA finishes some of the segment's columns
      const uint32_t ctas = cluster_size();
      if (ctas > 1)
        cluster_sync();
      else
        __syncthreads();
      const float v_scale = E4M3 ? p.v_scale[head] : 1.f;
      for (int i = cluster_rank() * kThreads + threadIdx.x; i < rows * LANES; i += ctas * kThreads) {
        const int r = i / LANES, c = 4 * (i % LANES);
        const uint32_t ml = smem_u32(&s_cta[r]), from = smem_u32(smem) + 4 * (r * C::ODIM + c);
        float high = -INFINITY, sum = 0.f;
        for (uint32_t k = 0; k < ctas; ++k) high = fmaxf(high, load_cluster2(in_cta(ml, k)).x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (uint32_t k = 0; k < ctas; ++k)
          add_part(acc, sum, high, load_cluster2(in_cta(ml, k)), load_cluster4(in_cta(from, k)));
        const float inv = sum == 0.f ? 0.f : v_scale / sum;
        const int64_t row = ((int64_t)b * p.Hkv + head) * p.nrows + row0 + r;
        *reinterpret_cast<uint2 *>(p.out + row * DV + c) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (c == 0) p.lse[row] = sum == 0.f ? -INFINITY : (high + log2f(sum)) * kLn2;
      }
      if (ctas > 1) cluster_sync();  // (no CTA ends while another reads its shared memory)
      return;
    }

    // ---- finished rows, or this warp's part of them
    const bool complete = from_start && change;
    const float v_scale = E4M3 ? p.v_scale[head] : 1.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int r = mt * 16 + quad + 8 * e;
        float sum = l[mt][e];
        sum += __shfl_xor_sync(~0u, sum, 1);
        sum += __shfl_xor_sync(~0u, sum, 2);
        if (r >= rows) continue;
        if (complete) {
          const float inv = sum == 0.f ? 0.f : v_scale / sum;
          const int64_t row = ((int64_t)b * p.Hkv + head) * p.nrows + row0 + r;
          if (tq == 0) p.lse[row] = sum == 0.f ? -INFINITY : (m[mt][e] + log2f(sum)) * kLn2;
          char *dst = reinterpret_cast<char *>(p.out + row * DV);
          if (E4M3) {
#pragma unroll
            for (int j = 0; j < DV / 16; ++j)
              *reinterpret_cast<uint2 *>(dst + 32 * j + 8 * tq) =
                  make_uint2(pack_bf16x2(o[mt][2 * j][2 * e] * inv, o[mt][2 * j + 1][2 * e] * inv),
                             pack_bf16x2(o[mt][2 * j][2 * e + 1] * inv, o[mt][2 * j + 1][2 * e + 1] * inv));
          } else {
#pragma unroll
            for (int j = 0; j < DV / 8; ++j)
              *reinterpret_cast<uint32_t *>(dst + 16 * j + 4 * tq) =
                  pack_bf16x2(o[mt][j][2 * e] * inv, o[mt][j][2 * e + 1] * inv);
          }
        } else {
          const int64_t row = (int64_t)part * p.part_rows + r;
          if (tq == 0) *reinterpret_cast<float2 *>(p.part_ml + 2 * row) = make_float2(m[mt][e], sum);
          store_row<C>(p.part_o + row * DV, o[mt], e, tq);
        }
      }
    part = 2 * wid + 1;  // what follows the first segment and is not complete is the last one
  } while (at.u < end);
  copy_wait<0>();
}

// Joins the parts of a row that several warps computed: with (m_c, l_c, o_c) of
// part c and m = max m_c: out = sum exp(m_c - m) o_c / sum exp(m_c - m) l_c.
// One CTA per row, its warps taking every fourth part.
template <int DV, int ROWS>
__global__ void __launch_bounds__(kThreads) paged_decode_join_kernel(const Params p, int warps) {
  __shared__ float s_o[kWarps][DV], s_sum[kWarps], s_top[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int PER = DV / 32;
  const int64_t row = blockIdx.x;  // (b, KV head, row)
  const int head_row = (int)(row % p.nrows), head = (int)(row / p.nrows % p.Hkv), b = (int)(row / p.nrows / p.Hkv);
  const int per_seq = p.Hkv * p.row_groups;
  grid_dependency();
  const Parts parts(p.before[p.B] * per_seq, warps);
  const int32_t entries = p.before[b + 1] - p.before[b];
  const int32_t u0 = p.before[b] * per_seq + entries * (head * p.row_groups + head_row / ROWS);
  const int c0 = parts.owner(u0), c1 = parts.owner(u0 + entries - 1);
  if (c0 == c1) return;  // written by that warp
  const int r = head_row % ROWS;
  // It is the first segment of warp c0 if nothing of the one before is that warp's.
  const int64_t first = (int64_t)2 * c0 + (parts.begin(c0) >= u0 ? 0 : 1);
  constexpr int AHEAD = 4;  // parts read at once
  float top = -INFINITY, sum = 0.f, acc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  for (int c = c0 + warp; c <= c1; c += kWarps * AHEAD) {
    float2 ml[AHEAD];
    float x[AHEAD][PER];
    float above = top;
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int ca = c + a * kWarps;
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
    for (int i = 0; i < PER; ++i) acc[i] *= f0;
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      if (c + a * kWarps > c1) break;
      const float f = ex2_approx(ml[a].x - ref);
      sum += f * ml[a].y;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] += f * x[a][i];
    }
    top = above;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) s_o[warp][i * 32 + lane] = acc[i];
  if (lane == 0) s_sum[warp] = sum, s_top[warp] = top;
  __syncthreads();
  float f[kWarps];
  top = -INFINITY;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_top[w]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = ex2_approx(s_top[w] - (top == -INFINITY ? 0.f : top));
    sum += f[w] * s_sum[w];
  }
  const float v_scale = p.v_scale != nullptr ? p.v_scale[head] : 1.f;
  const float inv = sum == 0.f ? 0.f : v_scale / sum;
  if ((int)threadIdx.x < DV / 2) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      x += f[w] * s_o[w][2 * threadIdx.x];
      y += f[w] * s_o[w][2 * threadIdx.x + 1];
    }
    reinterpret_cast<uint32_t *>(p.out + row * DV)[threadIdx.x] = pack_bf16x2(x * inv, y * inv);
  }
  if (threadIdx.x == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

int64_t align16(int64_t x) { return (x + 15) & ~(int64_t)15; }

// What the sizes of a call decide.
struct Plan {
  int rows;             // of a tile: 8, 16 or 32
  int64_t most;         // steps that a sequence can have, from its row of pages and the window
  int64_t segments;
  int cluster;          // CTAs per segment, 0: the list
  size_t workspace;
};

// Clusters or the list.  A cluster call has no scan and no second kernel, the
// list loads every SM alike however the lengths differ.  Measured (32 query, 8
// KV heads of 128, bf16; list -> clusters, us): 1 sequence of 64 keys
// 5.4 -> 3.1, 2048 keys 12.3 -> 6.6, 16384 keys 19.6 -> 17.2; 8 sequences of
// 2048 keys 13.9 -> 10.6, of 8192 keys 47.4 -> 42.9; 16 sequences through a
// window of 4096 keys 48.0 -> 42.7; 8 sequences of 1023 .. 8191 keys, 4 tokens
// each, 33.4 -> 32.6.  A sequence much longer than the others keeps its
// clusters running alone (2048 keys take a CTA 23 us), so the keys that a CTA may
// get are limited: 2048, and the ends of a window of that size per CTA.  (A block
// table with more columns takes the list.)  Other layouts take the same limits:
// 16 / 16 heads of 192: 1 sequence of 2048 keys 12.7 -> 11.5, of 16384 35.0 -> 43.3;
// 4 / 2 of 64: 7.5 -> 4.6, 24.7 -> 10.3; 4 tokens of 8 / 1 heads of 128: 20.9 -> 16.2,
// 96.2 -> 31.5; 32 / 8 heads of 128 in e4m3: 9.9 -> 6.7, 20.7 -> 16.3, but 8 sequences
// of 1023 .. 8191 keys 19.4 -> 24.7.
constexpr int kSlots = kMaxWarps / kWarps;  // CTAs that fill the GPU at two per SM
constexpr int kMaxCluster = 16;             // (with at most 8, 16384 keys of 1 sequence take 24.8 us)
constexpr int kClusterKeys = 2304;          // per CTA, at most
// The 32-row tile of 192-wide heads has one CTA per SM, so that its clusters may
// come in two waves.  That is better for sequences of mixed lengths (us, one wave
// or the list -> two waves: 20 sequences of 204 .. 4096 keys and 2 KV heads 47.7 ->
// 38.3, 100 of 20 .. 2048 67.7 -> 63.1) and worse for equal ones (50 of 2048 keys
// 47.9 -> 59.1, 100 of them 76.8 -> 93.7); the limit is the same for all tiles.

Plan plan(int32_t B, int32_t Hq, int32_t Hkv, int32_t Lq, int32_t dqk, int32_t dv, int32_t max_pages, int32_t page_size,
          int32_t type, int64_t window) {
  Plan x;
  const int64_t nrows = (int64_t)(Hq / Hkv) * Lq;
  x.rows = nrows <= 8 ? 8 : nrows <= 16 ? 16 : 32;
  const int64_t kw = keys_per_step((dqk + dv) * (type == SPLASH_CACHE_E4M3 ? 1 : 2));
  x.most = ((int64_t)max_pages * page_size + kw - 1) / kw;
  if (window >= 0) x.most = std::min(x.most, window / kw + 4);
  x.segments = (int64_t)B * Hkv * ((nrows + x.rows - 1) / x.rows);
  x.cluster = x.segments <= kSlots ? 1 : 0;
  while (x.cluster > 0 && x.cluster < kMaxCluster && 2 * x.cluster * x.segments <= kSlots && x.cluster * kWarps < x.most) x.cluster *= 2;
  if (x.most * kw > (int64_t)kClusterKeys * x.cluster) x.cluster = 0;
  const int64_t rows = std::min<int64_t>(nrows, x.rows);
  x.workspace = x.cluster > 0 ? 0 : (size_t)(align16(4 * ((int64_t)B + 1)) + (int64_t)2 * kMaxWarps * rows * 4 * (dv + 2));
  return x;
}

// The largest cluster that the current device can place.  More than 8 CTAs need
// not fit (a part of a GPU, say, may not have 16 SMs next to one another); a
// smaller one does the same with more keys per CTA.
template <class C>
int placeable() {
  int cluster = kMaxCluster;
  for (; cluster > 1; cluster /= 2) {
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(cluster);
    config.blockDim = dim3(kThreads);
    config.dynamicSmemBytes = C::SMEM;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    config.attrs = &attr;
    config.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, paged_decode_kernel<C, true>, &config) == cudaSuccess && clusters > 0) break;
    (void)cudaGetLastError();  // (what else is wrong shows at the launch)
  }
  return cluster;
}

// grid clusters of `cluster` CTAs each, or of fewer where that has no room.
template <class C, bool TOGETHER>
splash_status launch_kernel(int grid, int cluster, const Params &p, cudaStream_t stream) {
  static std::atomic<int8_t> most[64];  // per device: CTAs of a cluster that fits, 0: this kernel has not run there
  int dev = 0;
  SPLASH_CUDA_TRY(cudaGetDevice(&dev));
  std::atomic<int8_t> &fits = most[dev & 63];
  if (fits.load(std::memory_order_acquire) == 0) {
    SPLASH_CUDA_TRY(cudaFuncSetAttribute(paged_decode_kernel<C, TOGETHER>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
    int room = 1;
    if constexpr (TOGETHER) {
      SPLASH_CUDA_TRY(cudaFuncSetAttribute(paged_decode_kernel<C, TOGETHER>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
      room = placeable<C>();
    }
    fits.store((int8_t)room, std::memory_order_release);
  }
  cluster = std::min<int>(cluster, fits.load(std::memory_order_relaxed));
  SPLASH_CUDA_TRY(launch_dependent(paged_decode_kernel<C, TOGETHER>, dim3(grid * cluster), dim3(kThreads), C::SMEM, cluster, stream, p));
  splash_count_launches(1);
  return SPLASH_OK;
}

template <class C>
splash_status launch(const Plan &x, void *workspace, Params p, cudaStream_t stream) {
  p.row_groups = (p.nrows + C::ROWS - 1) / C::ROWS;
  p.part_rows = std::min(p.nrows, C::ROWS);
  if (x.cluster > 0) return launch_kernel<C, true>((int)x.segments, x.cluster, p, stream);
  char *ws = static_cast<char *>(workspace);
  p.before = reinterpret_cast<int32_t *>(ws);
  ws += align16(4 * ((int64_t)p.B + 1));
  p.part_ml = reinterpret_cast<float *>(ws);
  ws += (int64_t)2 * kMaxWarps * p.part_rows * 2 * 4;
  p.part_o = reinterpret_cast<float *>(ws);
  int dev = 0, sms = 0;
  SPLASH_CUDA_TRY(cudaGetDevice(&dev));
  SPLASH_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  const int ctas = (int)std::min<int64_t>({std::min<int64_t>(x.most, kMaxWarps) * x.segments, C::CTAS * (int64_t)sms,
                                           kMaxWarps / kWarps});
  const splash_status st = launch_kernel<C, false>(ctas, 1, p, stream);
  if (st != SPLASH_OK || x.most <= 1) return st;  // (no segment has more than one step: nothing to join)
  const dim3 rows((unsigned)((int64_t)p.B * p.Hkv * p.nrows));
  SPLASH_CUDA_TRY(launch_dependent(paged_decode_join_kernel<C::DV, C::ROWS>, rows, dim3(kThreads), 0, 1, stream, p, ctas * kWarps));
  splash_count_launches(1);
  return SPLASH_OK;
}

template <int DQK, int DV, int ROWS>
splash_status pick_queries(const Plan &x, void *workspace, const Params &p, cudaStream_t stream) {
  constexpr bool E4M3 = SPLASH_DECODE_E4M3 != 0;
  return p.Lq == 1 ? launch<Config<DQK, DV, E4M3, ROWS, false>>(x, workspace, p, stream)
                   : launch<Config<DQK, DV, E4M3, ROWS, true>>(x, workspace, p, stream);
}

template <int DQK, int DV>
splash_status pick(const splash_paged_decode_args &a, const Params &p, cudaStream_t stream) {
  const Plan x = plan(a.B, a.Hq, a.Hkv, a.Lq, a.dqk, a.dv, a.max_pages, a.page_size, a.cache_type, a.window_left);
  if (x.rows == 8) return pick_queries<DQK, DV, 8>(x, a.workspace, p, stream);
  if (x.rows == 16) return pick_queries<DQK, DV, 16>(x, a.workspace, p, stream);
  return pick_queries<DQK, DV, 32>(x, a.workspace, p, stream);
}

}  // namespace
}  // namespace splash

#if !SPLASH_DECODE_E4M3
size_t splash_paged_decode_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t Lq, int32_t dqk, int32_t dv,
                                           int32_t max_pages, int32_t page_size, int32_t type, int64_t window) {
  return splash::plan(B, Hq, Hkv, Lq, dqk, dv, max_pages, page_size, type, window).workspace;
}

splash_status splash_paged_decode_launch(const splash_paged_decode_args &a, cudaStream_t stream, uint32_t *err_word) {
  return a.cache_type == SPLASH_CACHE_E4M3 ? splash_paged_decode_launch_e4m3(a, stream, err_word)
                                           : splash_paged_decode_launch_bf16(a, stream, err_word);
}
#endif

#if SPLASH_DECODE_E4M3
splash_status splash_paged_decode_launch_e4m3(const splash_paged_decode_args &a, cudaStream_t stream, uint32_t *err_word) {
#else
splash_status splash_paged_decode_launch_bf16(const splash_paged_decode_args &a, cudaStream_t stream, uint32_t *err_word) {
#endif
  using namespace splash;
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
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  p.num_pages = a.num_pages;
  p.B = a.B;
  p.Hkv = a.Hkv;
  p.Lq = a.Lq;
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
  if (a.dqk == 64) return pick<64, 64>(a, p, stream);
  if (a.dqk == 128) return pick<128, 128>(a, p, stream);
  return pick<192, 128>(a, p, stream);
}
