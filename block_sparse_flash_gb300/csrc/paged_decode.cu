// paged_decode.cu -- attention of new tokens over a paged key/value cache
// (splash_paged_decode in splash.h).
//
// For a query row: s_j = scale q.k_j, m = max s_j, l = sum exp(s_j - m),
// out = sum exp(s_j - m) v_j / l, lse = m + ln l, in one pass over the keys.
// Every key and value is used by the Hq/Hkv * Lq rows of its head only, a few
// FLOP per byte: reading the cache bounds the call, so the kernel is built to
// keep the memory system full.
//
//  * Work.  The keys of each (sequence, KV head, group of rows) are cut into
//    tiles; all tiles form one list, and every CTA of a grid that fills the GPU
//    once takes an equal, contiguous part of it.  Long and short sequences
//    thus load every SM alike.  A (sequence, head) that one CTA covers is
//    finished there; parts of one that several CTAs share go to the workspace
//    as (sum, maximum, unnormalised output) and a second kernel joins them, in
//    the order of the keys, so that the result does not depend on timing.
//  * Loads.  Each warp takes its own keys of a tile (KW of them) and keeps its
//    own ring of stages in shared memory, filled by 16-byte asynchronous
//    copies: no barrier between warps in the loop.  Rows outside the keys that
//    some query sees are filled with zeros instead of being read, so that
//    whatever they hold cannot reach a product.
//  * Products.  16 rows x 16 keys per tensor instruction (mma.sync: with 4 to 32
//    rows a tile is memory-bound many times over, and the accumulators stay in
//    registers next to the softmax).  P goes to the second product from the
//    registers that the first one left it in.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "internal.h"
#include "sm103_ptx.cuh"

namespace splash {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kMaxGrid = 512;  // CTAs; the workspace holds two parts for each

// A running maximum is only moved when a score passes it by more than this
// (in powers of two): until then exp2(s - m) stays below 2^8, which neither
// the sums (fp32) nor P's 16-bit types mind, and no shuffles or rescaling of
// the output are needed.
constexpr float kSlack = 8.f;

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
  float *part_o, *part_ml;  // [2 * CTAs][rows][DV], [2 * CTAs][rows][2] (maximum, sum)
  int64_t *first_tile;      // [B + 1] tiles (of one head and row group) before each sequence
  int64_t num_pages;
  int32_t B, Hq, Hkv, Lq, G, nrows, row_groups;  // nrows = G * Lq rows per KV head
  int32_t max_pages, page_shift, window;         // window < 0: none
  float scale, cap;                              // cap <= 0: none
  uint32_t *err;
};

template <int DQK_, int DV_, bool E4M3_, int MT_>
struct Config {
  static constexpr int DQK = DQK_, DV = DV_, MT = MT_, ROWS = 16 * MT_;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int RK = DQK * (E4M3 ? 1 : 2), RV = DV * (E4M3 ? 1 : 2);  // bytes of a row
  static constexpr int NB = RK + RV >= 512 ? 1 : 2;                          // 16-key blocks per warp and step
  static constexpr int KW = 16 * NB, TILE = KW * kWarps;
  static constexpr int STAGE = KW * (RK + RV);
  static constexpr int STAGES = STAGE * kWarps >= 40960 ? 2 : STAGE * kWarps >= 32768 ? 3 : 6;
  static constexpr int RING = STAGES * STAGE;  // per warp
  static constexpr int ODIM = DV + 4;          // floats of a row of the warps' join
  static constexpr int QBYTES = ROWS * DQK * 2;
  static constexpr int SMEM = kWarps * RING + QBYTES;
  static_assert(RING >= ROWS * ODIM * 4, "the join of the warps reuses their rings");
};

// The keys of sequence b that its queries see, in tiles.
struct Span {
  int32_t n, lo;      // keys [lo, n) are visible to some query
  int32_t tile0, nt;  // tiles tile0 .. tile0 + nt - 1; at least one, so that empty rows are written too
};

template <int TILE>
__device__ __forceinline__ Span span_of(const Params &p, int b) {
  Span s;
  const int64_t most = (int64_t)p.max_pages << p.page_shift;
  const int32_t n = __ldg(p.seq_lens + b);
  s.n = n < 0 ? 0 : n > most ? (int32_t)most : n;
  s.lo = p.window < 0 ? 0 : max(0, s.n - p.Lq - p.window);
  s.tile0 = s.lo / TILE;
  s.nt = max(1, (s.n + TILE - 1) / TILE - s.tile0);
  return s;
}

// Equal contiguous parts of T tiles: CTA c takes [part(c), part(c + 1)).
struct Parts {
  int64_t each;
  int32_t more;  // the first `more` CTAs take one tile more
  __device__ __forceinline__ Parts(int64_t T, int32_t ctas) : each(T / ctas), more((int32_t)(T % ctas)) {}
  __device__ __forceinline__ int64_t begin(int32_t c) const { return each * c + min(c, more); }
  __device__ __forceinline__ int32_t owner(int64_t u) const {
    const int64_t cut = (each + 1) * more;
    return u < cut ? (int32_t)(u / (each + 1)) : more + (int32_t)((u - cut) / each);
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

// tanh|x| = (1 - e) / (1 + e), e = exp(-2|x|)
__device__ __forceinline__ float tanh_of(float x) {
  const float e = ex2_approx(-2.f * kLog2e * fabsf(x));
  return copysignf(__fdividef(1.f - e, 1.f + e), x);
}

// One warp's copies of its KW keys of a tile into a stage.
template <class C>
struct Loader {
  const Params &p;
  int b, head, lane;
  int32_t n, lo;
  const int32_t *pages;
  int32_t next[C::NB];  // page entries of the next step, read one step ahead

  __device__ __forceinline__ void look(int32_t key0) {
#pragma unroll
    for (int i = 0; i < C::NB; ++i) {
      const int32_t key = key0 + 16 * i;
      next[i] = key < n && key + 16 > lo ? __ldg(pages + (key >> p.page_shift)) : 0;
    }
  }

  template <int ROWB>
  __device__ __forceinline__ void block(uint32_t dst, const char *base, int64_t token, int32_t key, bool ok) const {
    constexpr int SEG = ROWB % 128 == 0 ? 128 : 64;  // a row's contiguous bytes per instruction
    constexpr int LPS = SEG / 16, RPI = 32 / LPS;
    const int r0 = lane / LPS, c0 = lane % LPS;
    const char *src = base + r0 * token + c0 * 16;
#pragma unroll
    for (int rg = 0; rg < 16 / RPI; ++rg) {
      const int r = rg * RPI + r0;
      const bool read = ok && key + r >= lo && key + r < n;
#pragma unroll
      for (int part = 0; part < ROWB / SEG; ++part)
        copy16(dst + chunk_at<ROWB>(r, part * LPS + c0), read ? src + rg * RPI * token + part * SEG : base, read);
    }
  }

  // the keys key0 .. key0 + KW - 1 (pages looked up before), and the pages of
  // the step after
  __device__ __forceinline__ void step(uint32_t stage, int32_t key0, int32_t key_next) {
    if (key0 < n && key0 + C::KW > lo) {
#pragma unroll
      for (int i = 0; i < C::NB; ++i) {
        const int32_t key = key0 + 16 * i, page = next[i];
        const bool ok = page >= 0 && page < p.num_pages;
        if (!ok && lane == 0) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
        const int32_t slot = key & ((1 << p.page_shift) - 1);
        const int64_t at = ok ? page : 0;
        block<C::RK>(stage + i * 16 * C::RK, p.k + at * p.k_page + head * p.k_head + slot * p.k_token, p.k_token, key, ok);
        block<C::RV>(stage + C::KW * C::RK + i * 16 * C::RV, p.v + at * p.v_page + head * p.v_head + slot * p.v_token,
                     p.v_token, key, ok);
      }
    }
    copy_commit();
    look(key_next);
  }
};

template <class C>
__global__ void __launch_bounds__(kThreads, 2) paged_decode_kernel(const Params p) {
  constexpr int DQK = C::DQK, DV = C::DV, MT = C::MT, NB = C::NB;
  constexpr bool E4M3 = C::E4M3;
  extern __shared__ __align__(1024) char smem[];
  __shared__ int64_t s_scan[kWarps], s_start[2];
  __shared__ float s_factor[C::ROWS], s_ml[kWarps][C::ROWS][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quad = lane >> 2, tq = lane & 3;
  char *q_smem = smem + kWarps * C::RING;
  char *ring = smem + warp * C::RING;
  const uint32_t ring_u = smem_u32(ring), q_u = smem_u32(q_smem);

  // the join may be launched; it waits for this grid before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's part of the list of tiles: a scan over the sequences
  const int per_seq = p.Hkv * p.row_groups;  // entries of the list per tile of a sequence
  int64_t T;
  {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    int64_t own = 0;
    for (int b = b0; b < b1; ++b) own += span_of<C::TILE>(p, b).nt;
    int64_t before = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(~0u, before, o);
      if (lane >= o) before += y;
    }
    if (lane == 31) s_scan[warp] = before;
    before -= own;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    T = total * per_seq;
    const int64_t u = Parts(T, gridDim.x).begin(blockIdx.x);
    if (blockIdx.x == 0 || (u >= before * per_seq && u < (before + own) * per_seq)) {
      int64_t at = before;
      for (int b = b0; b < b1; ++b) {
        const int64_t next = at + span_of<C::TILE>(p, b).nt;
        if (u >= at * per_seq && u < next * per_seq) s_start[0] = b, s_start[1] = at;
        if (blockIdx.x == 0) {
          p.first_tile[b] = at;
          if (b == p.B - 1) p.first_tile[p.B] = next;
        }
        at = next;
      }
    }
    if (blockIdx.x == 0)
      for (int b = b0; b < b1; ++b) {
        const int32_t n = p.seq_lens[b];
        if (n < 0 || n > (int64_t)p.max_pages << p.page_shift) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
      }
    __syncthreads();
  }
  const Parts parts(T, gridDim.x);
  int64_t u = parts.begin(blockIdx.x);
  const int64_t u_begin = u, u_end = parts.begin(blockIdx.x + 1);
  int b = (int)s_start[0];
  int64_t seq_u = s_start[1] * per_seq;  // first list entry of sequence b

  for (; u < u_end;) {
    Span sp = span_of<C::TILE>(p, b);
    if (u >= seq_u + (int64_t)sp.nt * per_seq) {
      seq_u += (int64_t)sp.nt * per_seq;
      ++b;
      continue;
    }
    const int seg = (int)((u - seq_u) / sp.nt);
    const int32_t t0 = (int32_t)((u - seq_u) % sp.nt);
    const int32_t t1 = (int32_t)min((int64_t)sp.nt, t0 + (u_end - u));
    const int head = seg / p.row_groups, row0 = (seg % p.row_groups) * C::ROWS;
    const int rows = min(C::ROWS, p.nrows - row0);

    // ---- queries to shared memory, rows g * Lq + l of the KV head's group.
    // For e4m3 they become fp16: scaled by a power of two that brings the
    // row's largest element into [1, 2), which is exact except for elements
    // 2^14 times smaller than it (their error, 2^-25 of the largest, is below
    // that of an fp32 sum); the factor goes to the row's scale.
    for (int r = warp; r < C::ROWS; r += kWarps) {
      constexpr int W = DQK / 64;  // words (two elements) per lane
      uint32_t x[W];
      if (r < rows) {
        const int g = (row0 + r) / p.Lq, l = (row0 + r) % p.Lq;
        const char *src = p.q + b * p.q_b + (int64_t)(head * p.G + g) * p.q_h + l * p.q_l;
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = __ldg(reinterpret_cast<const uint32_t *>(src) + i * 32 + lane);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = 0;
      }
      float f = p.cap > 0.f ? p.scale / p.cap : p.scale * kLog2e;
      if (E4M3) {
        uint32_t top = 0;  // exponent field of the largest element
#pragma unroll
        for (int i = 0; i < W; ++i) top = max(top, max((x[i] >> 7) & 255u, (x[i] >> 23) & 255u));
        top = __reduce_max_sync(~0u, top);
        top = top == 0 ? 1 : min(top, 253u);
        const float down = __uint_as_float((254u - top) << 23), up = __uint_as_float(top << 23);
#pragma unroll
        for (int i = 0; i < W; ++i)
          x[i] = pack2<true>(__uint_as_float(x[i] << 16) * down, __uint_as_float(x[i] & 0xffff0000u) * down);
        f *= up * __ldg(p.k_scale + head);
      }
      if (lane == 0) s_factor[r] = f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int d = 2 * (i * 32 + lane);
        // An ldmatrix of four e4m3 keys leaves elements 4t .. 4t+3 in the
        // thread that the product expects to hold 2t, 2t+1, 2t+8, 2t+9 of each
        // 16: the queries are stored in that order.
        const int at = E4M3 ? (d & ~15) + 2 * ((d & 15) >> 2) + ((d & 2) ? 8 : 0) : d;
        *reinterpret_cast<uint32_t *>(q_smem + chunk_at<DQK * 2>(r, at >> 3) + (at & 7) * 2) = x[i];
      }
    }

    // ---- the keys
    Loader<C> load{p, b, head, lane, sp.n, sp.lo, p.block_table + b * p.block_table_stride, {}};
    const int32_t key_base = (sp.tile0 + t0) * C::TILE + warp * C::KW;
    const int32_t steps = t1 - t0;
    load.look(key_base);
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) {
      if (s < steps)
        load.step(ring_u + s * C::STAGE, key_base + s * C::TILE, key_base + (s + 1) * C::TILE);
      else
        copy_commit();
    }
    __syncthreads();  // queries

    uint32_t qa[MT == 1 ? DQK / 16 : 1][4];
    const uint32_t q_row = (lane & 7) + ((lane >> 3) & 1) * 8;
    if (MT == 1) {
#pragma unroll
      for (int kk = 0; kk < DQK / 16; ++kk) ldsm4(qa[kk], q_u + chunk_at<DQK * 2>(q_row, 2 * kk + (lane >> 4)));
    }
    float factor[MT][2], m[MT][2], l[MT][2], o[MT][DV / 8][4];
    int32_t pos[MT][2];  // the row's position (rows past the last one see what the last query sees)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mt * 16 + quad + 8 * e;
        factor[mt][e] = s_factor[r];
        pos[mt][e] = sp.n - p.Lq + (r < rows ? (row0 + r) % p.Lq : p.Lq - 1);
        m[mt][e] = -INFINITY;
        l[mt][e] = 0.f;
      }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < DV / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][j][i] = 0.f;

    int slot = 0;
    for (int32_t t = 0; t < steps; ++t) {
      copy_wait<C::STAGES - 2>();
      __syncwarp();
      const int32_t key0 = key_base + t * C::TILE;
      const uint32_t ks = ring_u + slot * C::STAGE, vs = ks + C::KW * C::RK;
      {
        const int32_t ahead = t + C::STAGES - 1;
        const int into = slot == 0 ? C::STAGES - 1 : slot - 1;
        if (ahead < steps)
          load.step(ring_u + into * C::STAGE, key_base + ahead * C::TILE, key_base + (ahead + 1) * C::TILE);
        else
          copy_commit();
      }
      slot = slot == C::STAGES - 1 ? 0 : slot + 1;
      if (key0 >= sp.n || key0 + C::KW <= sp.lo) continue;  // (the same for the whole warp)

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
      const bool whole = key0 + C::KW <= sp.n - p.Lq + 1 && (p.window < 0 || key0 >= sp.n - 1 - p.window);
      bool move = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float y = s[mt][j][2 * e + i] * factor[mt][e];
              if (p.cap > 0.f) y = p.cap * kLog2e * tanh_of(y);
              if (!whole) {
                const int32_t behind = pos[mt][e] - (key0 + 8 * j + 2 * tq + i);
                if (behind < 0 || (p.window >= 0 && behind > p.window)) y = -INFINITY;
              }
              s[mt][j][2 * e + i] = y;
              top = fmaxf(top, y);
            }
          move |= top > m[mt][e] + kSlack;
        }
      if (__any_sync(~0u, move)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = m[mt][e];
#pragma unroll
            for (int j = 0; j < 2 * NB; ++j) top = fmax3(top, s[mt][j][2 * e], s[mt][j][2 * e + 1]);
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            const float alpha = top == -INFINITY ? 1.f : ex2_approx(m[mt][e] - top);
            m[mt][e] = top;
            l[mt][e] *= alpha;
#pragma unroll
            for (int j = 0; j < DV / 8; ++j) {
              o[mt][j][2 * e] *= alpha;
              o[mt][j][2 * e + 1] *= alpha;
            }
          }
      }

      // P (rounded to 16 bits for the product; its sum is taken before), O += P V
      uint32_t pa[MT][NB][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
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
          for (int i = 0; i < 4; ++i)
            pa[mt][nb][i] = pack2<E4M3>(s[mt][2 * nb + (i >> 1)][2 * (i & 1)], s[mt][2 * nb + (i >> 1)][2 * (i & 1) + 1]);
      }
      const int v_row = (lane & 7) + ((lane >> 3) & 1) * 8, v_chunk = lane >> 4;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int j = 0; j < DV / 16; j += E4M3 ? 2 : 1) {
          uint32_t vb[4];
          ldsm4_trans(vb, vs + nb * 16 * C::RV + chunk_at<C::RV>(v_row, (E4M3 ? j : 2 * j) + v_chunk));
          if (E4M3) {
            // Each word holds two neighbouring columns of two keys: the even
            // columns of 16 go to one product, the odd ones to the next.
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t b0, b1, c0, c1;
              widen(__byte_perm(vb[2 * x], 0, 0x3120), b0, c0);
              widen(__byte_perm(vb[2 * x + 1], 0, 0x3120), b1, c1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma<true>(o[mt][2 * (j + (E4M3 ? x : 0))], pa[mt][nb], b0, b1);
                mma<true>(o[mt][2 * (j + (E4M3 ? x : 0)) + 1], pa[mt][nb], c0, c1);
              }
            }
          } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma<false>(o[mt][2 * j], pa[mt][nb], vb[0], vb[1]);
              mma<false>(o[mt][2 * j + 1], pa[mt][nb], vb[2], vb[3]);
            }
          }
        }
      }
    }

    // ---- the warps' parts, joined through shared memory (each warp's ring
    // holds its own)
    copy_wait<0>();
    __syncwarp();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mt * 16 + quad + 8 * e;
        float sum = l[mt][e];
        sum += __shfl_xor_sync(~0u, sum, 1);
        sum += __shfl_xor_sync(~0u, sum, 2);
        if (tq == 0) {
          s_ml[warp][r][0] = m[mt][e];
          s_ml[warp][r][1] = sum;
        }
        float *row = reinterpret_cast<float *>(ring) + r * C::ODIM;
        if (E4M3) {
#pragma unroll
          for (int j = 0; j < DV / 16; ++j)
            *reinterpret_cast<float4 *>(row + 16 * j + 4 * tq) = make_float4(
                o[mt][2 * j][2 * e], o[mt][2 * j + 1][2 * e], o[mt][2 * j][2 * e + 1], o[mt][2 * j + 1][2 * e + 1]);
        } else {
#pragma unroll
          for (int j = 0; j < DV / 8; ++j)
            *reinterpret_cast<float2 *>(row + 8 * j + 2 * tq) = make_float2(o[mt][j][2 * e], o[mt][j][2 * e + 1]);
        }
      }
    __syncthreads();
    const bool complete = t0 == 0 && t1 == sp.nt;
    const int part = 2 * blockIdx.x + (u == u_begin ? 0 : 1);
    constexpr int LANES = DV / 4, STEP = kThreads / LANES;  // lanes per row, rows at a time
    const int col = 4 * (threadIdx.x % LANES);
    const float v_scale = E4M3 ? __ldg(p.v_scale + head) : 1.f;
    for (int r = threadIdx.x / LANES; r < rows; r += STEP) {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][r][0]);
      const float ref = top == -INFINITY ? 0.f : top;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(s_ml[w][r][0] - ref);
        sum += f * s_ml[w][r][1];
        const float4 x = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem + w * C::RING) + r * C::ODIM + col);
        acc.x += f * x.x;
        acc.y += f * x.y;
        acc.z += f * x.z;
        acc.w += f * x.w;
      }
      if (complete) {
        const float inv = sum == 0.f ? 0.f : v_scale / sum;
        const int64_t row = ((int64_t)b * p.Hkv + head) * p.nrows + row0 + r;
        *reinterpret_cast<uint2 *>(p.out + row * DV + col) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (col == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
      } else {
        *reinterpret_cast<float4 *>(p.part_o + ((int64_t)part * C::ROWS + r) * DV + col) = acc;
        if (col == 0) *reinterpret_cast<float2 *>(p.part_ml + ((int64_t)part * C::ROWS + r) * 2) = make_float2(top, sum);
      }
    }
    __syncthreads();
    u += t1 - t0;
  }
}

// Joins the parts of a row that several CTAs computed: with (m_c, l_c, o_c) of
// part c and m = max m_c: out = sum exp(m_c - m) o_c / sum exp(m_c - m) l_c.
// One CTA per row, its warps taking every fourth part.
template <int DV, int ROWS, int TILE>
__global__ void __launch_bounds__(kThreads) paged_decode_join_kernel(const Params p, int ctas) {
  __shared__ float s_o[kWarps][DV], s_sum[kWarps], s_top[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int PER = DV / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = blockIdx.x;  // (b, KV head, row)
  const int head_row = (int)(row % p.nrows), head = (int)(row / p.nrows % p.Hkv), b = (int)(row / p.nrows / p.Hkv);
  const int per_seq = p.Hkv * p.row_groups;
  const Parts parts(p.first_tile[p.B] * per_seq, ctas);
  const int64_t nt = p.first_tile[b + 1] - p.first_tile[b];
  const int64_t u0 = p.first_tile[b] * per_seq + nt * (head * p.row_groups + head_row / ROWS);
  const int c0 = parts.owner(u0), c1 = parts.owner(u0 + nt - 1);
  if (c0 == c1) return;  // written by that CTA
  const int r = head_row % ROWS;
  // A CTA's first part is the one its range begins with.
  const int64_t first = (int64_t)2 * c0 + (parts.begin(c0) >= u0 ? 0 : 1);
  float top = -INFINITY;
  for (int c = c0 + (int)threadIdx.x; c <= c1; c += kThreads)
    top = fmaxf(top, p.part_ml[((c == c0 ? first : (int64_t)2 * c) * ROWS + r) * 2]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_top[w]);
  const float ref = top == -INFINITY ? 0.f : top;
  float acc[PER], sum = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int c = c0 + warp; c <= c1; c += kWarps) {
    const int64_t at = (c == c0 ? first : (int64_t)2 * c) * ROWS + r;
    const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + at * 2);
    const float f = ex2_approx(ml.x - ref);
    sum += f * ml.y;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] += f * p.part_o[at * DV + i * 32 + lane];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) s_o[warp][i * 32 + lane] = acc[i];
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += s_sum[w];
  const float v_scale = p.v_scale != nullptr ? __ldg(p.v_scale + head) : 1.f;
  const float inv = sum == 0.f ? 0.f : v_scale / sum;
  if ((int)threadIdx.x < DV / 2) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      x += s_o[w][2 * threadIdx.x];
      y += s_o[w][2 * threadIdx.x + 1];
    }
    reinterpret_cast<uint32_t *>(p.out + row * DV)[threadIdx.x] = pack_bf16x2(x * inv, y * inv);
  }
  if (threadIdx.x == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

int64_t align16(int64_t x) { return (x + 15) & ~(int64_t)15; }

int row_tiles(int64_t nrows) { return nrows <= 16 ? 1 : 2; }

template <class C>
splash_status launch(const splash_paged_decode_args &a, Params p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  SPLASH_CUDA_TRY(cudaGetDevice(&dev));
  SPLASH_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  static std::atomic<uint64_t> ready{0};  // devices that allow this kernel its shared memory
  const uint64_t bit = (uint64_t)1 << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    SPLASH_CUDA_TRY(cudaFuncSetAttribute(paged_decode_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
    ready.fetch_or(bit, std::memory_order_release);
  }
  p.row_groups = (p.nrows + C::ROWS - 1) / C::ROWS;
  // tiles that a sequence can have at most, from the row of pages and the window
  int64_t most = (((int64_t)a.max_pages << p.page_shift) + C::TILE - 1) / C::TILE;
  if (p.window >= 0) most = std::min(most, ((int64_t)p.window + p.Lq) / C::TILE + 2);
  const int64_t all = std::min<int64_t>(most, kMaxGrid) * p.B * p.Hkv * p.row_groups;
  const int ctas = (int)std::min<int64_t>({all, 2 * (int64_t)sms, kMaxGrid});
  char *ws = static_cast<char *>(a.workspace);
  p.first_tile = reinterpret_cast<int64_t *>(ws);
  ws += align16(8 * ((int64_t)p.B + 1));
  p.part_ml = reinterpret_cast<float *>(ws);
  ws += (int64_t)2 * kMaxGrid * C::ROWS * 2 * 4;
  p.part_o = reinterpret_cast<float *>(ws);
  paged_decode_kernel<C><<<ctas, kThreads, C::SMEM, stream>>>(p);
  SPLASH_CUDA_TRY(cudaGetLastError());
  splash_count_launches(1);
  if (most <= 1) return SPLASH_OK;  // no sequence has more than one tile: nothing to join
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3((unsigned)((int64_t)p.B * p.Hkv * p.nrows));
  config.blockDim = dim3(kThreads);
  config.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &attr;
  config.numAttrs = 1;
  SPLASH_CUDA_TRY(cudaLaunchKernelEx(&config, paged_decode_join_kernel<C::DV, C::ROWS, C::TILE>, (const Params)p, ctas));
  splash_count_launches(1);
  return SPLASH_OK;
}

template <int DQK, int DV>
splash_status pick(const splash_paged_decode_args &a, const Params &p, cudaStream_t stream) {
  const bool one = row_tiles(p.nrows) == 1;
  if (a.cache_type == SPLASH_CACHE_E4M3)
    return one ? launch<Config<DQK, DV, true, 1>>(a, p, stream) : launch<Config<DQK, DV, true, 2>>(a, p, stream);
  return one ? launch<Config<DQK, DV, false, 1>>(a, p, stream) : launch<Config<DQK, DV, false, 2>>(a, p, stream);
}

}  // namespace
}  // namespace splash

size_t splash_paged_decode_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t Lq, int32_t dv) {
  using namespace splash;
  const int64_t rows = 16 * row_tiles((int64_t)(Hq / Hkv) * Lq);
  return (size_t)(align16(8 * ((int64_t)B + 1)) + (int64_t)2 * kMaxGrid * rows * 4 * (dv + 2));
}

splash_status splash_paged_decode_launch(const splash_paged_decode_args &a, cudaStream_t stream, uint32_t *err_word) {
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
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.Lq = a.Lq;
  p.G = a.Hq / a.Hkv;
  p.nrows = p.G * a.Lq;
  p.max_pages = a.max_pages;
  p.page_shift = __builtin_ctz((unsigned)a.page_size);
  // (differences of positions stay below 2^31 - 64)
  p.window = a.window_left < 0 ? -1 : (int32_t)std::min<int64_t>(a.window_left, INT32_MAX - 64);
  p.scale = a.scale;
  p.cap = a.softcap;
  p.err = err_word;
  if (a.dqk == 64) return pick<64, 64>(a, p, stream);
  if (a.dqk == 128) return pick<128, 128>(a, p, stream);
  return pick<192, 128>(a, p, stream);
}
