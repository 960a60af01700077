// rope.cu -- rotary positions, and appending rotated keys and values to a
// paged cache (splash_rope and splash_paged_append in splash.h).
//
// A pair (a, b) at position p turns by the angle whose cosine c and sine s
// are in the table: a' = a c - b s, b' = b c + a s; the transposed rotation
// (the gradient) has -s.  Both are 2 multiplications and 1 addition per
// element on data that is read once and written once, so HBM bounds them:
// q and k of 2 x 4096 tokens (32 + 8 heads of 128) take 27.5 us, 6.2 TB/s, the
// gradient of 128 + 128 heads of 192 dimensions 117 us, 6.9 TB/s, a packed
// prompt of 32768 tokens (16 + 8 + 8 heads, K and V to the cache) 99 us, 6.1 TB/s;
// the same with an e4m3 cache 133 us, 4.1 TB/s (a division per element and 8-byte
// stores of the keys).
// The next token of one request is a launch, 1.9 us.
//
// One thread takes 16 elements of a row as two 16-byte chunks: for rotated
// dimensions the chunks that hold 8 whole pairs (8 a's and the 8 b's half a
// rotation away, or 8 interleaved pairs side by side), so that the 8 cosines
// and 8 sines of a chunk are the same two aligned reads in both orders.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "dependent_launch.cuh"
#include "internal.h"
#include "sm103_ptx.cuh"

namespace splash {
namespace {

struct View {
  char *ptr;  // bytes
  int64_t b, h, l;  // byte strides
};

struct Cache {
  char *ptr;
  int64_t page, head, token;  // byte strides
};

struct Params {
  View q, q_out, k, k_out, v;
  Cache kc, vc;
  const float *k_scale, *v_scale;
  const int32_t *block_table, *positions, *seq_ids;
  int64_t block_table_stride, positions_stride, seq_ids_stride;
  const float *table;
  int64_t table_rows;
  int64_t num_pages;
  int32_t L, tokens, Hq, Hkv, heads;  // tokens = B * L; heads = rows per token (q, then k, then v)
  int32_t num_seqs, max_pages, page_shift;
  int32_t units, units_qk, units_v;  // threads per row: the larger, q / k, v
  int32_t rot, rot_offset;
  float sign;  // of the sines: -1 for the gradient
  uint32_t *err;
};

// Element offsets of a thread's two chunks in its row.
struct Chunks {
  int32_t c0, c1, pair;  // pair: index of the first cosine, -1 when the chunks are copied
};

template <bool INTERLEAVED>
__device__ __forceinline__ Chunks chunks_of(const Params &p, int u) {
  Chunks c;
  const int nrot = p.rot / 16;
  if (u < nrot) {
    c.pair = 8 * u;
    c.c0 = p.rot_offset + (INTERLEAVED ? 16 * u : 8 * u);
    c.c1 = c.c0 + (INTERLEAVED ? 8 : p.rot / 2);
  } else {
    // the dimensions that are not rotated, in order, 8 at a time
    const int e = 16 * (u - nrot);
    c.pair = -1;
    c.c0 = e < p.rot_offset ? e : e + p.rot;
    c.c1 = e + 8 < p.rot_offset ? e + 8 : e + 8 + p.rot;
  }
  return c;
}

struct Data {
  uint4 x0, x1;
};

__device__ __forceinline__ Data load(const char *row, const Chunks &c) {
  return {*reinterpret_cast<const uint4 *>(row + 2 * c.c0), *reinterpret_cast<const uint4 *>(row + 2 * c.c1)};
}

__device__ __forceinline__ void unpack(uint4 x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// The 8 cosines and sines of a thread's pairs.
struct Turn {
  float c[8], s[8];
};

__device__ __forceinline__ void load_turn(const Params &p, int64_t position, int pair, Turn &t) {
  const float *row = p.table + position * p.rot + pair;
  const float4 c0 = reinterpret_cast<const float4 *>(row)[0], c1 = reinterpret_cast<const float4 *>(row)[1];
  const float *srow = row + p.rot / 2;
  const float4 s0 = reinterpret_cast<const float4 *>(srow)[0], s1 = reinterpret_cast<const float4 *>(srow)[1];
  const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.c[i] = c[i];
    t.s[i] = p.sign * s[i];
  }
}

// y = the 16 elements in fp32, turned.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn(float (&y0)[8], float (&y1)[8], const Turn &t) {
  if (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = y0[2 * i], b = y0[2 * i + 1], d = y1[2 * i], e = y1[2 * i + 1];
      y0[2 * i] = a * t.c[i] - b * t.s[i];
      y0[2 * i + 1] = b * t.c[i] + a * t.s[i];
      y1[2 * i] = d * t.c[i + 4] - e * t.s[i + 4];
      y1[2 * i + 1] = e * t.c[i + 4] + d * t.s[i + 4];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = y0[i], b = y1[i];
      y0[i] = a * t.c[i] - b * t.s[i];
      y1[i] = b * t.c[i] + a * t.s[i];
    }
  }
}

// 8 values divided by the scale and rounded to e4m3 (nearest even, saturated;
// NaN stays NaN).  The division is the IEEE one: the stored value is the
// rounding of x / scale, not of x times a rounded reciprocal.
__device__ __forceinline__ uint2 to_e4m3(const float (&f)[8], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(f[4 * i], scale), __fdiv_rn(f[4 * i + 1], scale)), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(f[4 * i + 2], scale), __fdiv_rn(f[4 * i + 3], scale)), __NV_SATFINITE, __NV_E4M3);
    w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

// Block (units, tokens per block); grid.x over tokens, grid.y over groups of
// HEADS of a token's rows (q heads, k heads and with APPEND v heads).  All of
// a thread's rows are loaded before anything else: the reads of the data do
// not wait for those of the position and of the rotation, and HEADS rows use
// one rotation.
template <bool INTERLEAVED, bool APPEND, bool E4M3, int HEADS>
__global__ void __launch_bounds__(128) rope_kernel(const Params p) {
  grid_dependency();
  const int u = threadIdx.x;
  const int64_t token = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (token >= p.tokens) return;
  const int b = (int)(token / p.L), l = (int)(token - (int64_t)b * p.L);
  const int h0 = blockIdx.y * HEADS;
  const Chunks c = chunks_of<INTERLEAVED>(p, u), cv = {16 * u, 16 * u + 8, -1};
  Data x[HEADS];
  float scale[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = h0 + i;
    if (APPEND && E4M3 && h >= p.Hq && h < p.heads)
      scale[i] = h < p.Hq + p.Hkv ? p.k_scale[h - p.Hq] : p.v_scale[h - p.Hq - p.Hkv];
    if (h < p.Hq + p.Hkv) {
      const View &in = h < p.Hq ? p.q : p.k;
      if (u < p.units_qk) x[i] = load(in.ptr + b * in.b + (h < p.Hq ? h : h - p.Hq) * in.h + l * in.l, c);
    } else if (APPEND && h < p.heads && u < p.units_v) {
      x[i] = load(p.v.ptr + b * p.v.b + (h - p.Hq - p.Hkv) * p.v.h + l * p.v.l, cv);
    }
  }
  const int64_t pos = p.positions[b * p.positions_stride + l];
  bool bad = false;
  bool rotate = p.table != nullptr && pos >= 0;
  if (rotate && pos >= p.table_rows) rotate = false, bad = true;
  int64_t page = -1;
  if (APPEND && pos >= 0) {
    const int64_t seq = p.seq_ids != nullptr ? p.seq_ids[b * p.seq_ids_stride + l] : b;
    const int64_t col = pos >> p.page_shift;
    if (seq >= 0 && seq < p.num_seqs && col < p.max_pages && !bad) {
      page = p.block_table[seq * p.block_table_stride + col];
      if (page < 0 || page >= p.num_pages) page = -1;
    }
    bad = bad || page < 0;
  }
  if (bad && u == 0 && h0 == 0) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
  rotate = rotate && c.pair >= 0;
  Turn t;
  if (rotate) load_turn(p, pos, c.pair, t);
  const int64_t slot = APPEND ? pos & (((int64_t)1 << p.page_shift) - 1) : 0;

#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = h0 + i;
    if (h < p.Hq + p.Hkv) {
      if (u >= p.units_qk) continue;
      const bool is_q = h < p.Hq;
      const View &out = is_q ? p.q_out : p.k_out;
      const int hh = is_q ? h : h - p.Hq;
      uint4 o0 = x[i].x0, o1 = x[i].x1;
      float y0[8], y1[8];
      if (rotate || (APPEND && E4M3)) {
        unpack(o0, y0);
        unpack(o1, y1);
      }
      if (rotate) {
        turn<INTERLEAVED>(y0, y1, t);
        o0 = pack(y0);
        o1 = pack(y1);
      }
      if (!APPEND || out.ptr != nullptr) {
        char *row = out.ptr + b * out.b + hh * out.h + l * out.l;
        *reinterpret_cast<uint4 *>(row + 2 * c.c0) = o0;
        *reinterpret_cast<uint4 *>(row + 2 * c.c1) = o1;
      }
      if (APPEND && !is_q && page >= 0) {
        char *row = p.kc.ptr + page * p.kc.page + hh * p.kc.head + slot * p.kc.token;
        if (E4M3) {
          *reinterpret_cast<uint2 *>(row + c.c0) = to_e4m3(y0, scale[i]);
          *reinterpret_cast<uint2 *>(row + c.c1) = to_e4m3(y1, scale[i]);
        } else {
          *reinterpret_cast<uint4 *>(row + 2 * c.c0) = o0;
          *reinterpret_cast<uint4 *>(row + 2 * c.c1) = o1;
        }
      }
    } else if (APPEND && h < p.heads && u < p.units_v && page >= 0) {
      const int hh = h - p.Hq - p.Hkv;
      char *row = p.vc.ptr + page * p.vc.page + hh * p.vc.head + slot * p.vc.token;
      if (E4M3) {
        float y0[8], y1[8];
        unpack(x[i].x0, y0);
        unpack(x[i].x1, y1);
        const uint2 e0 = to_e4m3(y0, scale[i]), e1 = to_e4m3(y1, scale[i]);
        *reinterpret_cast<uint4 *>(row + 16 * u) = make_uint4(e0.x, e0.y, e1.x, e1.y);
      } else {
        *reinterpret_cast<uint4 *>(row + 2 * cv.c0) = x[i].x0;
        *reinterpret_cast<uint4 *>(row + 2 * cv.c1) = x[i].x1;
      }
    }
  }
}

View view(const splash_view &v) { return {static_cast<char *>(v.ptr), 2 * v.stride_b, 2 * v.stride_h, 2 * v.stride_l}; }

Cache cache(const splash_cache_view &v, int64_t size) {
  return {static_cast<char *>(v.ptr), size * v.stride_page, size * v.stride_head, size * v.stride_token};
}

template <bool APPEND, bool E4M3, int HEADS>
splash_status launch_heads(const Params &p, bool interleaved, cudaStream_t stream) {
  // 128 threads: a packed prompt of 32768 tokens 98 us, against 104 with 256 and 133 with 64
  const int ty = std::max(1, 128 / p.units);
  // (a call may have 2^31 - 1 tokens: adding to that would overflow)
  const dim3 block(p.units, ty), grid((p.tokens - 1) / ty + 1, (p.heads + HEADS - 1) / HEADS);
  SPLASH_CUDA_TRY(launch_dependent(interleaved ? rope_kernel<true, APPEND, E4M3, HEADS> : rope_kernel<false, APPEND, E4M3, HEADS>,
                                   grid, block, 0, 1, stream, p));
  splash_count_launches(1);
  return SPLASH_OK;
}

template <bool APPEND, bool E4M3>
splash_status launch(const Params &p, bool interleaved, cudaStream_t stream) {
  // Four rows per thread where that still gives every SM 1024 threads (152 x
  // 1024): q and k of 2 x 4096 tokens 27.8 us against 28.3 with one row, 128
  // heads of 192 dimensions 117.6 against 129 (fewer reads of the rotations per
  // row); 257 tokens of 4 heads 2.2 against 1.7 us.  Appending always takes
  // one: a prompt of 32768 tokens 99.2 us against 98.0 with four, the next token
  // of 256 requests 3.0 against 5.1.
  if constexpr (!APPEND) {
    if ((int64_t)p.tokens * p.units * ((p.heads + 3) / 4) >= 152 * 1024)
      return launch_heads<APPEND, E4M3, 4>(p, interleaved, stream);
  }
  return launch_heads<APPEND, E4M3, 1>(p, interleaved, stream);
}

}  // namespace
}  // namespace splash

splash_status splash_rope_launch(const splash_rope_args &a, cudaStream_t stream, uint32_t *err_word) {
  using namespace splash;
  Params p = {};
  p.q = view(a.q);
  p.q_out = view(a.q_out);
  p.k = view(a.k);
  p.k_out = view(a.k_out);
  p.positions = a.positions;
  p.positions_stride = a.positions_stride_b;
  p.table = a.table;
  p.table_rows = a.table_rows;
  p.L = (int32_t)a.L;
  p.tokens = (int32_t)(a.B * a.L);
  p.Hq = a.Hq;
  p.Hkv = a.k.ptr != nullptr ? a.Hkv : 0;
  p.heads = p.Hq + p.Hkv;
  p.units = p.units_qk = a.d / 16;
  p.rot = a.rot_dim;
  p.rot_offset = a.rot_offset;
  p.sign = a.inverse ? -1.f : 1.f;
  p.err = err_word;
  return launch<false, false>(p, a.interleaved != 0, stream);
}

splash_status splash_paged_append_launch(const splash_paged_append_args &a, cudaStream_t stream, uint32_t *err_word) {
  using namespace splash;
  const bool e4m3 = a.cache_type == SPLASH_CACHE_E4M3;
  Params p = {};
  p.q = view(a.q);
  p.q_out = view(a.q_out);
  p.k = view(a.k);
  p.k_out = view(a.k_out);
  p.v = view(a.v);
  p.kc = cache(a.k_cache, e4m3 ? 1 : 2);
  p.vc = cache(a.v_cache, e4m3 ? 1 : 2);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.block_table = a.block_table;
  p.block_table_stride = a.block_table_stride;
  p.positions = a.positions;
  p.positions_stride = a.positions_stride_b;
  p.seq_ids = a.seq_ids;
  p.seq_ids_stride = a.seq_ids_stride_b;
  p.table = a.table;
  p.table_rows = a.table_rows;
  p.num_pages = a.num_pages;
  p.L = (int32_t)a.L;
  p.tokens = (int32_t)(a.B * a.L);
  p.Hq = a.q.ptr != nullptr ? a.Hq : 0;
  p.Hkv = a.Hkv;
  p.heads = p.Hq + 2 * p.Hkv;
  p.num_seqs = a.num_seqs;
  p.max_pages = a.max_pages;
  p.page_shift = __builtin_ctz((unsigned)a.page_size);
  p.units_qk = a.dqk / 16;
  p.units_v = a.dv / 16;
  p.units = std::max(p.units_qk, p.units_v);
  p.rot = a.table != nullptr ? a.rot_dim : 0;
  p.rot_offset = a.table != nullptr ? a.rot_offset : 0;
  p.sign = 1.f;
  p.err = err_word;
  const bool inter = a.table != nullptr && a.interleaved != 0;
  return e4m3 ? launch<true, true>(p, inter, stream) : launch<true, false>(p, inter, stream);
}
