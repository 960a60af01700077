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
#include <cmath>

#include "dependent_launch.cuh"
#include "internal.h"
#include "sm103_ptx.cuh"

namespace splash {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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
  int64_t num_pages;
  int32_t B, Hq, Hkv, T, G, dqk, dv, max_pages, page_shift, window;  // window < 0: none
  float scale, cap;                                                 // cap <= 0: none
  uint32_t *err;
};

// A token's place in its tree: which tokens it sees (itself among them), and
// its depth; seen = 0 for padding.
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

// One warp per row: 32 keys at a time, a lane per key for the scores, then a
// lane per column for the values.
template <bool E4M3>
__global__ void __launch_bounds__(128) tree_decode_kernel(const Params p) {
  __shared__ float s_q[4][192];
  grid_dependency();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 4 + warp;  // (b, h, l)
  if (row >= (int64_t)p.B * p.Hq * p.T) return;
  const int l = (int)(row % p.T), h = (int)(row / p.T % p.Hq), b = (int)(row / p.T / p.Hq), g = h / p.G;
  bool bad = false;
  const int64_t most = (int64_t)p.max_pages << p.page_shift;
  const int32_t given = p.seq_lens[b];
  const int32_t n = given < 0 ? 0 : given > most ? (int32_t)most : given;
  bad |= n != given;
  const int ctx = n - p.T;
  const Branch me = branch_of(p.parents + b * p.parents_stride, l, max(0, -ctx), p.window, &bad);
  const char *q = p.q + b * p.q_b + h * p.q_h + l * p.q_l;
  for (int i = lane; i < p.dqk; i += 32) s_q[warp][i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(q)[i]);
  __syncwarp();
  const float ks = E4M3 ? p.k_scale[g] : 1.f, vs = E4M3 ? p.v_scale[g] : 1.f;
  const int64_t pos = (int64_t)ctx + me.depth;
  const int lo = p.window < 0 ? 0 : (int)max((int64_t)0, min((int64_t)ctx, pos - p.window));
  float m = -INFINITY, sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  auto value = [](const char *row, int i) {
    return E4M3 ? (float)reinterpret_cast<const __nv_fp8_e4m3 *>(row)[i]
                : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row)[i]);
  };
  for (int j0 = lo & ~31; j0 < n && me.seen != 0; j0 += 32) {
    const int j = j0 + lane;
    bool see = j < n && (j < ctx ? j >= lo : (me.seen >> (j - ctx) & 1u) != 0);
    int64_t page = 0;
    bool there = true;
    float s = -INFINITY;
    if (see) {
      page = p.block_table[b * p.block_table_stride + (j >> p.page_shift)];
      there = page >= 0 && page < p.num_pages;
      bad |= !there;
      s = 0.f;
      if (there) {
        const char *k = p.k + page * p.k_page + g * p.k_head + (j & ((1 << p.page_shift) - 1)) * p.k_token;
        for (int i = 0; i < p.dqk; ++i) s += s_q[warp][i] * value(k, i);
      }
      s *= p.scale * ks;
      if (p.cap > 0.f) s = p.cap * tanhf(s / p.cap);
      s *= kLog2e;
    }
    float top = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
    top = fmaxf(top, m);
    if (top == -INFINITY && !__any_sync(~0u, see)) continue;
    const float ref = top == -INFINITY ? 0.f : top, f = exp2f(m - ref);
    m = top;
    const float e = see ? exp2f(s - ref) : 0.f;
    float all = e;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) all += __shfl_xor_sync(~0u, all, x);
    sum = sum * f + all;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= f;
    const uint32_t seen = __ballot_sync(~0u, see && there);
    for (int k = 0; k < 32; ++k) {
      const float ek = __shfl_sync(~0u, e, k);
      const int64_t pk = __shfl_sync(~0u, page, k);
      if ((seen >> k & 1u) == 0) continue;
      const char *v = p.v + pk * p.v_page + g * p.v_head + ((j0 + k) & ((1 << p.page_shift) - 1)) * p.v_token;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (32 * i + lane < p.dv) o[i] += ek * value(v, 32 * i + lane);
    }
  }
  const bool empty = sum == 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (32 * i + lane < p.dv) p.out[row * p.dv + 32 * i + lane] = __float2bfloat16(empty ? 0.f : o[i] * vs / sum);
  if (lane == 0) p.lse[row] = empty ? -INFINITY : (m + log2f(sum)) * kLn2;
  if (bad) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
}

}  // namespace
}  // namespace splash

size_t splash_paged_tree_decode_workspace_bytes(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t,
                                                int64_t) {
  return 0;
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
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.block_table = a.block_table;
  p.block_table_stride = a.block_table_stride;
  p.seq_lens = a.seq_lens;
  p.parents = args.parents;
  p.parents_stride = args.parents_stride_b;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  p.num_pages = a.num_pages;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.T = a.Lq;
  p.G = a.Hq / a.Hkv;
  p.dqk = a.dqk;
  p.dv = a.dv;
  p.max_pages = a.max_pages;
  p.page_shift = __builtin_ctz((unsigned)a.page_size);
  // (differences of positions stay below 2^31 - 64)
  p.window = a.window_left < 0 ? -1 : (int32_t)std::min<int64_t>(a.window_left, INT32_MAX - 64);
  p.scale = a.scale;
  p.cap = a.softcap < 0x1p100f ? a.softcap : 0.f;
  p.err = err_word;
  const dim3 grid((unsigned)(((int64_t)a.B * a.Hq * a.Lq + 3) / 4));
  SPLASH_CUDA_TRY(launch_dependent(size == 1 ? tree_decode_kernel<true> : tree_decode_kernel<false>, grid, dim3(128), 0, 1, stream, p));
  splash_count_launches(1);
  return SPLASH_OK;
}
