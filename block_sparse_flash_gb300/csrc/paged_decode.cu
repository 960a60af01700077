// paged_decode.cu -- attention of new tokens over a paged key/value cache
// (splash_paged_decode in splash.h).
//
// For a query row: s_j = scale q.k_j, m = max s_j, l = sum exp(s_j - m),
// out = sum exp(s_j - m) v_j / l, lse = m + ln l, in one pass over the keys
// with the running maximum and sum in fp32.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "sm103_ptx.cuh"

namespace splash {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <bool E4M3>
__device__ __forceinline__ float element(const char *row, int i) {
  if (E4M3) {
    __nv_fp8_e4m3 x;
    x.__x = static_cast<__nv_fp8_storage_t>(row[i]);
    return static_cast<float>(x);
  }
  return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row)[i]);
}

// One CTA per query row: 128 keys at a time, one thread per key for the
// scores, one thread per output column for the values.
template <int DQK, int DV, bool E4M3>
__global__ void __launch_bounds__(128) paged_decode_kernel(const splash_paged_decode_args a, int page_shift, uint32_t *err) {
  __shared__ float q[DQK], prob[128], red[4];
  __shared__ const char *vrow[128];
  const int h = blockIdx.x / a.Lq, l = blockIdx.x % a.Lq, b = blockIdx.y, t = threadIdx.x;
  const int g = h / (a.Hq / a.Hkv);
  const int size = E4M3 ? 1 : 2;
  int64_t n = a.seq_lens[b];
  const int64_t most = (int64_t)a.max_pages << page_shift;
  if (n < 0 || n > most) {
    if (t == 0) atomicOr(err, SPLASH_DEV_BAD_TABLE);
    n = n < 0 ? 0 : most;
  }
  const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q.ptr) + b * a.q.stride_b + h * a.q.stride_h + l * a.q.stride_l;
  for (int i = t; i < DQK; i += 128) q[i] = __bfloat162float(qp[i]);
  __syncthreads();
  const int64_t p = n - a.Lq + l;
  const int64_t lo = a.window_left < 0 ? 0 : max((int64_t)0, p - a.window_left);
  float m = -INFINITY, sum = 0.f, acc = 0.f;
  const float factor = a.scale * (E4M3 ? a.k_scale[g] : 1.f);
  for (int64_t j0 = lo; j0 <= p; j0 += 128) {
    const int64_t j = j0 + t;
    float s = -INFINITY;
    vrow[t] = nullptr;
    if (j <= p) {
      const int64_t page = a.block_table[b * a.block_table_stride + (j >> page_shift)];
      s = 0.f;
      if (page < 0 || page >= a.num_pages) {
        atomicOr(err, SPLASH_DEV_BAD_TABLE);
      } else {
        const int64_t slot = j & ((1 << page_shift) - 1);
        const char *k = static_cast<const char *>(a.k_cache.ptr) +
                        size * (page * a.k_cache.stride_page + g * a.k_cache.stride_head + slot * a.k_cache.stride_token);
        vrow[t] = static_cast<const char *>(a.v_cache.ptr) +
                  size * (page * a.v_cache.stride_page + g * a.v_cache.stride_head + slot * a.v_cache.stride_token);
        for (int i = 0; i < DQK; ++i) s += q[i] * element<E4M3>(k, i);
      }
      s *= factor;
      if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
    }
    float top = s;
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
    if ((t & 31) == 0) red[t >> 5] = top;
    __syncthreads();
    const float m_new = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float ref = m_new == -INFINITY ? 0.f : m_new;
    prob[t] = exp2f((s - ref) * kLog2e);
    __syncthreads();
    const float alpha = exp2f((m - ref) * kLog2e);
    sum *= alpha;
    acc *= alpha;
    m = m_new;
    for (int x = 0; x < 128; ++x) {
      sum += prob[x];
      if (t < DV && vrow[x] != nullptr) acc += prob[x] * element<E4M3>(vrow[x], t);
    }
    __syncthreads();
  }
  const int64_t row = ((int64_t)b * a.Hq + h) * a.Lq + l;
  const float vs = E4M3 ? a.v_scale[g] : 1.f;
  if (t < DV) static_cast<__nv_bfloat16 *>(a.out)[row * DV + t] = __float2bfloat16(sum > 0.f ? acc / sum * vs : 0.f);
  if (t == 0) a.lse[row] = sum > 0.f ? m + kLn2 * log2f(sum) : -INFINITY;
}

template <int DQK, int DV>
splash_status launch(const splash_paged_decode_args &a, cudaStream_t stream, uint32_t *err) {
  const dim3 grid(a.Hq * a.Lq, a.B);
  const int shift = __builtin_ctz((unsigned)a.page_size);
  if (a.cache_type == SPLASH_CACHE_E4M3)
    paged_decode_kernel<DQK, DV, true><<<grid, 128, 0, stream>>>(a, shift, err);
  else
    paged_decode_kernel<DQK, DV, false><<<grid, 128, 0, stream>>>(a, shift, err);
  SPLASH_CUDA_TRY(cudaGetLastError());
  splash_count_launches(1);
  return SPLASH_OK;
}

}  // namespace
}  // namespace splash

size_t splash_paged_decode_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t Lq, int32_t dv) {
  (void)B, (void)Hq, (void)Hkv, (void)Lq, (void)dv;
  return 16;
}

splash_status splash_paged_decode_launch(const splash_paged_decode_args &a, cudaStream_t stream, uint32_t *err_word) {
  using namespace splash;
  if (a.dqk == 64) return launch<64, 64>(a, stream, err_word);
  if (a.dqk == 128) return launch<128, 128>(a, stream, err_word);
  return launch<192, 128>(a, stream, err_word);
}
