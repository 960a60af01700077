// api.cu -- the extern "C" boundary of libsplash.so (declared in splash.h):
// argument validation, MaskInfo handles, the device error word.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include "internal.h"

namespace {

// The device error word: kernels atomicOr error bits into it.  One copy per
// device (a __device__ variable); host code reaches it through
// cudaGetSymbolAddress, resolved once per device.
__device__ uint32_t g_error_word;

constexpr int kMaxDevices = 64;
uint32_t *g_error_addr[kMaxDevices];
std::mutex g_error_mu;

bool valid_block(int32_t b) { return b == 64 || b == 128; }
// query blocks may also be 256 rows tall (two 128-row tiles of one head)
bool valid_q_block(int32_t b) { return valid_block(b) || b == 256; }

splash_status check_spec(const splash_mask_spec *spec, int64_t Lq, int64_t Lk) {
  if (spec == nullptr) return SPLASH_ERR_INVALID_ARG;
  if (spec->causal != 0 && spec->causal != 1) return SPLASH_ERR_INVALID_ARG;
  if (spec->window_left < -1 || spec->window_right < -1) return SPLASH_ERR_INVALID_ARG;
  if (spec->q_segment_ids != nullptr) {
    if (spec->batch <= 0) return SPLASH_ERR_INVALID_ARG;
    if (spec->kv_segment_ids == nullptr && Lq != Lk) return SPLASH_ERR_SHAPE;
  } else if (spec->kv_segment_ids != nullptr) {
    return SPLASH_ERR_INVALID_ARG;
  }
  return SPLASH_OK;
}

splash_status check_geometry(int64_t Lq, int64_t Lk, int32_t bq, int32_t bk) {
  if (Lq <= 0 || Lk <= 0 || bq <= 0 || bk <= 0) return SPLASH_ERR_INVALID_ARG;
  if (!valid_q_block(bq) || !valid_block(bk)) return SPLASH_ERR_UNSUPPORTED;
  // ragged lengths are padded to whole blocks (the padding is masked)
  if ((Lq + bq - 1) / bq > 65535 || Lk > (int64_t)1 << 30 || Lq > (int64_t)1 << 30) return SPLASH_ERR_UNSUPPORTED;
  return SPLASH_OK;
}

}  // namespace

// Item order across heads.  The static schedule deals the items in rounds of
// `grid` (one per CTA), rows longest first, every head (pair) of a row
// together.  When rows reach across the keys (no window, no segments) and the
// K / V of all heads is larger than L2 can keep (budget 64 MB, about half of
// the 129 MB: each die has its own half), the CTAs of a round would stream it
// from DRAM for every row.  Then the items are ordered
// by groups of head_group heads whose K / V fits the budget, and among the
// group sizes from half that bound up to it, the one whose group fills whole
// rounds best (the fewest items left in a partial round; a group that ends
// mid-round leaves that round unbalanced).  Measured on the wide-head causal
// MHA workload (128 heads, K / V 335 MB): 19 heads per group (two whole
// rounds of 152) 0.468 ms, 32 heads 0.489 ms, all 128 heads 0.556 ms.
// (Windowed and document rows read short, overlapping key ranges; there the
// row-major order already keeps the K / V in L2, and grouping was measured a
// few per cent slower.)
int32_t splash_choose_head_group(bool dense_rows, int64_t items_per_head, int32_t npairs, int64_t kv_bytes, int64_t grid) {
  constexpr int64_t kBudget = 64ll << 20;
  if (!dense_rows || npairs <= 1 || kv_bytes <= kBudget) return npairs;
  const int32_t cap = std::max<int32_t>(1, (int32_t)((int64_t)npairs * kBudget / kv_bytes));
  int32_t best = cap;
  int64_t best_rem = LLONG_MAX;
  for (int32_t h = cap; h >= std::max<int32_t>(1, cap / 2); --h) {
    const int64_t rem = (items_per_head * h) % grid;
    if (rem < best_rem) {
      best_rem = rem;
      best = h;
      if (rem == 0) break;
    }
  }
  return best;
}

static std::atomic<uint64_t> g_launches{0};

void splash_count_launches(uint64_t n) { g_launches.fetch_add(n, std::memory_order_relaxed); }

uint32_t *splash_device_error_word(int device) {
  if (device < 0 || device >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_error_mu);
  if (g_error_addr[device] == nullptr) {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_error_word) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    g_error_addr[device] = static_cast<uint32_t *>(p);
  }
  return g_error_addr[device];
}

extern "C" {

const char *splash_status_string(splash_status s) {
  switch (s) {
    case SPLASH_OK: return "SPLASH_OK";
    case SPLASH_ERR_INVALID_ARG: return "SPLASH_ERR_INVALID_ARG: invalid argument";
    case SPLASH_ERR_SHAPE: return "SPLASH_ERR_SHAPE: inconsistent shapes";
    case SPLASH_ERR_UNSUPPORTED: return "SPLASH_ERR_UNSUPPORTED: shape or block size not supported by this build";
    case SPLASH_ERR_CUDA: return "SPLASH_ERR_CUDA: a CUDA call failed";
    case SPLASH_ERR_DEVICE_TIMEOUT: return "SPLASH_ERR_DEVICE_TIMEOUT: a kernel's bounded wait ran out";
    case SPLASH_ERR_OOM: return "SPLASH_ERR_OOM: device allocation failed";
    case SPLASH_ERR_DEVICE_CHECK: return "SPLASH_ERR_DEVICE_CHECK: a kernel rejected a table entry";
  }
  return "SPLASH_ERR_UNKNOWN";
}

const char *splash_version(void) { return "splash-gb300 0.1 sm_103a"; }

uint64_t splash_kernel_launches(void) { return g_launches.load(std::memory_order_relaxed); }

int32_t splash_schedule_head_group(int32_t dense_rows, int64_t items_per_head, int32_t npairs, int64_t kv_bytes,
                                   int64_t grid) {
  if (npairs < 1 || items_per_head < 1 || grid < 1 || kv_bytes < 0) return 0;
  return splash_choose_head_group(dense_rows != 0, items_per_head, npairs, kv_bytes, grid);
}

splash_status splash_shard_items(int32_t B, int32_t Hkv, int32_t world, int32_t rank, int64_t *begin,
                                int64_t *end) {
  if (begin == nullptr || end == nullptr) return SPLASH_ERR_INVALID_ARG;
  if (B <= 0 || Hkv <= 0 || world <= 0 || rank < 0 || rank >= world) return SPLASH_ERR_INVALID_ARG;
  // balanced contiguous ranges: rank r takes [floor(n r / G), floor(n (r+1) / G))
  const int64_t n = (int64_t)B * Hkv;
  *begin = n * rank / world;
  *end = n * (rank + 1) / world;
  return SPLASH_OK;
}

splash_status splash_mask_info_rebuild(splash_mask_info *mi, const splash_mask_spec *spec, int64_t Lq,
                                       int64_t Lk, int32_t bq, int32_t bk, void *cuda_stream) {
  if (mi == nullptr) return SPLASH_ERR_INVALID_ARG;
  splash_status st = check_spec(spec, Lq, Lk);
  if (st != SPLASH_OK) return st;
  if ((st = check_geometry(Lq, Lk, bq, bk)) != SPLASH_OK) return st;
  int dev = 0;
  SPLASH_CUDA_TRY(cudaGetDevice(&dev));
  if (mi->device >= 0 && mi->device != dev) return SPLASH_ERR_INVALID_ARG;
  mi->device = dev;
  st = splash_mask_info_build_into(mi, spec, Lq, Lk, bq, bk, static_cast<cudaStream_t>(cuda_stream));
  if (st != SPLASH_OK) {
    mi->num_active = mi->num_partial = mi->num_patterns = mi->allowed_pairs = 0;
    mi->nq = mi->nk = 0;
  }
  return st;
}

splash_status splash_build_mask_info(const splash_mask_spec *spec, int64_t Lq, int64_t Lk, int32_t bq,
                                     int32_t bk, void *cuda_stream, splash_mask_info **out) {
  if (out == nullptr) return SPLASH_ERR_INVALID_ARG;
  *out = nullptr;
  splash_status st = check_spec(spec, Lq, Lk);
  if (st != SPLASH_OK) return st;
  if ((st = check_geometry(Lq, Lk, bq, bk)) != SPLASH_OK) return st;
  splash_mask_info *mi = new (std::nothrow) splash_mask_info();
  if (mi == nullptr) return SPLASH_ERR_OOM;
  st = splash_mask_info_rebuild(mi, spec, Lq, Lk, bq, bk, cuda_stream);
  if (st != SPLASH_OK) {
    splash_mask_info_free_buffers(mi);
    delete mi;
    return st;
  }
  *out = mi;
  return SPLASH_OK;
}

splash_status splash_mask_info_shape(const splash_mask_info *mi, int32_t *batch_rows, int64_t *nq,
                                     int64_t *nk, int32_t *bq, int32_t *bk) {
  if (mi == nullptr) return SPLASH_ERR_INVALID_ARG;
  if (batch_rows) *batch_rows = mi->batch_rows;
  if (nq) *nq = mi->nq;
  if (nk) *nk = mi->nk;
  if (bq) *bq = mi->bq;
  if (bk) *bk = mi->bk;
  return SPLASH_OK;
}

splash_status splash_mask_info_counts(const splash_mask_info *mi, int64_t *num_active, int64_t *num_partial,
                                      int64_t *num_patterns, int64_t *allowed_pairs) {
  if (mi == nullptr) return SPLASH_ERR_INVALID_ARG;
  const splash_status st = splash_mask_info_sync_counts(const_cast<splash_mask_info *>(mi));
  if (st != SPLASH_OK) return st;
  if (num_active) *num_active = mi->num_active;
  if (num_partial) *num_partial = mi->num_partial;
  if (num_patterns) *num_patterns = mi->num_patterns;
  if (allowed_pairs) *allowed_pairs = mi->allowed_pairs;
  return SPLASH_OK;
}

splash_status splash_mask_info_set_pattern_source(splash_mask_info *mi, int32_t source) {
  if (mi == nullptr || (source != SPLASH_PATTERNS_STORED && source != SPLASH_PATTERNS_FROM_POSITIONS))
    return SPLASH_ERR_INVALID_ARG;
  mi->patterns_from_positions = source == SPLASH_PATTERNS_FROM_POSITIONS ? 1 : 0;
  return SPLASH_OK;
}

splash_status splash_mask_info_to_host(const splash_mask_info *mi, int8_t *block_mask, int32_t *row_ptr,
                                       int32_t *active_rows, int32_t *active_cols, int32_t *mask_next,
                                       uint8_t *bounds_start, uint8_t *bounds_end,
                                       uint8_t *partial_mask_blocks) {
  if (mi == nullptr || mi->nq <= 0) return SPLASH_ERR_INVALID_ARG;
  const splash_status st = splash_mask_info_sync_counts(const_cast<splash_mask_info *>(mi));
  if (st != SPLASH_OK) return st;
  const int64_t R = (int64_t)mi->batch_rows * mi->nq, A = mi->num_active;
  const int64_t P = mi->num_patterns;
  if (block_mask) SPLASH_CUDA_TRY(cudaMemcpy(block_mask, mi->block_mask, R * mi->nk, cudaMemcpyDeviceToHost));
  if (row_ptr) SPLASH_CUDA_TRY(cudaMemcpy(row_ptr, mi->row_ptr, 4 * (R + 1), cudaMemcpyDeviceToHost));
  if (A > 0) {
    if (active_rows) SPLASH_CUDA_TRY(cudaMemcpy(active_rows, mi->active_rows, 4 * A, cudaMemcpyDeviceToHost));
    if (active_cols) SPLASH_CUDA_TRY(cudaMemcpy(active_cols, mi->active_cols, 4 * A, cudaMemcpyDeviceToHost));
    if (mask_next) SPLASH_CUDA_TRY(cudaMemcpy(mask_next, mi->mask_next, 4 * A, cudaMemcpyDeviceToHost));
    if (bounds_start) SPLASH_CUDA_TRY(cudaMemcpy(bounds_start, mi->bounds_start, A, cudaMemcpyDeviceToHost));
    if (bounds_end) SPLASH_CUDA_TRY(cudaMemcpy(bounds_end, mi->bounds_end, A, cudaMemcpyDeviceToHost));
  }
  if (P > 0 && partial_mask_blocks) {
    // the device keeps the patterns bit-packed; expand them to one byte per element
    const int64_t words = mi->bk / 32, per = (int64_t)mi->bq * words;
    std::vector<uint32_t> bits((size_t)(P * per));
    SPLASH_CUDA_TRY(cudaMemcpy(bits.data(), mi->pattern_bits, bits.size() * sizeof(uint32_t), cudaMemcpyDeviceToHost));
    for (int64_t x = 0; x < P * mi->bq; ++x)
      for (int64_t j = 0; j < mi->bk; ++j)
        partial_mask_blocks[x * mi->bk + j] = (uint8_t)((bits[(size_t)(x * words + j / 32)] >> (j % 32)) & 1u);
  }
  return SPLASH_OK;
}

void splash_mask_info_destroy(splash_mask_info *mi) {
  if (mi == nullptr) return;
  splash_mask_info_free_buffers(mi);
  delete mi;
}

namespace {

// Argument checks shared by the attention entry points; on success *err is
// the device's error word.
splash_status check_attention(const void *q, const void *k, const void *v, int32_t B, int32_t Hq, int32_t Hkv,
                              int64_t Lq, int64_t Lk, int32_t dqk, int32_t dv, const splash_mask_info *mi,
                              float scale, float softcap, const void *out, const void *lse, uint32_t **err) {
  if (q == nullptr || k == nullptr || v == nullptr || out == nullptr || lse == nullptr || mi == nullptr)
    return SPLASH_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Lq <= 0 || Lk <= 0 || dqk <= 0 || dv <= 0)
    return SPLASH_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < INFINITY) || !(softcap == softcap) || softcap == INFINITY)
    return SPLASH_ERR_INVALID_ARG;  // scale must be positive and finite; NaN / inf cap rejected
  if (Hq % Hkv != 0) return SPLASH_ERR_SHAPE;
  if (mi->nq <= 0 || mi->Lq != Lq || mi->Lk != Lk) return SPLASH_ERR_SHAPE;
  if (mi->batch_rows != 1 && mi->batch_rows != B) return SPLASH_ERR_SHAPE;
  const uintptr_t mis = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
                        reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(out);
  if (mis & 15u) return SPLASH_ERR_INVALID_ARG;
  const bool shape_ok = ((dqk == 128 && dv == 128) || (dqk == 192 && dv == 128) || (dqk == 64 && dv == 64)) &&
                        (mi->bq == mi->bk || (mi->bq == 256 && mi->bk == 128));
  if (!shape_ok) return SPLASH_ERR_UNSUPPORTED;
  if (mi->bk == 64 && dqk == 192) return SPLASH_ERR_UNSUPPORTED;
  if ((int64_t)B * Hq * Lq >= ((int64_t)1 << 31) || (int64_t)B * Hkv * Lk >= ((int64_t)1 << 31))
    return SPLASH_ERR_UNSUPPORTED;
  int dev = 0;
  SPLASH_CUDA_TRY(cudaGetDevice(&dev));
  if (dev != mi->device) return SPLASH_ERR_INVALID_ARG;
  *err = splash_device_error_word(dev);
  if (*err == nullptr) return SPLASH_ERR_CUDA;
  return SPLASH_OK;
}

}  // namespace

splash_status splash_attention_fwd(const void *q, const void *k, const void *v, int32_t B, int32_t Hq,
                                   int32_t Hkv, int64_t Lq, int64_t Lk, int32_t dqk, int32_t dv,
                                   const int32_t *q_segment_ids, const int32_t *kv_segment_ids,
                                   const splash_mask_info *mi, float scale, float softcap, void *out,
                                   float *lse, void *cuda_stream) {
  uint32_t *err = nullptr;
  splash_status st = check_attention(q, k, v, B, Hq, Hkv, Lq, Lk, dqk, dv, mi, scale, softcap, out, lse, &err);
  if (st != SPLASH_OK) return st;
  return splash_attention_fwd_launch(q, k, v, B, Hq, Hkv, Lq, Lk, dqk, dv, q_segment_ids, kv_segment_ids, mi, scale,
                                     softcap, NAN, out, lse, 1, nullptr, nullptr,
                                     static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_attention_fwd_mle(const void *q, const void *k, const void *v, int32_t B, int32_t Hq,
                                       int32_t Hkv, int64_t Lq, int64_t Lk, int32_t dqk, int32_t dv,
                                       const int32_t *q_segment_ids, const int32_t *kv_segment_ids,
                                       const splash_mask_info *mi, float scale, float softcap, float max_logit,
                                       void *out, float *lse, void *cuda_stream) {
  if (!std::isfinite(max_logit)) return SPLASH_ERR_INVALID_ARG;
  uint32_t *err = nullptr;
  splash_status st = check_attention(q, k, v, B, Hq, Hkv, Lq, Lk, dqk, dv, mi, scale, softcap, out, lse, &err);
  if (st != SPLASH_OK) return st;
  return splash_attention_fwd_launch(q, k, v, B, Hq, Hkv, Lq, Lk, dqk, dv, q_segment_ids, kv_segment_ids, mi, scale,
                                     softcap, max_logit, out, lse, 1, nullptr, nullptr,
                                     static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_attention_fwd_host(const void *q_host, const void *k_host, const void *v_host, int32_t B,
                                        int32_t Hq, int32_t Hkv, int64_t Lq, int64_t Lk, int32_t dqk, int32_t dv,
                                        const int32_t *q_segment_ids, const int32_t *kv_segment_ids,
                                        const splash_mask_info *mi, float scale, float softcap, void *out_host,
                                        float *lse_host, void *q_dev, void *k_dev, void *v_dev, void *out_dev,
                                        float *lse_dev, void *cuda_stream) {
  if (q_host == nullptr || k_host == nullptr || v_host == nullptr || out_host == nullptr || lse_host == nullptr)
    return SPLASH_ERR_INVALID_ARG;
  uint32_t *err = nullptr;
  splash_status st =
      check_attention(q_dev, k_dev, v_dev, B, Hq, Hkv, Lq, Lk, dqk, dv, mi, scale, softcap, out_dev, lse_dev, &err);
  if (st != SPLASH_OK) return st;
  return splash_attention_fwd_host_launch(q_host, k_host, v_host, B, Hq, Hkv, Lq, Lk, dqk, dv, q_segment_ids,
                                          kv_segment_ids, mi, scale, softcap,
                                          out_host, lse_host, q_dev, k_dev, v_dev, out_dev, lse_dev, 8,
                                          static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_attention_bwd_workspace_size(int32_t B, int32_t Hq, int64_t Lq, int32_t dqk, size_t *bytes) {
  if (bytes == nullptr || B <= 0 || Hq <= 0 || Lq <= 0 || dqk <= 0) return SPLASH_ERR_INVALID_ARG;
  *bytes = splash_attention_bwd_workspace_bytes(B, Hq, Lq, dqk);
  return SPLASH_OK;
}

splash_status splash_attention_bwd(const void *q, const void *k, const void *v, const void *out, const float *lse,
                                   const void *dout, int32_t B, int32_t Hq, int32_t Hkv, int64_t Lq, int64_t Lk,
                                   int32_t dqk, int32_t dv, const int32_t *q_segment_ids,
                                   const int32_t *kv_segment_ids, splash_mask_info *mi, float scale, float softcap,
                                   void *dq, void *dk, void *dv_out, void *workspace, size_t workspace_bytes,
                                   void *cuda_stream) {
  (void)q_segment_ids;
  (void)kv_segment_ids;
  if (dout == nullptr || dq == nullptr || dk == nullptr || dv_out == nullptr || workspace == nullptr)
    return SPLASH_ERR_INVALID_ARG;
  uint32_t *err = nullptr;
  splash_status st = check_attention(q, k, v, B, Hq, Hkv, Lq, Lk, dqk, dv, mi, scale, softcap, out, lse, &err);
  if (st != SPLASH_OK) return st;
  const uintptr_t mis = reinterpret_cast<uintptr_t>(dout) | reinterpret_cast<uintptr_t>(dq) |
                        reinterpret_cast<uintptr_t>(dk) | reinterpret_cast<uintptr_t>(dv_out) |
                        reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(workspace);
  if (mis & 15u) return SPLASH_ERR_INVALID_ARG;
  if (workspace_bytes < splash_attention_bwd_workspace_bytes(B, Hq, Lq, dqk)) return SPLASH_ERR_INVALID_ARG;
  if (dqk != dv || (dqk != 64 && dqk != 128) || (mi->bq != 128 && mi->bq != 256) || mi->bk != 128)
    return SPLASH_ERR_UNSUPPORTED;
  return splash_attention_bwd_launch(q, k, v, out, lse, dout, B, Hq, Hkv, Lq, Lk, dqk, mi, scale, softcap, dq, dk,
                                     dv_out, workspace, static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_attention_fwd_split(const void *q, const void *k, const void *v, int32_t B, int32_t Hq,
                                         int32_t Hkv, int64_t Lq, int64_t Lk, int32_t dqk, int32_t dv,
                                         const int32_t *q_segment_ids, const int32_t *kv_segment_ids,
                                         const splash_mask_info *mi, float scale, float softcap,
                                         int32_t num_splits, float *o_part, float *lse_part, void *cuda_stream) {
  if (num_splits < 1 || num_splits > SPLASH_MAX_SPLITS) return SPLASH_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(o_part) & 31u) != 0) return SPLASH_ERR_INVALID_ARG;
  uint32_t *err = nullptr;
  splash_status st =
      check_attention(q, k, v, B, Hq, Hkv, Lq, Lk, dqk, dv, mi, scale, softcap, o_part, lse_part, &err);
  if (st != SPLASH_OK) return st;
  return splash_attention_fwd_launch(q, k, v, B, Hq, Hkv, Lq, Lk, dqk, dv, q_segment_ids, kv_segment_ids, mi, scale,
                                     softcap, NAN, nullptr, nullptr, num_splits, o_part, lse_part,
                                     static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_attention_merge(const float *o_part, const float *lse_part, int32_t num_splits, int64_t rows,
                                     int32_t dv, void *out, float *lse, void *cuda_stream) {
  if (o_part == nullptr || lse_part == nullptr || out == nullptr || lse == nullptr) return SPLASH_ERR_INVALID_ARG;
  if (num_splits < 1 || num_splits > SPLASH_MAX_SPLITS || rows < 0) return SPLASH_ERR_INVALID_ARG;
  if (dv != 64 && dv != 128) return SPLASH_ERR_UNSUPPORTED;
  if (((reinterpret_cast<uintptr_t>(o_part) | reinterpret_cast<uintptr_t>(out)) & 15u) != 0)
    return SPLASH_ERR_INVALID_ARG;
  return splash_attention_merge_launch(o_part, lse_part, num_splits, rows, dv, out, lse,
                                       static_cast<cudaStream_t>(cuda_stream));
}

splash_status splash_classify_blocks_noalloc(const splash_mask_spec *spec, int64_t Lq, int64_t Lk, int32_t bq,
                                             int32_t bk, int8_t *block_mask, int64_t *totals, void *cuda_stream) {
  if (block_mask == nullptr || totals == nullptr) return SPLASH_ERR_INVALID_ARG;
  splash_status st = check_spec(spec, Lq, Lk);
  if (st != SPLASH_OK) return st;
  if ((st = check_geometry(Lq, Lk, bq, bk)) != SPLASH_OK) return st;
  return splash_classify_blocks_noalloc_impl(spec, Lq, Lk, bq, bk, block_mask, totals,
                                             static_cast<cudaStream_t>(cuda_stream));
}

namespace {

// ---- the serving calls: rotary positions, paged append, paged decode

uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }

struct Dim {
  int64_t size, stride;
};

// Rows of d contiguous elements (`row_align` elements are 16 bytes) at up to
// three outer strides; the stride of a dimension of size 1 is not read.  An
// output's rows must not overlap: with the strides in ascending order, each
// must reach past everything the smaller ones span.
splash_status check_rows(const void *ptr, Dim a, Dim b, Dim c, int64_t d, int64_t row_align, bool output) {
  if (ptr == nullptr || (addr(ptr) & 15u) != 0) return SPLASH_ERR_INVALID_ARG;
  Dim dims[3] = {a, b, c};
  for (Dim &x : dims) {
    if (x.size == 1) x.stride = 0;
    if (x.stride < 0 || x.stride % row_align != 0 || x.stride > ((int64_t)1 << 40)) return SPLASH_ERR_INVALID_ARG;
  }
  if (!output) return SPLASH_OK;
  std::sort(dims, dims + 3, [](const Dim &x, const Dim &y) { return x.stride < y.stride; });
  int64_t span = d;
  for (const Dim &x : dims) {
    if (x.size == 1) continue;
    if (x.stride < span) return SPLASH_ERR_INVALID_ARG;
    // (sizes below 2^31 and strides below 2^41: the product may pass 2^63)
    if (x.stride > 0 && x.size - 1 > (((int64_t)1 << 62) - span) / x.stride) return SPLASH_ERR_UNSUPPORTED;
    span += (x.size - 1) * x.stride;
  }
  return SPLASH_OK;
}

splash_status check_view(const splash_view &v, int64_t B, int64_t H, int64_t L, int64_t d, bool output) {
  return check_rows(v.ptr, {B, v.stride_b}, {H, v.stride_h}, {L, v.stride_l}, d, 8, output);
}

// An output that is its input's own view is written in place.
splash_status check_out_view(const splash_view &out, const splash_view &in, int64_t B, int64_t H, int64_t L, int64_t d) {
  const splash_status st = check_view(out, B, H, L, d, true);
  if (st != SPLASH_OK || out.ptr != in.ptr) return st;
  const bool same = (B == 1 || out.stride_b == in.stride_b) && (H == 1 || out.stride_h == in.stride_h) &&
                    (L == 1 || out.stride_l == in.stride_l);
  return same ? SPLASH_OK : SPLASH_ERR_INVALID_ARG;
}

splash_status check_cache(const splash_cache_view &v, int64_t pages, int64_t Hkv, int64_t page_size, int64_t d,
                          int32_t type, bool output) {
  return check_rows(v.ptr, {pages, v.stride_page}, {Hkv, v.stride_head}, {page_size, v.stride_token}, d,
                    type == SPLASH_CACHE_E4M3 ? 16 : 8, output);
}

splash_status check_rotation(const float *table, int64_t table_rows, int32_t d, int32_t rot_dim, int32_t rot_offset,
                             int32_t interleaved) {
  if (table == nullptr || (addr(table) & 15u) != 0 || table_rows <= 0) return SPLASH_ERR_INVALID_ARG;
  if (rot_dim <= 0 || rot_offset < 0 || (interleaved != 0 && interleaved != 1)) return SPLASH_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0 || rot_offset % 8 != 0) return SPLASH_ERR_UNSUPPORTED;
  if (rot_dim > d || rot_offset > d - rot_dim) return SPLASH_ERR_SHAPE;
  return SPLASH_OK;
}

bool valid_head_dim(int32_t d) { return d % 16 == 0 && d <= 512; }

splash_status check_tokens(int32_t B, int64_t L, int64_t heads) {
  if (L > INT32_MAX || (int64_t)B * L > INT32_MAX || heads > 65535) return SPLASH_ERR_UNSUPPORTED;
  return SPLASH_OK;
}

// (positions leave room for the kernels' look ahead in 32 bits)
splash_status check_page_sizes(int32_t page_size, int32_t max_pages) {
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return SPLASH_ERR_UNSUPPORTED;
  return (int64_t)max_pages * page_size > INT32_MAX - 65535 ? SPLASH_ERR_UNSUPPORTED : SPLASH_OK;
}

splash_status check_pages(const splash_cache_view &k, const splash_cache_view &v, int64_t num_pages, int32_t Hkv,
                          int32_t page_size, int32_t dqk, int32_t dv, int32_t type, const float *k_scale,
                          const float *v_scale, const int32_t *block_table, int64_t block_table_stride, int64_t rows,
                          int32_t max_pages, bool output) {
  if (num_pages <= 0 || max_pages <= 0 || rows <= 0 || page_size <= 0 || block_table == nullptr)
    return SPLASH_ERR_INVALID_ARG;
  if ((addr(block_table) & 3u) != 0 || (rows > 1 && block_table_stride < 0)) return SPLASH_ERR_INVALID_ARG;
  if (type != SPLASH_CACHE_BF16 && type != SPLASH_CACHE_E4M3) return SPLASH_ERR_INVALID_ARG;
  if (type == SPLASH_CACHE_E4M3 &&
      (k_scale == nullptr || v_scale == nullptr || ((addr(k_scale) | addr(v_scale)) & 3u) != 0))
    return SPLASH_ERR_INVALID_ARG;
  if (num_pages > INT32_MAX) return SPLASH_ERR_UNSUPPORTED;
  splash_status st = check_page_sizes(page_size, max_pages);
  if (st != SPLASH_OK) return st;
  st = check_cache(k, num_pages, Hkv, page_size, dqk, type, output);
  if (st != SPLASH_OK) return st;
  return check_cache(v, num_pages, Hkv, page_size, dv, type, output);
}

splash_status check_rope(const splash_rope_args &a) {
  const bool has_k = a.k.ptr != nullptr;
  if (a.B <= 0 || a.Hq <= 0 || a.L <= 0 || a.d <= 0 || (has_k && a.Hkv <= 0)) return SPLASH_ERR_INVALID_ARG;
  if (a.positions == nullptr || (addr(a.positions) & 3u) != 0 || (a.B > 1 && a.positions_stride_b < 0))
    return SPLASH_ERR_INVALID_ARG;
  if (a.inverse != 0 && a.inverse != 1) return SPLASH_ERR_INVALID_ARG;
  if (!valid_head_dim(a.d)) return SPLASH_ERR_UNSUPPORTED;
  splash_status st = check_rotation(a.table, a.table_rows, a.d, a.rot_dim, a.rot_offset, a.interleaved);
  if (st != SPLASH_OK) return st;
  if ((st = check_tokens(a.B, a.L, (int64_t)a.Hq + (has_k ? a.Hkv : 0))) != SPLASH_OK) return st;
  if ((st = check_view(a.q, a.B, a.Hq, a.L, a.d, false)) != SPLASH_OK) return st;
  if ((st = check_out_view(a.q_out, a.q, a.B, a.Hq, a.L, a.d)) != SPLASH_OK) return st;
  if (has_k) {
    if ((st = check_view(a.k, a.B, a.Hkv, a.L, a.d, false)) != SPLASH_OK) return st;
    if ((st = check_out_view(a.k_out, a.k, a.B, a.Hkv, a.L, a.d)) != SPLASH_OK) return st;
  }
  return SPLASH_OK;
}

splash_status check_append(const splash_paged_append_args &a) {
  const bool has_q = a.q.ptr != nullptr;
  if (a.B <= 0 || a.Hkv <= 0 || a.L <= 0 || a.dqk <= 0 || a.dv <= 0 || (has_q && a.Hq <= 0))
    return SPLASH_ERR_INVALID_ARG;
  if (a.positions == nullptr || ((addr(a.positions) | addr(a.seq_ids)) & 3u) != 0) return SPLASH_ERR_INVALID_ARG;
  if (a.B > 1 && (a.positions_stride_b < 0 || (a.seq_ids != nullptr && a.seq_ids_stride_b < 0)))
    return SPLASH_ERR_INVALID_ARG;
  if (!valid_head_dim(a.dqk) || !valid_head_dim(a.dv)) return SPLASH_ERR_UNSUPPORTED;
  if (a.seq_ids == nullptr && a.num_seqs < a.B) return SPLASH_ERR_SHAPE;
  splash_status st = SPLASH_OK;
  if (a.table != nullptr &&
      (st = check_rotation(a.table, a.table_rows, a.dqk, a.rot_dim, a.rot_offset, a.interleaved)) != SPLASH_OK)
    return st;
  if ((st = check_tokens(a.B, a.L, (int64_t)(has_q ? a.Hq : 0) + 2 * (int64_t)a.Hkv)) != SPLASH_OK) return st;
  if ((st = check_pages(a.k_cache, a.v_cache, a.num_pages, a.Hkv, a.page_size, a.dqk, a.dv, a.cache_type, a.k_scale,
                        a.v_scale, a.block_table, a.block_table_stride, a.num_seqs, a.max_pages, true)) != SPLASH_OK)
    return st;
  if ((st = check_view(a.k, a.B, a.Hkv, a.L, a.dqk, false)) != SPLASH_OK) return st;
  if ((st = check_view(a.v, a.B, a.Hkv, a.L, a.dv, false)) != SPLASH_OK) return st;
  if (has_q) {
    if ((st = check_view(a.q, a.B, a.Hq, a.L, a.dqk, false)) != SPLASH_OK) return st;
    if ((st = check_out_view(a.q_out, a.q, a.B, a.Hq, a.L, a.dqk)) != SPLASH_OK) return st;
  } else if (a.q_out.ptr != nullptr) {
    return SPLASH_ERR_INVALID_ARG;
  }
  if (a.k_out.ptr != nullptr &&
      (st = check_out_view(a.k_out, a.k, a.B, a.Hkv, a.L, a.dqk)) != SPLASH_OK)
    return st;
  return SPLASH_OK;
}

splash_status check_axes(const uint8_t *axes, int32_t num_axes, int32_t rot_dim, const int32_t *positions, int64_t stride_a,
                         int64_t stride_b, int32_t B, int32_t reserved) {
  if (axes == nullptr || num_axes <= 0 || reserved != 0 || positions == nullptr || (addr(positions) & 3u) != 0)
    return SPLASH_ERR_INVALID_ARG;
  if ((num_axes > 1 && stride_a < 0) || (B > 1 && stride_b < 0)) return SPLASH_ERR_INVALID_ARG;
  if (num_axes > SPLASH_MAX_AXES) return SPLASH_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < rot_dim / 2; ++i)
    if (axes[i] >= num_axes) return SPLASH_ERR_INVALID_ARG;
  return SPLASH_OK;
}

// What the attention calls over a paged cache have in common; most: new tokens per sequence.
splash_status check_decode_sizes(int32_t B, int32_t Hq, int32_t Hkv, int32_t Lq, int32_t most, int32_t dqk, int32_t dv,
                                 int32_t max_pages, int32_t page_size, int32_t cache_type, int64_t window_left) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Lq <= 0 || dqk <= 0 || dv <= 0 || max_pages <= 0 || page_size <= 0 ||
      window_left < -1 || (cache_type != SPLASH_CACHE_BF16 && cache_type != SPLASH_CACHE_E4M3))
    return SPLASH_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return SPLASH_ERR_SHAPE;
  if (Lq > most || B > 65535 || Hq > 65535 || (int64_t)B * Hq * Lq > INT32_MAX) return SPLASH_ERR_UNSUPPORTED;
  if (!((dqk == 64 && dv == 64) || (dqk == 128 && dv == 128) || (dqk == 192 && dv == 128))) return SPLASH_ERR_UNSUPPORTED;
  return check_page_sizes(page_size, max_pages);
}

// paged_decode.cu's list: 16-key steps of every sequence, head and 16 rows, in 32 bits.
splash_status check_decode_list(int32_t B, int32_t Hq, int32_t Hkv, int32_t Lq, int32_t max_pages, int32_t page_size, int64_t window_left) {
  int64_t steps = (int64_t)max_pages * page_size / 16 + 1;
  if (window_left >= 0) steps = std::min(steps, window_left / 16 + 4);
  const int64_t segments = (int64_t)B * Hkv * (((int64_t)(Hq / Hkv) * Lq + 15) / 16);
  return steps > INT32_MAX / segments ? SPLASH_ERR_UNSUPPORTED : SPLASH_OK;
}

// need: bytes of workspace.
splash_status check_decode(const splash_paged_decode_args &a, size_t need) {
  if (need > 0 && (a.workspace == nullptr || a.workspace_bytes < need)) return SPLASH_ERR_INVALID_ARG;
  const splash_status st =
      check_pages(a.k_cache, a.v_cache, a.num_pages, a.Hkv, a.page_size, a.dqk, a.dv, a.cache_type, a.k_scale, a.v_scale,
                  a.block_table, a.block_table_stride, a.B, a.max_pages, false);
  if (st != SPLASH_OK) return st;
  return check_view(a.q, a.B, a.Hq, a.Lq, a.dqk, false);
}

// Whether two tables of int32 rows share an entry (conservative where their strides differ).
bool tables_overlap(const int32_t *x, int64_t rows_x, int64_t stride_x, const int32_t *y, int64_t rows_y, int64_t stride_y, int64_t cols) {
  if (rows_x == 0 || rows_y == 0) return false;
  if (rows_x == 1) stride_x = rows_y == 1 ? 0 : stride_y;
  if (rows_y == 1) stride_y = stride_x;
  const uintptr_t end_x = addr(x) + 4 * ((rows_x - 1) * stride_x + cols), end_y = addr(y) + 4 * ((rows_y - 1) * stride_y + cols);
  if (end_x <= addr(y) || end_y <= addr(x)) return false;
  if (stride_x != stride_y || stride_x < cols) return true;
  const int64_t off = (addr(y) > addr(x) ? addr(y) - addr(x) : addr(x) - addr(y)) / 4 % stride_x;  // columns of one buffer's rows
  return off < cols || off > stride_x - cols;
}

splash_status check_decode_values(const splash_paged_decode_args &a) {
  if (a.seq_lens == nullptr || a.out == nullptr || a.lse == nullptr || a.reserved != 0) return SPLASH_ERR_INVALID_ARG;
  if (((addr(a.out) | addr(a.workspace)) & 15u) != 0 || ((addr(a.seq_lens) | addr(a.lse)) & 3u) != 0)
    return SPLASH_ERR_INVALID_ARG;
  if (!(a.scale > 0.f) || !(a.scale < INFINITY) || !(a.softcap == a.softcap) || a.softcap == INFINITY)
    return SPLASH_ERR_INVALID_ARG;
  return SPLASH_OK;
}

splash_status current_error_word(uint32_t **err) {
  int dev = 0;
  SPLASH_CUDA_TRY(cudaGetDevice(&dev));
  *err = splash_device_error_word(dev);
  return *err != nullptr ? SPLASH_OK : SPLASH_ERR_CUDA;
}

}  // namespace

splash_status splash_rope(const splash_rope_args *args, void *cuda_stream) {
  if (args == nullptr || args->struct_bytes != sizeof *args) return SPLASH_ERR_INVALID_ARG;
  splash_status st = check_rope(*args);
  if (st != SPLASH_OK) return st;
  uint32_t *err = nullptr;
  if ((st = current_error_word(&err)) != SPLASH_OK) return st;
  return splash_rope_launch(*args, static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_paged_append(const splash_paged_append_args *args, void *cuda_stream) {
  if (args == nullptr || args->struct_bytes != sizeof *args) return SPLASH_ERR_INVALID_ARG;
  splash_status st = check_append(*args);
  if (st != SPLASH_OK) return st;
  uint32_t *err = nullptr;
  if ((st = current_error_word(&err)) != SPLASH_OK) return st;
  return splash_paged_append_launch(*args, static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_rope_axes(const splash_rope_axes_args *args, void *cuda_stream) {
  if (args == nullptr || args->struct_bytes != sizeof *args || args->rope.struct_bytes != sizeof args->rope)
    return SPLASH_ERR_INVALID_ARG;
  splash_status st = check_rope(args->rope);
  if (st != SPLASH_OK) return st;
  st = check_axes(args->axes, args->num_axes, args->rope.rot_dim, args->rope.positions, args->positions_stride_a,
                  args->rope.positions_stride_b, args->rope.B, args->reserved);
  if (st != SPLASH_OK) return st;
  uint32_t *err = nullptr;
  if ((st = current_error_word(&err)) != SPLASH_OK) return st;
  return splash_rope_axes_launch(*args, static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_paged_append_axes(const splash_paged_append_axes_args *args, void *cuda_stream) {
  if (args == nullptr || args->struct_bytes != sizeof *args || args->append.struct_bytes != sizeof args->append ||
      args->append.table == nullptr)
    return SPLASH_ERR_INVALID_ARG;
  splash_status st = check_append(args->append);
  if (st != SPLASH_OK) return st;
  st = check_axes(args->axes, args->num_axes, args->append.rot_dim, args->rot_positions, args->rot_positions_stride_a,
                  args->rot_positions_stride_b, args->append.B, args->reserved);
  if (st != SPLASH_OK) return st;
  uint32_t *err = nullptr;
  if ((st = current_error_word(&err)) != SPLASH_OK) return st;
  return splash_paged_append_axes_launch(*args, static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_paged_decode_workspace_size(int32_t B, int32_t Hq, int32_t Hkv, int32_t Lq, int32_t dqk, int32_t dv,
                                                 int32_t max_pages, int32_t page_size, int32_t cache_type,
                                                 int64_t window_left, size_t *bytes) {
  if (bytes == nullptr) return SPLASH_ERR_INVALID_ARG;
  splash_status st = check_decode_sizes(B, Hq, Hkv, Lq, SPLASH_MAX_NEW_TOKENS, dqk, dv, max_pages, page_size, cache_type, window_left);
  if (st != SPLASH_OK) return st;
  if ((st = check_decode_list(B, Hq, Hkv, Lq, max_pages, page_size, window_left)) != SPLASH_OK) return st;
  *bytes = splash_paged_decode_workspace_bytes(B, Hq, Hkv, Lq, dqk, dv, max_pages, page_size, cache_type, window_left);
  return SPLASH_OK;
}

splash_status splash_paged_decode(const splash_paged_decode_args *args, void *cuda_stream) {
  if (args == nullptr || args->struct_bytes != sizeof *args) return SPLASH_ERR_INVALID_ARG;
  const splash_paged_decode_args &a = *args;
  splash_status st = check_decode_values(a);
  if (st != SPLASH_OK) return st;
  size_t need = 0;
  st = splash_paged_decode_workspace_size(a.B, a.Hq, a.Hkv, a.Lq, a.dqk, a.dv, a.max_pages, a.page_size, a.cache_type,
                                          a.window_left, &need);
  if (st != SPLASH_OK) return st;
  if ((st = check_decode(a, need)) != SPLASH_OK) return st;
  uint32_t *err = nullptr;
  if ((st = current_error_word(&err)) != SPLASH_OK) return st;
  return splash_paged_decode_launch(a, static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_paged_tree_decode_workspace_size(int32_t B, int32_t Hq, int32_t Hkv, int32_t T, int32_t dqk, int32_t dv,
                                                      int32_t max_pages, int32_t page_size, int32_t cache_type,
                                                      int64_t window_left, size_t *bytes) {
  if (bytes == nullptr) return SPLASH_ERR_INVALID_ARG;
  splash_status st = check_decode_sizes(B, Hq, Hkv, T, SPLASH_MAX_TREE_TOKENS, dqk, dv, max_pages, page_size, cache_type, window_left);
  if (st != SPLASH_OK) return st;
  if (splash_paged_tree_decode_few_rows(Hq, Hkv, T) &&
      (st = check_decode_list(B, Hq, Hkv, T, max_pages, page_size, window_left)) != SPLASH_OK)
    return st;
  if (splash_paged_tree_decode_entries(B, Hq, Hkv, T, max_pages, page_size, window_left) > INT32_MAX) return SPLASH_ERR_UNSUPPORTED;
  *bytes = splash_paged_tree_decode_workspace_bytes(B, Hq, Hkv, T, dqk, dv, max_pages, page_size, cache_type, window_left);
  return SPLASH_OK;
}

splash_status splash_paged_tree_decode(const splash_paged_tree_decode_args *args, void *cuda_stream) {
  if (args == nullptr || args->struct_bytes != sizeof *args || args->decode.struct_bytes != sizeof args->decode)
    return SPLASH_ERR_INVALID_ARG;
  const splash_paged_decode_args &a = args->decode;
  splash_status st = check_decode_values(a);
  if (st != SPLASH_OK) return st;
  if (args->parents == nullptr || (addr(args->parents) & 3u) != 0 || (a.B > 1 && args->parents_stride_b < 0))
    return SPLASH_ERR_INVALID_ARG;
  size_t need = 0;
  st = splash_paged_tree_decode_workspace_size(a.B, a.Hq, a.Hkv, a.Lq, a.dqk, a.dv, a.max_pages, a.page_size, a.cache_type,
                                               a.window_left, &need);
  if (st != SPLASH_OK) return st;
  if ((st = check_decode(a, need)) != SPLASH_OK) return st;
  // what a tensor map holds
  const int64_t size = a.cache_type == SPLASH_CACHE_E4M3 ? 1 : 2;
  for (const splash_cache_view *v : {&a.k_cache, &a.v_cache})
    for (const Dim x : {Dim{a.num_pages, v->stride_page}, Dim{a.Hkv, v->stride_head}, Dim{2, v->stride_token}})
      if (x.size > 1 && size * x.stride >= (int64_t)1 << 40) return SPLASH_ERR_UNSUPPORTED;
  if (a.k_cache.stride_token == 0 || a.v_cache.stride_token == 0) return SPLASH_ERR_UNSUPPORTED;
  uint32_t *err = nullptr;
  if ((st = current_error_word(&err)) != SPLASH_OK) return st;
  return splash_paged_tree_decode_launch(*args, static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_paged_compact(const splash_paged_compact_args *args, void *cuda_stream) {
  if (args == nullptr || args->struct_bytes != sizeof *args) return SPLASH_ERR_INVALID_ARG;
  const splash_paged_compact_args &a = *args;
  if (a.B <= 0 || a.Hkv <= 0 || a.dqk <= 0 || a.dv <= 0 || a.moves <= 0 || a.reserved != 0) return SPLASH_ERR_INVALID_ARG;
  if (a.k_cache.ptr == a.v_cache.ptr) return SPLASH_ERR_INVALID_ARG;  // (rows would move twice)
  if (a.src == nullptr || a.start == nullptr || ((addr(a.src) | addr(a.start)) & 3u) != 0 || (a.B > 1 && a.src_stride < 0))
    return SPLASH_ERR_INVALID_ARG;
  if (!valid_head_dim(a.dqk) || !valid_head_dim(a.dv) || a.Hkv > 65535 || a.moves > INT32_MAX) return SPLASH_ERR_UNSUPPORTED;
  // (the scales are not used: values move as they are)
  const float *scale = reinterpret_cast<const float *>(a.src);
  splash_status st = check_pages(a.k_cache, a.v_cache, a.num_pages, a.Hkv, a.page_size, a.dqk, a.dv, a.cache_type, scale, scale,
                                 a.block_table, a.block_table_stride, a.B, a.max_pages, true);
  if (st != SPLASH_OK) return st;
  uint32_t *err = nullptr;
  if ((st = current_error_word(&err)) != SPLASH_OK) return st;
  return splash_paged_compact_launch(a, static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_paged_remap_workspace_size(int64_t num_pages, int32_t new_rows, size_t *bytes) {
  if (bytes == nullptr || num_pages <= 0 || new_rows <= 0) return SPLASH_ERR_INVALID_ARG;
  if (num_pages > INT32_MAX) return SPLASH_ERR_UNSUPPORTED;
  *bytes = splash_paged_remap_workspace_bytes(num_pages, new_rows);
  return SPLASH_OK;
}

splash_status splash_paged_remap(const splash_paged_remap_args *args, void *cuda_stream) {
  if (args == nullptr || args->struct_bytes != sizeof *args) return SPLASH_ERR_INVALID_ARG;
  const splash_paged_remap_args &a = *args;
  if (a.num_rows < 0 || a.new_rows <= 0 || a.max_pages <= 0 || a.page_size <= 0 || a.num_pages <= 0) return SPLASH_ERR_INVALID_ARG;
  if ((a.num_rows > 0 && a.block_table == nullptr) || a.new_table == nullptr || a.parents == nullptr || a.keep == nullptr ||
      a.room == nullptr || a.refs == nullptr || a.refs_out == nullptr || a.copies == nullptr || a.short_pages == nullptr ||
      a.workspace == nullptr)
    return SPLASH_ERR_INVALID_ARG;
  if (((addr(a.block_table) | addr(a.new_table) | addr(a.parents) | addr(a.keep) | addr(a.room) | addr(a.refs) | addr(a.refs_out) |
        addr(a.copies) | addr(a.short_pages)) & 3u) != 0 ||
      (addr(a.workspace) & 15u) != 0)
    return SPLASH_ERR_INVALID_ARG;
  if ((a.num_rows > 1 && a.block_table_stride < 0) || (a.new_rows > 1 && a.new_table_stride < a.max_pages))
    return SPLASH_ERR_INVALID_ARG;
  splash_status st = check_page_sizes(a.page_size, a.max_pages);
  if (st != SPLASH_OK) return st;
  if ((int64_t)a.num_rows * a.max_pages > INT32_MAX || (int64_t)a.new_rows * a.max_pages > INT32_MAX) return SPLASH_ERR_UNSUPPORTED;
  if ((a.num_rows > 1 && a.block_table_stride > ((int64_t)1 << 29)) || (a.new_rows > 1 && a.new_table_stride > ((int64_t)1 << 29)))
    return SPLASH_ERR_UNSUPPORTED;
  size_t need = 0;
  if ((st = splash_paged_remap_workspace_size(a.num_pages, a.new_rows, &need)) != SPLASH_OK) return st;
  if (a.workspace_bytes < need) return SPLASH_ERR_INVALID_ARG;
  if (tables_overlap(a.block_table, a.num_rows, a.block_table_stride, a.new_table, a.new_rows, a.new_table_stride, a.max_pages) ||
      (a.refs != a.refs_out && tables_overlap(a.refs, 1, 0, a.refs_out, 1, 0, a.num_pages)))
    return SPLASH_ERR_INVALID_ARG;
  uint32_t *err = nullptr;
  if ((st = current_error_word(&err)) != SPLASH_OK) return st;
  return splash_paged_remap_launch(a, static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_paged_copy(const splash_paged_copy_args *args, void *cuda_stream) {
  if (args == nullptr || args->struct_bytes != sizeof *args) return SPLASH_ERR_INVALID_ARG;
  const splash_paged_copy_args &a = *args;
  if (a.count <= 0 || a.Hkv <= 0 || a.dqk <= 0 || a.dv <= 0 || a.copies == nullptr || (addr(a.copies) & 3u) != 0)
    return SPLASH_ERR_INVALID_ARG;
  if (!valid_head_dim(a.dqk) || !valid_head_dim(a.dv) || a.Hkv > 65535) return SPLASH_ERR_UNSUPPORTED;
  const float *scale = reinterpret_cast<const float *>(a.copies);  // (not used)
  splash_status st = check_pages(a.k_cache, a.v_cache, a.num_pages, a.Hkv, a.page_size, a.dqk, a.dv, a.cache_type, scale, scale,
                                 a.copies, 0, 1, 1, true);
  if (st != SPLASH_OK) return st;
  uint32_t *err = nullptr;
  if ((st = current_error_word(&err)) != SPLASH_OK) return st;
  return splash_paged_copy_launch(a, static_cast<cudaStream_t>(cuda_stream), err);
}

splash_status splash_last_device_error(void *cuda_stream) {
  int dev = 0;
  SPLASH_CUDA_TRY(cudaGetDevice(&dev));
  SPLASH_CUDA_TRY(cudaStreamSynchronize(static_cast<cudaStream_t>(cuda_stream)));
  uint32_t *addr = splash_device_error_word(dev);
  if (addr == nullptr) return SPLASH_ERR_CUDA;
  uint32_t word = 0;
  SPLASH_CUDA_TRY(cudaMemcpy(&word, addr, sizeof word, cudaMemcpyDeviceToHost));
  if (word != 0) SPLASH_CUDA_TRY(cudaMemset(addr, 0, sizeof word));
  if (word & (SPLASH_DEV_TIMEOUT_PRODUCER | SPLASH_DEV_TIMEOUT_MMA | SPLASH_DEV_TIMEOUT_SOFTMAX |
              SPLASH_DEV_TIMEOUT_DRAIN | SPLASH_DEV_TIMEOUT_SELFTEST | SPLASH_DEV_TIMEOUT_BUILD))
    return SPLASH_ERR_DEVICE_TIMEOUT;
  if (word & (SPLASH_DEV_BAD_TABLE | SPLASH_DEV_SMEM_ALIGN)) return SPLASH_ERR_DEVICE_CHECK;
  return SPLASH_OK;
}

splash_status splash_debug_wait_selftest(uint64_t timeout_ns, void *cuda_stream) {
  if (timeout_ns == 0 || timeout_ns > 2000000000ull) return SPLASH_ERR_INVALID_ARG;
  int dev = 0;
  SPLASH_CUDA_TRY(cudaGetDevice(&dev));
  uint32_t *err = splash_device_error_word(dev);
  if (err == nullptr) return SPLASH_ERR_CUDA;
  splash_status st = splash_wait_selftest_launch(timeout_ns, static_cast<cudaStream_t>(cuda_stream), err);
  if (st != SPLASH_OK) return st;
  return splash_last_device_error(cuda_stream);
}

}  // extern "C"
