// pages.cu -- the upkeep of a paged cache: remapping block tables (forks,
// growth, truncation, release), copying pages and compacting sequences
// (splash_paged_remap, splash_paged_copy and splash_paged_compact in splash.h).
//
// None of them computes; they read and write each byte once, so HBM bounds the
// large ones and the chain of dependent reads the small ones.  Measured (device time, 8 KV
// heads of 128, bf16): 8192 of 16384 tokens of 8 sequences moved 95 us, 5.6 TB/s, of 1
// sequence 54 us, 1.3 TB/s; the 5 accepted drafts of one 1.9 us; 16 requests of 4 beams, up to
// 2000 tokens, forked and their pages copied 12.0 us; 64 prompts into 8 samples each, pages of
// 128 tokens, 30 us, of which the remap 14; 64 requests of 4 beams, up to 16384 tokens in a pool of
// 134000 pages, 73 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "cluster.cuh"
#include "dependent_launch.cuh"
#include "internal.h"

namespace splash {
namespace {

struct Cache {
  char *ptr;
  int64_t page, head, token;  // byte strides
  int32_t chunks;             // 16-byte chunks of a row
};

Cache cache(const splash_cache_view &v, int64_t size, int32_t d) {
  return {static_cast<char *>(v.ptr), size * v.stride_page, size * v.stride_head, size * v.stride_token, (int32_t)(d * size / 16)};
}

// ------------------------------------------------------------------ compact
constexpr int kMoveThreads = 256, kMoveRows = 256;  // most tokens of a batch
constexpr int kMovesEach = 4;                       // chunks that a thread has in flight

struct CompactParams {
  Cache k, v;
  int32_t k_slices, v_slices;  // groups of up to 8 chunk columns
  const int32_t *block_table, *src, *start;
  int64_t block_table_stride, src_stride, num_pages;
  int64_t moves;
  int32_t max_pages, page_shift;
  uint32_t *err;
};

// A move's places: byte offsets of the rows, from < 0: nothing to do.
struct Move {
  int64_t from, to;
};

// CTA (sequence, head, slice): the slice's columns of all moves in order, in
// batches.  A batch is read into registers before any of it is written; what it
// overwrites (start + m <= src[m]) was read in it or before, and what later
// batches read (src > src[m]) is not overwritten by it, so that one barrier per
// batch is enough.  The places of the next batch (three dependent reads) are
// looked up while this one's data is on the way.  Slices of 8 chunks, 128 bytes of a row, or of 4
// where there are few: the half of 8 sequences' tokens 129 us with 8 chunks, 95 with 4.  The
// batches of a list follow one another: 32 of 256 moves take one sequence 54 us on 64 CTAs, with
// one KV head 36 us on 8, where HBM would take 10 and 1.
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const CompactParams p) {
  __shared__ Move s_move[2][kMoveRows];
  __shared__ int s_end[2];
  grid_dependency();
  const int tid = threadIdx.x, head = blockIdx.y;
  const int64_t b = blockIdx.x;
  const bool is_v = (int)blockIdx.z >= p.k_slices;
  const Cache &c = is_v ? p.v : p.k;
  const int slices = is_v ? p.v_slices : p.k_slices, slice = is_v ? blockIdx.z - p.k_slices : blockIdx.z;
  const int width = (c.chunks + slices - 1) / slices;  // columns of a slice
  const int column = slice * width + tid % width, lane = tid / width, lanes = kMoveThreads / width;
  const int batch = min(kMovesEach * lanes, kMoveRows);
  const bool works = lane < lanes && column < c.chunks;
  char *base = c.ptr + head * c.head + column * 16;
  const int32_t *src = p.src + b * p.src_stride, *pages = p.block_table + b * p.block_table_stride;
  const int64_t first = p.start[b], limit = (int64_t)p.max_pages << p.page_shift;
  const int32_t in_page = (1 << p.page_shift) - 1;
  const bool reports = head == 0 && blockIdx.z == 0;

  // Move m of the list; *stop: the list ends here, *bad: for a reason that is reported.
  auto place = [&](int64_t m, bool *stop, bool *bad) {
    Move x = {-1, -1};
    *stop = true;
    *bad = false;
    const int32_t s = src[m];
    if (s < 0) return x;
    const int64_t d = first + m;
    *bad = first < 0 || s < d || s >= limit || (m > 0 && src[m - 1] >= s);
    if (*bad) return x;
    const int64_t from = pages[s >> p.page_shift], to = pages[d >> p.page_shift];
    *bad = from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages;
    if (*bad) return x;
    *stop = false;
    if (s == d) return x;
    x.from = from * c.page + (s & in_page) * c.token;
    x.to = to * c.page + (d & in_page) * c.token;
    return x;
  };
  // The places of batch [m0, m0 + batch) into s_move[half]; s_end[half]: the list's end in it.
  auto look = [&](int64_t m0, int half) {
    if (tid >= batch || m0 + tid >= p.moves) return;
    bool stop, bad;
    const Move x = place(m0 + tid, &stop, &bad);
    s_move[half][tid] = x;
    // (an entry behind the list's end is not reported: the first one that ends it is)
    if (stop) atomicMin(&s_end[half], 2 * tid + (bad ? 1 : 0));
  };

  if (tid < 2) s_end[tid] = INT_MAX;
  __syncthreads();
  look(0, 0);
  __syncthreads();
  int half = 0;
  for (int64_t m0 = 0; m0 < p.moves; m0 += batch) {
    const int end = s_end[half];  // 2 * index + reported, INT_MAX: none
    const int n = (int)min((int64_t)batch, p.moves - m0);
    const int count = end == INT_MAX ? n : end >> 1;
    uint4 x[kMovesEach];
    bool live[kMovesEach];
    int64_t to[kMovesEach];
#pragma unroll
    for (int i = 0; i < kMovesEach; ++i) {
      const int m = i * lanes + lane;
      live[i] = works && m < count && m < batch;
      if (live[i]) {
        const Move y = s_move[half][m];
        live[i] = y.from >= 0;
        to[i] = y.to;
        if (live[i]) x[i] = *reinterpret_cast<const uint4 *>(base + y.from);
      }
    }
    const bool more = end == INT_MAX && m0 + batch < p.moves;
    if (more) look(m0 + batch, half ^ 1);
    if (end != INT_MAX && (end & 1) && reports && tid == 0) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
    __syncthreads();  // everything of this batch is read, the next one's places are known
#pragma unroll
    for (int i = 0; i < kMovesEach; ++i)
      if (live[i]) *reinterpret_cast<uint4 *>(base + to[i]) = x[i];
    if (!more) return;
    half ^= 1;
  }
}

// ------------------------------------------------------------------ copy
constexpr int kCopyThreads = 256, kCopyEach = 4;

struct CopyParams {
  Cache k, v;
  const int32_t *copies;
  int64_t num_pages;
  int32_t page_size;
  uint32_t *err;
};

// CTA (entry, head, K or V): the rows of a page, 16 bytes a thread and four of them in flight.
// (512 entries of pages of up to 128 rows, 8 heads: 16 us.  140 MB pass L2, at 36 % of its rate, 15 MB
// HBM: what it waits for is each CTA's own chain, the entry and one or two rounds of reads.)
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyParams p) {
  grid_dependency();
  const int32_t *entry = p.copies + 3 * (int64_t)blockIdx.x;
  const int32_t from = entry[0], to = entry[1], rows = entry[2];
  if (from < 0 || to < 0 || rows <= 0) return;
  if (from >= p.num_pages || to >= p.num_pages || rows > p.page_size) {
    if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
    return;
  }
  if (from == to) return;
  const Cache &c = blockIdx.z == 0 ? p.k : p.v;
  const char *src = c.ptr + from * c.page + blockIdx.y * c.head;
  char *dst = c.ptr + to * c.page + blockIdx.y * c.head;
  const int n = rows * c.chunks;  // (at most 1024 rows of 64)
  for (int i0 = threadIdx.x; i0 < n; i0 += kCopyThreads * kCopyEach) {
    uint4 x[kCopyEach];
    int64_t at[kCopyEach];
#pragma unroll
    for (int k = 0; k < kCopyEach; ++k) {
      const int i = i0 + k * kCopyThreads;
      if (i < n) {
        const int row = i / c.chunks;
        at[k] = row * c.token + (i - row * c.chunks) * 16;
        x[k] = *reinterpret_cast<const uint4 *>(src + at[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kCopyEach; ++k)
      if (i0 + k * kCopyThreads < n) *reinterpret_cast<uint4 *>(dst + at[k]) = x[k];
  }
}

// ------------------------------------------------------------------ remap
constexpr int kMapThreads = 1024, kMapCtas = 8, kMapWarps = kMapThreads / 32;
constexpr int kPagesEach = 4;    // pages of a thread in a scan's round
constexpr int kSharedRows = 4096;  // new rows whose needs every CTA adds up by itself

struct RemapParams {
  const int32_t *block_table;
  int64_t block_table_stride;
  int32_t *new_table;
  int64_t new_table_stride;
  const int32_t *parents, *keep, *room, *refs;
  int32_t *refs_out, *copies, *short_pages;
  // workspace: per page its uses, the rows that keep part of it and the first of them; the
  // free pages in order; per row the fresh pages before it
  int32_t *uses, *parts, *first, *fresh, *before;
  int32_t *totals;  // [2][kMapCtas]: free pages, needed pages of each CTA's share
  int64_t num_pages;
  int32_t num_rows, new_rows, max_pages, page_shift;
  uint32_t *err;
};

// Sum over the CTA's threads before this one, and *all of them.
__device__ __forceinline__ int32_t scan(int32_t x, int32_t *s_warp, int32_t *all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t z = __shfl_up_sync(~0u, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) s_warp[warp] = y;
  __syncthreads();
  int32_t w = s_warp[lane], total = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t z = __shfl_up_sync(~0u, total, o);
    if (lane >= o) total += z;
  }
  *all = __shfl_sync(~0u, total, 31);
  const int32_t base = __shfl_sync(~0u, total - w, warp);
  __syncthreads();  // (s_warp is used again)
  return base + y - x;
}

// What a new row takes over, in tokens and columns.
struct Row {
  int32_t parent;           // -1: none
  int32_t keep, cols_kept;  // columns that hold kept tokens
  int32_t cols;             // of the row
  bool part;                // the last kept column holds other tokens too
  bool bad;
};

__device__ __forceinline__ Row row_of(const RemapParams &p, int i) {
  Row r;
  const int32_t limit = p.max_pages << p.page_shift;  // (the host keeps it below 2^31)
  r.parent = p.parents[i];
  int32_t keep = p.keep[i], room = p.room[i];
  r.bad = r.parent >= p.num_rows || keep < 0 || keep > limit || room > limit;
  if (r.parent < 0 || r.parent >= p.num_rows) r.parent = -1;
  r.keep = r.parent < 0 ? 0 : max(0, min(keep, limit));
  room = max(r.keep, min(room, limit));
  const int32_t up = (1 << p.page_shift) - 1;
  r.cols_kept = (int32_t)(((int64_t)r.keep + up) >> p.page_shift);
  r.cols = (int32_t)(((int64_t)room + up) >> p.page_shift);
  r.part = (r.keep & up) != 0;
  return r;
}

__device__ __forceinline__ bool is_page(const RemapParams &p, int32_t x) { return x >= 0 && x < p.num_pages; }

// Whether row i's last kept page, of which it keeps a part, has to be copied
// (after all uses are counted, each shared page once for every row that keeps it).
__device__ __forceinline__ bool copied(const RemapParams &p, int i, int32_t page) {
  const int32_t uses = __ldcg(p.uses + page), parts = __ldcg(p.parts + page), first = __ldcg(p.first + page);
  return uses != parts || first != i;
}

// Fresh pages that row i needs.
__device__ __forceinline__ int32_t need_of(const RemapParams &p, int i) {
  const Row r = row_of(p, i);
  int32_t need = r.cols - r.cols_kept;
  if (r.part) {
    const int32_t x = p.block_table[r.parent * p.block_table_stride + r.cols_kept - 1];
    if (is_page(p, x) && copied(p, i, x)) ++need;
  }
  return need;
}

// One cluster: its 8192 threads hold the counters of a usual pool in one or two
// rounds, and the phases are barriers of the cluster instead of launches.  What
// bounds it is the chain of dependent reads: counts; entries, and the counts that they
// change; last pages and their counts; fresh pages (fork of 16 requests of 4 beams: 10 us; with four
// barriers and units of 128 columns the fork and its copies took 19.7 us, now 12).  All sums are of
// integers, so that the order of the atomics does not show.
__global__ void __launch_bounds__(kMapThreads) remap_kernel(const RemapParams p) {
  __shared__ int32_t s_warp[32], s_before[kSharedRows];
  grid_dependency();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  bool bad = false;
  // ---- this CTA's pages: counters, and how many are free
  const int64_t per_cta = (p.num_pages + kMapCtas - 1) / kMapCtas;
  const int64_t page0 = min(p.num_pages, cta * per_cta), page1 = min(p.num_pages, page0 + per_cta);
  int32_t free_pages = 0;
  for (int64_t x = page0 + tid; x < page1; x += kMapThreads) {
    const int32_t n = p.refs[x];
    p.uses[x] = n;
    p.parts[x] = 0;
    p.first[x] = INT_MAX;
    free_pages += n == 0;
  }
  int32_t all_free;
  scan(free_pages, s_warp, &all_free);
  if (tid == 0) p.totals[cta] = all_free;
  cluster_sync();

  // ---- uses: a warp per 32 columns of a row of either table
  const uint32_t chunks = (uint32_t)(p.max_pages + 31) / 32, all_warps = kMapCtas * kMapWarps, gw = cta * kMapWarps + warp;
  const uint32_t old_units = p.num_rows * chunks, new_units = p.new_rows * chunks;  // (below 2^31)
  for (uint32_t unit = gw; unit < old_units; unit += all_warps) {
    const int32_t i = unit / chunks, j = (unit - i * chunks) * 32 + lane;
    const int32_t x = j < p.max_pages ? p.block_table[i * p.block_table_stride + j] : -1;
    if (is_page(p, x)) atomicSub(p.uses + x, 1);
  }
  for (uint32_t unit = gw; unit < new_units; unit += all_warps) {
    const int32_t i = unit / chunks, j = (unit - i * chunks) * 32 + lane;
    const Row r = row_of(p, i);
    bad |= r.bad;
    if (j >= r.cols_kept) continue;
    const int32_t x = p.block_table[r.parent * p.block_table_stride + j];
    if (!is_page(p, x)) {
      bad = true;
      continue;
    }
    atomicAdd(p.uses + x, 1);
    if (r.part && j == r.cols_kept - 1) {
      atomicAdd(p.parts + x, 1);
      atomicMin(p.first + x, i);
    }
  }
  // (and, meanwhile, the free pages in order)
  int64_t total_free = 0;
  int32_t free_before = 0;
#pragma unroll
  for (int k = 0; k < kMapCtas; ++k) {
    const int32_t f = __ldcg(p.totals + k);
    if (k < cta) free_before += f;
    total_free += f;
  }
  const int32_t rank0 = free_before;
  for (int64_t x0 = page0; x0 < page1; x0 += kMapThreads * kPagesEach) {
    const int64_t mine = x0 + (int64_t)tid * kPagesEach;
    int32_t n[kPagesEach], here = 0, all;
#pragma unroll
    for (int k = 0; k < kPagesEach; ++k) {
      n[k] = mine + k < page1 ? p.refs[mine + k] : 1;
      here += n[k] == 0;
    }
    int32_t rank = free_before + scan(here, s_warp, &all);
#pragma unroll
    for (int k = 0; k < kPagesEach; ++k)
      if (n[k] == 0) p.fresh[rank++] = (int32_t)(mine + k);
    free_before += all;
  }
  cluster_sync();

  // ---- the fresh pages that each row needs, and those before it: every CTA for all rows, or where
  // there are many, its share of them, joined by another barrier
  int64_t all_needed = 0;
  const bool shared = p.new_rows <= kSharedRows;
  const int32_t rows_each = shared ? p.new_rows : (int32_t)(((int64_t)p.new_rows + kMapCtas - 1) / kMapCtas);
  const int32_t row0 = shared ? 0 : (int32_t)min((int64_t)p.new_rows, (int64_t)cta * rows_each), row1 = min(p.new_rows, row0 + rows_each);
  int32_t needed = 0;
  for (int32_t i0 = row0; i0 < row1; i0 += kMapThreads) {
    const int i = i0 + tid;
    int32_t all;
    const int32_t at = needed + scan(i < row1 ? need_of(p, i) : 0, s_warp, &all);
    if (i < row1) (shared ? s_before : p.before)[i] = at;
    needed += all;
  }
  if (shared) {
    all_needed = needed;
    __syncthreads();
  } else {
    if (tid == 0) p.totals[kMapCtas + cta] = needed;
    cluster_sync();
    for (int k = 0; k < kMapCtas; ++k) all_needed += __ldcg(p.totals + kMapCtas + k);
  }
  const int64_t given = min(all_needed, total_free);
  if (cta == 0 && tid == 0) *p.short_pages = (int32_t)(all_needed - given);

  // ---- the new table: a warp per 32 columns of a row
  for (uint32_t unit = gw; unit < new_units; unit += all_warps) {
    const int32_t i = unit / chunks, c = unit - i * chunks, j = c * 32 + lane;
    const Row r = row_of(p, i);
    const int32_t *old = p.block_table + (int64_t)max(r.parent, 0) * p.block_table_stride;
    const int32_t kept = j < r.cols_kept ? old[j] : -1, last = r.part ? old[r.cols_kept - 1] : -1;
    int64_t rank = shared ? s_before[i] : __ldcg(p.before + i);
    if (!shared)
      for (int k = 0; k < i / rows_each; ++k) rank += __ldcg(p.totals + kMapCtas + k);
    const bool copy = r.part && is_page(p, last) && copied(p, i, last);
    const int32_t held = r.cols_kept - (copy ? 1 : 0);
    int32_t x = -1;
    if (j < held) {
      x = is_page(p, kept) ? kept : -1;
    } else if (j < r.cols && (copy || j >= r.cols_kept)) {
      const int64_t k = rank + (j - held);
      if (k < given) x = __ldcg(p.fresh + k);
    }
    if (j < p.max_pages) p.new_table[i * p.new_table_stride + j] = x;
    if (c == 0 && lane < 3) {
      const int32_t to = copy && rank < given ? __ldcg(p.fresh + rank) : -1;
      const int32_t y = lane == 0 ? last : lane == 1 ? to : r.keep & ((1 << p.page_shift) - 1);
      p.copies[3 * (int64_t)i + lane] = to >= 0 ? y : lane == 2 ? 0 : -1;
    }
  }
  // ---- counts out (in place: nobody reads refs any more but this thread)
  free_before = rank0;
  for (int64_t x0 = page0; x0 < page1; x0 += kMapThreads * kPagesEach) {
    const int64_t mine = x0 + (int64_t)tid * kPagesEach;
    int32_t n[kPagesEach], here = 0, all;
#pragma unroll
    for (int k = 0; k < kPagesEach; ++k) {
      n[k] = mine + k < page1 ? p.refs[mine + k] : 1;
      here += n[k] == 0;
    }
    int32_t rank = free_before + scan(here, s_warp, &all);
#pragma unroll
    for (int k = 0; k < kPagesEach; ++k) {
      const int64_t x = mine + k;
      if (x >= page1) continue;
      const int32_t parts = __ldcg(p.parts + x);
      int32_t uses = __ldcg(p.uses + x);
      bad |= uses < 0;
      uses -= parts > 0 && uses == parts ? parts - 1 : parts;  // (copied: not kept)
      if (n[k] == 0 && rank++ < given) ++uses;
      p.refs_out[x] = uses;
    }
    free_before += all;
  }
  if (bad) atomicOr(p.err, SPLASH_DEV_BAD_TABLE);
}

}  // namespace
}  // namespace splash

splash_status splash_paged_compact_launch(const splash_paged_compact_args &a, cudaStream_t stream, uint32_t *err_word) {
  using namespace splash;
  const int64_t size = a.cache_type == SPLASH_CACHE_E4M3 ? 1 : 2;
  CompactParams p = {};
  p.k = cache(a.k_cache, size, a.dqk);
  p.v = cache(a.v_cache, size, a.dv);
  // slices of 128 bytes of a row, or of 64 where those leave an SM with fewer than four CTAs
  int width = 8;
  if ((int64_t)a.B * a.Hkv * ((p.k.chunks + 7) / 8 + (p.v.chunks + 7) / 8) < 4 * 152) width = 4;
  p.k_slices = (p.k.chunks + width - 1) / width;
  p.v_slices = (p.v.chunks + width - 1) / width;
  p.block_table = a.block_table;
  p.block_table_stride = a.block_table_stride;
  p.src = a.src;
  p.src_stride = a.src_stride;
  p.start = a.start;
  p.num_pages = a.num_pages;
  p.moves = a.moves;
  p.max_pages = a.max_pages;
  p.page_shift = __builtin_ctz((unsigned)a.page_size);
  p.err = err_word;
  const dim3 grid((unsigned)a.B, (unsigned)a.Hkv, (unsigned)(p.k_slices + p.v_slices));
  SPLASH_CUDA_TRY(launch_dependent(compact_kernel, grid, dim3(kMoveThreads), 0, 1, stream, p));
  splash_count_launches(1);
  return SPLASH_OK;
}

splash_status splash_paged_copy_launch(const splash_paged_copy_args &a, cudaStream_t stream, uint32_t *err_word) {
  using namespace splash;
  const int64_t size = a.cache_type == SPLASH_CACHE_E4M3 ? 1 : 2;
  CopyParams p = {};
  p.k = cache(a.k_cache, size, a.dqk);
  p.v = cache(a.v_cache, size, a.dv);
  p.copies = a.copies;
  p.num_pages = a.num_pages;
  p.page_size = a.page_size;
  p.err = err_word;
  const dim3 grid((unsigned)a.count, (unsigned)a.Hkv, 2);
  SPLASH_CUDA_TRY(launch_dependent(copy_kernel, grid, dim3(kCopyThreads), 0, 1, stream, p));
  splash_count_launches(1);
  return SPLASH_OK;
}

size_t splash_paged_remap_workspace_bytes(int64_t num_pages, int32_t new_rows) {
  return (size_t)(4 * (4 * num_pages + (int64_t)new_rows + 2 * splash::kMapCtas) + 15) & ~(size_t)15;
}

splash_status splash_paged_remap_launch(const splash_paged_remap_args &a, cudaStream_t stream, uint32_t *err_word) {
  using namespace splash;
  RemapParams p = {};
  p.block_table = a.block_table;
  p.block_table_stride = a.block_table_stride;
  p.new_table = a.new_table;
  p.new_table_stride = a.new_table_stride;
  p.parents = a.parents;
  p.keep = a.keep;
  p.room = a.room;
  p.refs = a.refs;
  p.refs_out = a.refs_out;
  p.copies = a.copies;
  p.short_pages = a.short_pages;
  p.uses = static_cast<int32_t *>(a.workspace);
  p.parts = p.uses + a.num_pages;
  p.first = p.parts + a.num_pages;
  p.fresh = p.first + a.num_pages;
  p.before = p.fresh + a.num_pages;
  p.totals = p.before + a.new_rows;
  p.num_pages = a.num_pages;
  p.num_rows = a.num_rows;
  p.new_rows = a.new_rows;
  p.max_pages = a.max_pages;
  p.page_shift = __builtin_ctz((unsigned)a.page_size);
  p.err = err_word;
  SPLASH_CUDA_TRY(launch_dependent(remap_kernel, dim3(kMapCtas), dim3(kMapThreads), 0, kMapCtas, stream, p));
  splash_count_launches(1);
  return SPLASH_OK;
}
